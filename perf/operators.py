"""The operators of the paged 4-bit KV cache, as they are measured.

Three operators share one cache.  A layer's cache is a pool of pages of `page` positions
each; K and V are NVFP4 (E2M1 codes two per byte, the even element in the low nibble, one
E4M3 scale per 16 elements of a head, one fp32 scale per kv head):
    codes  [pages][kv_heads][page][head_dim / 2]      scales [pages][kv_heads][page][head_dim / 16]

plan    block tables and slot maps from the requests' lengths: which pages a step's new
        tokens take from the free list, where each token goes, what finished requests return
append  the new tokens' K and V rows quantised into their slots
attn    causal attention of the new tokens over the cache: one token a request (decode), a
        few (draft tokens), or long chunks of a prompt, in one ragged batch

A case is plain values; lengths follow from it alone, values from the seed.
"""
import math
import zlib

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------- cases

def _plan(name, n, page, width, old, new_lo, new_hi, release):
    return dict(name=name, kind="plan", n_seqs=n, page=page, width=width, old=old, new_lo=new_lo,
                new_hi=new_hi, release=release)


def _append(name, tokens, kv_heads, head_dim, page, dtype, fused, padded):
    return dict(name=name, kind="append", tokens=tokens, kv_heads=kv_heads, head_dim=head_dim,
                page=page, dtype=dtype, fused=fused, padded=padded)


def _attn(name, n, len_lo, len_hi, new_lo, new_hi, heads, kv_heads, head_dim, page, dtype, idle=0,
          fused=False):
    return dict(name=name, kind="attn", n_seqs=n, len_lo=len_lo, len_hi=len_hi, new_lo=new_lo,
                new_hi=new_hi, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
                dtype=dtype, idle=idle, fused=fused)


def listed():
    return [
        # one decode step of a small batch: one new token a request, latency alone
        _plan("plan_decode_8", 8, 16, 256, 4000, 1, 1, 0),
        # a busy server admits prompts while others decode or finish: ragged, thousands of requests
        _plan("plan_prompts_2048", 2048, 32, 128, 1900, 1, 200, 7),
        # the K and V rows of one decode step, from bf16 projections, some slots of the batch padded
        _append("append_decode_bf16", 64, 4, 128, 16, "bf16", False, 5),
        # a long prompt's rows, F32, read in place from the side-by-side Q/K/V rows
        _append("append_prompt_f32", 16384, 4, 128, 64, "f32", True, 0),
        # the batch-1 decode layer of the framework's own 48-layer step: 4096 positions, F32
        _attn("decode_1x4096_f32", 1, 4096, 4096, 1, 1, 32, 4, 128, 16, "f32"),
        # an ordinary serving batch: ragged contexts, some slots idle
        _attn("decode_64_ragged_bf16", 64, 100, 8192, 1, 1, 32, 4, 128, 32, "bf16", idle=9),
        # few requests with very long contexts: work has to be split along the context
        _attn("decode_4x131072_f16", 4, 131072, 131072, 1, 1, 32, 4, 128, 64, "f16"),
        # odd head layout (7 query heads a kv head, 64 wide), odd lengths
        _attn("decode_37_odd_f16", 37, 1, 5003, 1, 1, 28, 4, 64, 16, "f16", idle=6),
        # checking a few draft tokens a request
        _attn("draft_16x5_bf16", 16, 700, 6001, 5, 5, 32, 4, 128, 16, "bf16"),
        # a prompt from its first token, F32 rows
        _attn("prompt_777_f32", 1, 777, 777, 777, 777, 32, 4, 128, 32, "f32", fused=True),
        # continuous batching: decoding requests and prompt chunks in one call
        _attn("mixed_24_bf16", 24, 300, 6000, 1, 500, 32, 4, 128, 32, "bf16"),
        # long prompts in chunks of 2048 tokens, bound by the matrix products
        _attn("chunk_4x2048_bf16", 4, 8192, 16384, 2048, 2048, 32, 4, 128, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = ((32, 4), (28, 4), (40, 8), (64, 4), (10, 10), (8, 1), (6, 2))


def draw(rng):
    kind = rng.choice(["plan", "append", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "plan":
        n = _log(rng, 1, 4096)
        old = _log(rng, 1, 4096)
        hi = max(1, min(_log(rng, 1, 4096), 200000 // n))
        lo = rng.choice([0, 1, hi])
        width = (old + hi) // page + 1 + rng.randrange(8)
        return {k: v for k, v in _plan("", n, page, width, old, min(lo, hi), hi, rng.choice([0, 3, 10])).items()
                if k != "name"}
    head_dim = rng.choice([64, 128, 256])
    heads, kv_heads = rng.choice(HEADS)
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind == "append":
        tokens = _log(rng, 1, 16384)
        c = _append("", tokens, kv_heads, head_dim, page, dtype, rng.random() < 0.5, rng.choice([0, min(3, tokens - 1)]))
        return {k: v for k, v in c.items() if k != "name"}
    most = max(_cost(c) for c in listed())
    form = rng.choice(["decode", "draft", "chunk", "mixed"])
    n = _log(rng, 1, 256 if form == "decode" else 64 if form == "draft" else 16)
    hi = _log(rng, 1 if rng.random() < 0.2 else 40, 65536 if n < 8 else 16384)
    lo = max(1, hi // rng.choice([1, 3, 50]))
    new = {"decode": (1, 1), "draft": (2, 9), "chunk": (hi, hi), "mixed": (1, hi)}[form]
    cap = _log(rng, 16, 2048)
    new = tuple(max(1, min(x, cap, hi)) for x in new)
    while True:
        c = _attn("", n, lo, hi, new[0], new[1], heads, kv_heads, head_dim, page, dtype,
                  idle=rng.choice([0, 5]), fused=rng.random() < 0.3)
        # the plain form works on the padded batch: keep its scores and rows within a few GB
        if _cost(c) <= most / 2 and n * heads * new[1] * hi < 3e9 and n * hi * kv_heads * head_dim < 1e9:
            return {k: v for k, v in c.items() if k != "name"}
        hi = max(1, hi * 2 // 3)
        lo, new = min(lo, hi), tuple(min(x, hi) for x in new)
        n = max(1, n * 3 // 4)


def _numbers(case):
    """The case's own stream of lengths: the same for every seed."""
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return np.random.RandomState(zlib.crc32(text.encode()) & 0x7FFFFFFF)


def _log_uniform(rs, lo, hi, n):
    return np.floor(np.exp(rs.uniform(np.log(lo), np.log(hi + 1), n))).astype(np.int64).clip(lo, hi)


def _lengths(case):
    """(context length with the new tokens, new tokens) of each request of an attention case."""
    rs = _numbers(case)
    n = case["n_seqs"]
    length = _log_uniform(rs, case["len_lo"], case["len_hi"], n)
    new = _log_uniform(rs, case["new_lo"], case["new_hi"], n)
    if case["new_hi"] >= 16 and case["new_lo"] == 1 and n > 2:
        new[rs.uniform(size=n) < 0.7] = 1            # most requests decode, some bring a prompt
    length[0], new[0] = case["len_hi"], case["new_hi"]
    new = np.minimum(new, length)
    if case["idle"]:
        length[case["idle"] - 1::case["idle"]] = 0   # padded slots: a row with nothing to attend to
        new[case["idle"] - 1::case["idle"]] = 1
    return length, new


def _pairs(length, new):
    """Visible (token, position) pairs of each request: token i sees length - new + i + 1 positions."""
    first = np.maximum(length - new + 1, 0)
    return np.where(length > 0, (first + length) * new // 2, 0)


def _requests(case):
    """(length so far, tokens that arrive; -1: the request has finished) of each request of a plan case."""
    rs = _numbers(case)
    n = case["n_seqs"]
    old = _log_uniform(rs, 1, case["old"], n)
    new = rs.randint(case["new_lo"], case["new_hi"] + 1, n).astype(np.int64)
    if case["release"]:
        new[case["release"] - 1::case["release"]] = -1
    return old, new


def work(case):
    if case["kind"] == "plan":
        old, new = _requests(case)
        page = case["page"]
        add, gone = np.maximum(new, 0), new < 0
        have = -(-old // page)
        pages = int((-(-(old + add) // page) - have)[~gone].sum())
        back = int(have[gone].sum())
        # lengths in and out, offsets, position and slot of each token, pages taken and returned
        return {"bytes": 16 * case["n_seqs"] + 4 + 12 * int(add.sum()) + 8 * pages + 4 * back + 8, "flops": 0}
    if case["kind"] == "append":
        row = case["kv_heads"] * case["head_dim"]
        size = DTYPES[case["dtype"]].itemsize
        t = case["tokens"]
        # rows in, codes and scales out, the rows as the cache holds them out, slots in
        return {"bytes": t * (2 * row * size + 8 * row + 8) + (t - case["padded"]) * 2 * row * 9 // 16,
                "flops": 4 * t * row}
    length, new = _lengths(case)
    size = DTYPES[case["dtype"]].itemsize
    rows = int(new.sum()) * case["heads"]
    cache = int(length.sum()) * case["kv_heads"] * case["head_dim"] * 9 // 8
    table = 4 * int((-(-length // case["page"])).sum())
    return {"bytes": cache + rows * (2 * size * case["head_dim"] + 4) + table + 8 * case["n_seqs"],
            "flops": 4 * case["head_dim"] * case["heads"] * int(_pairs(length, new).sum())}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# --------------------------------------------------------------------------- inputs

def _quantise(x, g):
    """x [..., kv_heads, head_dim] in fp32 -> (codes, scales): per 16 elements the E4M3 scale nearest
    to max|x| / (6 g), then the E2M1 code nearest to x / (scale g), ties to the even code."""
    b = x.unflatten(-1, (-1, 16))
    g = g[:, None]
    s = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0)
    s = torch.where(g > 0, s, torch.zeros_like(s)).to(torch.float8_e4m3fn)
    d = (s.float() * g)[..., None]
    v = torch.where(d > 0, b / d, torch.zeros_like(b))
    a = v.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (m + 8 * torch.signbit(v)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], s.view(torch.uint8)


def _values(codes, scales, g):
    """The values that codes [..., kv_heads, head_dim/2] and scales stand for, fp32."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = table[c.int()].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]
    return v.flatten(-2) * g[:, None]


def _fill(codes, scales, g, gen, spread):
    """Quantised rows of every page, a few pages at a time: normal values, some channels wider."""
    pages, kv_heads, page, half = codes.shape
    step = max(1, (1 << 25) // (kv_heads * page * half * 2))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, page, kv_heads, 2 * half, device="cuda", generator=gen) * spread
        c, s = _quantise(x, g)
        codes[p:p + n] = c.transpose(1, 2)
        scales[p:p + n] = s.transpose(1, 2)


def _cache(pages, kv_heads, page, head_dim):
    c = torch.zeros(pages, kv_heads, page, head_dim // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(pages, kv_heads, page, head_dim // 16, dtype=torch.uint8, device="cuda")
    return c, s


class _Handle:
    """The framework's cache handle, freed with the state that keeps it."""

    def __init__(self, heads, kv_heads, head_dim, page, pages, seqs, tokens, width):
        import quantized_mixture_experts_f32_gb300 as q
        self.q = q
        self.h = q.qmoe_kv4_create(q.make_kv4_config(
            heads, kv_heads, head_dim, page, pages, seqs, tokens, width,
            torch.cuda.current_stream().cuda_stream))

    def __del__(self):
        if getattr(self, "h", None):
            self.q.qmoe_kv4_destroy(self.h)
            self.h = None


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"kind": case["kind"], "dtype": case.get("dtype", "").upper()}
    if case["kind"] == "plan":
        return _prepare_plan(case, gen, s)
    kv_heads, head_dim, page = case["kv_heads"], case["head_dim"], case["page"]
    dtype = DTYPES[case["dtype"]]
    g = torch.rand(2, kv_heads, device="cuda", generator=gen) * 0.5 + 0.75
    s["k_global"], s["v_global"] = (g[0] * 7.0 / 2688.0), (g[1] * 5.0 / 2688.0)
    spread = torch.exp(0.4 * torch.randn(head_dim, device="cuda", generator=gen))
    if case["kind"] == "append":
        t = case["tokens"]
        pages = -(-t // page) + 3
        slots = torch.randperm(pages * page, device="cuda", generator=gen)[:t]
        slots[t - case["padded"]:] = -1
        s["slots"], s["pages"], s["page"] = slots, pages, page
        rows = torch.randn(t, 3, kv_heads * head_dim, device="cuda", generator=gen)
        rows[:, 1] = (rows[:, 1].unflatten(-1, (kv_heads, head_dim)) * spread).flatten(1)
        rows = rows.to(dtype)
        if not case["fused"]:
            rows = rows.transpose(0, 1).contiguous().transpose(0, 1)
        s["k"], s["v"] = rows[:, 1], rows[:, 2]
        # one page more than the cache has: the plain form's place for rows that go nowhere
        for n in ("k", "v"):
            s[n + "_codes"], s[n + "_scales"] = _cache(pages + 1, kv_heads, page, head_dim)
        if own:
            s["handle"] = _Handle(kv_heads, kv_heads, head_dim, page, pages, 1, t, pages)
        return s
    length, new = _lengths(case)
    need = -(-length // page)
    width, pages = int(need.max()) + 1, int(need.sum()) + 5
    perm = torch.randperm(pages, device="cuda", generator=gen).int()
    col = torch.arange(width, device="cuda")
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(need)[:-1]])).cuda()
    at = first[:, None] + col
    live = col < torch.from_numpy(need).cuda()[:, None]
    s["table"] = torch.where(live, perm[at.clamp(max=pages - 1)], torch.full_like(at, -1, dtype=torch.int32))
    s["length"] = torch.from_numpy(length).int().cuda()
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).int().cuda()
    for n, sp in (("k", spread), ("v", torch.ones_like(spread))):
        s[n + "_codes"], s[n + "_scales"] = _cache(pages, kv_heads, page, head_dim)
        _fill(s[n + "_codes"], s[n + "_scales"], s[n + "_global"], gen, sp)
    t = int(new.sum())
    heads = case["heads"]
    row = heads * head_dim
    q = torch.randn(t, row + (2 * kv_heads * head_dim if case["fused"] else 0), device="cuda", generator=gen)
    s["q"] = q.to(dtype)[:, :row]
    s["heads"], s["kv_heads"], s["head_dim"], s["page"] = heads, kv_heads, head_dim, page
    s["tokens"], s["max_new"], s["max_len"] = t, int(new.max()), max(1, int(length.max()))
    if own:
        s["handle"] = _Handle(heads, kv_heads, head_dim, page, pages, case["n_seqs"], t, width)
    return s


def _prepare_plan(case, gen, s):
    old, new = _requests(case)
    page, width, n = case["page"], case["width"], case["n_seqs"]
    have = -(-old // page)
    pages = int(have.sum()) + int((-(-(old + np.maximum(new, 0)) // page) - have).sum()) + 11
    perm = torch.randperm(pages, device="cuda", generator=gen).int()
    col = torch.arange(width, device="cuda")
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(have)[:-1]])).cuda()
    live = col < torch.from_numpy(have).cuda()[:, None]
    at = (first[:, None] + col).clamp(max=pages - 1)
    s["table"] = torch.where(live, perm[at], torch.full_like(at, -1, dtype=torch.int32))
    used = int(have.sum())
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    s["free"][:pages - used] = perm[used:]
    s["n_free"] = torch.tensor([pages - used], dtype=torch.int32, device="cuda")
    s["old"] = torch.from_numpy(old).int().cuda()
    s["new"] = torch.from_numpy(new).int().cuda()
    s["cap"] = int(np.maximum(new, 0).sum()) + 5
    s["page"], s["pages"] = page, pages
    if own:
        s["handle"] = _Handle(1, 1, 64, page, pages, n, s["cap"], width)
    return s


# --------------------------------------------------------------------------- one pass

def run(state):
    return {"plan": _run_plan, "append": _run_append, "attn": _run_attn}[state["kind"]](state)


def _run_plan(s):
    n, cap = s["old"].numel(), s["cap"]
    if own:
        q = s["handle"].q
        i32 = dict(dtype=torch.int32, device="cuda")
        length, n_free = torch.empty(n, **i32), torch.empty(1, **i32)
        cu, pos = torch.empty(n + 1, **i32), torch.empty(cap, **i32)
        slots = torch.empty(cap, dtype=torch.int64, device="cuda")
        q.qmoe_kv4_plan(s["handle"].h, n, s["old"], s["new"], s["table"], s["free"], s["n_free"], cap,
                        length, n_free, cu, pos, slots)
        return dict(length=length, n_free=n_free, cu=cu, pos=pos, slots=slots, table=s["table"], free=s["free"])
    page, pages = s["page"], s["pages"]
    old, new = s["old"].long(), s["new"].long()
    gone, add = new < 0, new.clamp(min=0)
    have = (old + page - 1) // page
    need = torch.where(gone, 0, (old + add + page - 1) // page - have)
    cu = torch.nn.functional.pad(add.cumsum(0), (1, 0))
    first = need.cumsum(0) - need
    # the pages that finished requests return, in the order of requests and columns
    col = torch.arange(s["table"].shape[1], device="cuda")
    back = gone[:, None] & (col < have[:, None])
    order = torch.where(back, back.flatten().cumsum(0).view_as(back) - 1, pages)
    stack = torch.zeros(pages + 1, dtype=torch.int32, device="cuda").scatter_(0, order.flatten(), s["table"].flatten())
    n_back, n_need, n_free = back.sum(), need.sum(), s["n_free"][0].long()
    # pages are taken from the top: the returned ones first (the last returned before the others)
    k = first[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    page_id = torch.where(k < n_back, stack[(n_back - 1 - k).clamp(0, pages)],
                          s["free"][(n_free - 1 - (k - n_back)).clamp(0, pages - 1)])
    table = torch.where(fresh, page_id, s["table"])
    i = torch.arange(pages, device="cuda") - n_free
    free = torch.where((i >= 0) & (i < n_back - n_need), stack[i.clamp(0, pages)], s["free"])
    t = torch.arange(cap, device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True).clamp(max=n - 1)
    live = t < cu[n]
    pos = torch.where(live, old[seq] + t - cu[seq], -1)
    where = torch.where(live, table[seq, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page, -1)
    s["table"].copy_(table)
    s["free"].copy_(free)
    return dict(length=torch.where(gone, 0, old + add).int(), n_free=(n_free + n_back - n_need).int().reshape(1),
                cu=cu.int(), pos=pos.int(), slots=where, table=s["table"], free=s["free"])


def _run_append(s):
    k, v, pages, page = s["k"], s["v"], s["pages"], s["page"]
    t, kv_heads, head_dim = k.shape[0], s["k_global"].numel(), 2 * s["k_codes"].shape[-1]
    out = {n: s[n][:pages] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    if own:
        q = s["handle"].q
        hat = torch.empty(2, t, kv_heads, head_dim, dtype=torch.float32, device="cuda")
        cache = q.make_kv4_cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["k_global"], s["v_global"])
        q.qmoe_kv4_append(s["handle"].h, cache, k, v, q.DTYPE[s["dtype"]], t, k.stride(0), v.stride(0), s["slots"],
                          hat[0], hat[1])
        return dict(out, k_hat=hat[0], v_hat=hat[1])
    to = torch.where(s["slots"] >= 0, s["slots"], pages * page)
    p, off = to // page, to % page
    ck, sk = _quantise(k.float().unflatten(1, (kv_heads, head_dim)), s["k_global"])
    cv, sv = _quantise(v.float().unflatten(1, (kv_heads, head_dim)), s["v_global"])
    s["k_codes"][p, :, off], s["k_scales"][p, :, off] = ck, sk
    s["v_codes"][p, :, off], s["v_scales"][p, :, off] = cv, sv
    return dict(out, k_hat=_values(ck, sk, s["k_global"]), v_hat=_values(cv, sv, s["v_global"]))


def _run_attn(s):
    heads, kv_heads, head_dim, t = s["heads"], s["kv_heads"], s["head_dim"], s["tokens"]
    n, q = s["length"].numel(), s["q"]
    if own:
        m = s["handle"].q
        out = torch.empty(t, heads * head_dim, dtype=q.dtype, device="cuda")
        lse = torch.empty(t, heads, dtype=torch.float32, device="cuda")
        cache = m.make_kv4_cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["k_global"], s["v_global"])
        m.qmoe_kv4_attention(s["handle"].h, cache, q, m.DTYPE[s["dtype"]], q.stride(0), n, t, s["max_new"], s["cu"],
                             s["length"], s["table"], head_dim ** -0.5, out, m.DTYPE[s["dtype"]], out.stride(0), lse)
        return dict(out=out, lse=lse)
    page, group, length = s["page"], heads // kv_heads, s["length"].long()
    at = torch.arange(s["max_len"], device="cuda")
    seen = at < length[:, None]
    p = torch.where(seen, s["table"][:, at // page].long(), 0)
    k = _values(s["k_codes"][p, :, at % page], s["k_scales"][p, :, at % page], s["k_global"])
    v = _values(s["v_codes"][p, :, at % page], s["v_scales"][p, :, at % page], s["v_global"])
    # the new tokens as a padded batch: token i of request b is row cu[b] + i
    cu = s["cu"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(s["max_new"], device="cuda")
    row = (cu[:-1, None] + i).clamp(max=t - 1)
    x = q.float().unflatten(1, (kv_heads, group, head_dim))[row]             # [n, new, kv, group, dim]
    x = x.permute(0, 2, 3, 1, 4).flatten(2, 3)                               # [n, kv, group * new, dim]
    z = torch.matmul(x, k.permute(0, 2, 3, 1)) * head_dim ** -0.5
    z = z.unflatten(2, (group, s["max_new"]))
    mask = at <= (length - new)[:, None, None] + i[:, None]                  # [n, new, len]
    z = z.masked_fill(~(mask & seen[:, None])[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z = torch.exp(z - top)
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.flatten(2, 3), v.transpose(1, 2)).unflatten(2, (group, s["max_new"]))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + torch.log(total))[..., 0]
    b = torch.searchsorted(cu[1:], torch.arange(t, device="cuda"), right=True)
    r = torch.arange(t, device="cuda") - cu[b]
    return dict(out=o[b, :, :, r].reshape(t, heads * head_dim).to(q.dtype), lse=lse[b, :, :, r].reshape(t, heads))


# --------------------------------------------------------------------------- 64 bits

def _float32(x):
    """x rounded to 24 bits: for a quotient of 32-bit numbers the same as the 32-bit division."""
    return x.float().double()


def _e2m1_64(code):
    """An E2M1 code's value by its fields: sign, two exponent bits, one bit of fraction."""
    e, f = (code >> 1) & 3, (code & 1).double()
    size = torch.where(e > 0, (1.0 + 0.5 * f) * torch.pow(2.0, (e - 1).double()), 0.5 * f)
    return torch.where(code >= 8, -size, size)


def _e4m3_64(code):
    e, f = (code >> 3) & 15, (code & 7).double()
    return torch.where(e > 0, (1.0 + f / 8) * torch.pow(2.0, (e - 7).double()), f / 512)


def _nearest(v, grid):
    """The index of the grid value nearest to each v >= 0, ties to the even index."""
    hi = torch.searchsorted(grid, v).clamp(1, grid.numel() - 1)
    lo = hi - 1
    a, b = v - grid[lo], grid[hi] - v
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _quantise_64(x, g):
    """(codes, scales, values) of x [t, kv_heads, head_dim]: the quotients are defined in 32 bits."""
    b = x.double().unflatten(-1, (-1, 16))
    g = g.double()[:, None]
    scales = _e4m3_64(torch.arange(127, device=x.device))
    at = _nearest(_float32(b.abs().amax(-1) / _float32(6.0 * g)).clamp(max=448.0), scales)
    d = _float32(scales[at] * g)[..., None]
    v = _float32(torch.where(d > 0, b / d.clamp(min=1e-300), torch.zeros_like(b)))
    c = _nearest(v.abs().clamp(max=6.0), torch.tensor(E2M1, dtype=torch.float64, device=x.device))
    c = c + 8 * torch.signbit(v)
    value = _e2m1_64(c) * scales[at][..., None] * g[..., None]
    c = c.flatten(-2)
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8), at.to(torch.uint8), value.flatten(-2)


def exact(case, seed):
    if case["kind"] == "plan":
        return None
    s = prepare(case, seed)
    if case["kind"] == "append":
        got, page = {}, s["page"]
        for n in ("k", "v"):
            kv_heads = s[n + "_global"].numel()
            c, sc, got[n + "_hat"] = _quantise_64(s[n].unflatten(1, (kv_heads, -1)), s[n + "_global"])
            put = s["slots"] >= 0
            p, off = s["slots"][put] // page, s["slots"][put] % page
            s[n + "_codes"][p, :, off], s[n + "_scales"][p, :, off] = c[put], sc[put]
            got[n + "_codes"], got[n + "_scales"] = s[n + "_codes"][:s["pages"]], s[n + "_scales"][:s["pages"]]
        return got
    heads, kv_heads, head_dim, page = s["heads"], s["kv_heads"], s["head_dim"], s["page"]
    group, t = heads // kv_heads, s["tokens"]
    length, new = _lengths(case)
    if float((length * new).sum()) * heads * head_dim > 2e12:
        return None
    out = torch.zeros(t, kv_heads, group, head_dim, dtype=torch.float64, device="cuda")
    lse = torch.full((t, kv_heads, group), -math.inf, dtype=torch.float64, device="cuda")
    q = s["q"].double().unflatten(1, (kv_heads, group, head_dim))
    first = 0
    for b in range(len(length)):
        n_pos, n_new = int(length[b]), int(new[b])
        if n_pos:
            pages = s["table"][b, :-(-n_pos // page)].long()
            for h in range(kv_heads):
                kv = []
                for n in ("k", "v"):
                    c = s[n + "_codes"][pages, h].flatten(0, 1)[:n_pos].long()
                    sc = s[n + "_scales"][pages, h].flatten(0, 1)[:n_pos].long()
                    c = _e2m1_64(torch.stack((c & 15, c >> 4), -1).flatten(-2)).unflatten(-1, (-1, 16))
                    kv.append((c * _e4m3_64(sc)[..., None]).flatten(-2) * s[n + "_global"][h].double())
                for i in range(0, n_new, 128):
                    m = min(128, n_new - i)
                    z = torch.einsum("igd,pd->igp", q[first + i:first + i + m, h], kv[0]) / math.sqrt(head_dim)
                    last = torch.arange(i, i + m, device="cuda") + (n_pos - n_new)
                    z = torch.where(torch.arange(n_pos, device="cuda") <= last[:, None, None], z, -math.inf)
                    lse[first + i:first + i + m, h] = torch.logsumexp(z, -1)
                    out[first + i:first + i + m, h] = torch.softmax(z, -1) @ kv[1]
        first += n_new
    return dict(out=out.flatten(1), lse=lse.flatten(1))
