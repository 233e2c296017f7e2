"""The operators of a decoder layer's 8-bit path around the paged 4-bit cache, as they are measured.

norm    h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, as 16- or 32-bit values or in 8 bits:
        E4M3 codes with one fp32 scale per 128 elements of a row (max / 448)
quant   rows into the same 8-bit form without the norm (the attention's output on its way to the O product)
linear  act(x W^T + bias) + residual, x in that form, W in E4M3 with one scale per 128 x 128 block
rope    rotary positions on rows of heads: halves or interleaved pairs, part of the head, scaled frequencies,
        each head normalised first on demand
append  the K and V rows of new tokens into the paged 4-bit cache, K normalised and rotated on the way, and
        the q rows beside them

A case is plain values; inputs come from the seed.  An operator on 8- or 4-bit data decides its codes in
fp32, each step rounded once; the plain forms and `exact` follow the same steps.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# --------------------------------------------------------------------------- cases

def _norm(name, rows, dim, dtype, residual, out):
    return dict(name=name, kind="norm", rows=rows, dim=dim, dtype=dtype, residual=residual, out=out)


def _quant(name, rows, dim, dtype, fused):
    return dict(name=name, kind="quant", rows=rows, dim=dim, dtype=dtype, fused=fused)


def _linear(name, tokens, k, n, out, bias, act, residual):
    return dict(name=name, kind="linear", tokens=tokens, k=k, n=n, out=out, bias=bias, act=act, residual=residual)


def _rope(name, tokens, heads, head_dim, rot, layout, scaling, n_pos, dtype, norm, fused):
    return dict(name=name, kind="rope", tokens=tokens, heads=heads, head_dim=head_dim, rot=rot, layout=layout,
                scaling=scaling, n_pos=n_pos, dtype=dtype, norm=norm, fused=fused)


def _append(name, tokens, heads, kv_heads, head_dim, rot, layout, scaling, n_pos, dtype, norm, page, padded):
    return dict(name=name, kind="append", tokens=tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim, rot=rot,
                layout=layout, scaling=scaling, n_pos=n_pos, dtype=dtype, norm=norm, page=page, padded=padded)


def listed():
    return [
        # one token between two layers of a decode step: the residual's addition, the norm, 8 bits; latency alone
        _norm("norm_1x2048_e4m3", 1, 2048, "f32", "f32", "e4m3"),
        # a long prompt's rows: a bf16 product added to the fp32 residual, normalised into 8 bits
        _norm("norm_16384x2048_e4m3", 16384, 2048, "bf16", "f32", "e4m3"),
        # the attention's output of one decode step of a batch
        _quant("quant_64x4096_bf16", 64, 4096, "bf16", False),
        # an odd number of fp32 rows, read in place from wider ones
        _quant("quant_5003x4096_f32", 5003, 4096, "f32", True),
        # the Q/K/V product of one token: the weights' bytes alone
        _linear("linear_1x2048x5120_bf16", 1, 2048, 5120, "bf16", False, "none", ""),
        # the O product of a decode step, added to the fp32 residual
        _linear("linear_64x4096x2048_f32", 64, 4096, 2048, "f32", False, "none", "f32"),
        # odd sizes with bias and activation: a ragged batch through a small head, the last block of k and of n cut
        _linear("linear_777x2000x1003_f16", 777, 2000, 1003, "f16", True, "gelu", ""),
        # the Q/K/V product of a long prompt, bound by the matrix products
        _linear("linear_16384x2048x5120_bf16", 16384, 2048, 5120, "bf16", True, "none", ""),
        # q of a decode step, each head normalised, halves, whole heads
        _rope("rope_64x32_bf16", 64, 32, 128, 128, "half", "none", 40960, "bf16", True, False),
        # a long prompt at far positions: interleaved pairs, half of each head, scaled by parts, in place in wider rows
        _rope("rope_8191x40_f16", 8191, 40, 128, 64, "interleaved", "parts", 131072, "f16", False, True),
        # a decode step's rows from one Q/K/V product, some of the batch padding
        _append("append_rope_64_bf16", 64, 32, 4, 128, 128, "half", "none", 40960, "bf16", True, 16, 5),
        # a long prompt's rows
        _append("append_rope_16384_bf16", 16384, 32, 4, 128, 128, "half", "none", 40960, "bf16", True, 64, 0),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


HEADS = ((32, 4), (28, 4), (40, 8), (64, 4), (10, 10), (8, 1), (6, 2))


def draw(rng):
    while True:
        c = _drawn(rng)
        if _cost(c) <= max(_cost(x) for x in listed() if x["kind"] == c["kind"]):
            return {k: v for k, v in c.items() if k != "name"}


def _drawn(rng):
    kind = rng.choice(["norm", "quant", "linear", "linear", "rope", "append"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind == "norm":
        out = rng.choice(["e4m3", "e4m3", "f32", "f16", "bf16"])
        return _norm("", _log(rng, 1, 16384), _log(rng, 64, 16384, 16), dtype, rng.choice(["", "f32", "bf16"]), out)
    if kind == "quant":
        return _quant("", _log(rng, 1, 16384), _log(rng, 64, 16384, 16), dtype, rng.random() < 0.5)
    if kind == "linear":
        return _linear("", _log(rng, 1, 16384), _log(rng, 64, 16384, 16), _log(rng, 1, 16384), dtype, rng.random() < 0.5,
                       rng.choice(["none", "relu", "silu", "gelu"]), rng.choice(["", dtype]))
    head_dim = rng.choice([64, 128, 256])
    rot = rng.choice([32, head_dim // 2, head_dim])
    more = dict(rot=rot, layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "parts"]),
                n_pos=_log(rng, 1000, 131072), dtype=dtype, norm=rng.random() < 0.5)
    heads, kv_heads = rng.choice(HEADS)
    tokens = _log(rng, 1, 16384)
    if kind == "rope":
        return _rope("", tokens, heads, head_dim, fused=rng.random() < 0.5, **more)
    return _append("", tokens, heads, kv_heads, head_dim, page=rng.choice([16, 32, 64, 128]),
                   padded=rng.choice([0, min(3, tokens - 1)]), **more)


def _size(dtype):
    return 1 if dtype == "e4m3" else DTYPES[dtype].itemsize


def work(case):
    kind = case["kind"]
    if kind in ("norm", "quant"):
        n = case["rows"] * case["dim"]
        out = case.get("out", "e4m3")
        b = n * (_size(case["dtype"]) + _size(out))
        b += 4 * case["rows"] * -(-case["dim"] // 128) if out == "e4m3" else 0
        if case.get("residual"):
            b += 2 * n * _size(case["residual"])         # the residual in, the sum out
        b += 4 * case["dim"] if kind == "norm" else 0
        return {"bytes": b, "flops": 6 * n}
    t = case["tokens"]
    if kind == "linear":
        k, n = case["k"], case["n"]
        blocks = -(-k // 128)
        b = t * k + n * k + 4 * blocks * (t + -(-n // 128)) + t * n * _size(case["out"])
        b += t * n * _size(case["residual"]) if case["residual"] else 0
        b += 4 * n if case["bias"] else 0
        return {"bytes": b, "flops": 2 * t * n * k}
    size = _size(case["dtype"])
    q = t * case["heads"] * case["head_dim"]
    b = 2 * q * size + t * (4 + 4 * case["rot"])         # q in and out, positions, the table's rows
    if kind == "rope":
        return {"bytes": b, "flops": 6 * q}
    row = case["kv_heads"] * case["head_dim"]
    # K and V in, their values out, codes and scales out, slots
    b += t * (2 * row * size + 8 * row + 8) + (t - case["padded"]) * 2 * row * 9 // 16
    return {"bytes": b, "flops": 6 * q + 14 * t * row}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# --------------------------------------------------------------------------- inputs

class _Handle:
    """The framework's context, and its cache handle where one is wanted, freed with the state that keeps them."""

    def __init__(self, cache=None):
        import quantized_mixture_experts_f32_gb300 as q
        self.q, self.kv = q, None
        stream = torch.cuda.current_stream().cuda_stream
        self.ctx = q.qmoe_create(q.make_config(256, 1, 1, 256, 1, stream=stream))
        if cache:
            self.kv = q.qmoe_kv4_create(q.make_kv4_config(*cache, stream=stream))

    def __del__(self):
        if getattr(self, "kv", None):
            self.q.qmoe_kv4_destroy(self.kv)
        if getattr(self, "ctx", None):
            self.q.qmoe_destroy(self.ctx)
        self.kv = self.ctx = None


def _rows(gen, rows, width, of, dtype, at=0):
    """`width` columns of rows `of` columns wide: normal values, some channels much larger, as hidden states are."""
    x = torch.randn(rows, of, device="cuda", generator=gen)
    x *= torch.exp(0.7 * torch.randn(of, device="cuda", generator=gen))
    return x.to(dtype)[:, at:at + width]


def _inv_freq(case, device="cuda"):
    """The angle a position turns each pair by, in 64 bits, and the factor of cosines and sines."""
    rot, base = case["rot"], 1e6
    j = torch.arange(rot // 2, dtype=torch.float64, device=device)
    f = base ** (-2.0 * j / rot)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "parts":
        lo, hi = (rot * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        ramp = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / 4.0 * ramp, 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def _table(case):
    """(cosine, sine) of each position and pair, fp32 from 64 bits."""
    f, m = _inv_freq(case)
    angle = torch.arange(case["n_pos"], dtype=torch.float64, device="cuda")[:, None] * f
    return torch.stack((torch.cos(angle) * m, torch.sin(angle) * m), -1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    s = dict(case)
    if kind in ("norm", "quant"):
        rows, dim = case["rows"], case["dim"]
        x = _rows(gen, rows, dim, dim + (256 if case.get("fused") else 0), DTYPES[case["dtype"]])
        s["x"], blocks = x, -(-dim // 128)
        if kind == "norm":
            s["weight"] = 1 + 0.2 * torch.randn(dim, device="cuda", generator=gen)
            if case["residual"]:
                s["res"] = _rows(gen, rows, dim, dim, DTYPES[case["residual"]]) * 3
                s["sum"] = torch.empty_like(s["res"])
        out = case.get("out", "e4m3")
        s["y"] = torch.empty(rows, dim, dtype=E4M3 if out == "e4m3" else DTYPES[out], device="cuda")
        s["scale"] = torch.empty(rows, blocks, device="cuda")
    elif kind == "linear":
        t, k, n = case["tokens"], case["k"], case["n"]
        kb, nb = -(-k // 128), -(-n // 128)
        # activations as the norm leaves them; weights uniform in sign, their sizes spread as trained ones are
        x = _rows(gen, t, k, k, torch.float32)
        pad = torch.nn.functional.pad(x, (0, kb * 128 - k)).unflatten(1, (kb, 128))
        s["xs"] = pad.abs().amax(-1) / 448
        s["xc"] = (pad / s["xs"][..., None]).clamp(-448, 448).flatten(1)[:, :k].to(E4M3).contiguous()
        w = torch.randn(n, k, device="cuda", generator=gen) * 60
        s["wc"] = w.clamp(-448, 448).to(E4M3)
        s["ws"] = (torch.rand(nb, kb, device="cuda", generator=gen) + 0.5) / (60 * math.sqrt(k))
        s["bias_row"] = torch.randn(n, device="cuda", generator=gen) if case["bias"] else None
        # rows of 16 bytes' multiples, as a user lays them out
        wide = -(-n // 16) * 16
        s["res"] = torch.randn(t, wide, device="cuda", generator=gen).to(DTYPES[case["out"]])[:, :n] if case["residual"] else None
        s["y"] = torch.empty(t, wide, dtype=DTYPES[case["out"]], device="cuda")[:, :n]
    else:
        t, heads, hd = case["tokens"], case["heads"], case["head_dim"]
        kv = case.get("kv_heads", 0)
        of = (heads + 2 * kv) * hd if kind == "append" else heads * hd + (4 * hd if case["fused"] else 0)
        rows = _rows(gen, t, of, of, DTYPES[case["dtype"]])
        s["pos"] = torch.randint(0, case["n_pos"], (t,), device="cuda", generator=gen, dtype=torch.int32)
        s["q"] = rows[:, :heads * hd]
        s["q_norm"], s["k_norm"] = (1 + 0.2 * torch.randn(hd, device="cuda", generator=gen) if case["norm"] else None for _ in "qk")
        s["q_out"] = torch.zeros(t, heads * hd, dtype=DTYPES[case["dtype"]], device="cuda")
        if kind == "append":
            page, row = case["page"], kv * hd
            pages = -(-t // page) + 3
            slots = torch.randperm(pages * page, device="cuda", generator=gen)[:t]
            if case["padded"]:
                slots[t - case["padded"]:] = -1
                s["pos"][t - case["padded"]:] = -1
            s["slots"], s["pages"] = slots, pages
            s["k"], s["v"] = rows[:, heads * hd:heads * hd + row], rows[:, heads * hd + row:]
            g = torch.rand(2, kv, device="cuda", generator=gen) * 0.5 + 0.75
            s["k_global"], s["v_global"] = g[0] * 9.0 / 2688.0, g[1] * 12.0 / 2688.0
            # one page more than the cache has: the plain form's place for rows that go nowhere
            for n in ("k", "v"):
                s[n + "_codes"] = torch.zeros(pages + 1, kv, page, hd // 2, dtype=torch.uint8, device="cuda")
                s[n + "_scales"] = torch.zeros(pages + 1, kv, page, hd // 16, dtype=torch.uint8, device="cuda")
            s["hat"] = torch.zeros(2, t, kv, hd, device="cuda")
    if own:
        h = s["handle"] = _Handle((case["heads"], case["kv_heads"], case["head_dim"], case["page"], s["pages"], 1,
                                   case["tokens"], s["pages"]) if kind == "append" else None)
        if kind in ("rope", "append"):
            s["table"] = torch.empty(case["n_pos"], case["rot"] // 2, 2, device="cuda")
            f = dict(none={}, linear=dict(scaling=h.q.QMOE_ROPE_LINEAR, factor=4.0),
                     parts=dict(scaling=h.q.QMOE_ROPE_PARTS, factor=4.0, orig_ctx=32768, beta_fast=32.0, beta_slow=1.0))
            s["rope"] = h.q.make_rope(case["rot"], 1e6, case["n_pos"], s["table"],
                                      layout=h.q.ROPE_LAYOUT[case["layout"]], **f[case["scaling"]])
            h.q.qmoe_rope_table(h.ctx, s["rope"])
        if kind == "append":
            s["cache"] = h.q.make_kv4_cache(*(s[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_global", "v_global")))
    elif kind in ("rope", "append"):
        s["table"] = _table(case)
    return s


# --------------------------------------------------------------------------- one pass

def run(state):
    f = {"norm": (_plain_norm, _own_norm), "quant": (_plain_quant, _own_quant), "linear": (_plain_linear, _own_linear),
         "rope": (_plain_rope, _own_rope), "append": (_plain_append, _own_append)}[state["kind"]]
    return f[bool(own)](state)


def _own_norm(s):
    h = s["handle"]
    q, x, res, y = h.q, s["x"], s.get("res"), s["y"]
    fp8 = y.dtype == E4M3
    q.qmoe_rmsnorm(h.ctx, x, q.DTYPE[s["dtype"].upper()], x.stride(0), res, q.DTYPE[(s["residual"] or "f32").upper()], 0,
                   s.get("sum"), s["weight"], EPS, x.shape[0], x.shape[1], y, q.DTYPE[s["out"].upper()], 0,
                   s["scale"] if fp8 else None)
    return dict(y=y, **({"scale": s["scale"]} if fp8 else {}), **({"sum": s["sum"]} if res is not None else {}))


def _own_quant(s):
    h, x = s["handle"], s["x"]
    h.q.qmoe_fp8_quantize(h.ctx, x, h.q.DTYPE[s["dtype"].upper()], x.stride(0), x.shape[0], x.shape[1], s["y"], s["scale"])
    return dict(y=s["y"], scale=s["scale"])


def _own_linear(s):
    h, y, res = s["handle"], s["y"], s["res"]
    q = h.q
    q.qmoe_linear_fp8(h.ctx, s["xc"], s["xs"], s["tokens"], s["k"], s["wc"], s["ws"], s["n"], s["bias_row"],
                      q.ACT[s["act"].upper()], res, 0 if res is None else res.stride(0), y, q.DTYPE[s["out"].upper()], y.stride(0))
    return y


def _own_rope(s):
    h, x, y = s["handle"], s["q"], s["q_out"]
    h.q.qmoe_rope(h.ctx, s["rope"], x, h.q.DTYPE[s["dtype"].upper()], x.stride(0), s["tokens"], s["heads"], s["head_dim"],
                  s["pos"], s["q_norm"], EPS, y, y.stride(0))
    return y


def _own_append(s):
    h, x, k, v, y = s["handle"], s["q"], s["k"], s["v"], s["q_out"]
    h.q.qmoe_kv4_append_rope(h.kv, s["cache"], s["rope"], x, k, v, h.q.DTYPE[s["dtype"].upper()], s["tokens"], x.stride(0),
                             k.stride(0), v.stride(0), s["pos"], s["slots"], s["q_norm"], s["k_norm"], EPS, y, y.stride(0),
                             s["hat"][0], s["hat"][1])
    return _appended(s, y, s["hat"][0], s["hat"][1])


def _appended(s, q, k_hat, v_hat):
    got = {n: s[n][:s["pages"]] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    return dict(got, q=q, k_hat=k_hat, v_hat=v_hat)


def _to_e4m3(y):
    """Codes and scales of y [rows, dim], fp32."""
    rows, dim = y.shape
    blocks = -(-dim // 128)
    b = torch.nn.functional.pad(y, (0, blocks * 128 - dim)).unflatten(1, (blocks, 128))
    scale = b.abs().amax(-1) / 448
    c = torch.where(scale[..., None] > 0, b / scale[..., None], torch.zeros_like(b)).clamp(-448, 448)
    return c.flatten(1)[:, :dim].to(E4M3), scale


def _plain_norm(s):
    h = s["x"].float()
    out = {}
    if s["residual"]:
        h = h + s["res"].float()
        out["sum"] = h.to(s["res"].dtype)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    if s["out"] == "e4m3":
        out["y"], out["scale"] = _to_e4m3(y)
    else:
        out["y"] = y.to(DTYPES[s["out"]])
    return out


def _plain_quant(s):
    y, scale = _to_e4m3(s["x"].float())
    return dict(y=y, scale=scale)


def _activate(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2.0)))
    return z


def _plain_linear(s):
    k, n = s["k"], s["n"]
    x = s["xc"].float() * s["xs"].repeat_interleave(128, 1)[:, :k]
    w = s["wc"].float() * s["ws"].repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
    z = torch.matmul(x, w.t())
    if s["bias_row"] is not None:
        z = z + s["bias_row"]
    z = _activate(z, s["act"])
    if s["res"] is not None:
        z = z + s["res"].float()
    return z.to(DTYPES[s["out"]])


def _heads(x, hd, norm):
    """Rows as [tokens, heads, hd] in fp32, each head normalised on demand (its mean square in 64 bits)."""
    x = x.float().unflatten(1, (-1, hd))
    if norm is None:
        return x
    r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + EPS).float()
    return x * r * norm


def _rotate(x, table, pos, rot, layout):
    cs = table[pos.long().clamp(min=0)][:, None]                             # [tokens, 1, rot / 2, 2]
    c, n = cs[..., 0], cs[..., 1]
    part = x[..., :rot]
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * c - b * n, b * c + a * n), -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rope(s):
    x = _heads(s["q"], s["head_dim"], s["q_norm"])
    return _rotate(x, s["table"], s["pos"], s["rot"], s["layout"]).flatten(1).to(s["q"].dtype)


def _quantise4(x, g):
    """x [tokens, kv_heads, head_dim] in fp32 -> (codes, scales, values): per 16 elements the E4M3 scale nearest to
    max|x| / (6 g), then the E2M1 code nearest to x / (scale g), ties to the even code."""
    b = x.unflatten(-1, (-1, 16))
    g = g[:, None]
    scale = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(E4M3)
    d = (scale.float() * g)[..., None]
    v = torch.where(d > 0, b / d, torch.zeros_like(b))
    a = v.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = m + 8 * torch.signbit(v)
    grid = torch.tensor(E2M1 + tuple(-e for e in E2M1), device=x.device)
    value = (grid[code.int()] * scale.float()[..., None]).flatten(-2) * g
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], scale.view(torch.uint8), value


def _plain_append(s):
    hd, page = s["head_dim"], s["page"]
    live = (s["pos"] >= 0)[:, None, None]
    q = _rotate(_heads(s["q"], hd, s["q_norm"]), s["table"], s["pos"], s["rot"], s["layout"])
    k = _rotate(_heads(s["k"], hd, s["k_norm"]), s["table"], s["pos"], s["rot"], s["layout"])
    v = _heads(s["v"], hd, None)
    to = torch.where(s["slots"] >= 0, s["slots"], s["pages"] * page)
    p, off = to // page, to % page
    hat = []
    for n, x in (("k", k), ("v", v)):
        c, sc, value = _quantise4(x, s[n + "_global"])
        s[n + "_codes"][p, :, off], s[n + "_scales"][p, :, off] = c, sc
        hat.append(torch.where(live, value, 0.0))
    return _appended(s, torch.where(live, q, 0.0).flatten(1).to(s["q"].dtype), *hat)


# --------------------------------------------------------------------------- 64 bits

def _r32(x):
    """x rounded to 24 bits."""
    return x.float().double()


def _code_e4m3(v):
    """The E4M3 value nearest to each v, ties to the even code: a step is 2^(e-3), 2^-9 below 2^-6."""
    a = v.abs().clamp(max=448.0)
    step = torch.pow(2.0, torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(max=8) - 3)
    step = torch.where(a < 2.0 ** -6, torch.full_like(a, 2.0 ** -9), step)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def _exact_e4m3(y):
    rows, dim = y.shape
    c, scale = torch.empty_like(y), torch.empty(rows, -(-dim // 128), dtype=torch.float64, device=y.device)
    for b in range(scale.shape[1]):
        part = y[:, 128 * b:128 * b + 128]
        scale[:, b] = part.abs().amax(1) / 448
        d = scale[:, b:b + 1]
        c[:, 128 * b:128 * b + 128] = torch.where(d > 0, _code_e4m3(part / d.clamp(min=1e-300)), torch.zeros_like(part))
    return c, scale


def _exact_heads(s, x, norm):
    """The heads' rows after norm and rotation; the steps before a 4-bit decision round to fp32 as they are defined to."""
    hd, rot = s["head_dim"], s["rot"]
    x = x.double().unflatten(1, (-1, hd))
    if norm is not None:
        r = _r32(1 / torch.sqrt((x * x).sum(-1, keepdim=True) / hd + EPS))
        x = _r32(_r32(x * r) * norm.double())
    f, m = _inv_freq(s)
    angle = s["pos"].double().clamp(min=0)[:, None] * f
    c, n = _r32(torch.cos(angle) * m)[:, None], _r32(torch.sin(angle) * m)[:, None]
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if s["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., first].clone(), x[..., second].clone()
    x[..., first] = _r32(_r32(a * c) - _r32(b * n))
    x[..., second] = _r32(_r32(b * c) + _r32(a * n))
    return x


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quant":
        y, scale = _exact_e4m3(s["x"].double())
        return dict(y=y, scale=scale)
    if kind == "norm":
        h, got = s["x"].double(), {}
        if case["residual"]:
            h = got["sum"] = h + s["res"].double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + EPS) * s["weight"].double()
        if case["out"] == "e4m3":
            got["y"], got["scale"] = _exact_e4m3(y)
        else:
            got["y"] = y
        return got
    if kind == "linear":
        k, n = case["k"], case["n"]
        z = torch.zeros(case["tokens"], n, dtype=torch.float64, device="cuda")
        for b in range(-(-k // 128)):
            at = slice(128 * b, min(k, 128 * b + 128))
            w = s["wc"][:, at].double() * s["ws"][:, b].double().repeat_interleave(128)[:n, None]
            z += (s["xc"][:, at].double() * s["xs"][:, b:b + 1].double()) @ w.t()
        if s["bias_row"] is not None:
            z += s["bias_row"].double()
        z = {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z * torch.sigmoid(z),
             "gelu": lambda: z * 0.5 * torch.erfc(-z / math.sqrt(2.0))}[case["act"]]()
        return z if s["res"] is None else z + s["res"].double()
    q = _exact_heads(s, s["q"], s["q_norm"])
    if kind == "rope":
        return q.flatten(1)
    live = (s["pos"] >= 0).double()[:, None, None]
    got = dict(q=(q * live).flatten(1), k_codes=None, k_scales=None, v_codes=None, v_scales=None)
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for n, x in (("k", _exact_heads(s, s["k"], s["k_norm"])), ("v", s["v"].double().unflatten(1, (-1, case["head_dim"])))):
        g = s[n + "_global"].double()[:, None]
        b = x.unflatten(-1, (-1, 16))
        scale = _code_e4m3(_r32(b.abs().amax(-1) / _r32(6 * g)))
        d = _r32(scale * g)[..., None]
        v = _r32(torch.where(d > 0, b / d.clamp(min=1e-300), torch.zeros_like(b)))
        a = v.abs().clamp(max=6.0)
        hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
        low, up = a - grid[hi - 1], grid[hi] - a
        at = torch.where((low < up) | ((low == up) & (hi % 2 == 1)), hi - 1, hi)
        value = torch.copysign(grid[at], v) * scale[..., None] * g[..., None]
        got[n + "_hat"] = value.flatten(-2) * live
    return got
