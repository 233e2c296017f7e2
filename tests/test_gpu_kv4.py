"""The paged 4-bit KV cache on the GPU, through the C ABI, against the numpy forms of
tests/kv4_ref.py: the plan (whole numbers, equal), the append (codes, scales and values bit
for bit) and the attention (within the bound that attention_bound derives)."""
import numpy as np
import pytest

from tests import kv4_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TORCH = {"F32": torch.float32, "F16": torch.float16, "BF16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import quantized_mixture_experts_f32_gb300 as q
    return q


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Kv:
    """A handle with one layer's cache, codes and scales filled with bytes that must not matter."""

    def __init__(self, q, nq=8, nkv=2, hd=128, page=16, n_pages=40, seqs=8, tokens=256, width=12, stream=0,
                 seed=0):
        self.q, self.nq, self.nkv, self.hd, self.page, self.n_pages, self.width = q, nq, nkv, hd, page, n_pages, width
        self.tokens, self.stream = tokens, stream
        self.h = q.qmoe_kv4_create(q.make_kv4_config(nq, nkv, hd, page, n_pages, seqs, tokens, width, stream))
        self.t = {}
        for n in ("k", "v"):
            self.t[n + "_codes"] = torch.full((n_pages, nkv, page, hd // 2), 0x5A, dtype=torch.uint8, device="cuda")
            self.t[n + "_scales"] = torch.full((n_pages, nkv, page, hd // 16), 0x7F, dtype=torch.uint8, device="cuda")
        rng = np.random.default_rng(seed)
        self.g = rng.uniform(0.8, 1.3, (2, nkv)).astype(np.float32) * np.float32(5 / 2688)
        self.kg, self.vg = cuda(self.g[0]), cuda(self.g[1])
        self.cache = q.make_kv4_cache(self.t["k_codes"], self.t["k_scales"], self.t["v_codes"], self.t["v_scales"],
                                      self.kg, self.vg)

    def close(self):
        self.q.qmoe_kv4_destroy(self.h)

    def ready(self):
        """What the current stream made is there for a handle on another one."""
        if self.stream:
            torch.cuda.current_stream().synchronize()

    def status(self):
        return self.q.qmoe_kv4_get_status(self.h)

    def plan(self, seq_len, new_len, table, free, n_free, cap, inplace=False):
        d = dict(len=cuda(seq_len), new=cuda(new_len), table=cuda(table), free=cuda(free),
                 n=cuda(np.array([n_free], np.int32)))
        n = len(seq_len)
        i32 = dict(dtype=torch.int32, device="cuda")
        out_len = d["len"] if inplace else torch.full((n,), -7, **i32)
        out_n = d["n"] if inplace else torch.full((1,), -7, **i32)
        cu, pos = torch.full((n + 1,), -7, **i32), torch.full((cap,), -7, **i32)
        slots = torch.full((cap,), -7, dtype=torch.int64, device="cuda")
        self.q.qmoe_kv4_plan(self.h, n, d["len"], d["new"], d["table"], d["free"], d["n"], cap, out_len, out_n,
                             cu, pos, slots)
        st = self.status()
        nf = int(out_n[0])
        return st, dict(seq_len=out_len.cpu().numpy(), n_free=nf, cu=cu.cpu().numpy(), pos=pos.cpu().numpy(),
                        slots=slots.cpu().numpy(), table=d["table"].cpu().numpy(),
                        stack=d["free"].cpu().numpy()[:max(nf, 0)])

    def append(self, k, v, slots, dtype="F32", k_hat=None, v_hat=None, n=None, ks=0, vs=0):
        self.q.qmoe_kv4_append(self.h, self.cache, k, v, self.q.DTYPE[dtype], n or k.shape[0], ks, vs, slots, k_hat,
                               v_hat)

    def attention(self, x, cu, seq_len, table, dtype, out_t=None, scale=None, lse=True, max_new=None, qs=0, os=0,
                  out=None):
        t = x.shape[0]
        out_t = out_t or dtype
        if out is None:
            out = torch.full((t, self.nq * self.hd), 77.0, dtype=TORCH[out_t], device="cuda")
        ls = torch.full((t, self.nq), 77.0, dtype=torch.float32, device="cuda") if lse else None
        scale = self.hd ** -0.5 if scale is None else scale
        dev = [cuda(np.asarray(v, np.int32)) for v in (cu, seq_len, table)]
        self.ready()
        self.q.qmoe_kv4_attention(self.h, self.cache, x, self.q.DTYPE[dtype], qs, len(seq_len), t,
                                  max_new or max(1, int(np.diff(cu).max())), *dev, scale, out, self.q.DTYPE[out_t], os,
                                  ls)
        return out, ls

    def values(self):
        """The cache as it stands, in 64 bits: k, v [pages, nkv, page, hd]."""
        got = []
        for n, g in (("k", self.g[0]), ("v", self.g[1])):
            c = R.unpack(self.t[n + "_codes"].cpu().numpy()).transpose(0, 2, 1, 3)
            s = self.t[n + "_scales"].cpu().numpy().transpose(0, 2, 1, 3)
            got.append(R.values_of(c, s, g).transpose(0, 2, 1, 3))
        return got


# --------------------------------------------------------------------------- plan

def _tables(rng, seq_len, width, page, n_pages):
    need = -(-seq_len // page)
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(seq_len), width), -1, np.int32)
    at = 0
    for s, c in enumerate(need):
        table[s, :c] = perm[at:at + c]
        at += c
    free = np.full(n_pages, -9, np.int32)
    free[:n_pages - at] = perm[at:]
    return table, free, n_pages - at


def _same_plan(got, want, table_before):
    for n in ("seq_len", "cu", "pos", "slots", "table", "stack"):
        assert np.array_equal(got[n], want[n]), n
    assert got["n_free"] == want["n_free"]


@pytest.mark.parametrize("n,page,old,new,inplace", [
    (1, 16, 0, 1, False), (1, 16, 16, 1, True), (1, 256, 255, 2, False), (3, 32, 40, 0, False),
    (7, 16, 100, 33, True), (33, 64, 300, 5, False), (511, 16, 50, 3, True), (513, 32, 70, 9, False),
    (4096, 16, 40, 5, True), (4095, 128, 300, 2, False)])
def test_plan_against_the_plain_form(q, n, page, old, new, inplace):
    rng = np.random.default_rng(n + page)
    width = -(-(old + new) // page) + 2
    seq_len = rng.integers(0, old + 1, n).astype(np.int32)
    new_len = rng.integers(0, new + 1, n).astype(np.int32)
    new_len[rng.uniform(size=n) < 0.2] = -1
    if n == 1:
        seq_len[:], new_len[:] = old, new
    n_pages = int((-(-(seq_len + np.maximum(new_len, 0)) // page)).sum()) + 3
    table, free, n_free = _tables(rng, seq_len, width, page, n_pages)
    cap = int(np.maximum(new_len, 0).sum()) + 4
    kv = Kv(q, 1, 1, 64, page, n_pages, n, cap, width)
    try:
        want = R.plan(seq_len, new_len, table, free, n_free, page, n_pages, cap)
        for _ in range(2):
            st, got = kv.plan(seq_len, new_len, table, free, n_free, cap, inplace)
            assert st == 0
            _same_plan(got, want, table)
    finally:
        kv.close()


@pytest.mark.parametrize("what,status", [
    ("negative length", 8), ("length past the row", 8), ("n_free negative", 8), ("n_free too large", 8),
    ("too many returned", 8), ("row too short", 4), ("too many tokens", 4), ("huge counts", 4), ("no pages", 5)])
def test_plan_refuses_a_step_as_a_whole(q, what, status):
    page, width, n_pages, cap = 16, 4, 12, 40
    seq_len = np.array([17, 3, 30], np.int32)
    new_len = np.array([2, -1, 5], np.int32)
    rng = np.random.default_rng(3)
    table, free, n_free = _tables(rng, seq_len, width, page, n_pages)
    if what == "negative length":
        seq_len[1] = -1
    elif what == "length past the row":
        seq_len[1] = 65
    elif what == "n_free negative":
        n_free = -1
    elif what == "n_free too large":
        n_free = 13
    elif what == "too many returned":
        n_free = 12
        new_len[0] = 0
        new_len[2] = 0
    elif what == "row too short":
        new_len[2] = 35
    elif what == "too many tokens":
        new_len[:] = [21, 0, 20]
    elif what == "huge counts":
        new_len[:] = [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    elif what == "no pages":
        n_free = 1
        new_len[:] = [31, 0, 5]
    assert R.plan(seq_len, new_len, table, free, n_free, page, n_pages, cap) == status
    kv = Kv(q, 1, 1, 64, page, n_pages, 3, cap, width)
    try:
        st, got = kv.plan(seq_len, new_len, table, free, n_free, cap)
        assert st == status
        assert np.array_equal(got["seq_len"], seq_len) and got["n_free"] == n_free
        assert not got["cu"].any() and (got["pos"] == -1).all() and (got["slots"] == -1).all()
        assert np.array_equal(got["table"], table)
        assert kv.status() == 0                                   # read once, cleared
        seq_ok = np.array([17, 3, 30], np.int32)                  # the handle serves the next step
        table, free, n_free = _tables(np.random.default_rng(3), seq_ok, width, page, n_pages)
        one = np.ones(3, np.int32)
        st, got = kv.plan(seq_ok, one, table, free, n_free, cap)
        assert st == 0
        _same_plan(got, R.plan(seq_ok, one, table, free, n_free, page, n_pages, cap), table)
    finally:
        kv.close()


@pytest.mark.parametrize("n", [1024, 1025, 2047, 2048])
def test_plan_of_a_thousand_requests_and_more(q, n):
    """As many requests as a thread scans two and four of."""
    rng = np.random.default_rng(n)
    page, width = 32, 5
    seq_len = rng.integers(0, 71, n).astype(np.int32)
    new_len = rng.integers(-1, 40, n).astype(np.int32)
    n_pages = int((-(-(seq_len + np.maximum(new_len, 0)) // page)).sum()) + 3
    table, free, n_free = _tables(rng, seq_len, width, page, n_pages)
    cap = int(np.maximum(new_len, 0).sum()) + 4
    kv = Kv(q, 1, 1, 64, page, n_pages, n, cap, width)
    try:
        st, got = kv.plan(seq_len, new_len, table, free, n_free, cap)
        assert st == 0
        _same_plan(got, R.plan(seq_len, new_len, table, free, n_free, page, n_pages, cap), table)
    finally:
        kv.close()


@pytest.mark.parametrize("n", [3, 700])
@pytest.mark.parametrize("where", ["free", "returned", "returned and taken", "cached"])
@pytest.mark.parametrize("bad", [-1, "n_pages", -2 ** 31, 2 ** 31 - 1])
def test_plan_reports_pages_out_of_range(q, bad, where, n):
    """In the free stack, among a finished request's pages, or where a request's next token goes: the id is
    handed on as it is, its tokens have no slot, and the status word says so; all else as ever."""
    rng = np.random.default_rng(n)
    page, width, cap = 16, 4, 40 + 8 * n
    seq_len = rng.integers(1, 32, n).astype(np.int32)
    new_len = rng.integers(0, 9, n).astype(np.int32)
    seq_len[:3], new_len[:3] = [20, 33, 16], [3, -1, 17 if where == "returned and taken" else 1]
    if where == "returned":
        new_len[0], new_len[2:] = 0, 0
    elif where == "free":
        new_len[1] = 1
    n_pages = 3 * n + 9
    table, free, n_free = _tables(rng, seq_len, width, page, n_pages)
    bad = n_pages if bad == "n_pages" else bad
    if where == "free":
        free[:n_free] = bad
    elif where == "cached":
        table[0, 1] = bad
    else:
        table[1, 2 if where == "returned and taken" else 0] = bad
    want = R.plan(seq_len, new_len, table, free, n_free, page, n_pages, cap)
    out = (want["slots"] // page < 0) | (want["slots"] // page >= n_pages)
    assert where == "returned" or (out & (want["pos"] >= 0)).any()
    want["slots"][out] = -1
    kv = Kv(q, 1, 1, 64, page, n_pages, n, cap, width)
    try:
        st, got = kv.plan(seq_len, new_len, table, free, n_free, cap)
        assert st == 8
        _same_plan(got, want, table)
        assert kv.status() == 0
        table[0, 3] = table[1, 3] = bad                            # columns that nothing looks up
        table[0, 1], table[1, :3], free[:n_free] = 0, [1, 2, 3], np.arange(n_free)
        st, got = kv.plan(seq_len, new_len, table, free, n_free, cap)
        assert st == 0
    finally:
        kv.close()


# --------------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", ["F32", "F16", "BF16"])
@pytest.mark.parametrize("t,nkv,hd,page,fused,hat", [
    (1, 1, 64, 16, False, True), (5, 2, 128, 32, True, False), (37, 3, 256, 16, False, True),
    (130, 4, 128, 64, True, True), (9, 10, 64, 256, False, False)])
def test_append_bit_for_bit(q, dtype, t, nkv, hd, page, fused, hat):
    rng = np.random.default_rng(t + hd)
    n_pages = -(-t // page) + 2
    kv = Kv(q, nkv, nkv, hd, page, n_pages, 1, t, n_pages, seed=t)
    try:
        rows = rng.normal(size=(3, t, nkv * hd)) * np.exp(rng.normal(size=(3, t, 1)) * 2)
        rows[1, 0, :16] = 0.0                                     # an all-zero block
        rows[2, 0, :16] = -0.0
        rows[1, -1, :16] = 1e-30                                  # far below the smallest scale
        rows[2, -1, 3] = 3e4                                      # far above the largest
        x = torch.from_numpy(rows).cuda().to(TORCH[dtype])
        if fused:
            x = x.transpose(0, 1).contiguous().transpose(0, 1)
        stride = x.stride(1)
        slots = rng.permutation(n_pages * page)[:t].astype(np.int64)
        if t > 3:
            slots[[1, t - 1]] = [-1, -5]
        kh = torch.full((t, nkv * hd), 5.0, device="cuda") if hat else None
        vh = torch.full((t, nkv * hd), 5.0, device="cuda") if hat else None
        before = {n: a.cpu().numpy().copy() for n, a in kv.t.items()}
        kv.append(x[1], x[2], cuda(slots), dtype, kh, vh, t, stride if fused else 0, stride if fused else 0)
        assert kv.status() == 0
        put = slots >= 0
        p, o = slots[put] // page, slots[put] % page
        for n, i, g, h in (("k", 1, kv.g[0], kh), ("v", 2, kv.g[1], vh)):
            c, s, val = R.quantise(x[i].float().cpu().numpy().reshape(t, nkv, hd), g)
            wc, ws = before[n + "_codes"].copy(), before[n + "_scales"].copy()
            wc[p, :, o], ws[p, :, o] = c[put], s[put]
            assert np.array_equal(kv.t[n + "_codes"].cpu().numpy(), wc)
            assert np.array_equal(kv.t[n + "_scales"].cpu().numpy(), ws)
            if hat:   # code * scale is exact, the global scale multiplies with one rounding
                assert np.array_equal(h.cpu().numpy(), val.reshape(t, -1).astype(np.float32))
    finally:
        kv.close()


def test_append_zero_global_and_slots_past_the_cache(q):
    kv = Kv(q, 2, 2, 64, 16, 3, 1, 8, 3)
    try:
        kv.kg[1] = 0.0
        kv.g[0][1] = 0.0
        x = torch.randn(4, 128, device="cuda")
        before = kv.t["v_codes"].cpu().numpy().copy()
        kv.append(x, x, cuda(np.array([0, 17, 48, 2 ** 40], np.int64)))
        assert kv.status() == 8
        c, s, _ = R.quantise(x.cpu().numpy().reshape(4, 2, 64), kv.g[0])
        got = kv.t["k_codes"].cpu().numpy()
        assert np.array_equal(got[0, :, 0], c[0]) and np.array_equal(got[1, :, 1], c[1])
        assert not got[0, 1, 0].any() and not kv.t["k_scales"].cpu().numpy()[0, 1, 0].any()
        after = kv.t["v_codes"].cpu().numpy()
        same = np.ones((3, 16), bool)
        same[0, 0] = same[1, 1] = False
        assert np.array_equal(after.transpose(0, 2, 1, 3)[same], before.transpose(0, 2, 1, 3)[same])
    finally:
        kv.close()


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -60, 2.0 ** -100, 2.0 ** 60, 2.0 ** 100])
def test_append_at_and_beside_every_border(q, scale):
    """Quotients on a border between two codes, one step of x above and below it, and random ones, for
    small, ordinary and large global scales."""
    rng = np.random.default_rng(4)
    t, nkv, hd, page = 256, 2, 128, 64
    kv = Kv(q, nkv, nkv, hd, page, 5, 1, t, 5)
    try:
        f = np.float32
        kv.g = (rng.uniform(0.7, 1.4, (2, nkv)) * scale).astype(f)
        kv.kg.copy_(cuda(kv.g[0]))
        kv.vg.copy_(cuda(kv.g[1]))
        borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], f)
        rows = []
        for g in kv.g:
            sv = R.e4m3_values()[rng.integers(1, 127, (t, nkv, hd // 16))].astype(f)
            d = (sv * g[:, None]).astype(f)[..., None]
            x = (borders[rng.integers(0, 7, (t, nkv, hd // 16, 16))] * d).astype(f)
            x = np.where(rng.uniform(size=x.shape) < 0.33, np.nextafter(x, f(0)),
                         np.where(rng.uniform(size=x.shape) < 0.5, np.nextafter(x, f(np.inf)), x)).astype(f)
            x[..., 8:12] = (rng.uniform(0, 6, x[..., 8:12].shape) * d).astype(f)
            x[..., 15] = (f(6) * d[..., 0]).astype(f)              # the largest: the block's scale is sv
            x *= rng.choice([-1, 1], x.shape).astype(f)
            rows.append(x.reshape(t, nkv, hd))
        x = [cuda(r.reshape(t, -1)) for r in rows]
        hat = torch.empty(2, t, nkv * hd, device="cuda")
        kv.append(x[0], x[1], cuda(np.arange(t)), "F32", hat[0], hat[1])
        assert kv.status() == 0
        p, o = np.arange(t) // page, np.arange(t) % page
        for i, n in enumerate("kv"):
            c, s, val = R.quantise(rows[i], kv.g[i])
            assert np.array_equal(kv.t[n + "_codes"].cpu().numpy()[p, :, o], c)
            assert np.array_equal(kv.t[n + "_scales"].cpu().numpy()[p, :, o], s)
            assert np.array_equal(hat[i].cpu().numpy(), val.reshape(t, -1).astype(f))
    finally:
        kv.close()


def test_append_of_what_is_not_finite_keeps_scales_finite(q):
    kv = Kv(q, 1, 1, 64, 16, 1, 1, 8, 1)
    try:
        x = torch.randn(4, 64, device="cuda")
        x[0, 3], x[1, 20], x[2, :] = float("nan"), float("inf"), float("nan")
        kv.append(x, x, cuda(np.arange(4)))
        assert kv.status() == 0
        assert ((kv.t["k_scales"].cpu().numpy()[0, 0, :4] & 0x7F) != 0x7F).all()
        c, s, _ = R.quantise(x[3:].cpu().numpy().reshape(1, 1, 64), kv.g[0])
        assert np.array_equal(kv.t["k_codes"].cpu().numpy()[0, 0, 3], c[0, 0])
    finally:
        kv.close()


@pytest.mark.parametrize("dtype", ["F32", "BF16"])
@pytest.mark.parametrize("nkv,hd", [(10, 256), (33, 64), (17, 128)])
def test_append_of_rows_a_cta_takes_in_turns(q, nkv, hd, dtype):
    """More than 2048 elements a row, the last turn of a row partly filled."""
    rng = np.random.default_rng(hd)
    t, page, n_pages = 7, 16, 2
    kv = Kv(q, nkv, nkv, hd, page, n_pages, 1, t, n_pages, seed=3)
    try:
        x = torch.from_numpy(rng.normal(size=(2, t, nkv * hd))).cuda().to(TORCH[dtype])
        slots = rng.permutation(n_pages * page)[:t].astype(np.int64)
        hat = torch.full((2, t + 1, nkv * hd), 5.0, device="cuda")
        kv.append(x[0], x[1], cuda(slots), dtype, hat[0], hat[1])
        assert kv.status() == 0
        p, o = slots // page, slots % page
        for i, n in enumerate("kv"):
            c, sc, val = R.quantise(x[i].float().cpu().numpy().reshape(t, nkv, hd), kv.g[i])
            wc, ws = np.full((n_pages, nkv, page, hd // 2), 0x5A, np.uint8), np.full((n_pages, nkv, page, hd // 16), 0x7F, np.uint8)
            wc[p, :, o], ws[p, :, o] = c, sc
            assert np.array_equal(kv.t[n + "_codes"].cpu().numpy(), wc)
            assert np.array_equal(kv.t[n + "_scales"].cpu().numpy(), ws)
            assert np.array_equal(hat[i, :t].cpu().numpy(), val.reshape(t, -1).astype(np.float32)) and (hat[i, t] == 5.0).all()
    finally:
        kv.close()


def test_append_of_infinity_under_a_large_global_keeps_scales_finite(q):
    """6 * global past fp32's range: infinity over infinity is no scale."""
    kv = Kv(q, 1, 1, 64, 16, 1, 1, 8, 1)
    try:
        kv.kg.fill_(1e38)
        kv.vg.fill_(3e38)
        x = torch.randn(3, 64, device="cuda")
        x[0, 3], x[1, 20] = float("inf"), float("-inf")
        x[1, 40] = float("nan")
        kv.append(x, x, cuda(np.arange(3)))
        assert kv.status() == 0
        for n in ("k_scales", "v_scales"):
            assert ((kv.t[n].cpu().numpy()[0, 0, :3] & 0x7F) != 0x7F).all()
    finally:
        kv.close()


# --------------------------------------------------------------------------- attention

def _filled(q, lens, news, nq, nkv, hd, page, dtype, seed, width=None, extra=3, stream=0):
    """A cache whose visible positions are appended rows and whose other slots are bytes that decode
    to NaN, with the requests' tables; returns kv, q rows, cu, table."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    width = width or max(1, int((-(-lens // page)).max()) + 1)
    n_pages = int((-(-lens // page)).sum()) + extra
    t = int(np.sum(news))
    kv = Kv(q, nq, nkv, hd, page, n_pages, len(lens), max(t, int(lens.sum()), 1), width, stream, seed)
    table, _, _ = _tables(rng, lens, width, page, n_pages)
    slots = np.array([int(table[s, p // page]) * page + p % page for s in range(len(lens)) for p in range(lens[s])],
                     np.int64)
    if len(slots):
        rows = torch.from_numpy(rng.normal(size=(2, len(slots), nkv * hd)).astype(np.float32)).cuda()
        rows[0] *= torch.from_numpy(np.exp(0.4 * rng.normal(size=nkv * hd)).astype(np.float32)).cuda()
        slots = cuda(slots)
        kv.ready()
        kv.append(rows[0], rows[1], slots)
        assert kv.status() == 0
    x = torch.from_numpy(rng.normal(size=(t, nq * hd)).astype(np.float32) * 1.5).cuda().to(TORCH[dtype])
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return kv, x, cu, table


def _check(kv, x, out, lse, cu, lens, table, scale=None, out_t=None):
    t = int(cu[-1])
    scale = kv.hd ** -0.5 if scale is None else scale
    xq = x[:t].double().cpu().numpy().reshape(t, kv.nq, kv.hd)
    want, wl, vmax, zabs, seen = R.attention(xq, kv.values(), cu, lens, table, scale, kv.page)
    half = torch.finfo(out.dtype).eps / 2
    ob, lb = R.attention_bound(want, vmax, zabs, seen, kv.hd, x.dtype != torch.float32, half)
    got = out[:t].double().cpu().numpy().reshape(t, kv.nq, kv.hd)
    assert np.isfinite(got).all()
    over = np.abs(got - want) / ob
    assert over.max() <= 1, f"{over.max():.3g} times the bound at {np.unravel_index(over.argmax(), over.shape)}"
    if lse is not None:
        gl = lse[:t].double().cpu().numpy()
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(gl), empty)
        assert (np.abs(gl[~empty] - wl[~empty]) <= lb[~empty]).all()


LAYOUTS = [(8, 2, 128, 16), (4, 4, 64, 32), (14, 2, 64, 16), (32, 1, 128, 64), (6, 2, 256, 16), (10, 10, 128, 128),
           (20, 1, 256, 256), (9, 3, 64, 64)]


@pytest.mark.parametrize("dtype", ["F32", "F16", "BF16"])
@pytest.mark.parametrize("nq,nkv,hd,page", LAYOUTS)
def test_decode_rows(q, nq, nkv, hd, page, dtype):
    lens = [1, 2, 15, 16, 17, 0, 130, 257, 333]
    news = [1] * len(lens)
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, hd, page, dtype, nq + hd)
    try:
        out, lse = kv.attention(x, cu, lens, table, dtype)
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table)
        again, lse2 = kv.attention(x, cu, lens, table, dtype)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    finally:
        kv.close()


@pytest.mark.parametrize("dtype", ["F32", "F16", "BF16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("nq,nkv,new", [(32, 2, [1]), (26, 2, [1]), (8, 2, [3, 1, 4]), (32, 2, [1, 0, 40])])
def test_many_sequences_of_more_than_eight_rows(q, nq, nkv, new, hd, dtype):
    """Items of 16 rows, some short of them, alone and beside prompts."""
    lens = ([1, 33, 0, 700, 16, 257, 5, 1500, 64, 90] * 3)[:24]
    news = [min(x, max(n, 1)) for x, n in zip(new * 24, lens)]
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, hd, 32, dtype, hd + nq)
    try:
        out, lse = kv.attention(x, cu, lens, table, dtype)
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table)
    finally:
        kv.close()


@pytest.mark.parametrize("dtype", ["F32", "F16", "BF16"])
@pytest.mark.parametrize("nq,nkv,hd,page", LAYOUTS)
def test_several_new_tokens(q, nq, nkv, hd, page, dtype):
    lens = [5, 70, 0, 33, 129, 40, 3]
    news = [5, 3, 2, 0, 9, 40, 7]          # a prompt from its start, draft tokens, rows before the first position
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, hd, page, dtype, nq * hd)
    try:
        out, lse = kv.attention(x, cu, lens, table, dtype)
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table)
    finally:
        kv.close()


@pytest.mark.parametrize("dtype", ["F32", "BF16", "F16"])
@pytest.mark.parametrize("nq,nkv,hd,page,lens,news", [
    (8, 1, 128, 32, [300, 140, 1, 77], [300, 100, 1, 13]),
    (8, 2, 64, 16, [513], [257]), (2, 2, 256, 64, [200, 450], [130, 1]), (12, 4, 128, 16, [260, 31], [129, 31])])
def test_prompt_chunks(q, nq, nkv, hd, page, lens, news, dtype):
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, hd, page, dtype, hd + len(lens))
    try:
        out, lse = kv.attention(x, cu, lens, table, dtype)
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table)
        again, lse2 = kv.attention(x, cu, lens, table, dtype)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    finally:
        kv.close()


@pytest.mark.parametrize("nq,nkv,hd", [(8, 1, 128), (4, 2, 64)])
def test_a_long_context_split_over_the_gpu(q, nq, nkv, hd):
    lens, news = [20011, 3, 9000], [1, 1, 2]
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, hd, 64, "F32", 11)
    try:
        out, lse = kv.attention(x, cu, lens, table, "F32")
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table)
    finally:
        kv.close()


@pytest.mark.parametrize("q_t,out_t", [("F32", "F16"), ("F32", "BF16"), ("BF16", "F32"), ("F16", "F32")])
@pytest.mark.parametrize("news", [[1, 1, 1], [40, 3, 30]])
def test_strides_and_types_apart(q, q_t, out_t, news):
    lens, nq, nkv, hd = [45, 100, 61], 4, 2, 128
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, hd, 16, q_t, 5)
    try:
        t, row = x.shape
        wide = torch.full((t + 2, row + 24), float("nan"), dtype=x.dtype, device="cuda")
        wide[:t, 16:16 + row] = x
        out = torch.full((t + 2, row + 8), 9.0, dtype=TORCH[out_t], device="cuda")
        view = wide[:t, 16:16 + row]
        kv.attention(view, cu, lens, table, q_t, out_t, qs=row + 24, os=row + 8, out=out, lse=False)
        assert kv.status() == 0
        _check(kv, x, out[:t, :row], None, cu, lens, table)
        assert (out[t:] == 9.0).all() and (out[:, row:] == 9.0).all()
    finally:
        kv.close()


@pytest.mark.parametrize("news", [[1, 1], [20, 30]])
def test_rows_behind_the_last_sequence_stay(q, news):
    lens = [40, 70]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 9)
    try:
        pad = torch.cat([x, torch.full((5, x.shape[1]), float("nan"), device="cuda")])
        out, lse = kv.attention(pad, cu, lens, table, "F32")
        assert kv.status() == 0
        t = x.shape[0]
        _check(kv, x, out[:t], lse[:t], cu, lens, table)
        assert (out[t:] == 77.0).all() and (lse[t:] == 77.0).all()
    finally:
        kv.close()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("news", [[1, 1], [33, 20]])
def test_any_finite_scale(q, scale, news):
    lens = [40, 70]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 2)
    try:
        out, lse = kv.attention(x, cu, lens, table, "F32", scale=scale)
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table, scale=scale)
    finally:
        kv.close()


@pytest.mark.parametrize("dtype", ["F32", "F16", "BF16"])
@pytest.mark.parametrize("scale,sign", [(-0.2, 1), (0.0, 1), (0.125, -1), (-0.125, -1)])
@pytest.mark.parametrize("news", [[1, 1], [33, 20]])
def test_signs_of_scale_and_global(q, scale, sign, news, dtype):
    lens = [40, 70]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, dtype, 2)
    try:
        kv.g[0][1] *= sign                                         # the second kv head's keys
        kv.kg.copy_(cuda(kv.g[0]))
        out, lse = kv.attention(x, cu, lens, table, dtype, scale=scale)
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table, scale=scale)
    finally:
        kv.close()


@pytest.mark.parametrize("dtype", ["F32", "F16", "BF16"])
@pytest.mark.parametrize("kg,mag", [(3e38, 1.0), (1e-42, 1.0), (2.0 ** -100, 2.0 ** -14), (2.0 ** 126, 2.0 ** -14), (2.0 ** -149, 2.0 ** 10)])
@pytest.mark.parametrize("news", [[1, 1], [33, 20]])
def test_scale_and_global_at_opposite_ends(q, news, kg, mag, dtype):
    """Scores of ordinary size from a scale and a global of which either leaves fp32's range together with a
    constant or with the row's size."""
    lens = [40, 70]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, dtype, 2)
    try:
        kv.g[0][:] = kg
        kv.kg.copy_(cuda(kv.g[0]))
        x = x * mag
        scale = float(np.float32(0.125 * (5 / 2688) / np.float64(np.float32(kg)) / mag))
        assert 0 < scale < 3.4e38
        out, lse = kv.attention(x, cu, lens, table, dtype, scale=scale)
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table, scale=scale)
    finally:
        kv.close()


def test_scores_of_zero_under_a_factor_past_the_range(q):
    """q.k is 0 whatever scale * global is."""
    lens = [40, 70]
    for news in ([1, 1], [33, 20]):
        kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 2)
        try:
            kv.kg.fill_(1e30)
            kv.t["k_codes"].zero_()
            kv.t["k_scales"].fill_(0x38)
            out, lse = kv.attention(x, cu, lens, table, "F32", scale=1e30)
            kv.t["k_codes"].fill_(0x11)
            want, wl = kv.attention(x, cu, lens, table, "F32", scale=0.0)
            assert kv.status() == 0 and torch.equal(out, want) and torch.equal(lse, wl)
        finally:
            kv.close()


@pytest.mark.parametrize("dtype", ["F32", "F16", "BF16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("scale", [1e5, -1e8, 1e12, 1e30])
@pytest.mark.parametrize("news", [[1, 1, 1], [33, 20, 3], [3, 150, 1]])
def test_scores_far_past_the_exponential(q, news, scale, hd, dtype):
    """Scores whose rounding alone is more than the exponential's whole range: the largest one takes all."""
    lens = [40, 700, 9]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, hd, 16, dtype, 2)
    try:
        out, lse = kv.attention(x, cu, lens, table, dtype, scale=scale)
        assert kv.status() == 0
        t = x.shape[0]
        xq = x.double().cpu().numpy().reshape(t, 8, hd)
        k, v = kv.values()
        want, wl, vmax, zabs, seen = R.attention(xq, (k, v), cu, lens, table, scale, kv.page)
        got, gl = out.double().cpu().numpy().reshape(t, 8, hd), lse.double().cpu().numpy()
        half = float(torch.finfo(out.dtype).eps) / 2
        # two weights of a mean at least, each within 2^-22 + (seen + 8) roundings, one fp16 term of 16-bit rows' weights
        w = 2.0 ** -22 + (seen[:, None] + 8) * R.EPS32 + (0 if dtype == "F32" else 2.0 ** -11 + seen[:, None] * 2.0 ** -25)
        assert np.isfinite(got).all() and (np.abs(got) <= (vmax * (1 + 2 * w + half))[..., None]).all()
        dz = (hd + 12) * R.EPS32 * zabs + 2.0 ** -22 * zabs
        assert (np.abs(gl - wl) <= dz + 4 * R.EPS32 * zabs + 7).all()   # 7: ln(seen), which a row's rounding may lose
        clear = 0
        for s in range(3):
            L = lens[s]
            cols = table[s, :-(-L // 16)].astype(np.int64)
            for i in range(news[s]):
                r, n = int(cu[s]) + i, L - news[s] + i + 1
                for h in range(8):
                    kk, vv = k[cols, h // 4].reshape(-1, hd)[:n], v[cols, h // 4].reshape(-1, hd)[:n]
                    z = np.sort(scale * (kk @ xq[r, h]))[::-1]
                    if n == 1 or z[0] - z[1] > 2 * dz[r, h] + 40:  # no rounding makes another one the largest
                        clear += 1
                        top = vv[np.argmax(scale * (kk @ xq[r, h]))]
                        assert (np.abs(got[r, h] - top) <= 2 * w[r] * vmax[r, h] + half * np.abs(top)).all(), (r, h)
        assert clear > 0.8 * t * 8
    finally:
        kv.close()


@pytest.mark.parametrize("dtype", ["F32", "BF16"])
def test_scores_far_past_the_exponential_split_over_the_gpu(q, dtype):
    """The same where parts of a context are joined: whichever the parts, one position takes all."""
    for lens, news, nkv in (([9000], [1], 1), ([5000], [40], 1)):
        kv, x, cu, table = _filled(q, lens, news, 8, nkv, 64, 16, dtype, 4)
        try:
            out, lse = kv.attention(x, cu, lens, table, dtype, scale=1e12)
            assert kv.status() == 0 and torch.isfinite(out.float()).all()
            t = x.shape[0]
            xq = x.double().cpu().numpy().reshape(t, 8, 64)
            want, wl, vmax, zabs, seen = R.attention(xq, kv.values(), cu, lens, table, 1e12, 16)
            got = out.double().cpu().numpy().reshape(t, 8, 64)
            same = (np.abs(got - want) <= 2.0 ** -7 * vmax[..., None]).all(-1)
            assert same.mean() > 0.9                               # but for rows whose two largest are near each other
            assert (np.abs(lse.double().cpu().numpy() - wl) <= (64 + 16) * R.EPS32 * zabs + 2.0 ** -22 * zabs + 10).all()
        finally:
            kv.close()


@pytest.mark.parametrize("dtype", ["F32", "F16", "BF16"])
@pytest.mark.parametrize("vg", [2.0 ** -80, -0.01, 2.0 ** 100])
@pytest.mark.parametrize("lens,news", [([40, 70], [1, 1]), ([40, 70], [33, 20]), ([6000], [24])])
def test_small_large_and_negative_globals_of_v(q, lens, news, vg, dtype):
    nq, nkv = (8, 1) if len(lens) == 1 else (8, 2)
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, 64, 16, dtype, 2)
    try:
        kv.g[1][:] = vg
        kv.vg.copy_(cuda(kv.g[1]))
        out, lse = kv.attention(x, cu, lens, table, dtype, "F32")
        assert kv.status() == 0
        t = x.shape[0]
        xq = x.double().cpu().numpy().reshape(t, nq, 64)
        want, wl, vmax, zabs, seen = R.attention(xq, kv.values(), cu, lens, table, 0.125, 16)
        ob, lb = R.attention_bound(want / vg, vmax / abs(vg), zabs, seen, 64, dtype != "F32", 2.0 ** -24)
        got = out.double().cpu().numpy().reshape(t, nq, 64)
        assert (np.abs(got - want) <= ob * abs(vg)).all()
        assert (np.abs(lse.double().cpu().numpy() - wl) <= lb).all()
    finally:
        kv.close()


@pytest.mark.parametrize("mag", [1e-6, 1e4, 1e18])
@pytest.mark.parametrize("news", [[1, 1], [33, 20]])
def test_rows_of_any_size(q, mag, news):
    lens = [40, 70]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 21)
    try:
        x = x * mag
        out, lse = kv.attention(x, cu, lens, table, "F32", scale=0.125 / mag)
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table, scale=0.125 / mag)
    finally:
        kv.close()


@pytest.mark.parametrize("dtype", ["F32", "F16", "BF16"])
@pytest.mark.parametrize("news", [[1, 1], [33, 20]])
def test_rows_at_the_ends_of_their_type(q, news, dtype):
    """Rows of subnormals and rows with the type's largest values: scaled before they are products' operands.
    (The sums of products stay below fp32's largest number: few elements of the largest rows are not zero.)"""
    lens = [40, 70]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 23)
    try:
        info = torch.finfo(TORCH[dtype])
        x = x.reshape(-1, 8, 64)
        x[:, :4] *= info.smallest_normal / 2                       # heads 0 .. 3: some multiples of the smallest step
        x[:, 4:, 2:] = 0
        x[:, 4:, :2] = x[:, 4:, :2].sign() * info.max
        x = x.reshape(-1, 512).to(TORCH[dtype])
        assert torch.isfinite(x).all() and (x != 0).any(1).all()
        for scale in (2.0 / float(x.abs().max()), min(1.0 / float(info.smallest_normal), 3e38)):
            out, lse = kv.attention(x, cu, lens, table, dtype, scale=scale)
            assert kv.status() == 0
            heads = range(8) if scale < 1 else range(4)            # the largest rows' z overflow with the second
            xq = x.double().cpu().numpy().reshape(-1, 8, 64)
            if scale > 1:
                xq[:, 4:] = 0
            want, wl, vmax, zabs, seen = R.attention(xq, kv.values(), cu, lens, table, scale, kv.page)
            ob, lb = R.attention_bound(want, vmax, zabs, seen, 64, dtype != "F32", info.eps / 2)
            got, gl = out.double().cpu().numpy().reshape(-1, 8, 64), lse.double().cpu().numpy()
            for h in heads:
                assert (np.abs(got[:, h] - want[:, h]) <= ob[:, h] + float(info.smallest_normal)).all(), (h, scale)
                assert (np.abs(gl[:, h] - wl[:, h]) <= lb[:, h]).all(), (h, scale)
    finally:
        kv.close()


@pytest.mark.parametrize("news", [[1, 1, 1], [20, 30, 3]])
def test_one_row_that_is_not_finite_harms_no_other(q, news):
    lens = [40, 70, 9]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 8)
    try:
        x[int(cu[1]), 2 * 64 + 5] = float("nan")                 # one head of one row
        out, _ = kv.attention(x, cu, lens, table, "F32")
        clean = x.clone()
        clean[int(cu[1]), 2 * 64 + 5] = 0.0
        want, _ = kv.attention(clean, cu, lens, table, "F32")
        bad = torch.zeros_like(out, dtype=torch.bool)
        bad[int(cu[1]), 2 * 64:3 * 64] = True
        assert torch.equal(out[~bad], want[~bad]) and torch.isnan(out[bad]).all()
    finally:
        kv.close()


@pytest.mark.parametrize("news", [[1, 1, 1], [20, 30, 3]])
def test_bad_pages_count_as_not_visible(q, news):
    lens = [40, 70, 9]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 8)
    try:
        table[0, 1], table[1, 4], table[2, 0] = -1, 2 ** 30, kv.n_pages
        out, lse = kv.attention(x, cu, lens, table, "F32")
        assert kv.status() == 8
        _check(kv, x, out, lse, cu, lens, table)
        assert kv.status() == 0
    finally:
        kv.close()


@pytest.mark.parametrize("news", [[1, 1, 1], [20, 30, 3]])
def test_sequences_out_of_range_are_skipped(q, news):
    lens = np.array([40, 70, 9], np.int32)
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 8)
    t = x.shape[0]
    try:
        want, wl = kv.attention(x, cu, lens, table, "F32")
        cases = [(cu, np.array([40, -1, 9]), 1), (cu, np.array([40, 2 ** 31 - 1, 9]), 1),
                 (np.array([0, cu[1], cu[2], t + 1]), lens, 2), (np.array([-1, cu[1], cu[2], t]), lens, 0)]
        for c, ln, skipped in cases:
            out, lse = kv.attention(x, c, ln, table, "F32", max_new=max(news))
            assert kv.status() == 8
            for s in range(3):
                rows = slice(int(cu[s]), int(cu[s + 1]))
                if s == skipped:
                    assert (out[rows] == 77.0).all() and (lse[rows] == 77.0).all()
                else:
                    assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], wl[rows])
        if max(news) > 1:                                          # more new tokens than max_new says
            out, lse = kv.attention(x, cu, lens, table, "F32", max_new=max(news) - 1)
            assert kv.status() == 8
            big = int(np.argmax(news))
            assert (out[int(cu[big]):int(cu[big + 1])] == 77.0).all()
    finally:
        kv.close()


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [20, 30, 3, 40]])
def test_descending_offsets_compute_nothing(q, news):
    lens = [40, 70, 9, 50]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 8)
    try:
        for bad in ([0, cu[2], cu[1], cu[3], cu[4]], [cu[4], 0, cu[4], 0, cu[4]], [0, -3, cu[2], cu[3], cu[4]]):
            out, lse = kv.attention(x, np.array(bad, np.int32), lens, table, "F32", max_new=x.shape[0])
            assert kv.status() == 8
            assert (out == 77.0).all() and (lse == 77.0).all()
        out, lse = kv.attention(x, cu, lens, table, "F32")
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table)
    finally:
        kv.close()


@pytest.mark.parametrize("seed", range(4))
def test_device_arrays_of_any_content_are_safe(q, seed):
    """Offsets, lengths, tables and slots of any bits: nothing out of range is followed, rows of the
    sequences that are in order are right, and the handle serves the next call."""
    rng = np.random.default_rng(seed)
    lens, news = [40, 70, 9, 50, 33], [1, 30, 3, 1, 17]
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 8)
    try:
        want, wl = kv.attention(x, cu, lens, table, "F32")
        wild = lambda n: rng.integers(-2 ** 31, 2 ** 31, n).astype(np.int32)  # noqa: E731
        kv.attention(x, wild(6), wild(5), wild(table.size).reshape(table.shape), "F32", max_new=x.shape[0])
        kv.attention(x, np.sort(wild(6)), wild(5), wild(table.size).reshape(table.shape), "F32", max_new=x.shape[0])
        kv.attention(x, cu, wild(5), wild(table.size).reshape(table.shape), "F32")
        kv.status()
        good = rng.permutation(5)[:2]
        ln, tb = wild(5), wild(table.size).reshape(table.shape)
        ln = np.where(ln > 0, -ln, ln)
        ln[good], tb[good] = np.array(lens)[good], table[good]
        out, lse = kv.attention(x, cu, ln, tb, "F32")
        assert kv.status() == 8
        for s in range(5):
            rows = slice(int(cu[s]), int(cu[s + 1]))
            if s in good:
                assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], wl[rows])
            else:
                assert (out[rows] == 77.0).all()
        before = {n: t.clone() for n, t in kv.t.items()}
        kv.append(x[:, :128], x[:, 128:256], cuda(rng.integers(2 ** 40, 2 ** 62, x.shape[0])), ks=512, vs=512)
        assert kv.status() == 8
        assert all(torch.equal(kv.t[n], before[n]) for n in before)
        kv.plan(wild(5), wild(5), wild(table.size).reshape(table.shape), wild(kv.n_pages), int(wild(1)[0]), 50)
        kv.status()
        again, _ = kv.attention(x, cu, lens, table, "F32")
        assert kv.status() == 0 and torch.equal(again, want)
    finally:
        kv.close()


@pytest.mark.parametrize("dtype", ["F32", "BF16"])
@pytest.mark.parametrize("nq,nkv,hd,page,lens,news", [
    (8, 1, 128, 64, [6000], [24]), (4, 2, 64, 16, [5000, 90], [70, 40]), (2, 2, 256, 32, [2900], [130]),
    (32, 1, 64, 16, [4100, 7, 2000], [5, 1, 9])])
def test_chunks_of_a_long_context_split_over_the_gpu(q, nq, nkv, hd, page, lens, news, dtype):
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, hd, page, dtype, 77)
    try:
        out, lse = kv.attention(x, cu, lens, table, dtype)
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table)
        for _ in range(10):                                        # whichever CTA comes last
            again, lse2 = kv.attention(x, cu, lens, table, dtype)
            assert torch.equal(out, again) and torch.equal(lse, lse2)
        last = (lens[0] - 1) // page
        table[0, 3], table[0, last // 2], table[0, last] = -1, kv.n_pages, -2 ** 31
        out, lse = kv.attention(x, cu, lens, table, dtype)
        assert kv.status() == 8
        _check(kv, x, out, lse, cu, lens, table)
    finally:
        kv.close()


def test_parts_that_come_late_are_reported_and_forgotten(q):
    """The CTA that joins a split item gives up on parts that come too late; what they count afterwards is not
    taken for the next call's parts, whose own come late, but in time."""
    lens, news, nq, nkv, hd = [6000], [24], 8, 1, 128
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, hd, 64, "BF16", 5)
    try:
        y = x.flip(0).contiguous()
        want, wl = kv.attention(y, cu, lens, table, "BF16")
        assert kv.status() == 0
        for _ in range(2):
            q.qmoe_kv4_debug_stall_next(kv.h, 400_000_000)
            out, lse = kv.attention(x, cu, lens, table, "BF16")
            assert kv.status() == 7                                # QMOE_ERR_TIMEOUT, and no row of it
            assert (out == 77.0).all() and (lse == 77.0).all()
            for wait in (20_000_000, 0, 1_000_000):
                if wait:
                    q.qmoe_kv4_debug_stall_next(kv.h, wait)
                out, lse = kv.attention(y, cu, lens, table, "BF16")
                assert kv.status() == 0
                assert torch.equal(out, want) and torch.equal(lse, wl)
        assert q.lib.qmoe_kv4_debug_stall_next(kv.h, 0) == 1 and q.lib.qmoe_kv4_debug_stall_next(None, 5) == 1
        assert q.lib.qmoe_kv4_debug_stall_next(kv.h, 2_000_000_000) == 1
    finally:
        kv.close()


def test_the_most_sequences(q):
    rng = np.random.default_rng(3)
    n = 4096
    lens = rng.integers(0, 40, n)
    news = np.where(rng.uniform(size=n) < 0.9, 1, rng.integers(0, 20, n))
    kv, x, cu, table = _filled(q, lens, news, 4, 1, 64, 16, "BF16", 6)
    try:
        out, lse = kv.attention(x, cu, lens, table, "BF16")
        assert kv.status() == 0
        _check(kv, x, out, lse, cu, lens, table)
    finally:
        kv.close()


@pytest.mark.parametrize("news", [[1, 1, 1], [20, 30, 3]])
def test_caches_past_32_bits(q, news):
    """5.2e9 bytes of codes each for K and V: the same rows as from a small cache, bit for bit."""
    lens, nq, nkv, hd, page, n_pages = [40, 170, 9], 16, 2, 128, 64, 640_000
    kv, x, cu, table = _filled(q, lens, news, nq, nkv, hd, page, "F16", 8)
    big = Kv(q, nq, nkv, hd, page, n_pages, 3, 300, kv.width, 0, 8)
    try:
        assert big.t["k_codes"].numel() > 2 ** 32
        far = np.where(table >= 0, n_pages - 1 - 70_000 * table, -1).astype(np.int32)
        slots = lambda t: np.array([int(t[s, p // page]) * page + p % page  # noqa: E731
                                    for s in range(3) for p in range(lens[s])], np.int64)
        rows = torch.randn(2, sum(lens), nkv * hd, device="cuda")
        kv.append(rows[0], rows[1], cuda(slots(table)))
        big.append(rows[0], rows[1], cuda(slots(far)))
        want, wl = kv.attention(x, cu, lens, table, "F16")
        out, lse = big.attention(x, cu, lens, far, "F16")
        assert kv.status() == 0 and big.status() == 0
        assert torch.equal(out, want) and torch.equal(lse, wl)
        st, r = big.plan(np.array([60, 0, 0], np.int32), np.array([10, 70, 1], np.int32),
                         np.where(np.arange(kv.width) == 0, far[0, 0], -1) * np.ones((3, 1), np.int32),
                         np.array([5, n_pages - 2, 6, n_pages - 1] + [-9] * (n_pages - 4), np.int32), 4, 81)
        assert st == 0 and r["slots"][[4, 10, 80]].tolist() == [(n_pages - 1) * 64, 6 * 64, 5 * 64]
    finally:
        kv.close()
        big.close()


@pytest.mark.parametrize("nq,new", [(8, 1), (64, 2)])
def test_rows_past_32_bits_apart(q, nq, new):
    lens, nkv, hd, far = [40, 70], 1, 64, 2 ** 31 + 8
    kv, x, cu, table = _filled(q, lens, [new, new], nq, nkv, hd, 16, "F16", 5)
    try:
        want, _ = kv.attention(x, cu, lens, table, "F16")
        t, row = x.shape
        wide = torch.empty((t - 1) * far + row, dtype=x.dtype, device="cuda")
        view = wide.as_strided((t, row), (far, 1))
        view.copy_(x)
        out = torch.empty_like(wide)
        kv.attention(view, cu, lens, table, "F16", qs=far, os=far, out=out, lse=False)
        assert kv.status() == 0 and torch.equal(out.as_strided((t, row), (far, 1)), want)
        rows = torch.randn(2, t, hd, device="cuda").to(x.dtype)
        hat = torch.empty(4, t, hd, device="cuda")
        slots = cuda(np.arange(t))
        kv.append(rows[0], rows[1], slots, "F16", hat[0], hat[1])
        a, b = wide.as_strided((t, hd), (far, 1)), out.as_strided((t, hd), (far, 1))
        a.copy_(rows[0])
        b.copy_(rows[1])
        kv.append(a, b, slots, "F16", hat[2], hat[3], ks=far, vs=far)
        assert kv.status() == 0 and torch.equal(hat[:2], hat[2:])
    finally:
        kv.close()


def test_two_handles_on_two_streams(q):
    lens, news = [2000, 70, 900], [1, 30, 5]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = [_filled(q, lens, news, 8, 2, 64, 16, "BF16", 8 + i, stream=s.cuda_stream) for i, s in enumerate(streams)]
    try:
        want = []
        for kv, x, cu, table in sets:
            torch.cuda.synchronize()
            want.append(kv.attention(x, cu, lens, table, "BF16"))
            assert kv.status() == 0
        dev = [(cuda(cu), cuda(np.array(lens, np.int32)), cuda(table)) for _, _, cu, table in sets]
        outs = [[(torch.empty_like(w[0]), torch.empty_like(w[1])) for _ in range(40)] for w in want]
        torch.cuda.synchronize()
        for i in range(40):
            for (kv, x, _, _), d, o in zip(sets, dev, outs):
                q.qmoe_kv4_attention(kv.h, kv.cache, x, q.DTYPE["BF16"], 0, 3, x.shape[0], 30, *d, kv.hd ** -0.5,
                                     o[i][0], q.DTYPE["BF16"], 0, o[i][1])
        for (kv, *_), w, o in zip(sets, want, outs):
            assert kv.status() == 0
            assert all(torch.equal(a, w[0]) and torch.equal(b, w[1]) for a, b in o)
    finally:
        for kv, *_ in sets:
            kv.close()


def test_a_handle_that_only_decodes(q):
    """max_tokens of few rows: no room for parts of prompt chunks, and none is needed."""
    nq, nkv, hd, page = 8, 2, 128, 16
    lens = [3000 + 16 * i for i in range(20)]
    kv, x, cu, table = _filled(q, lens, [1] * 4 + [0] * 16, nq, nkv, hd, page, "F32", 8)
    small = Kv(q, nq, nkv, hd, page, kv.n_pages, 20, 4, kv.width)
    assert q.qmoe_kv4_workspace_bytes(q.make_kv4_config(nq, nkv, hd, page, 9, 20, 4, 9)) < 8 << 20
    try:
        for n in (20, 2):
            c, ln = cu[:n + 1].copy(), lens[:n]
            c[-1] = 4
            if n == 2:
                c[1] = 1                                           # one and three new tokens
            want, wl = kv.attention(x, c, ln, table, "F32")
            q.qmoe_kv4_attention(small.h, kv.cache, x, 0, 0, n, 4, 4, cuda(c), cuda(np.array(ln, np.int32)),
                                 cuda(table), hd ** -0.5, want2 := torch.empty_like(want), 0, 0, None)
            assert kv.status() == 0 and small.status() == 0 and torch.equal(want2, want)
            _check(kv, x, want, wl, c, ln, table)
    finally:
        kv.close()
        small.close()


# --------------------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", ["F32", "BF16"])
def test_steps_of_a_serving_loop(q, dtype):
    """plan -> append -> attention over several steps: prompts admitted in chunks, decoding, finishing,
    all lengths and tables on the device; every step against the plain forms."""
    nq, nkv, hd, page, n, width, n_pages, cap = 8, 2, 128, 16, 5, 10, 40, 96
    rng = np.random.default_rng(1)
    kv = Kv(q, nq, nkv, hd, page, n_pages, n, cap, width)
    try:
        i32 = dict(dtype=torch.int32, device="cuda")
        ln, nf = torch.zeros(n, **i32), torch.tensor([n_pages], **i32)
        table = torch.full((n, width), -1, **i32)
        free = torch.arange(n_pages, **i32)
        cu, pos = torch.empty(n + 1, **i32), torch.empty(cap, **i32)
        slots = torch.empty(cap, dtype=torch.int64, device="cuda")
        r = dict(seq_len=np.zeros(n, np.int32), table=table.cpu().numpy(), n_free=n_pages)
        stack = np.arange(n_pages, dtype=np.int32)
        for new in ([30, 17, 0, 1, 0], [1, 1, 60, 1, 0], [1, -1, 20, 1, 5], [1, 40, 1, -1, 1], [-1, 1, 3, 2, 1]):
            new = np.array(new, np.int32)
            q.qmoe_kv4_plan(kv.h, n, ln, cuda(new), table, free, nf, cap, ln, nf, cu, pos, slots)
            rows = torch.from_numpy(rng.normal(size=(cap, (nq + 2 * nkv) * hd))).cuda().to(TORCH[dtype])
            stride = rows.shape[1]
            kv.append(rows[:, nq * hd:], rows[:, (nq + nkv) * hd:], slots, dtype, n=cap, ks=stride, vs=stride)
            out = torch.full((cap, nq * hd), 77.0, dtype=TORCH[dtype], device="cuda")
            q.qmoe_kv4_attention(kv.h, kv.cache, rows, q.DTYPE[dtype], stride, n, cap, 64, cu, ln, table, hd ** -0.5,
                                 out, q.DTYPE[dtype], 0, None)
            assert kv.status() == 0
            r = R.plan(r["seq_len"], new, r["table"], stack, r["n_free"], page, n_pages, cap)
            stack[:r["n_free"]] = r["stack"]
            assert np.array_equal(ln.cpu().numpy(), r["seq_len"]) and np.array_equal(table.cpu().numpy(), r["table"])
            assert np.array_equal(slots.cpu().numpy(), r["slots"]) and int(nf[0]) == r["n_free"]
            t = int(r["cu"][-1])
            x = rows[:, :nq * hd]
            _check(kv, x, out, None, r["cu"], r["seq_len"], r["table"])
            assert (out[t:] == 77.0).all()
    finally:
        kv.close()


@pytest.mark.parametrize("captured", [False, True])
def test_what_follows_prompts_beside_decoding_sees_every_row(q, captured):
    """The attention's two kernels overlap: an append of its output right behind it, and the next attention into
    the same rows, find them complete, call after call and replay after replay."""
    s = torch.cuda.Stream()
    lens, news = [3000, 900, 40, 2500, 300, 17] * 4, [200, 1, 40, 1, 1, 17] * 4
    kv, x, cu, table = _filled(q, lens, news, 8, 2, 64, 16, "F32", 31, stream=s.cuda_stream)
    t = x.shape[0]
    to = Kv(q, 8, 8, 64, 16, t // 16 + 1, 1, t, 1, s.cuda_stream)
    try:
        slots, dev = cuda(np.arange(t)), (cuda(cu), cuda(np.array(lens, np.int32)), cuda(table))
        hat, n = torch.empty(2, t, 512, device="cuda"), 6
        want, out = torch.empty(t, 512, device="cuda"), torch.empty(t, 512, device="cuda")
        hats = torch.empty(n, 2, t, 512, device="cuda")
        torch.cuda.synchronize()                                   # what the default stream made is there
        q.qmoe_kv4_attention(kv.h, kv.cache, x, 0, 0, len(lens), t, 200, *dev, 0.125, want, 0, 0, None)
        torch.cuda.synchronize()
        to.append(want, want, slots, "F32", hat[0], hat[1])
        assert kv.status() == 0 and to.status() == 0

        def run():
            for i in range(n):
                out.fill_(float("nan"))
                q.qmoe_kv4_attention(kv.h, kv.cache, x, 0, 0, len(lens), t, 200, *dev, 0.125, out, 0, 0, None)
                to.append(out, out, slots, "F32", hats[i][0], hats[i][1])

        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            if captured:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=s):
                    run()
            for _ in range(5):
                g.replay() if captured else run()
        torch.cuda.synchronize()
        assert kv.status() == 0 and to.status() == 0
        assert torch.equal(out, want) and all(torch.equal(h, hat) for h in hats)
    finally:
        kv.close()
        to.close()


def test_prompts_among_many_that_decode(q):
    """Far fewer pieces than the host has to fear, as lengths change from call to call."""
    rng = np.random.default_rng(9)
    n = 600
    for big in (1, 40, 0, 3):
        news = np.ones(n, int)
        news[rng.permutation(n)[:big]] = rng.integers(9, 150, big)
        lens = news + rng.integers(0, 60, n)
        kv, x, cu, table = _filled(q, lens, news, 4, 1, 64, 16, "F16", big)
        try:
            for k in range(3):
                out, lse = kv.attention(x, cu, lens, table, "F16", max_new=150)
                assert kv.status() == 0
                if k in (0, 2):
                    _check(kv, x, out, lse, cu, lens, table)
                else:                                              # the same handle, every second request idle
                    half = np.where(np.arange(n) % 2, 0, lens)
                    out, lse = kv.attention(x, cu, half, table, "F16", max_new=150)
                    assert kv.status() == 0
                    _check(kv, x, out, lse, cu, half, table)
        finally:
            kv.close()


def test_a_captured_step_replayed_while_lengths_grow(q):
    nq, nkv, hd, page, n, width, n_pages, cap = 8, 2, 64, 16, 4, 6, 24, 4
    s = torch.cuda.Stream()
    kv = Kv(q, nq, nkv, hd, page, n_pages, n, cap, width, s.cuda_stream)
    try:
        i32 = dict(dtype=torch.int32, device="cuda")
        ln, nf = torch.zeros(n, **i32), torch.tensor([n_pages], **i32)
        table, free = torch.full((n, width), -1, **i32), torch.arange(n_pages, **i32)
        new = torch.ones(n, **i32)
        cu, pos = torch.empty(n + 1, **i32), torch.empty(cap, **i32)
        slots = torch.empty(cap, dtype=torch.int64, device="cuda")
        rows = torch.empty(cap, (nq + 2 * nkv) * hd, device="cuda")
        out = torch.empty(cap, nq * hd, device="cuda")
        stride = rows.shape[1]

        def step():
            q.qmoe_kv4_plan(kv.h, n, ln, new, table, free, nf, cap, ln, nf, cu, pos, slots)
            kv.append(rows[:, nq * hd:], rows[:, (nq + nkv) * hd:], slots, n=cap, ks=stride, vs=stride)
            q.qmoe_kv4_attention(kv.h, kv.cache, rows, 0, stride, n, cap, 1, cu, ln, table, hd ** -0.5, out, 0, 0,
                                 None)

        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step()
        torch.cuda.synchronize()
        assert int(ln.sum()) == 0                                  # captured, not run
        for i in range(40):
            rows.copy_(torch.from_numpy(np.random.default_rng(i).normal(size=tuple(rows.shape))))
            if i == 20:
                new.copy_(torch.tensor([1, 0, -1, 1]))
            if i == 21:
                new.fill_(1)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert kv.status() == 0
            lens, cus = ln.cpu().numpy(), cu.cpu().numpy()
            if i % 7 == 0 or i in (20, 21, 22):
                _check(kv, rows[:, :nq * hd], out, None, cus, lens, table.cpu().numpy())
        assert lens.tolist() == [40, 39, 19, 40]
    finally:
        kv.close()


def test_refused_arguments(q):
    kv = Kv(q, 4, 2, 64, 16, 6, 2, 8, 3)
    L = q.lib
    try:
        i = torch.zeros(64, dtype=torch.int32, device="cuda")
        j = torch.zeros(64, dtype=torch.int64, device="cuda")
        x = torch.zeros(16 * 1024, device="cuda")

        def plan(**c):
            a = dict(n=2, len=i, new=i[8:], table=i[16:], free=i[24:], nf=i[32:], cap=8, lo=i[36:], no=i[40:],
                     cu=i[44:], pos=i[48:], slots=j)
            a.update(c)
            return L.qmoe_kv4_plan(kv.h, a["n"], *[q._ptr(a[k]) for k in ("len", "new", "table", "free", "nf")],
                                   a["cap"], *[q._ptr(a[k]) for k in ("lo", "no", "cu", "pos", "slots")])

        assert plan(n=0) == 4 and plan(n=3) == 4 and plan(cap=0) == 4 and plan(cap=9) == 4
        for k in ("len", "new", "table", "free", "nf", "lo", "no", "cu", "pos", "slots"):
            assert plan(**{k: None}) == 1
        assert plan(lo=i[8:]) == 1 and plan(cu=i) == 1
        assert plan(slots=j.data_ptr() + 4) == 2 and plan(len=i.data_ptr() + 2) == 2

        def append(**c):
            a = dict(cache=kv.cache, k=x, v=x, t=0, n=2, ks=0, vs=0, slots=j, kh=None, vh=None)
            a.update(c)
            return L.qmoe_kv4_append(kv.h, a["cache"] and q.C.byref(a["cache"]), q._ptr(a["k"]), q._ptr(a["v"]),
                                     a["t"], a["n"], a["ks"], a["vs"], q._ptr(a["slots"]), q._ptr(a["kh"]),
                                     q._ptr(a["vh"]))

        assert append(n=0) == 4 and append(n=9) == 4 and append(t=3) == 1 and append(ks=127) == 4
        assert append(vs=-128) == 4 and append(ks=129) == 2 and append(k=x.data_ptr() + 4) == 2
        assert append(t=1, vs=132) == 2 and append(cache=None) == 1 and append(slots=None) == 1
        assert append(k=None) == 1 and append(v=None) == 1 and append(kh=x.data_ptr() + 8) == 2
        odd = q.make_kv4_cache(kv.t["k_codes"].data_ptr() + 8, kv.t["k_scales"], kv.t["v_codes"], kv.t["v_scales"],
                               kv.kg, kv.vg)
        none = q.make_kv4_cache(kv.t["k_codes"], kv.t["k_scales"], kv.t["v_codes"], None, kv.kg, kv.vg)
        assert append(cache=odd) == 2 and append(cache=none) == 1

        def attn(**c):
            a = dict(cache=kv.cache, q=x, t=0, qs=0, n=2, tok=2, mx=1, cu=i, len=i, table=i, scale=1.0, out=x[8192:],
                     ot=0, os=0, lse=None)
            a.update(c)
            return L.qmoe_kv4_attention(kv.h, a["cache"] and q.C.byref(a["cache"]), q._ptr(a["q"]), a["t"], a["qs"],
                                        a["n"], a["tok"], a["mx"], q._ptr(a["cu"]), q._ptr(a["len"]),
                                        q._ptr(a["table"]), a["scale"], q._ptr(a["out"]), a["ot"], a["os"],
                                        q._ptr(a["lse"]))

        assert attn(n=0) == 4 and attn(n=3) == 4 and attn(tok=0) == 4 and attn(tok=9) == 4
        assert attn(mx=0) == 4 and attn(mx=3) == 4 and attn(t=7) == 1 and attn(ot=-1) == 1
        assert attn(scale=float("nan")) == 1 and attn(scale=float("inf")) == 1 and attn(out=x) == 1
        assert attn(qs=255) == 4 and attn(os=257) == 2 and attn(q=x.data_ptr() + 4) == 2
        for k in ("q", "cu", "len", "table", "out"):
            assert attn(**{k: None}) == 1
        assert attn(cache=odd) == 2 and attn(cache=none) == 1 and attn(lse=x.data_ptr() + 2) == 2
        assert "lse" in q.qmoe_kv4_last_error(kv.h)
        torch.cuda.synchronize()
        assert kv.status() == 0
    finally:
        kv.close()


def test_allocation_failure_is_reported(q):
    q.qmoe_debug_fail_alloc(1)
    try:
        with pytest.raises(q.QmoeError) as e:
            q.qmoe_kv4_create(q.make_kv4_config(8, 2, 128, 16, 4, 1, 1, 1))
        assert e.value.status == 5 and "allocation" in str(e.value)
    finally:
        q.qmoe_debug_fail_alloc(0)
