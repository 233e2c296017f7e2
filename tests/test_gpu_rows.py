"""The 8-bit path's row operators on the GPU against their plain forms in 64 bits."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as K4
from tests import rows_ref as R
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

TORCH = {"F32": torch.float32, "F16": torch.float16, "BF16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import quantized_mixture_experts_f32_gb300 as q
    return q


def make_ctx(q, stream=None):
    stream = stream or torch.cuda.current_stream(dev())
    return q.qmoe_create(q.make_config(256, 1, 1, 256, 1, stream=stream.cuda_stream))


@pytest.fixture(scope="module")
def ctx(q):
    c = make_ctx(q)
    yield c
    assert q.qmoe_get_status(c) == q.QMOE_OK, q.qmoe_last_error(c)
    q.qmoe_destroy(c)


def host(t):
    return (t.float() if t.dtype in (torch.float16, torch.bfloat16) else t).cpu().numpy()


def rand_rows(rows, cols, dtype, seed, stride=None, lead=0):
    """Device rows of `dtype`, `stride` elements apart, behind `lead` elements."""
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    stride = stride or cols
    x = torch.randn(rows, stride, device=dev(), generator=g) * torch.exp(torch.randn(1, stride, device=dev(), generator=g))
    return x.to(TORCH[dtype])[:, lead:lead + cols]


def guarded(rows, cols, dtype, stride=None, value=7.0):
    """Rows in a buffer filled with `value`, and the buffer."""
    buf = torch.full((rows + 2, stride or cols), value, dtype=dtype, device=dev())
    return buf[1:-1, :cols], buf


def assert_guard(buf, rows, cols, value=7.0):
    b = buf.clone().float()
    b[1:1 + rows, :cols] = value
    assert (b == value).all()


# ---------------------------------------------------------------------------- norm and 8 bits

# fp32 error of y, relative: a thread's sum of at most 64 squares, 5 shuffles and 32 warps' parts
# (101 roundings, halved by the root), h itself, mean, root and two products
NORM_ERR = 64 * R.U


def check_codes(codes, scale, y, slack):
    """8-bit rows of y (64 bits), whose fp32 form is `slack` off, relative."""
    b = R._blocks(y)
    want = np.abs(b).max(-1) / 448
    assert (np.abs(scale - want) <= (slack + R.U) * want).all()
    v = R.e4m3_decode(codes)
    s = np.repeat(want, 128, 1)[:, :y.shape[1]]
    u = np.where(s > 0, y / np.where(s > 0, s, 1), 0)
    best = R.GRID[R._nearest_even(np.minimum(np.abs(u), 448.0), R.GRID)]
    assert (np.abs(np.abs(v) - np.abs(u)) <= np.abs(best - np.abs(u)) + 2 * (2 * slack + 4 * R.U) * np.abs(u)).all()
    assert (v * u >= 0).all()


NORM_CASES = [  # rows, dim, x, residual, out, x stride, in place
    (1, 2048, "F32", "F32", "E4M3", 0, "sum"), (1, 16, "F32", None, "F32", 0, ""), (3, 16, "BF16", "BF16", "E4M3", 24, ""),
    (7, 128, "F16", "F32", "F16", 0, "y"), (33, 144, "BF16", "F32", "BF16", 160, "sum"), (5, 768, "F32", None, "E4M3", 1024, ""),
    (257, 2048, "BF16", "F32", "E4M3", 0, ""), (2, 2064, "F16", "F16", "F32", 0, "x"), (9, 4096, "BF16", None, "BF16", 0, "y"),
    (4, 5008, "F32", "BF16", "E4M3", 5012, ""), (3, 16384, "BF16", "F32", "E4M3", 0, ""), (2, 32768, "F16", "F32", "E4M3", 0, ""),
    (1, 32752, "F32", "F32", "F32", 0, ""), (2000, 256, "F32", "F32", "F32", 0, ""), (4099, 64, "BF16", None, "E4M3", 0, ""),
    (1500, 512, "BF16", "BF16", "BF16", 0, "x"),
]


@pytest.mark.parametrize("rows,dim,x_t,res_t,y_t,stride,alias", NORM_CASES)
@pytest.mark.parametrize("weighted", [True, False])
def test_rmsnorm(q, ctx, rows, dim, x_t, res_t, y_t, stride, alias, weighted):
    x = rand_rows(rows, dim, x_t, 1, stride, 0)
    res = rand_rows(rows, dim, res_t, 2) * 3 if res_t else None
    w = (1 + 0.3 * torch.randn(dim, device=dev())) if weighted else None
    xh, rh = host(x), None if res is None else host(res)
    h, y64 = R.rmsnorm(xh, rh, None if w is None else host(w), EPS)
    total = None
    if res is not None:
        total = res if alias == "sum" else x if alias == "x" and x_t == res_t else torch.empty_like(res)
    fp8 = y_t == "E4M3"
    if alias == "y" and x_t == y_t:
        y, guard = x, None
    else:
        y, guard = guarded(rows, dim, torch.uint8 if fp8 else TORCH[y_t])
    scale, sguard = guarded(rows, -(-dim // 128), torch.float32)
    q.qmoe_rmsnorm(ctx, x, q.DTYPE[x_t], x.stride(0), res, q.DTYPE[res_t or "F32"],
                   res.stride(0) if res is not None and alias != "x" else (x.stride(0) if alias == "x" and x_t == res_t else 0),
                   total, w, EPS, rows, dim, y, q.DTYPE[y_t], 0 if fp8 else y.stride(0), scale if fp8 else None)
    torch.cuda.synchronize()
    if total is not None:
        t = host(total).astype(np.float64)
        assert (np.abs(t - h) <= (R.HALF[res_t] + R.U) * np.abs(h) + 2.0 ** -25).all()
    if fp8:
        check_codes(host(y), host(scale), y64, NORM_ERR)
        assert_guard(sguard, rows, scale.shape[1])
    else:
        err = np.abs(host(y).astype(np.float64) - y64)
        half = 0 if y_t == "F32" else R.HALF[y_t]
        assert (err <= (NORM_ERR + half) * np.abs(y64) + (2.0 ** -25 if y_t == "F16" else 0)).all()
    if guard is not None:
        assert_guard(guard, rows, dim)


@pytest.mark.parametrize("rows,cols,x_t,stride", [
    (1, 16, "F32", 0), (1, 4096, "BF16", 0), (64, 4096, "BF16", 0), (3, 144, "F16", 152), (17, 2000, "F32", 2048),
    (5003, 272, "F32", 300), (2, 32768, "BF16", 0), (700, 128, "F16", 0), (11, 1040, "BF16", 0)])
def test_fp8_quantize_is_bit_exact(q, ctx, rows, cols, x_t, stride):
    x = rand_rows(rows, cols, x_t, 3, stride)
    x[0, :16] = 0
    if rows > 2:
        x[1] = 0
        x[2] *= 1e-30 if x_t != "F16" else 1e-4
    codes, guard = guarded(rows, cols, torch.uint8)
    scale, sguard = guarded(rows, -(-cols // 128), torch.float32)
    q.qmoe_fp8_quantize(ctx, x, q.DTYPE[x_t], x.stride(0), rows, cols, codes, scale)
    torch.cuda.synchronize()
    c, s = R.quantise8(host(x))
    assert np.array_equal(host(scale), s)
    assert np.array_equal(host(codes), c)
    assert_guard(guard, rows, cols)
    assert_guard(sguard, rows, scale.shape[1])


def test_fp8_quantize_at_and_beside_every_border(q, ctx):
    """Rows whose block maximum is 448 s, so that the scale is s, and elements at and next to every border."""
    mid = (R.GRID[1:] + R.GRID[:-1]) / 2
    for s in (1.0, 2.0 ** -20, 1.7e-3, 3e20, 2.0 ** -100):
        v = np.concatenate([mid, R.GRID[1:]]).astype(np.float32)
        v = np.concatenate([v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(1e9))]) * np.float32(s)
        v = np.minimum(v, np.float32(448 * s))
        v = np.pad(v, (0, -len(v) % 127)).reshape(-1, 127)
        x = np.concatenate([np.full((len(v), 1), 448 * s, np.float32), v], 1)
        x = np.concatenate([x, -x])
        t = torch.from_numpy(x).to(dev())
        codes, scale = torch.empty(len(x), 128, dtype=torch.uint8, device=dev()), torch.empty(len(x), 1, device=dev())
        q.qmoe_fp8_quantize(ctx, t, q.QMOE_F32, 0, len(x), 128, codes, scale)
        torch.cuda.synchronize()
        c, sc = R.quantise8(x)
        assert np.array_equal(host(scale), sc)
        # the sign of a zero is the element's
        assert np.array_equal(host(codes) & 127, c & 127)
        assert np.array_equal((host(codes) >> 7)[x != 0], (c >> 7)[x != 0])


def test_8_bit_rows_of_values_that_are_not_finite(q, ctx):
    x = torch.ones(4, 256, device=dev())
    x[0, 5], x[1, 7], x[2, 130] = float("nan"), float("inf"), -float("inf")
    x[3, :128] = float("nan")
    codes, scale = torch.empty(4, 256, dtype=torch.uint8, device=dev()), torch.empty(4, 2, device=dev())
    q.qmoe_fp8_quantize(ctx, x, q.QMOE_F32, 0, 4, 256, codes, scale)
    c, s = host(codes), host(scale)
    one = np.float32(1) / np.float32(448)
    assert c[0, 5] & 127 == 127 and (np.delete(c[0], 5) == 126).all() and (s[0] == one).all()
    assert c[1, 7] & 127 == 127 and not np.delete(c[1, :128], 7).any() and np.isinf(s[1, 0]) and s[1, 1] == one
    assert c[2, 130] & 127 == 127 and np.isinf(s[2, 1]) and s[2, 0] == one
    assert (c[3, :128] & 127 == 127).all() and s[3, 0] == 0 and (c[3, 128:] == 126).all()


# ---------------------------------------------------------------------------- linear

def linear_inputs(T, K, N, seed):
    rng = np.random.default_rng(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    xc = rng.integers(0, 256, (T, K), dtype=np.uint8)
    wc = rng.integers(0, 256, (N, K), dtype=np.uint8)
    for c in (xc, wc):
        c[(c & 127) == 127] = 0
    xs = (np.exp(rng.normal(size=(T, kb)) * 2) * 1e-3).astype(np.float32)
    ws = (np.exp(rng.normal(size=(nb, kb)) * 2) * 1e-3).astype(np.float32)
    return xc, xs, wc, ws


def linear_bound(size, kb, out, half, act):
    """Each block's 128 products of eight bits' fraction are exact and summed in fp32 (at most a step, two
    half steps, lost an addition), the blocks' scaled sums added in kb roundings, scale and bias in three;
    the activation's slope is at most 1.13, its own error four steps of its argument."""
    rel = (2 * 128 + kb + 4) * R.U * size
    return (1.13 * rel + 8 * R.U * (size + np.abs(out)) if act != "NONE" else rel) + (R.U + half) * np.abs(out) + 2.0 ** -25


def run_linear(q, ctx, T, K, N, out_t="F32", act="NONE", bias=False, residual="", seed=0, pad=0, sync=True):
    xc, xs, wc, ws = linear_inputs(T, K, N, 1000 + seed)
    d = [torch.from_numpy(a).to(dev()) for a in (xc, xs, wc, ws)]
    want_size = R.linear(xc, xs, wc, ws, None, "NONE", None)[1]
    unit = float(np.median(want_size))
    b = torch.randn(N, device=dev()) * unit if bias else None
    step = 4 if out_t == "F32" else 8
    stride = -(-N // step) * step + pad
    out, guard = guarded(T, N, TORCH[out_t], stride)
    res = None
    if out_t == "F16":                                   # keep the results in fp16's range
        d[1] *= 1 / unit
        xs = host(d[1])
        b = None if b is None else b / unit
        unit = 1.0
    if residual:
        r = (torch.randn(T, N, device=dev()) * unit).to(TORCH[out_t])
        if residual == "place":
            out.copy_(r)
            res = out
        else:
            res = torch.zeros(T, stride + 8, dtype=TORCH[out_t], device=dev())[:, :N]
            res.copy_(r)
    ref, size = R.linear(xc, xs, wc, ws, None if b is None else host(b).astype(np.float64), act, host(r) if residual else None)
    q.qmoe_linear_fp8(ctx, d[0], d[1], T, K, d[2], d[3], N, b, q.ACT[act], res, 0 if res is None else res.stride(0), out,
                      q.DTYPE[out_t], out.stride(0))
    if not sync:
        return out, ref
    torch.cuda.synchronize()
    err = np.abs(host(out).astype(np.float64) - ref)
    bound = linear_bound(size, -(-K // 128), ref, 0 if out_t == "F32" else R.HALF[out_t], act)
    assert (err <= bound).all(), (err / bound).max()
    assert_guard(guard, T, N)
    return out


LINEAR_CASES = [  # T, K, N, out, act, bias, residual, pad
    (1, 16, 1, "F32", "NONE", False, "", 0), (1, 2048, 5120, "BF16", "NONE", False, "", 0),
    (1, 4096, 2048, "F32", "NONE", True, "place", 0), (2, 144, 130, "F16", "GELU", True, "apart", 8),
    (3, 1008, 257, "BF16", "SILU", False, "apart", 0), (8, 2048, 640, "F32", "RELU", True, "", 4),
    (9, 128, 128, "F32", "NONE", False, "", 0), (15, 256, 1000, "F16", "NONE", False, "place", 0),
    (16, 2048, 512, "BF16", "NONE", True, "", 0), (17, 400, 129, "F32", "SILU", True, "apart", 12),
    (31, 1024, 384, "BF16", "GELU", False, "place", 0), (32, 528, 2000, "F32", "NONE", False, "", 0),
    (33, 2048, 256, "F16", "RELU", True, "", 0), (64, 4096, 2048, "F32", "NONE", False, "place", 0),
    (65, 112, 127, "BF16", "NONE", True, "apart", 0), (100, 1536, 300, "F32", "GELU", True, "", 0),
    (127, 256, 255, "F16", "SILU", False, "", 8), (128, 384, 256, "F32", "NONE", False, "", 0),
    (129, 640, 131, "BF16", "NONE", False, "place", 0), (200, 16, 700, "F32", "NONE", True, "", 0),
    (255, 1040, 384, "F32", "RELU", False, "apart", 0), (256, 2048, 512, "BF16", "GELU", True, "", 0),
    (257, 2048, 640, "F32", "NONE", False, "", 0), (511, 896, 1003, "F16", "GELU", True, "", 0),
    (777, 2000, 1003, "F16", "GELU", True, "", 0), (1000, 256, 2049, "BF16", "SILU", True, "place", 0),
    (2048, 512, 384, "F32", "NONE", False, "apart", 0), (2049, 2048, 640, "BF16", "NONE", True, "", 0),
    (1, 16384, 200, "F32", "NONE", False, "", 0), (5, 20000, 64, "BF16", "NONE", False, "", 0),
    (4, 64, 20001, "F32", "NONE", False, "", 0), (300, 8192, 130, "F32", "NONE", False, "", 0),
]


@pytest.mark.parametrize("T,K,N,out_t,act,bias,residual,pad", LINEAR_CASES)
def test_linear(q, ctx, T, K, N, out_t, act, bias, residual, pad):
    run_linear(q, ctx, T, K, N, out_t, act, bias, residual, T + K + N, pad)


@pytest.mark.parametrize("T,K,N,out_t,act,bias,residual", [(1, 528, 20011, "F32", "SILU", True, "place"), (7, 144, 40001, "BF16", "NONE", False, ""),
                                                          (8, 1040, 20000, "F16", "GELU", True, "apart"),
                                                          (16, 400, 5121, "F32", "RELU", False, "apart"), (30, 2064, 4999, "BF16", "SILU", True, "place"),
                                                          (1, 2048, 8192, "BF16", "NONE", False, ""), (12, 272, 30001, "F16", "NONE", True, "")])
def test_linear_few_tokens_many_features(q, ctx, T, K, N, out_t, act, bias, residual):
    run_linear(q, ctx, T, K, N, out_t, act, bias, residual, T + K + N)


SHARED_CASES = [  # tiles whose k is shared by two to four pairs of CTAs: tokens, K, N as above
    (100, 2048, 2500, "BF16", "NONE", False, "", 0), (777, 2000, 1100, "F32", "SILU", True, "place", 0),
    (256, 4096, 2048, "F32", "NONE", False, "place", 0), (199, 4112, 2047, "F16", "GELU", True, "apart", 0),
    (200, 4096, 1400, "BF16", "RELU", True, "", 8), (256, 16368, 513, "F32", "GELU", True, "apart", 4),
    (257, 6160, 1001, "BF16", "NONE", True, "place", 0), (513, 8208, 300, "F16", "NONE", False, "", 0),
    (1500, 10000, 129, "BF16", "SILU", False, "apart", 0), (140, 1552, 2560, "F32", "NONE", True, "", 0)]


@pytest.mark.parametrize("T,K,N,out_t,act,bias,residual,pad", SHARED_CASES)
def test_linear_shared_k(q, ctx, T, K, N, out_t, act, bias, residual, pad):
    run_linear(q, ctx, T, K, N, out_t, act, bias, residual, T + K + N, pad)


@pytest.mark.parametrize("T,K,N", [(256, 4096, 2048), (200, 4096, 1400), (100, 2048, 2500)])
def test_linear_shared_k_on_two_streams_and_again(q, T, K, N):
    """Two handles at once, many calls, the results the same bits each time."""
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    ctx = [make_ctx(q, s) for s in st]
    d = [torch.from_numpy(a).to(dev()) for a in linear_inputs(T, K, N, 3)]
    out = [[torch.zeros(T, -(-N // 4) * 4, device=dev())[:, :N] for _ in range(8)] for _ in st]
    torch.cuda.synchronize()
    for i in range(8):
        for c, o in zip(ctx, out):
            q.qmoe_linear_fp8(c, d[0], d[1], T, K, d[2], d[3], N, None, 0, None, 0, o[i], q.QMOE_F32, o[i].stride(0))
    torch.cuda.synchronize()
    for c, o in zip(ctx, out):
        assert q.qmoe_get_status(c) == q.QMOE_OK
        assert all(torch.equal(out[0][0], x) for x in o)
    want, size = R.linear(*linear_inputs(T, K, N, 3), None, "NONE", None)
    assert (np.abs(host(out[0][0]) - want) <= linear_bound(size, -(-K // 128), want, 0, "NONE")).all()
    for c in ctx:
        q.qmoe_destroy(c)


@pytest.mark.parametrize("T", [1, 300])
@pytest.mark.parametrize("act", ["RELU", "SILU", "GELU"])
def test_linear_activations_over_their_range(q, ctx, act, T):
    """Products of zeros, so that a bias is what is activated: tiny, ordinary, huge."""
    z = np.concatenate([np.linspace(-12, 12, 1501), np.geomspace(1e-38, 1e30, 300), -np.geomspace(1e-38, 1e30, 300)]).astype(np.float32)
    N, K = len(z), 128
    zero = torch.zeros(max(T, N), K, dtype=torch.uint8, device=dev())
    one = torch.ones(max(T, N), device=dev())
    bias = torch.from_numpy(z).to(dev())
    wide = -(-N // 4) * 4
    out = torch.zeros(T, wide, device=dev())[:, :N]
    q.qmoe_linear_fp8(ctx, zero, one, T, K, zero, one, N, bias, q.ACT[act], None, 0, out, q.QMOE_F32, wide)
    want = R.activate(z.astype(np.float64), act)
    # exponentials and their arguments to some four steps, times a slope below 1.2
    assert (np.abs(host(out) - want) <= 8 * R.U * np.abs(z) + 1e-37).all()


def test_linear_products_are_summed_in_32_bits(q, ctx):
    """Blocks whose large products cancel: what is left is exact where 24 bits hold every partial sum."""
    T, K, N = 40, 256, 160
    rng = np.random.default_rng(5)
    big, small = 0x7e, 0x38                                             # 448 and 1
    xc, wc = np.full((T, K), small, np.uint8), np.full((N, K), small, np.uint8)
    xc[:, 0::2] = big                                                   # 448
    wc[:, 0::4], wc[:, 2::4] = big, big | 0x80                          # 448 * (448 - 448)
    flip = rng.integers(0, 2, (N, K // 2)).astype(np.uint8) << 7
    wc[:, 1::2] |= flip
    xs, ws = np.ones((T, 2), np.float32), np.ones((2, 2), np.float32)
    ref, _ = R.linear(xc, xs, wc, ws, None, "NONE", None)
    d = [torch.from_numpy(a).to(dev()) for a in (xc, xs, wc, ws)]
    out = torch.empty(T, N, device=dev())
    q.qmoe_linear_fp8(ctx, d[0], d[1], T, K, d[2], d[3], N, None, 0, None, 0, out, q.QMOE_F32, 0)
    # partial sums are below 32 * 448^2 < 2^23: whole numbers stay exact in 24 bits
    assert np.array_equal(host(out), ref.astype(np.float32))


@pytest.mark.parametrize("T,K,N", [(2000, 256, 256), (600, 1024, 5120), (256, 4096, 2048), (16, 4096, 128)])
def test_linear_products_are_summed_in_32_bits_by_every_kernel(q, ctx, T, K, N):
    """As above on tcgen05, both tiles, k shared or not: 448 * 448 and its negative beside ones."""
    rng = np.random.default_rng(7)
    x = np.full((1, K), 0x38, np.uint8)
    x[:, 0::2] = 0x7e
    w = np.full((N, K), 0x38, np.uint8)
    w[:, 0::4], w[:, 2::4] = 0x7e, 0x7e | 0x80
    w[:, 1::2] |= rng.integers(0, 2, (N, K // 2)).astype(np.uint8) << 7
    ref = (1 - 2 * (w[:, 1::2] >> 7).astype(np.float64)).sum(1).astype(np.float32)
    d = [torch.from_numpy(a).to(dev()) for a in (np.repeat(x, T, 0), w)]
    xs, ws = torch.ones(T, -(-K // 128), device=dev()), torch.ones(-(-N // 128), -(-K // 128), device=dev())
    out = torch.empty(T, N, device=dev())
    q.qmoe_linear_fp8(ctx, d[0], xs, T, K, d[1], ws, N, None, 0, None, 0, out, q.QMOE_F32, 0)
    assert (host(out) == ref).all()


def test_linear_not_finite_stays_in_its_row(q, ctx):
    T, K, N = 20, 256, 200
    xc, xs, wc, ws = linear_inputs(T, K, N, 9)
    xc[3, 200] = 0x7f
    xs[5, 0] = np.inf
    d = [torch.from_numpy(a).to(dev()) for a in (xc, xs, wc, ws)]
    out = torch.empty(T, N, device=dev())
    for act in ("NONE", "RELU", "SILU", "GELU"):
        q.qmoe_linear_fp8(ctx, d[0], d[1], T, K, d[2], d[3], N, None, q.ACT[act], None, 0, out, q.QMOE_F32, 0)
        o = host(out)
        assert np.isnan(o[3]).all()
        rest = np.delete(o, (3, 5), 0)
        assert np.isfinite(rest).all()


def test_linear_results_do_not_change_from_run_to_run(q, ctx):
    for T, K, N in ((1, 4096, 2048), (40, 2048, 640), (600, 2048, 900)):
        first = None
        for _ in range(4):
            out = run_linear(q, ctx, T, K, N, seed=3)
            if first is None:
                first = out.clone()
            assert torch.equal(first, out)


# ---------------------------------------------------------------------------- rotary positions

def make_table(q, ctx, rot, n_pos, layout="half", scaling="plain", base=1e6, **more):
    table = torch.full((n_pos + 1, 2, rot // 2), 9.0, device=dev())
    kind = {"plain": q.QMOE_ROPE_PLAIN, "linear": q.QMOE_ROPE_LINEAR, "parts": q.QMOE_ROPE_PARTS}[scaling]
    rope = q.make_rope(rot, base, n_pos, table, layout=q.ROPE_LAYOUT[layout], scaling=kind, **more)
    q.qmoe_rope_table(ctx, rope)
    torch.cuda.synchronize()
    assert (table[n_pos] == 9).all()
    return rope, table


@pytest.mark.parametrize("rot,n_pos,base,scaling,more", [
    (128, 40960, 1e6, "plain", {}), (16, 3, 1e4, "plain", {}), (64, 200001, 1e7, "linear", dict(factor=8.0)),
    (128, 131072, 1e6, "parts", dict(factor=4.0, orig_ctx=32768.0)), (256, 1000, 500.0, "parts", dict(factor=2.0, orig_ctx=100.0, mscale=0.5)),
    (32, 1000, 1e4, "parts", dict(factor=0.5, orig_ctx=7.0, beta_fast=1e9, beta_slow=1e8))])
def test_rope_table(q, ctx, rot, n_pos, base, scaling, more):
    rope, table = make_table(q, ctx, rot, n_pos, scaling=scaling, base=base, **more)
    f, m = R.rope_freq(rot, base, scaling, **more)
    ang = np.arange(n_pos, dtype=np.longdouble)[:, None] * f.astype(np.longdouble)
    got = table[:n_pos].cpu().numpy()
    # half a step of a value in size at most m, and the frequency's and the product's rounding times the position
    tol = R.U * max(1.0, m) + n_pos * f.max() * 2.0 ** -50
    for j, fn in enumerate((np.cos, np.sin)):
        assert np.abs(got[:, j] - (fn(ang) * m).astype(np.float64)).max() <= tol


ROPE_CASES = [  # tokens, heads, hd, rot, layout, dtype, norm, stride beyond, in place
    (1, 1, 64, 16, "half", "F32", False, 0, False), (1, 32, 128, 128, "half", "BF16", True, 0, True),
    (5, 7, 64, 64, "interleaved", "F16", True, 8, False), (64, 32, 128, 128, "half", "BF16", True, 1024, True),
    (33, 3, 256, 256, "half", "F32", True, 4, False), (9, 10, 128, 48, "half", "F32", False, 0, True),
    (700, 5, 64, 32, "interleaved", "BF16", False, 64, False), (3, 1024, 64, 64, "half", "F16", False, 0, False),
    (2, 100, 256, 128, "interleaved", "F32", True, 0, True), (1001, 1, 128, 112, "half", "F16", True, 0, False)]


@pytest.mark.parametrize("T,heads,hd,rot,layout,dtype,norm,more,place", ROPE_CASES)
def test_rope(q, ctx, T, heads, hd, rot, layout, dtype, norm, more, place):
    n_pos = 5000
    rope, table = make_table(q, ctx, rot, n_pos, layout)
    cols = heads * hd
    x = rand_rows(T, cols, dtype, 11, cols + more)
    pos = torch.randint(0, n_pos, (T,), device=dev(), dtype=torch.int32)
    pos[T // 2:T // 2 + 1] = n_pos - 1
    if T > 4:
        pos[3] = -1
        pos[T - 1] = -(2 ** 31)
    w = 1 + 0.3 * torch.randn(hd, device=dev()) if norm else None
    xh, ph = host(x).astype(np.float32), host(pos)
    out, guard = (x, None) if place else guarded(T, cols, TORCH[dtype], cols + 8)
    before = host(out).copy()
    q.qmoe_rope(ctx, rope, x, q.DTYPE[dtype], x.stride(0), T, heads, hd, pos, w, EPS, out, out.stride(0))
    torch.cuda.synchronize()
    assert q.qmoe_get_status(ctx) == q.QMOE_OK
    cs = host(table)[np.maximum(ph, 0)]
    n = R.rope_heads(xh, hd, None if w is None else host(w), EPS)
    want = R.rope(n, cs, rot, layout).reshape(T, cols)
    live = ph >= 0
    # the same fp32 steps; rounded to the rows' type as torch rounds
    want = host(torch.from_numpy(want).to(TORCH[dtype]))
    assert np.array_equal(host(out)[live], want[live])
    assert np.array_equal(host(out)[~live], before[~live])
    if guard is not None:
        assert_guard(guard, T, cols)


def test_rope_position_past_the_table(q, ctx):
    rope, table = make_table(q, ctx, 64, 100)
    x = rand_rows(3, 128, "F32", 5)
    pos = torch.tensor([99, 100, 2 ** 31 - 1], dtype=torch.int32, device=dev())
    out = torch.full((3, 128), 7.0, device=dev())
    q.qmoe_rope(ctx, rope, x, q.QMOE_F32, 0, 3, 2, 64, pos, None, 0.0, out, 0)
    assert q.qmoe_get_status(ctx) == 8
    assert (out[1:] == 7).all() and not (out[0] == 7).any()
    assert q.qmoe_get_status(ctx) == q.QMOE_OK


@pytest.mark.parametrize("dtype", ["F32", "F16"])
def test_rope_norm_of_small_large_and_zero_heads(q, ctx, dtype):
    rope, _ = make_table(q, ctx, 128, 10)
    x = rand_rows(6, 128, dtype, 6)
    x[0] = 0
    x[1] *= 1e-3
    x[2] *= 1e3
    if dtype == "F32":
        x[3] *= 1e-25
        x[4] *= 1e18
    pos = torch.zeros(6, dtype=torch.int32, device=dev())
    w = torch.ones(128, device=dev())
    out = torch.empty_like(x)
    for eps in (1e-6, 1e-12):
        q.qmoe_rope(ctx, rope, x, q.DTYPE[dtype], 0, 6, 1, 128, pos, w, eps, out, 0)
        want = R.rope_heads(host(x), 128, host(w), eps).reshape(6, 128)
        # (an approximate root of two steps outside 1e-30 .. 1e30)
        err = np.abs(host(out).astype(np.float64) - want)
        assert (err <= (R.HALF[dtype] * 1.01 + 6 * R.U) * np.abs(want) + (2.0 ** -25 if dtype == "F16" else 1e-44)).all()


@pytest.mark.parametrize("eps", [1e-44, 1e-25, 1e-3, 0.5, 1e10, 3e38])
def test_rope_norm_of_any_eps(q, ctx, eps):
    """eps far from 1, heads far from eps: the same inverse root as from 64 bits, to two steps."""
    rope, _ = make_table(q, ctx, 64, 10)
    x = rand_rows(8, 64, "F32", 16)
    for i, f in enumerate((1e-30, 1e-22, 1e-18, 1e-15, 1.0, 1e10, 1e15, 1e18)):
        x[i] *= f
    pos = torch.zeros(8, dtype=torch.int32, device=dev())
    out = torch.empty_like(x)
    q.qmoe_rope(ctx, rope, x, q.QMOE_F32, 0, 8, 1, 64, pos, torch.ones(64, device=dev()), eps, out, 0)
    d = host(x).astype(np.float64)
    want = d / np.sqrt((d * d).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    assert (np.abs(host(out) - want) <= 6 * R.U * np.abs(want) + 1e-44).all()


@pytest.mark.parametrize("hd,eps,chunks", [(64, 1e-6, 20), (64, 1e-12, 16), (128, 1e-6, 10), (128, 1e-3, 10), (256, 1e-6, 6)])
@pytest.mark.parametrize("constant", [False, True])
def test_rope_roots_are_nearest_or_next_to_a_border(q, ctx, hd, eps, chunks, constant):
    """2^20 F32 heads a chunk at position 0: every inverse root is the fp32 number nearest to the one in 64 bits, or
    the other where that lies within 2^-34 of the border between the two.

    The mean of n squares in two words, relative to it: a square's loss is at most 2^-22 (half a step of a
    power of two up to four times the sum) and is rounded itself (n 2^-46); eight of one sign add up to
    35 2^-46 of rounding in each of n/8 sums (n 4.4 2^-46); pairs, lanes (four levels at most) and the two
    last sums another n 2^-46 each, 7 at most.  n 12.4 2^-46 is below 2^-34 at n = 256; half of it in the
    root, and 2^-44 of its last step.  Constant heads are those where losses have one sign."""
    heads = 1 << 20
    rope, table = make_table(q, ctx, 16, 1)
    g = torch.Generator(device=dev())
    g.manual_seed(hd)
    w, pos = torch.ones(hd, device=dev()), torch.zeros(heads // 16, dtype=torch.int32, device=dev())
    others = 0
    for chunk in range(2 if constant else chunks):
        x = torch.randn(heads, 1 if constant else hd, device=dev(), generator=g) * torch.exp(2 * torch.randn(heads, 1, device=dev(), generator=g))
        x = x.expand(heads, hd).contiguous()
        out = torch.empty_like(x)
        q.qmoe_rope(ctx, rope, x, q.QMOE_F32, 0, heads // 16, 16, hd, pos, w, eps, out, 0)
        d = x.double()
        r = 1 / torch.sqrt((d * d).sum(1, keepdim=True) / hd + float(np.float32(eps)))
        low, high = (x * (r * (1 + o)).float() for o in (-2.0 ** -34, 2.0 ** -34))
        assert ((out == low).all(1) | (out == high).all(1)).all(), chunk
        others += int((out != x * r.float()).any(1).sum())
    print("not the nearest:", others, "of", (chunk + 1) * heads)
    assert (table[0, 0] == 1).all() and not table[0, 1].any()


# ---------------------------------------------------------------------------- the append

APPEND_CASES = [  # tokens, heads, kv heads, hd, rot, layout, dtype, q norm, k norm, page, padded, with q
    (1, 32, 4, 128, 128, "half", "BF16", True, True, 16, 0, True), (64, 32, 4, 128, 128, "half", "BF16", True, True, 16, 5, True),
    (7, 6, 2, 64, 32, "interleaved", "F32", False, True, 32, 2, True), (33, 10, 10, 256, 64, "half", "F16", True, False, 128, 0, True),
    (500, 8, 1, 64, 64, "half", "F32", True, True, 64, 3, True), (19, 28, 4, 128, 96, "half", "F32", False, False, 256, 1, False),
    (129, 40, 8, 128, 64, "interleaved", "F16", True, True, 16, 0, True), (2, 64, 4, 256, 256, "interleaved", "BF16", False, True, 16, 0, False)]


def append_rig(q, T, heads, kv, hd, page, dtype, seed=0, stream=None):
    pages = -(-T // page) + 3
    stream = stream or torch.cuda.current_stream(dev())
    h = q.qmoe_kv4_create(q.make_kv4_config(heads, kv, hd, page, pages, 4, T, pages, stream.cuda_stream))
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    bufs = []
    for _ in "kv":
        bufs += [torch.full((pages + 1, kv, page, hd // 2), 0xA5, dtype=torch.uint8, device=dev()),
                 torch.full((pages + 1, kv, page, hd // 16), 0x5A, dtype=torch.uint8, device=dev())]
    glob = (torch.rand(2, kv, device=dev(), generator=g) + 0.5) * 8 / 2688
    cache = q.make_kv4_cache(bufs[0], bufs[1], bufs[2], bufs[3], glob[0], glob[1])
    slots = torch.randperm(pages * page, device=dev(), generator=g)[:T].contiguous()
    return h, cache, bufs, glob, slots, pages


@pytest.mark.parametrize("T,heads,kv,hd,rot,layout,dtype,qn,kn,page,padded,with_q", APPEND_CASES)
@pytest.mark.parametrize("fused", [True, False])
def test_append_rope(q, ctx, T, heads, kv, hd, rot, layout, dtype, qn, kn, page, padded, with_q, fused):
    h, cache, bufs, glob, slots, pages = append_rig(q, T, heads, kv, hd, page, dtype, T)
    n_pos = 9000
    rope, table = make_table(q, ctx, rot, n_pos, layout, "parts", factor=3.0, orig_ctx=2000.0)
    nq, nk = heads * hd, kv * hd
    rows = rand_rows(T, nq + 2 * nk, dtype, 21)
    parts = rows[:, :nq], rows[:, nq:nq + nk], rows[:, nq + nk:]
    if not fused:
        parts = tuple(p.contiguous() for p in parts)
    x, k, v = parts
    pos = torch.randint(0, n_pos, (T,), device=dev(), dtype=torch.int32)
    if padded:
        pos[T - padded:] = -1
        slots[T - padded:] = -1
    if T > 30:
        slots[11] = -1                                       # turned, its values given, but not stored
    w = [1 + 0.3 * torch.randn(hd, device=dev()) if on else None for on in (qn and with_q, kn)]
    ref = [host(p).astype(np.float32).copy() for p in parts]
    q_out = x if fused else torch.full((T, nq), 7.0, dtype=TORCH[dtype], device=dev())
    before = host(q_out).copy()
    hats = [torch.full((T, nk), 7.0, device=dev()) for _ in "kv"]
    q.qmoe_kv4_append_rope(h, cache, rope, x if with_q else None, k, v, q.DTYPE[dtype], T, x.stride(0) if with_q else 0,
                           k.stride(0), v.stride(0), pos, slots, w[0], w[1], EPS, q_out if with_q else None,
                           q_out.stride(0) if with_q else 0, hats[0], hats[1])
    torch.cuda.synchronize()
    assert q.qmoe_kv4_get_status(h) == q.QMOE_OK, q.qmoe_kv4_last_error(h)
    ph, sh = host(pos), host(slots)
    live = ph >= 0
    cs = host(table)[np.maximum(ph, 0)]
    if with_q:
        want = R.rope(R.rope_heads(ref[0], hd, None if w[0] is None else host(w[0]), EPS), cs, rot, layout).reshape(T, nq)
        want = host(torch.from_numpy(want).to(TORCH[dtype]))
        assert np.array_equal(host(q_out)[live], want[live])
    assert np.array_equal(host(q_out)[~live], before[~live]) or not with_q
    turned = (R.rope(R.rope_heads(ref[1], hd, None if w[1] is None else host(w[1]), EPS), cs, rot, layout),
              ref[2].reshape(T, kv, hd))
    for i, rows64 in enumerate(turned):
        codes, scales, val = K4.quantise(rows64, host(glob[i]))
        want_c = np.full(tuple(bufs[2 * i].shape), 0xA5, np.uint8)
        want_s = np.full(tuple(bufs[2 * i + 1].shape), 0x5A, np.uint8)
        for t in range(T):
            if live[t] and sh[t] >= 0:
                want_c[sh[t] // page, :, sh[t] % page] = codes[t]
                want_s[sh[t] // page, :, sh[t] % page] = scales[t]
        assert np.array_equal(host(bufs[2 * i + 1]), want_s)
        assert np.array_equal(host(bufs[2 * i]), want_c)
        hat = host(hats[i]).astype(np.float64)
        assert (np.abs(hat - val.reshape(T, nk))[live] <= 2 * R.U * np.abs(val.reshape(T, nk))[live]).all()
        assert (hat[~live] == 7).all()
    q.qmoe_kv4_destroy(h)


def test_append_rope_without_turning_is_the_append(q, ctx):
    """At position 0 without norms the rows are as they were: codes and scales are qmoe_kv4_append's."""
    T, kv, hd = 77, 4, 128
    h, cache, bufs, glob, slots, pages = append_rig(q, T, 8, kv, hd, 32, "BF16", 4)
    rope, _ = make_table(q, ctx, 128, 4)
    k, v = rand_rows(T, kv * hd, "BF16", 31), rand_rows(T, kv * hd, "BF16", 32)
    q.qmoe_kv4_append(h, cache, k, v, q.QMOE_BF16, T, 0, 0, slots)
    torch.cuda.synchronize()
    want = [b.clone() for b in bufs]
    for b in bufs:
        b.fill_(0)
    pos = torch.zeros(T, dtype=torch.int32, device=dev())
    q.qmoe_kv4_append_rope(h, cache, rope, None, k, v, q.QMOE_BF16, T, 0, 0, 0, pos, slots, None, None, 0.0, None, 0)
    torch.cuda.synchronize()
    at, off = slots // 32, slots % 32
    for a, b in zip(want, bufs):
        assert torch.equal(a[at, :, off], b[at, :, off])
    q.qmoe_kv4_destroy(h)


def test_append_rope_slots_and_positions_out_of_range(q, ctx):
    T, kv, hd = 6, 2, 64
    h, cache, bufs, glob, slots, pages = append_rig(q, T, 4, kv, hd, 16, "F32", 8)
    rope, _ = make_table(q, ctx, 64, 50)
    k, v = rand_rows(T, kv * hd, "F32", 1), rand_rows(T, kv * hd, "F32", 2)
    x = rand_rows(T, 4 * hd, "F32", 3)
    for bad_slot, bad_pos in ((pages * 16, None), (2 ** 62, None), (None, 50), (None, 2 ** 31 - 1)):
        for b, val in zip(bufs, (0xA5, 0x5A, 0xA5, 0x5A)):
            b.fill_(val)
        s, p = slots.clone(), torch.arange(T, device=dev(), dtype=torch.int32)
        if bad_slot is not None:
            s[2] = bad_slot
        else:
            p[2] = bad_pos
        out = torch.full_like(x, 7.0)
        q.qmoe_kv4_append_rope(h, cache, rope, x, k, v, q.QMOE_F32, T, 0, 0, 0, p, s, None, None, 0.0, out, 0)
        assert q.qmoe_kv4_get_status(h) == 8
        assert q.qmoe_kv4_get_status(h) == q.QMOE_OK
        assert (out[2] == 7).all() == (bad_pos is not None) and not (out[3] == 7).any()
        assert (bufs[0][slots[2] // 16, :, slots[2] % 16] == 0xA5).all()     # its own slot was not written
        assert not (bufs[1][slots[3] // 16, :, slots[3] % 16] == 0x5A).all()
    q.qmoe_kv4_destroy(h)


# ---------------------------------------------------------------------------- refusals

def refused(q, status, f, *args):
    with pytest.raises(q.QmoeError) as e:
        f(*args)
    assert e.value.status == status, str(e.value)
    assert len(str(e.value)) > 20


INVALID, MISALIGNED, SHAPE = 1, 2, 4


def test_rmsnorm_refusals(q, ctx):
    x, r, y = (torch.zeros(4, 128, device=dev()) for _ in range(3))
    w, c, s = torch.ones(128, device=dev()), torch.zeros(4, 128, dtype=torch.uint8, device=dev()), torch.zeros(4, device=dev())
    ok = dict(x=x, x_t=0, xs=0, r=r, r_t=0, rs=0, sum=None, w=w, eps=EPS, n=4, d=128, y=y, y_t=0, ys=0, sc=None)

    def call(**k):
        q.qmoe_rmsnorm(ctx, *{**ok, **k}.values())

    call()
    for status, k in [(INVALID, dict(x=None)), (INVALID, dict(y=None)), (SHAPE, dict(n=0)), (SHAPE, dict(n=(1 << 24) + 1)),
                      (SHAPE, dict(d=0)), (SHAPE, dict(d=120)), (SHAPE, dict(d=32784)), (INVALID, dict(x_t=3)),
                      (INVALID, dict(r_t=3)), (INVALID, dict(y_t=4)), (SHAPE, dict(xs=64)), (MISALIGNED, dict(xs=130)),
                      (MISALIGNED, dict(x=x.data_ptr() + 4)), (MISALIGNED, dict(r=r.data_ptr() + 8)), (SHAPE, dict(rs=-128)),
                      (MISALIGNED, dict(w=w.data_ptr() + 4)), (INVALID, dict(eps=0.0)), (INVALID, dict(eps=-1.0)),
                      (INVALID, dict(eps=float("inf"))), (INVALID, dict(eps=float("nan"))), (INVALID, dict(r=None, sum=y)),
                      (INVALID, dict(sum=y)), (INVALID, dict(sc=s)), (INVALID, dict(y_t=3, y=c)),
                      (SHAPE, dict(y_t=3, y=c, sc=s, ys=256)), (INVALID, dict(y=r)), (INVALID, dict(y=x, ys=256)),
                      (INVALID, dict(y_t=3, y=x, sc=s)), (INVALID, dict(y=x, y_t=1)), (INVALID, dict(sum=x, rs=132)),
                      (MISALIGNED, dict(y=y.data_ptr() + 4)), (MISALIGNED, dict(y_t=3, y=c.data_ptr() + 1, sc=s))]:
        refused(q, status, lambda: call(**k))
    call(w=None)


def test_quantize_refusals(q, ctx):
    x, c, s = torch.zeros(4, 256, device=dev()), torch.zeros(4, 256, dtype=torch.uint8, device=dev()), torch.zeros(4, 2, device=dev())
    ok = dict(x=x, t=0, xs=0, n=4, d=256, c=c, s=s)

    def call(**k):
        q.qmoe_fp8_quantize(ctx, *{**ok, **k}.values())

    call()
    for status, k in [(INVALID, dict(x=None)), (INVALID, dict(c=None)), (INVALID, dict(s=None)), (SHAPE, dict(n=0)),
                      (SHAPE, dict(d=8)), (SHAPE, dict(d=250)), (SHAPE, dict(d=1 << 16)), (INVALID, dict(t=3)),
                      (SHAPE, dict(xs=128)), (MISALIGNED, dict(xs=258)), (MISALIGNED, dict(c=c.data_ptr() + 8)),
                      (MISALIGNED, dict(s=s.data_ptr() + 2)), (INVALID, dict(c=x))]:
        refused(q, status, lambda: call(**k))


def test_linear_refusals(q, ctx):
    T, K, N = 4, 256, 64
    d = [torch.from_numpy(a).to(dev()) for a in linear_inputs(T, K, N, 1)]
    out = torch.zeros(T, N, device=dev())
    b = torch.zeros(N, device=dev())
    ok = dict(x=d[0], xs=d[1], T=T, K=K, w=d[2], ws=d[3], N=N, b=b, act=0, r=None, rs=0, o=out, ot=0, os=0)

    def call(**k):
        q.qmoe_linear_fp8(ctx, *{**ok, **k}.values())

    call()
    for status, k in [(INVALID, dict(x=None)), (INVALID, dict(xs=None)), (INVALID, dict(w=None)), (INVALID, dict(ws=None)),
                      (INVALID, dict(o=None)), (SHAPE, dict(T=0)), (SHAPE, dict(T=-1)), (SHAPE, dict(N=0)), (SHAPE, dict(K=8)),
                      (SHAPE, dict(K=250)), (SHAPE, dict(K=(1 << 20) + 16)), (INVALID, dict(act=4)), (INVALID, dict(act=-1)),
                      (INVALID, dict(ot=3)), (MISALIGNED, dict(x=d[0].data_ptr() + 8)), (MISALIGNED, dict(w=d[2].data_ptr() + 1)),
                      (MISALIGNED, dict(b=b.data_ptr() + 2)), (MISALIGNED, dict(xs=d[1].data_ptr() + 2)), (SHAPE, dict(os=32)),
                      (MISALIGNED, dict(os=66)), (MISALIGNED, dict(N=63)), (INVALID, dict(r=out, rs=128)),
                      (MISALIGNED, dict(r=out.data_ptr() + 4)), (INVALID, dict(o=d[0])), (SHAPE, dict(os=1 << 38))]:
        refused(q, status, lambda: call(**k))
    call(b=None, r=out)


def test_rope_refusals(q, ctx):
    table = torch.zeros(10, 2, 32, device=dev())
    x, pos, w = torch.zeros(4, 128, device=dev()), torch.zeros(4, dtype=torch.int32, device=dev()), torch.ones(64, device=dev())

    def made(rot=64, base=1e4, n_pos=10, t=table, **k):
        q.qmoe_rope_table(ctx, q.make_rope(rot, base, n_pos, t, **k))

    made()
    for status, k in [(SHAPE, dict(rot=0)), (SHAPE, dict(rot=24)), (SHAPE, dict(rot=272)), (SHAPE, dict(n_pos=0)),
                      (INVALID, dict(base=1.0)), (INVALID, dict(base=float("inf"))), (INVALID, dict(t=None)),
                      (MISALIGNED, dict(t=table.data_ptr() + 8)), (INVALID, dict(layout=2)), (INVALID, dict(scaling=3)),
                      (INVALID, dict(scaling=1, factor=0.0)), (INVALID, dict(scaling=2, factor=2.0)),
                      (INVALID, dict(scaling=2, factor=2.0, orig_ctx=8.0, beta_fast=1.0)), (INVALID, dict(mscale=-1.0)),
                      (INVALID, dict(mscale=float("nan")))]:
        refused(q, status, lambda: made(**k))
    rope = q.make_rope(64, 1e4, 10, table)
    out = torch.zeros_like(x)
    ok = dict(rope=rope, x=x, t=0, xs=0, T=4, h=2, hd=64, pos=pos, w=w, eps=EPS, out=out, os=0)

    def call(**k):
        q.qmoe_rope(ctx, *{**ok, **k}.values())

    call()
    for status, k in [(INVALID, dict(x=None)), (INVALID, dict(pos=None)), (INVALID, dict(out=None)), (SHAPE, dict(T=0)),
                      (SHAPE, dict(h=0)), (SHAPE, dict(h=1025)), (SHAPE, dict(hd=96)), (SHAPE, dict(hd=32)), (INVALID, dict(t=3)),
                      (SHAPE, dict(rope=q.make_rope(128, 1e4, 10, table))), (MISALIGNED, dict(xs=130)), (SHAPE, dict(os=64)),
                      (INVALID, dict(out=x, os=256)), (INVALID, dict(eps=0.0)), (MISALIGNED, dict(w=w.data_ptr() + 4)),
                      (MISALIGNED, dict(pos=pos.data_ptr() + 2))]:
        refused(q, status, lambda: call(**k))
    call(w=None, eps=0.0, out=x)


def test_append_rope_refusals(q, ctx):
    T, heads, kv, hd = 4, 4, 2, 64
    h, cache, bufs, glob, slots, pages = append_rig(q, T, heads, kv, hd, 16, "F32")
    rope, table = make_table(q, ctx, 64, 10)
    x, k, v = (torch.zeros(T, n * hd, device=dev()) for n in (heads, kv, kv))
    pos, w = torch.zeros(T, dtype=torch.int32, device=dev()), torch.ones(hd, device=dev())
    out = torch.zeros_like(x)
    ok = dict(cache=cache, rope=rope, q=x, k=k, v=v, t=0, T=T, qs=0, ks=0, vs=0, pos=pos, slots=slots, qn=w, kn=w, eps=EPS,
              out=out, os=0, kh=None, vh=None)

    def call(**m):
        q.qmoe_kv4_append_rope(h, *{**ok, **m}.values())

    call()
    none = q.make_kv4_cache(None, *bufs[1:], glob[0], glob[1])
    for status, m in [(INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(pos=None)), (INVALID, dict(slots=None)),
                      (INVALID, dict(q=None)), (INVALID, dict(out=None)), (INVALID, dict(q=None, out=None)), (SHAPE, dict(T=0)),
                      (SHAPE, dict(T=5)), (INVALID, dict(t=3)), (SHAPE, dict(rope=q.make_rope(48, 1e4, 10, table))),
                      (SHAPE, dict(rope=q.make_rope(128, 1e4, 10, table))), (SHAPE, dict(ks=64)), (MISALIGNED, dict(vs=130)),
                      (MISALIGNED, dict(q=x.data_ptr() + 4)), (INVALID, dict(out=x, os=512)), (INVALID, dict(out=k)),
                      (INVALID, dict(eps=0.0)), (MISALIGNED, dict(kn=w.data_ptr() + 4)), (INVALID, dict(cache=none)),
                      (MISALIGNED, dict(slots=slots.data_ptr() + 4)), (MISALIGNED, dict(kh=k.data_ptr() + 4))]:
        refused(q, status, lambda: call(**m))
    call(q=None, out=None, qn=None)
    assert q.qmoe_kv4_get_status(h) == q.QMOE_OK
    q.qmoe_kv4_destroy(h)


# ---------------------------------------------------------------------------- streams, graphs, long strides

LINEAR_PATHS = [(1, 512, 300), (12, 256, 200), (30, 640, 260), (64, 2048, 700), (150, 1024, 2048), (700, 512, 900), (1500, 768, 4096)]


@pytest.mark.parametrize("T,K,N", LINEAR_PATHS)
def test_linear_in_a_graph_follows_its_inputs(q, T, K, N):
    """Captured once, replayed over other codes and scales: the results of calls of their own."""
    st = torch.cuda.Stream()
    ctx = make_ctx(q, st)
    sets = []
    for seed in (1, 2):
        xc, xs, wc, ws = (torch.from_numpy(a).to(dev()) for a in linear_inputs(T, K, N, seed))
        sets.append((xc, xs, wc, ws))
    buf = [t.clone() for t in sets[0]]
    wide = -(-N // 8) * 8
    out = torch.zeros(T, wide, device=dev())[:, :N]
    torch.cuda.synchronize()

    def call():
        q.qmoe_linear_fp8(ctx, buf[0], buf[1], T, K, buf[2], buf[3], N, None, q.ACT["SILU"], None, 0, out, q.QMOE_F32, wide)

    with torch.cuda.stream(st):
        call()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):                               # kernels that overlap the ones before
                call()
        got = []
        for s in (sets[1], sets[0], sets[1]):
            for b, t in zip(buf, s):
                b.copy_(t)
            out.fill_(0)
            g.replay()
            got.append(out.clone())
        for s, o in zip((sets[1], sets[0], sets[1]), got):
            for b, t in zip(buf, s):
                b.copy_(t)
            out.fill_(0)
            call()
            assert torch.equal(out, o)
        st.synchronize()
    assert q.qmoe_get_status(ctx) == q.QMOE_OK
    q.qmoe_destroy(ctx)


def test_two_contexts_on_two_streams(q):
    """Products, norms and turned rows of two contexts that run at the same time are those of each alone."""
    T, K, N, dim = 600, 1024, 1300, 2048
    streams = [torch.cuda.Stream() for _ in range(2)]
    ctxs = [make_ctx(q, s) for s in streams]
    rope, _ = make_table(q, ctxs[0], 128, 4000)
    work = []
    for i in range(2):
        d = [torch.from_numpy(a).to(dev()) for a in linear_inputs(T, K, N, 40 + i)]
        x, pos = rand_rows(3000, dim, "BF16", 50 + i), torch.randint(0, 4000, (3000,), device=dev(), dtype=torch.int32)
        work.append((d, x, pos, torch.zeros(T, 1304, device=dev())[:, :N], torch.zeros(3000, dim, dtype=torch.uint8, device=dev()),
                     torch.zeros(3000, dim // 128, device=dev()), torch.zeros(3000, dim, dtype=torch.bfloat16, device=dev())))
    torch.cuda.synchronize()

    def go(i):
        d, x, pos, out, codes, scale, turned = work[i]
        q.qmoe_linear_fp8(ctxs[i], d[0], d[1], T, K, d[2], d[3], N, None, 0, None, 0, out, q.QMOE_F32, 1304)
        q.qmoe_rmsnorm(ctxs[i], x, q.QMOE_BF16, 0, None, 0, 0, None, None, EPS, 3000, dim, codes, q.QMOE_E4M3, 0, scale)
        q.qmoe_rope(ctxs[i], rope, x, q.QMOE_BF16, 0, 3000, dim // 128, 128, pos, None, 0.0, turned, 0)

    alone = []
    for i in range(2):
        go(i)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in work[i][3:]])
        for t in work[i][3:]:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            go(i)
    torch.cuda.synchronize()
    for i in range(2):
        assert q.qmoe_get_status(ctxs[i]) == q.QMOE_OK
        for a, b in zip(alone[i], work[i][3:]):
            assert torch.equal(a, b)
        q.qmoe_destroy(ctxs[i])


def test_rows_further_apart_than_32_bits(q, ctx):
    """Three rows 2^30 + 8 F32 elements apart: offsets past 2^32 bytes, and past 2^31 elements."""
    stride, dim = (1 << 30) + 8, 128
    buf = torch.empty(2 * stride + dim, device=dev())
    x = torch.as_strided(buf, (3, dim), (stride, 1))
    x.copy_(rand_rows(3, dim, "F32", 60))
    want_c, want_s = R.quantise8(host(x))
    codes, scale = torch.empty(3, dim, dtype=torch.uint8, device=dev()), torch.empty(3, 1, device=dev())
    q.qmoe_fp8_quantize(ctx, x, q.QMOE_F32, stride, 3, dim, codes, scale)
    assert np.array_equal(host(codes), want_c) and np.array_equal(host(scale), want_s)
    rope, table = make_table(q, ctx, 64, 100)
    pos = torch.tensor([3, 99, 50], dtype=torch.int32, device=dev())
    want = R.rope(host(x).reshape(3, 2, 64), host(table)[host(pos)], 64, "half").reshape(3, dim)
    q.qmoe_rope(ctx, rope, x, q.QMOE_F32, stride, 3, 2, 64, pos, None, 0.0, x, stride)
    assert np.array_equal(host(x), want)
    _, y = R.rmsnorm(host(x), None, None, EPS)
    q.qmoe_rmsnorm(ctx, x, q.QMOE_F32, stride, None, 0, 0, None, None, EPS, 3, dim, x, q.QMOE_F32, stride, None)
    assert (np.abs(host(x) - y) <= NORM_ERR * np.abs(y)).all()
    # products into rows as far apart, from the kernel for few tokens
    d = [torch.from_numpy(a).to(dev()) for a in linear_inputs(3, 256, 100, 61)]
    want, size = R.linear(*linear_inputs(3, 256, 100, 61), None, "NONE", host(x)[:, :100])
    q.qmoe_linear_fp8(ctx, d[0], d[1], 3, 256, d[2], d[3], 100, None, 0, x, stride, x, q.QMOE_F32, stride)
    assert (np.abs(host(x)[:, :100] - want) <= linear_bound(size, 2, want, 0, "NONE") + 2 * R.U * np.abs(want)).all()


def test_linear_rows_far_apart_on_pairs_of_ctas(q, ctx):
    T, K, N, stride = 300, 128, 40, 1 << 23                 # the last rows' offsets are past 2^31 elements
    buf = torch.empty((T - 1) * stride + N, dtype=torch.bfloat16, device=dev())
    out = torch.as_strided(buf, (T, N), (stride, 1))
    near = torch.empty(T, N, dtype=torch.bfloat16, device=dev())
    d = [torch.from_numpy(a).to(dev()) for a in linear_inputs(T, K, N, 62)]
    for o in (out, near):
        q.qmoe_linear_fp8(ctx, d[0], d[1], T, K, d[2], d[3], N, None, 0, None, 0, o, q.QMOE_BF16, o.stride(0))
    assert torch.equal(out, near)


@pytest.mark.parametrize("T", [3, 20, 50, 300])
def test_linear_scales_that_are_not_16_byte_aligned(q, ctx, T):
    K, N = 512, 140
    xc, xs, wc, ws = linear_inputs(T, K, N, 63)
    pad = torch.zeros(T * 4 + 1, device=dev())
    pad[1:] = torch.from_numpy(xs).to(dev()).flatten()
    d = [torch.from_numpy(a).to(dev()) for a in (xc, wc, ws)]
    out = torch.empty(T, N, device=dev())
    q.qmoe_linear_fp8(ctx, d[0], pad.data_ptr() + 4, T, K, d[1], d[2], N, None, 0, None, 0, out, q.QMOE_F32, 0)
    ref, size = R.linear(xc, xs, wc, ws, None, "NONE", None)
    assert (np.abs(host(out) - ref) <= linear_bound(size, 4, ref, 0, "NONE")).all()
