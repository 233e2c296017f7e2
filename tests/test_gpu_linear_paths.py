"""qmoe_linear_fp8 on pairs of CTAs: both tiles, k shared or not, one and several tiles a pair, every type and
activation of each, against the plain form in 64 bits.  Each size says which kernel it is for, and the test asks
whether it still goes there."""
import os
import subprocess
import sys
import time

import numpy as np
import pytest
import torch

from tests import rows_ref as R
from tests.gpu_util import dev
from tests.test_gpu_rows import assert_guard, ctx, guarded, host, linear_bound, linear_inputs, make_ctx, q, run_linear  # noqa: F401

pytestmark = pytest.mark.gpu

# sizes for each kernel: tokens, k, features, (tile, pairs that share its k)
T128, T256, SHARED = (300, 1024, 1003, (128, 1)), (513, 912, 5003, (256, 1)), (300, 2048, 1003, (128, 2))
FEW = (33, 256, 200, (0, 1))


def check_path(q, T, K, N, want, per_pair=0):  # noqa: F811
    sms = torch.cuda.get_device_properties(dev()).multi_processor_count
    assert q.qmoe_debug_linear_choice(sms, T, K, N) == want
    if per_pair:
        assert -(-T // 256) * -(-N // want[0]) > (per_pair - 1) * (sms // 2)


# every kernel there is: a tile's two blocks of features have scales of their own, tokens and features are cut
@pytest.mark.parametrize("size", [T128, T256, SHARED], ids=["128", "256", "shared"])
@pytest.mark.parametrize("act", ["NONE", "RELU", "SILU", "GELU"])
@pytest.mark.parametrize("out_t,residual", [("F32", "apart"), ("F16", "place"), ("BF16", "apart")])
def test_every_kernel(q, ctx, size, act, out_t, residual):  # noqa: F811
    T, K, N, want = size
    check_path(q, T, K, N, want)
    run_linear(q, ctx, T, K, N, out_t, act, True, residual, T + K + N, 8)


PATHS = [  # tokens, K, N, (tile, shared by), tiles that some pair takes, out, act, bias, residual, stride beyond
    (1281, 464, 4999, (256, 1), 2, "F32", "NONE", True, "place", 0),
    (1281, 512, 4999, (256, 1), 2, "BF16", "GELU", True, "apart", 16),
    (1100, 1040, 7001, (256, 1), 2, "F16", "NONE", False, "place", 0),
    (2049, 272, 5400, (256, 1), 3, "F32", "SILU", False, "apart", 4),
    (2500, 528, 4867, (256, 1), 3, "BF16", "RELU", True, "place", 0),
    (2304, 640, 5377, (256, 1), 3, "F16", "NONE", True, "", 8),
    (700, 1024, 4500, (256, 1), 1, "BF16", "NONE", False, "", 0),
    (3000, 16, 1500, (128, 1), 2, "F32", "NONE", True, "apart", 0),
    (2100, 128, 4001, (128, 1), 4, "BF16", "SILU", False, "place", 0),
    (2500, 256, 1101, (128, 1), 2, "F16", "GELU", True, "apart", 8),
    (3000, 640, 2051, (128, 1), 3, "F32", "RELU", True, "place", 4),
    (1300, 400, 3001, (128, 1), 2, "BF16", "NONE", False, "", 0),
    (5000, 144, 771, (128, 1), 2, "F16", "NONE", True, "place", 0),
    (2049, 528, 4099, (128, 1), 4, "F32", "GELU", False, "apart", 0),
    (4000, 48, 900, (128, 1), 2, "F32", "SILU", True, "", 0),
    (300, 1536, 1003, (128, 3), 0, "F16", "SILU", True, "apart", 0),
    (257, 4096, 700, (128, 4), 0, "BF16", "GELU", True, "place", 8),
    (300, 2048, 1003, (128, 2), 0, "F32", "NONE", False, "", 0)]


@pytest.mark.parametrize("T,K,N,want,per_pair,out_t,act,bias,residual,pad", PATHS)
def test_paths(q, ctx, T, K, N, want, per_pair, out_t, act, bias, residual, pad):  # noqa: F811
    check_path(q, T, K, N, want, per_pair)
    run_linear(q, ctx, T, K, N, out_t, act, bias, residual, T + K + N, pad)


@pytest.mark.parametrize("size", [FEW, T128, T256, SHARED], ids=["few", "128", "256", "shared"])
def test_not_finite_stays_in_its_row_and_column(q, ctx, size):  # noqa: F811
    T, K, N, want = size
    check_path(q, T, K, N, want)
    xc, xs, wc, ws = linear_inputs(T, K, N, 19)
    xc[3, 200], xs[5, 0], wc[7, 50] = 0x7f, np.inf, 0xff
    b = np.random.default_rng(4).normal(size=N).astype(np.float32)
    b[9] = np.inf
    d = [torch.from_numpy(a).to(dev()) for a in (xc, xs, wc, ws, b)]
    out, guard = guarded(T, N, torch.float32, -(-N // 4) * 4)
    rows, cols = np.arange(T)[:, None], np.arange(N)[None]
    kept = (rows != 3) & (rows != 5) & (cols != 7) & (cols != 9)
    with np.errstate(invalid="ignore"):
        z, size = R.linear(xc, xs, wc, ws, b, "NONE", None)
    for act in ("NONE", "RELU", "SILU", "GELU"):
        out.fill_(7.0)
        q.qmoe_linear_fp8(ctx, d[0], d[1], T, K, d[2], d[3], N, d[4], q.ACT[act], None, 0, out, q.QMOE_F32, out.stride(0))
        o = host(out)
        assert np.isnan(o[3]).all() and np.isnan(o[:, 7]).all()
        assert (np.delete(o[:, 9], (3, 5)) == np.inf).all()
        ref = R.activate(z[kept], act)
        assert (np.abs(o[kept] - ref) <= linear_bound(size[kept], -(-K // 128), ref, 0, act)).all()
        assert_guard(guard, T, N)


@pytest.mark.parametrize("size", [(700, 512, 900, (128, 1)), (513, 1024, 5003, (256, 1)), SHARED], ids=["128", "256", "shared"])
def test_scales_that_are_not_16_byte_aligned(q, ctx, size):  # noqa: F811
    """Four blocks' scales are loaded at once where they lie on 16 bytes, else one by one: the same bits."""
    T, K, N, want = size
    check_path(q, T, K, N, want)
    assert -(-K // 128) % 4 == 0
    xc, xs, wc, ws = linear_inputs(T, K, N, 63)
    pad = torch.zeros(xs.size + 1, device=dev())
    pad[1:] = torch.from_numpy(xs).to(dev()).flatten()
    d = [torch.from_numpy(a).to(dev()) for a in (xc, xs, wc, ws)]
    got = []
    for scales in (d[1], pad.data_ptr() + 4):
        out = torch.empty(T, -(-N // 4) * 4, device=dev())[:, :N]
        q.qmoe_linear_fp8(ctx, d[0], scales, T, K, d[2], d[3], N, None, 0, None, 0, out, q.QMOE_F32, out.stride(0))
        got.append(out)
    assert torch.equal(*got)
    ref, size = R.linear(xc, xs, wc, ws, None, "NONE", None)
    assert (np.abs(host(got[1]) - ref) <= linear_bound(size, -(-K // 128), ref, 0, "NONE")).all()


@pytest.mark.parametrize("size,stride", [(T128, 1 << 23), (T256, 1 << 22)], ids=["128", "256"])
def test_rows_far_apart(q, ctx, size, stride):  # noqa: F811
    """In place, the last rows past 2^31 elements, features behind the last whole 16 bytes; what lies behind a row stays."""
    T, K, N, want = size
    check_path(q, T, K, N, want)
    assert (T - 1) * stride + N > 2 ** 31 and N % 8
    buf = torch.empty((T - 1) * stride + N + 64, dtype=torch.bfloat16, device=dev())
    wide = torch.as_strided(buf, (T, N + 64), (stride, 1))
    wide.fill_(7.0)
    out = wide[:, :N]
    xc, xs, wc, ws = linear_inputs(T, K, N, 62)
    d = [torch.from_numpy(a).to(dev()) for a in (xc, xs, wc, ws)]
    bias = torch.randn(N, device=dev())
    res = torch.randn(T, N, device=dev()).to(torch.bfloat16)
    out.copy_(res)
    ref, size = R.linear(xc, xs, wc, ws, host(bias).astype(np.float64), "NONE", host(res))
    q.qmoe_linear_fp8(ctx, d[0], d[1], T, K, d[2], d[3], N, bias, 0, out, stride, out, q.QMOE_BF16, stride)
    assert (np.abs(host(out) - ref) <= linear_bound(size, -(-K // 128), ref, R.HALF["BF16"], "NONE")).all()
    assert (wide[:, N:] == 7).all()


@pytest.mark.parametrize("size", [FEW, T128, T256, SHARED], ids=["few", "128", "256", "shared"])
def test_gelu_is_as_exact_as_it_says(q, ctx, size):  # noqa: F811
    """2e-7 |z|, over a fine grid: one product of ones under a token's scale, a bias a feature, z their rounded sum."""
    T, K, N, want = size
    check_path(q, T, K, N, want)
    xc, wc = torch.zeros(T, K, dtype=torch.uint8, device=dev()), torch.zeros(N, K, dtype=torch.uint8, device=dev())
    xc[:, 5], wc[:, 5] = 0x38, 0x38
    ws = torch.ones(-(-N // 128), -(-K // 128), device=dev())
    out = torch.empty(T, -(-N // 4) * 4, device=dev())[:, :N]
    half = np.geomspace(1e-30, 1e4, N // 2)
    for scales, bias in [(np.linspace(0, 16 / N, T), np.linspace(-8, 8, N)), (np.zeros(T), np.append(half, -half)),
                         (np.geomspace(1e-6, 1, T), np.append(half, -half))]:
        bias = np.resize(bias.astype(np.float32), N)
        xs = torch.zeros(T, -(-K // 128), device=dev())
        xs[:, 0] = torch.from_numpy(scales.astype(np.float32))
        q.qmoe_linear_fp8(ctx, xc, xs, T, K, wc, ws, N, torch.from_numpy(bias).to(dev()), q.ACT["GELU"], None, 0, out, q.QMOE_F32, out.stride(0))
        z = (scales.astype(np.float32)[:, None] + bias[None]).astype(np.float64)      # rounded to fp32 once
        ref = z * 0.5 * torch.erfc(torch.from_numpy(-z / np.sqrt(2))).numpy()
        err = np.abs(host(out) - ref)
        with np.errstate(divide="ignore", invalid="ignore"):
            print("largest error over |z|", np.nanmax(err / np.abs(z)), "absolute below 0", err[z < 0].max())
        assert (err <= 2e-7 * np.abs(z)).all()


# ---------------------------------------------------------------------------- waits that run out

LATE = [(128, 128, 2500, (128, 1)), (1281, 464, 4999, (256, 1)), (3000, 640, 2051, (128, 1)), T128, T256, SHARED,
        (300, 1536, 1003, (128, 3)), (257, 4096, 700, (128, 4))]


@pytest.mark.parametrize("T,K,N,want", LATE)
def test_scales_that_come_late(q, T, K, N, want):  # noqa: F811
    """One CTA's scales later than the limit: the status says so, and the next call on the context is right; later than
    usual within it: nothing but time."""
    check_path(q, T, K, N, want)
    c = make_ctx(q)
    data = linear_inputs(T, K, N, 71)
    d = [torch.from_numpy(a).to(dev()) for a in data]
    res = torch.randn(T, -(-N // 4) * 4, device=dev())[:, :N]
    ref, size = R.linear(*data, None, "NONE", host(res))
    out, guard = guarded(T, N, torch.float32, -(-N // 4) * 4)

    def call():
        out.fill_(7.0)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        q.qmoe_linear_fp8(c, d[0], d[1], T, K, d[2], d[3], N, None, 0, res, res.stride(0), out, q.QMOE_F32, out.stride(0))
        torch.cuda.synchronize()
        return time.perf_counter() - t0

    def right():
        assert q.qmoe_get_status(c) == q.QMOE_OK, q.qmoe_last_error(c)
        assert (np.abs(host(out) - ref) <= linear_bound(size, -(-K // 128), ref, 0, "NONE")).all()
        assert_guard(guard, T, N)

    for wait in (400_000_000, 20_000_000, 250_000_000):
        q.qmoe_debug_stall_linear_next(c, wait)
        took = call()
        print(f"{wait / 1e9} s late: {took:.3f} s")
        assert took > 0.9e-9 * wait
        if wait > 200_000_000:
            assert q.qmoe_get_status(c) == 7 and "status 7" in q.qmoe_last_error(c)
            assert_guard(guard, T, N)
            call()                                       # the hook is spent
        right()
    for bad in (0, 1_000_000_001):
        with pytest.raises(q.QmoeError):
            q.qmoe_debug_stall_linear_next(c, bad)
    assert q.lib.qmoe_debug_stall_linear_next(None, 5) == 1
    q.qmoe_destroy(c)


# ---------------------------------------------------------------------------- the first call

FIRST = """
import sys
import torch
sys.path.insert(0, {root!r})
import quantized_mixture_experts_f32_gb300 as q
from tests.test_gpu_rows import linear_inputs, make_ctx
T, K, N = {size}
st = torch.cuda.Stream()
c, other = make_ctx(q, st), make_ctx(q, st)
d = [torch.from_numpy(a).cuda() for a in linear_inputs(T, K, N, 5)]
out = [torch.zeros(T, -(-N // 4) * 4, device="cuda") for _ in range(3)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=st):
    q.qmoe_linear_fp8(c, d[0], d[1], T, K, d[2], d[3], N, None, 0, None, 0, out[0], 0, out[0].stride(0))
g.replay()
q.qmoe_linear_fp8(c, d[0], d[1], T, K, d[2], d[3], N, None, 0, None, 0, out[1], 0, out[1].stride(0))
q.qmoe_linear_fp8(other, d[0], d[1], T, K, d[2], d[3], N, None, 0, None, 0, out[2], 0, out[2].stride(0))
torch.cuda.synchronize()
assert q.qmoe_get_status(c) == 0 and q.qmoe_get_status(other) == 0
assert out[0].abs().sum() > 0 and torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
print("first call right")
"""


@pytest.mark.parametrize("size", [T128, T256, SHARED], ids=["128", "256", "shared"])
def test_a_kernels_first_call_may_be_captured(q, size):  # noqa: F811
    """A process's first call of a kernel, which sets it up, inside a graph's capture; then calls of two contexts."""
    check_path(q, *size)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, size=size[:3])], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first call right" in r.stdout, r.stderr[-2000:]
