"""The plain forms of the row operators against definitions and library functions (CPU)."""
import os
import re

import numpy as np
import pytest
import torch

from tests import rows_ref as R


def test_every_code_comes_back():
    v = R.GRID[np.newaxis, :]                            # 0 .. 448: the scale is 1
    c, s = R.quantise8(np.concatenate([v, -v], 0))
    assert (s == 1).all()
    assert np.array_equal(c[0], np.arange(127)) and np.array_equal(c[1, 1:], 128 + np.arange(1, 127))


def test_quantise8_is_the_nearest_and_torchs():
    rng = np.random.default_rng(1)
    y = (rng.normal(size=(7, 400)) * np.exp(rng.normal(size=(7, 1)) * 5)).astype(np.float32)
    y[3, 128:256] = 0
    c, s = R.quantise8(y)
    assert s.shape == (7, 4) and s[3, 1] == 0 and not c[3, 128:256].any()
    d = np.repeat(s, 128, 1)[:, :400]
    q = np.where(d > 0, y / np.where(d > 0, d, 1), 0).astype(np.float32)
    t = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(c & 127, t & 127)
    assert (np.abs(R.values8(c, s) - y) <= np.maximum(np.abs(y) * 2.0 ** -4, d * 2.0 ** -10) * (1 + 4 * R.U)).all()


def test_linear_is_the_product_of_the_values():
    rng = np.random.default_rng(2)
    xc, wc = rng.integers(0, 127, (3, 144), dtype=np.uint8), rng.integers(0, 127, (130, 144), dtype=np.uint8)
    xs, ws = rng.random((3, 2)).astype(np.float32), rng.random((2, 2)).astype(np.float32)
    z, _ = R.linear(xc, xs, wc, ws, None, "NONE", None)
    at = [(0, 0), (2, 127), (1, 128), (2, 129)]
    for t, n in at:
        want = sum(R.GRID[xc[t, k]] * float(xs[t, k // 128]) * R.GRID[wc[n, k]] * float(ws[n // 128, k // 128]) for k in range(144))
        assert abs(z[t, n] - want) <= 1e-12 * abs(want)


@pytest.mark.parametrize("act,f", [("RELU", torch.relu), ("SILU", torch.nn.functional.silu), ("GELU", torch.nn.functional.gelu)])
def test_activations_are_torchs(act, f):
    z = np.linspace(-9, 9, 501)
    assert np.allclose(R.activate(z, act), f(torch.from_numpy(z)).numpy(), rtol=1e-12, atol=1e-15)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_turns_pairs_and_keeps_their_distance(layout):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(4, 2, 64)).astype(np.float32)
    f, m = R.rope_freq(32, 1e4)
    pos = np.array([0, 1, 77, 100000])
    ang = pos[:, None] * f
    cs = np.stack([np.cos(ang) * m, np.sin(ang) * m], 1).astype(np.float32)
    y = R.rope(x, cs, 32, layout)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
    a, b = (slice(0, 16), slice(16, 32)) if layout == "half" else (slice(0, 32, 2), slice(1, 32, 2))
    z, w = x[..., a] + 1j * x[..., b], y[..., a] + 1j * y[..., b]
    assert np.allclose(w, z * np.exp(1j * ang)[:, None], atol=4e-6)


def test_frequencies_by_parts_are_between_plain_and_linear():
    plain, lin = R.rope_freq(128, 1e6)[0], R.rope_freq(128, 1e6, "linear", 4.0)[0]
    parts, m = R.rope_freq(128, 1e6, "parts", 4.0, 32768.0)
    assert np.array_equal(lin, plain / 4) and abs(m - (0.1 * np.log(4) + 1)) < 1e-15
    assert parts[0] == plain[0] and parts[-1] == lin[-1]
    assert (parts <= plain).all() and (parts >= lin).all() and (np.diff(parts) < 0).all()


def test_rmsnorm_of_constant_rows():
    h, y = R.rmsnorm(np.full((2, 32), 3.0), np.full((2, 32), -1.0), None, 1e-30)
    assert (h == 2).all() and np.allclose(y, 1, rtol=1e-15)


def test_calls_select_their_device_before_they_reach_it():
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                            "quantized_mixture_experts_f32_gb300", "csrc", "rows_api.cu")).read()
    bodies = {m.group(1): m.group(2) for m in re.finditer(r"^[\w ]+?[ *](\w+)\([^;{]*?\) \{\n(.*?)^\}", src, flags=re.S | re.M)}
    names = [n for n in bodies if re.search(r"\blaunch_\w+\(", bodies[n])]
    assert len(names) == 5                     # rmsnorm and quantise share one
    for n in names:
        guard = re.search(r"\bOnDevice dev\(\w+\.device\);", bodies[n])
        assert guard and guard.start() < re.search(r"\blaunch_\w+\(", bodies[n]).start(), n


def test_calls_without_a_handle_are_refused():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_mixture_experts_f32_gb300 as q
    rope = q.make_rope(64, 1e4, 1, 16)
    assert q.lib.qmoe_rmsnorm(None, 16, 0, 0, None, 0, 0, None, None, 1.0, 1, 16, 16, 0, 0, None) == 1
    assert q.lib.qmoe_fp8_quantize(None, 16, 0, 0, 1, 16, 16, 16) == 1
    assert q.lib.qmoe_linear_fp8(None, 16, 16, 1, 16, 16, 16, 1, None, 0, None, 0, 16, 0, 0) == 1
    assert q.lib.qmoe_rope_table(None, rope) == 1
    assert q.lib.qmoe_rope(None, rope, 16, 0, 0, 1, 1, 64, 16, None, 1.0, 16, 0) == 1
    cache = q.make_kv4_cache(16, 16, 16, 16, 16, 16)
    assert q.lib.qmoe_kv4_append_rope(None, cache, rope, None, 16, 16, 0, 1, 0, 0, 0, 16, 16, None, None, 1.0, None, 0, None, None) == 1


def test_cluster_barriers_are_met_by_whole_warps():
    """barrier.cluster's aligned forms want every lane of a warp at the same instruction: a lane that had something
    of its own to do (the status of a wait that ran out) meets the others first."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_mixture_experts_f32_gb300", "csrc")
    seen = 0
    for f in os.listdir(csrc):
        src = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, f)).read())
        for m in re.finditer(r'asm volatile\("barrier\.cluster\.arrive\.aligned', src):
            assert re.search(r"__syncwarp\(\);\s*$", src[:m.start()]), f
            seen += 1
    assert seen == 1
