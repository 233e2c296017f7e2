"""CPU: the plain forms the cache's GPU tests compare with, against the pinned oracle and by their
own properties, and the refusals that need no device."""
import ctypes

import numpy as np
import pytest

import oracle
from tests import kv4_ref as R


def test_quantise_matches_the_pinned_quantiser(oracle_lib):
    import synth
    bits = synth.bf16_matrix(5, 48, 128)
    x = (bits.astype(np.uint32) << 16).view(np.float32)
    amax = np.abs(x).max()
    c, s, v = R.quantise(x[:, None, :], np.array([amax / np.float32(2688)], np.float32))
    oc, os_, og = oracle.nvfp4_quantize(bits)
    assert np.array_equal(c[:, 0].ravel(), np.asarray(oc).ravel())
    assert np.array_equal(s[:, 0].ravel(), np.asarray(os_).ravel())
    assert np.array_equal(R.values_of(R.unpack(c), s, np.array([og], np.float32)), v)


def test_e2m1_times_e4m3_is_an_fp16_number():
    p = np.outer(R.E2M1, R.e4m3_values())
    assert np.array_equal(p, p.astype(np.float16).astype(np.float64))


@pytest.mark.parametrize("seed", range(6))
def test_plan_keeps_every_page_once(seed):
    rng = np.random.default_rng(seed)
    page, n, width, n_pages = 16, 9, 12, 80
    seq_len = np.zeros(n, np.int32)
    table = np.full((n, width), -1, np.int32)
    free, n_free = np.arange(n_pages, dtype=np.int32), n_pages
    for _ in range(30):
        new = rng.integers(-1, 40, n).astype(np.int32)
        r = R.plan(seq_len, new, table, free, n_free, page, n_pages, 400)
        if not isinstance(r, dict):
            new = np.full(n, -1, np.int32)
            r = R.plan(seq_len, new, table, free, n_free, page, n_pages, 400)
        seq_len, table, n_free = r["seq_len"], r["table"], r["n_free"]
        free[:n_free] = r["stack"]
        held = [table[s, c] for s in range(n) for c in range(-(-int(seq_len[s]) // page))]
        assert sorted(held + free[:n_free].tolist()) == list(range(n_pages))


def test_attention_of_equal_keys_is_the_mean():
    rng = np.random.default_rng(0)
    k = np.ones((2, 1, 16, 64))
    v = rng.normal(size=(2, 1, 16, 64))
    q = rng.normal(size=(1, 1, 64))
    out, lse, *_ = R.attention(q, (k, v), [0, 1], [20], np.array([[1, 0]]), 0.125, 16)
    want = np.concatenate([v[1, 0], v[0, 0, :4]]).mean(0)
    assert np.abs(out[0, 0] - want).max() < 1e-12
    assert abs(lse[0, 0] - (0.125 * q.sum() + np.log(20))) < 1e-12


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_mixture_experts_f32_gb300 as q
    return q


GOOD = dict(n_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=10, max_seqs=4, max_tokens=32,
            max_pages_per_seq=5)


@pytest.mark.parametrize("change", [
    dict(n_heads=0), dict(n_heads=7), dict(n_heads=2048, n_kv_heads=2), dict(n_kv_heads=0), dict(head_dim=96),
    dict(head_dim=192), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(n_pages=0),
    dict(n_pages=(1 << 30) + 1), dict(max_seqs=0), dict(max_seqs=4097), dict(max_tokens=0),
    dict(max_tokens=(1 << 20) + 1), dict(max_pages_per_seq=0), dict(max_pages_per_seq=(1 << 26) + 1)])
def test_bad_configs_are_refused_before_touching_cuda(q, change):
    assert q.qmoe_kv4_workspace_bytes(q.make_kv4_config(**GOOD)) > 0
    cfg = q.make_kv4_config(**{**GOOD, **change})
    assert q.qmoe_kv4_workspace_bytes(cfg) == 0
    with pytest.raises(q.QmoeError) as e:
        q.qmoe_kv4_create(cfg)
    assert e.value.status == 1 and list(change)[0] in str(e.value)


def test_null_handles_are_refused(q):
    L = q.lib
    assert L.qmoe_kv4_plan(None, 1, *[None] * 5, 1, *[None] * 5) == 1
    cache = q.make_kv4_cache(None, None, None, None, None, None)
    assert L.qmoe_kv4_append(None, ctypes.byref(cache), None, None, 0, 1, 0, 0, None, None, None) == 1
    assert L.qmoe_kv4_attention(None, ctypes.byref(cache), None, 0, 0, 1, 1, 1, None, None, None, 1.0, None, 0, 0,
                                None) == 1
    assert L.qmoe_kv4_get_status(None) == 1 and L.qmoe_kv4_set_stream(None, None) == 1
    L.qmoe_kv4_destroy(None)
