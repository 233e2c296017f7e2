"""A decoder layer over FP8 weights and the paged 4-bit cache, put together from the row operators: norm into
8 bits, Q/K/V product, the append that rotates, attention, quantisation, O product into the residual, norm,
and the FP8 experts.  Each step is compared with its plain form in 64 bits on what the step before gave."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests import kv4_ref as K4
from tests import rows_ref as R
from tests.compare import TOL_FP32, ids_match, rel_err, tie_bound
from tests.gpu_util import dev, to_dev
from tests.test_gpu_rows import EPS, NORM_ERR, check_codes, host, linear_bound, linear_inputs, make_table, q  # noqa: F401

pytestmark = pytest.mark.gpu

NQ, NKV, HD, PAGE = 8, 2, 64, 16
LENS, NEWS = [40, 17, 5], [1, 9, 5]               # with the new tokens: one decodes, one brings a chunk, one its prompt
PAD = 2                                           # rows behind the last sequence


class Layer:
    """Everything one layer keeps, on a stream of its own."""

    def __init__(self, q, seed=1):
        rng = np.random.default_rng(seed)
        self.q, self.st = q, torch.cuda.Stream()
        self.moe = synth.moe_inputs_fp8(synth.FP8_CONFIGS["tiny_fp8"], T=sum(NEWS) + PAD)
        m = self.moe
        self.H, self.T = m["H"], sum(NEWS) + PAD
        self.ctx = q.qmoe_create(q.make_config(self.H, m["E"], m["K"], m["F"], self.T, 1, stream=self.st.cuda_stream))
        self.pages = 12
        self.kv = q.qmoe_kv4_create(q.make_kv4_config(NQ, NKV, HD, PAGE, self.pages, 3, self.T, 4, self.st.cuda_stream))
        self.qkv_n = (NQ + 2 * NKV) * HD
        _, _, wc, ws = linear_inputs(1, self.H, self.qkv_n, seed + 1)
        _, _, oc, os_ = linear_inputs(1, NQ * HD, self.H, seed + 2)
        self.wnp = [wc, ws * np.float32(2e-3), oc, os_ * np.float32(2e-3)]
        self.w = [to_dev(a) for a in self.wnp]
        self.norm = to_dev((1 + 0.2 * rng.normal(size=self.H)).astype(np.float32))
        self.qn, self.kn = (to_dev((1 + 0.2 * rng.normal(size=HD)).astype(np.float32)) for _ in "qk")
        self.rope, self.table = make_table(q, self.ctx, HD, 64)
        self.cache_t = []
        for _ in "kv":
            self.cache_t += [torch.zeros(self.pages, NKV, PAGE, HD // 2, dtype=torch.uint8, device=dev()),
                             torch.zeros(self.pages, NKV, PAGE, HD // 16, dtype=torch.uint8, device=dev())]
        self.glob = to_dev(np.full((2, NKV), 4 / 2688, np.float32))
        self.cache = q.make_kv4_cache(*self.cache_t, self.glob[0], self.glob[1])
        self.table_np = np.arange(12, dtype=np.int32).reshape(3, 4)
        self.blocks = to_dev(self.table_np)
        self.cu = to_dev(np.concatenate([[0], np.cumsum(NEWS)]).astype(np.int32))
        self.lens = to_dev(np.array(LENS, np.int32))
        pos, slots = [], []
        for s, (L, n) in enumerate(zip(LENS, NEWS)):
            for p in range(L - n, L):
                pos.append(p)
                slots.append(int(self.table_np[s, p // PAGE]) * PAGE + p % PAGE)
        self.pos, self.slots = to_dev(np.array(pos + [-1] * PAD, np.int32)), to_dev(np.array(slots + [-1] * PAD, np.int64))
        z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device=dev())  # noqa: E731
        T, H = self.T, self.H
        self.h, self.h2, self.h3 = z(T, H), z(T, H), z(T, H)
        self.c1, self.s1 = z(T, H, dtype=torch.uint8), z(T, -(-H // 128))
        self.rows, self.q_out = z(T, self.qkv_n, dtype=torch.bfloat16), z(T, NQ * HD, dtype=torch.bfloat16)
        self.att, self.c2, self.s2 = z(T, NQ * HD, dtype=torch.bfloat16), z(T, NQ * HD, dtype=torch.uint8), z(T, NQ * HD // 128)
        self.ids, self.wts = z(T, m["K"], dtype=torch.int32), z(T, m["K"])
        self.experts = {n: to_dev(m[n]) for n in ("router", "gate", "gate_scale", "up", "up_scale", "down", "down_scale")}
        torch.cuda.synchronize()

    def run(self):
        q, T, H, w = self.q, self.T, self.H, self.w
        nq = NQ * HD
        q.qmoe_rmsnorm(self.ctx, self.h, q.QMOE_F32, 0, None, 0, 0, None, self.norm, EPS, T, H, self.c1, q.QMOE_E4M3, 0, self.s1)
        q.qmoe_linear_fp8(self.ctx, self.c1, self.s1, T, H, w[0], w[1], self.qkv_n, None, 0, None, 0, self.rows, q.QMOE_BF16, 0)
        k, v = self.rows[:, nq:nq + NKV * HD], self.rows[:, nq + NKV * HD:]
        q.qmoe_kv4_append_rope(self.kv, self.cache, self.rope, self.rows, k, v, q.QMOE_BF16, T, self.qkv_n, self.qkv_n, self.qkv_n,
                               self.pos, self.slots, self.qn, self.kn, EPS, self.q_out, 0)
        q.qmoe_kv4_attention(self.kv, self.cache, self.q_out, q.QMOE_BF16, 0, 3, T, max(NEWS), self.cu, self.lens, self.blocks,
                             HD ** -0.5, self.att, q.QMOE_BF16, 0)
        q.qmoe_fp8_quantize(self.ctx, self.att, q.QMOE_BF16, 0, T, nq, self.c2, self.s2)
        q.qmoe_linear_fp8(self.ctx, self.c2, self.s2, T, nq, w[2], w[3], H, None, 0, self.h, H, self.h2, q.QMOE_F32, 0)
        q.qmoe_rmsnorm(self.ctx, self.h2, q.QMOE_F32, 0, None, 0, 0, None, None, EPS, T, H, self.h3, q.QMOE_F32, 0)
        e = self.experts
        self.out = getattr(self, "out", torch.zeros(T, H, device=dev()))
        q.qmoe_forward_fp8(self.ctx, self.h3, e["router"], e["gate"], e["gate_scale"], e["up"], e["up_scale"], e["down"],
                           e["down_scale"], T, self.out, self.ids, self.wts)

    def close(self):
        assert self.q.qmoe_get_status(self.ctx) == self.q.QMOE_OK, self.q.qmoe_last_error(self.ctx)
        assert self.q.qmoe_kv4_get_status(self.kv) == self.q.QMOE_OK, self.q.qmoe_kv4_last_error(self.kv)
        self.q.qmoe_kv4_destroy(self.kv)
        self.q.qmoe_destroy(self.ctx)


def hidden(T, H, seed):
    return to_dev(np.random.default_rng(seed).normal(size=(T, H)).astype(np.float32))


def test_an_fp8_layer_step_by_step(q):  # noqa: F811
    la = Layer(q)
    T, H, live = la.T, la.H, sum(NEWS)
    la.h.copy_(hidden(T, H, 5))
    # what the cache holds of earlier tokens
    for c in la.cache_t[::2]:
        c.copy_(to_dev(np.random.default_rng(7).integers(0, 256, c.shape, dtype=np.uint8)))
    for s in la.cache_t[1::2]:
        s.fill_(0x38)                                        # 1
    torch.cuda.synchronize()
    with torch.cuda.stream(la.st):
        la.run()
    torch.cuda.synchronize()
    _, y = R.rmsnorm(host(la.h), None, host(la.norm), EPS)
    check_codes(host(la.c1), host(la.s1), y, NORM_ERR)
    ref, size = R.linear(host(la.c1), host(la.s1), la.wnp[0], la.wnp[1], None, "NONE", None)
    rows = host(la.rows)
    assert (np.abs(rows - ref) <= linear_bound(size, H // 128, ref, R.HALF["BF16"], "NONE")).all()
    nq, pos = NQ * HD, host(la.pos)
    cs = host(la.table)[np.maximum(pos, 0)]
    want = R.rope(R.rope_heads(rows[:, :nq], HD, host(la.qn), EPS), cs, HD, "half").reshape(T, nq)
    assert np.array_equal(host(la.q_out)[:live], host(torch.from_numpy(want).to(torch.bfloat16))[:live])
    assert not host(la.q_out)[live:].any()
    kk = R.rope(R.rope_heads(rows[:, nq:nq + NKV * HD], HD, host(la.kn), EPS), cs, HD, "half")
    slots = host(la.slots)
    for i, x in enumerate((kk, rows[:, nq + NKV * HD:].reshape(T, NKV, HD))):
        codes, scales, _ = K4.quantise(x.astype(np.float32), host(la.glob[i]))
        for t in range(live):
            p, o = slots[t] // PAGE, slots[t] % PAGE
            assert np.array_equal(host(la.cache_t[2 * i])[p, :, o], codes[t])
            assert np.array_equal(host(la.cache_t[2 * i + 1])[p, :, o], scales[t])
    vals = [K4.values_of(K4.unpack(host(la.cache_t[2 * i])).swapaxes(1, 2), host(la.cache_t[2 * i + 1]).swapaxes(1, 2),
                         host(la.glob[i])).swapaxes(1, 2) for i in range(2)]
    o, _, vmax, zabs, seen = K4.attention(host(la.q_out).astype(np.float64).reshape(T, NQ, HD)[:live], vals, host(la.cu), LENS,
                                          la.table_np, HD ** -0.5, PAGE)
    bound, _ = K4.attention_bound(o, vmax, zabs, seen, HD, True, R.HALF["BF16"])
    assert (np.abs(host(la.att)[:live].reshape(o.shape) - o) <= bound).all()
    c, s = R.quantise8(host(la.att))
    assert np.array_equal(host(la.c2), c) and np.array_equal(host(la.s2), s)
    ref, size = R.linear(c, s, la.wnp[2], la.wnp[3], None, "NONE", host(la.h))
    assert (np.abs(host(la.h2) - ref) <= linear_bound(size, nq // 128, ref, 0, "NONE")).all()
    _, y = R.rmsnorm(host(la.h2), None, None, EPS)
    assert (np.abs(host(la.h3) - y) <= NORM_ERR * np.abs(y)).all()
    m, x = la.moe, host(la.h3)
    logits, ids, wts, _ = oracle.route(x, m["router"], m["K"])
    ok, ties = ids_match(host(la.ids), ids, logits, tie_bound(logits))
    assert ok and not ties
    ref = oracle.moe_ffn_fp8(x, ids, wts, m["gate"], m["gate_scale"], m["up"], m["up_scale"], m["down"], m["down_scale"], m["F"], m["E"])
    assert rel_err(host(la.out), ref) <= TOL_FP32
    la.close()


def test_an_fp8_layer_in_a_graph(q):  # noqa: F811
    """Captured once and replayed over other hidden rows: as called one by one, bit for bit."""
    la = Layer(q, 3)
    with torch.cuda.stream(la.st):
        la.h.copy_(hidden(la.T, la.H, 8))
        la.run()
        la.st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=la.st):
            la.run()
        for seed in (9, 10, 9):
            got = []
            for run in (g.replay, la.run):
                la.h.copy_(hidden(la.T, la.H, seed))
                for t in (la.rows, la.q_out, la.att, la.out, *la.cache_t):
                    t.zero_()
                run()
                la.st.synchronize()
                got.append([t.clone() for t in (la.rows, la.q_out, la.h2, la.out, *la.cache_t)] + [la.att[:sum(NEWS)].clone()])
            assert all(torch.equal(a, b) for a, b in zip(*got))
            assert got[0][3].abs().max() > 0
    la.close()
