"""qmoe_step_kv4: ragged batches through whole decoder layers over paged 4-bit caches, planned by
qmoe_kv4_plan, against the oracle's pieces.

Each layer is compared on the kernel's own input to it and over the cache as the kernel left it
(so that neither one layer's fp16 projections nor a code decided the other way by them count
twice): the cached K and V within a quantisation step of the oracle's rows, the hidden state
within the half-precision bound of the batched prefill (the same projections and MoE), expert
ids as there.  The call over all layers must give what one layer per call gives, bit for bit.
"""
import numpy as np
import pytest

import oracle
import synth
from tests import kv4_ref as R
from tests.compare import TOL_BF16, rel_err
from tests.test_gpu_prefill_layer import ID_SLACK, QWEN3, SMALL, _layer_struct, _upload

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import quantized_mixture_experts_f32_gb300 as q
    return q


class Server:
    """A context, a cache handle, and the layers' weights and caches."""

    def __init__(self, q, geo, n, page, width, n_pages, cap, stream=0):
        self.q, self.geo, self.n, self.page, self.width, self.cap, self.n_pages = q, geo, n, page, width, cap, n_pages
        L, hd, nkv = geo["n_layers"], geo["head_dim"], geo["n_kv"]
        dev = torch.device("cuda:0")
        self.keep, self.small, self.structs = [], [], []
        for l in range(L):
            small, d = _upload(geo, l, dev)
            s = _layer_struct(q, d, small["down_t"])
            s.k_cache = s.v_cache = None                          # not used by this path
            self.keep.append(d)
            self.small.append(small)
            self.structs.append(s)
        self.layers = (q.qmoe_layer_weights * L)(*self.structs)
        self.ctx = q.qmoe_create(q.make_config(geo["H"], geo["E"], geo["K"], geo["F"], cap, 1, stream,
                                               n_heads=geo["n_heads"], n_kv_heads=nkv, head_dim=hd, max_ctx=1,
                                               rope_base=geo["rope_base"], rms_eps=geo["eps"]))
        self.kv = q.qmoe_kv4_create(q.make_kv4_config(geo["n_heads"], nkv, hd, page, n_pages, n, cap, width, stream))
        g = np.full(nkv, 2.0 ** -9, np.float32)
        self.g = torch.from_numpy(g).cuda()
        self.buf = [{"k_codes": torch.zeros(n_pages, nkv, page, hd // 2, dtype=torch.uint8, device=dev),
                     "k_scales": torch.full((n_pages, nkv, page, hd // 16), 0x7F, dtype=torch.uint8, device=dev),
                     "v_codes": torch.zeros(n_pages, nkv, page, hd // 2, dtype=torch.uint8, device=dev),
                     "v_scales": torch.full((n_pages, nkv, page, hd // 16), 0x7F, dtype=torch.uint8, device=dev)}
                    for _ in range(L)]
        self.caches = (q.qmoe_kv4_cache * L)(*[
            q.make_kv4_cache(b["k_codes"], b["k_scales"], b["v_codes"], b["v_scales"], self.g, self.g) for b in self.buf])
        i32 = dict(dtype=torch.int32, device=dev)
        self.len, self.nf = torch.zeros(n, **i32), torch.tensor([n_pages], **i32)
        self.table, self.free = torch.full((n, width), -1, **i32), torch.arange(n_pages, **i32)
        self.cu, self.pos = torch.zeros(n + 1, **i32), torch.zeros(cap, **i32)
        self.slots = torch.zeros(cap, dtype=torch.int64, device=dev)

    def close(self):
        self.q.qmoe_kv4_destroy(self.kv)
        self.q.qmoe_destroy(self.ctx)

    def plan(self, new):
        self.q.qmoe_kv4_plan(self.kv, self.n, self.len, new, self.table, self.free, self.nf, self.cap, self.len, self.nf,
                             self.cu, self.pos, self.slots)

    def step(self, hidden, n_tokens, max_new, layer=None, ids=None):
        one = layer is not None
        self.q.qmoe_step_kv4(self.ctx, self.kv, (self.q.qmoe_layer_weights * 1)(self.structs[layer]) if one else self.layers,
                             (self.q.qmoe_kv4_cache * 1)(self.caches[layer]) if one else self.caches,
                             1 if one else self.geo["n_layers"], self.n, n_tokens, max_new, self.cu, self.len, self.table,
                             self.pos, self.slots, hidden, ids)

    def ok(self):
        assert self.q.qmoe_get_status(self.ctx) == 0 and self.q.qmoe_kv4_get_status(self.kv) == 0

    def values(self, l):
        out = []
        for n in "kv":
            c = R.unpack(self.buf[l][n + "_codes"].cpu().numpy()).transpose(0, 2, 1, 3)
            s = self.buf[l][n + "_scales"].cpu().numpy().transpose(0, 2, 1, 3)
            out.append(R.values_of(c, s, self.g.cpu().numpy()).transpose(0, 2, 1, 3))
        return out


def _layer(sv, l, h, ids_gpu, cu, lens, table, pos, slots):
    """The oracle's layer over the kernel's cache; checks the cached rows."""
    geo, small = sv.geo, sv.small[l]
    H, hd, nq, nkv, eps = geo["H"], geo["head_dim"], geo["n_heads"], geo["n_kv"], geo["eps"]
    W = {n: oracle.dequant_matrix("Q4_K", small[n], r, c) for n, r, c in
         (("wq", nq * hd, H), ("wk", nkv * hd, H), ("wv", nkv * hd, H), ("wo", H, nq * hd))}
    T = len(pos)
    K, V = sv.values(l)
    qs = np.zeros((T, nq, hd))
    for t in range(T):
        x = oracle.rmsnorm(h[t], small["attn_norm"], eps)
        qv, kv, vv = W["wq"] @ x, W["wk"] @ x, W["wv"] @ x
        for i in range(nq):
            qs[t, i] = oracle.rope_neox(oracle.rmsnorm(qv[i * hd:(i + 1) * hd], small["q_norm"], eps), int(pos[t]), geo["rope_base"])
        p, o = slots[t] // sv.page, slots[t] % sv.page
        for g in range(nkv):
            k = oracle.rope_neox(oracle.rmsnorm(kv[g * hd:(g + 1) * hd], small["k_norm"], eps), int(pos[t]), geo["rope_base"])
            for got, ref, n in ((K[p, g, o], k, "k"), (V[p, g, o], vv[g * hd:(g + 1) * hd], "v")):
                code = sv.buf[l][n + "_scales"][int(p), g, int(o)].cpu().numpy()
                d = np.repeat(R.e4m3_values()[code] * 2.0 ** -9, 16)
                # half of the widest step (4 to 6), and the projections' fp16 error; block scales stop
                # at 448, so that values stop at 6 * 448 globals
                near = np.clip(ref, -2688 * 2.0 ** -9, 2688 * 2.0 ** -9)
                assert (np.abs(got - near) <= d + TOL_BF16 * max(1.0, np.abs(ref).max())).all(), (l, n, t)
    att, *_ = R.attention(qs, (K, V), cu, lens, table, hd ** -0.5, sv.page)
    h1 = h + att.reshape(T, -1) @ W["wo"].T
    x2 = np.stack([oracle.rmsnorm(h1[t], small["ffn_norm"], eps) for t in range(T)])
    ex = synth.step_layer_experts(geo, l)
    inp = dict(x=x2.astype(np.float32), router=small["router"], K=geo["K"], gate=ex["gate"], up=ex["up"], down=ex["down"],
               gate_t="Q4_K", up_t="Q4_K", down_t=small["down_t"], F=geo["F"], E=geo["E"])
    r = oracle.moe_forward(inp)
    bad = [t for t in range(T) if not np.array_equal(r["ids"][t], ids_gpu[t])]
    for t in bad:
        lg = r["logits"][t].astype(np.float64)
        kth = lg[r["ids"][t]].min()
        changed = set(r["ids"][t].tolist()) ^ set(ids_gpu[t].tolist())
        assert all(abs(lg[e] - kth) <= ID_SLACK * np.abs(lg).max() for e in changed), (t, r["ids"][t], ids_gpu[t])
    assert len(bad) <= max(1, T // 10)
    if bad:
        r = oracle.moe_forward(inp, force=ids_gpu)
    return h1 + (r["out"] - inp["x"].astype(np.float64))


STEPS = {"small": (SMALL, 4, 16, 5, 14, 48, [[13, 5, 0, 1], [1, 20, 2, 1], [1, 1, -1, 1], [30, 1, 3, 1]]),
         "qwen3": (QWEN3, 3, 32, 3, 8, 40, [[33, 0, 1], [1, 5, 1]])}


@pytest.mark.parametrize("name", list(STEPS))
def test_steps_of_whole_layers(q, name):
    geo, n, page, width, n_pages, cap, steps = STEPS[name]
    sv = Server(q, geo, n, page, width, n_pages, cap)
    worst = 0.0
    try:
        for i, new in enumerate(steps):
            sv.plan(torch.tensor(new, dtype=torch.int32, device="cuda"))
            before = [{k: b.clone() for k, b in x.items()} for x in sv.buf]
            cu, lens = sv.cu.cpu().numpy(), sv.len.cpu().numpy()
            T = int(cu[-1])
            pad = T if i == 0 else min(cap, T + 3)                # later steps carry rows behind the last token
            h0 = synth.prefill_input(dict(geo, input_seed=geo["input_seed"] + i), pad)
            h0[T:] = np.nan
            mx = max(1, max(new))
            hidden = torch.from_numpy(h0.copy()).cuda()
            ids_all = torch.full((geo["n_layers"], pad, geo["K"]), -1, dtype=torch.int32, device="cuda")
            sv.step(hidden, pad, mx, None, ids_all)
            sv.ok()
            h_all = hidden.cpu().numpy()
            caches_all = [{k: b.cpu().numpy() for k, b in x.items()} for x in sv.buf]
            for x, b in zip(sv.buf, before):
                for k in x:
                    x[k].copy_(b[k])
            hidden = torch.from_numpy(h0.copy()).cuda()
            for l in range(geo["n_layers"]):
                h_in = hidden.cpu().numpy()
                ids = torch.full((1, pad, geo["K"]), -1, dtype=torch.int32, device="cuda")
                sv.step(hidden, pad, mx, l, ids)
                sv.ok()
                got = hidden.cpu().numpy()
                assert np.isnan(got[T:]).all()                    # left as they were
                idl = ids.cpu().numpy()[0, :T]
                assert np.array_equal(idl, ids_all.cpu().numpy()[l, :T])
                want = _layer(sv, l, h_in[:T].astype(np.float64), idl, cu, lens, sv.table.cpu().numpy(),
                              sv.pos.cpu().numpy()[:T], sv.slots.cpu().numpy()[:T])
                err = rel_err(got[:T], want)
                worst = max(worst, err)
                assert err <= TOL_BF16, f"step {i} layer {l}: hidden rel err {err:.3e}"
                for k in sv.buf[l]:
                    assert np.array_equal(sv.buf[l][k].cpu().numpy(), caches_all[l][k]), k
            assert np.array_equal(hidden.cpu().numpy()[:T], h_all[:T])
    finally:
        sv.close()
    print(f"{name}: rel err {worst:.2e}")


@pytest.mark.parametrize("n", [4, 300])
def test_rows_that_no_sequence_serves_stay(q, n):
    """Sequences that the attention skips, rows before the first and behind the last one, offsets that descend:
    their rows are left as they were, the others' are what they are without them."""
    geo, page, width = SMALL, 16, 3
    new = np.ones(n, np.int32)
    new[:4] = [5, 3, 1, 9]
    T = int(new.sum())
    sv = Server(q, geo, n, page, width, n * 3, T + 4)
    try:
        sv.plan(torch.from_numpy(new).cuda())
        sv.ok()
        x = torch.from_numpy(synth.prefill_input(geo, T + 4)).cuda()
        cu, lens = sv.cu.clone(), sv.len.clone()
        want = x.clone()
        sv.step(want, T + 4, 9)
        sv.ok()
        served = torch.ones(T + 4, dtype=torch.bool, device="cuda")
        served[T:] = False
        assert torch.equal(want[~served], x[~served]) and not torch.equal(want[:T], x[:T])

        def stay(first, last, mx=9):
            h = x.clone()
            sv.step(h, T + 4, mx)
            assert q.qmoe_get_status(sv.ctx) == 0 and q.qmoe_kv4_get_status(sv.kv) == 8
            keep = ~served
            keep[first:last] = True
            assert torch.equal(h[keep], x[keep]) and torch.equal(h[~keep], want[~keep])
            sv.cu.copy_(cu)
            sv.len.copy_(lens)

        sv.len[1] = -1                                             # sequence 1, rows 5 .. 7
        stay(5, 8)
        sv.len[n - 1] = width * page + 1                           # the last one
        stay(T - new[n - 1], T)
        stay(9, 18, 8)                                             # more new tokens than max_new says: sequence 3
        sv.cu[0] = -1                                              # no such row
        stay(0, 5)
        sv.cu[2] = 4                                               # sequence 1 ends before it begins
        stay(0, T)
        sv.cu[:2] = 5                                              # rows before the first sequence's
        h = x.clone()
        sv.step(h, T + 4, 9)
        sv.ok()
        assert torch.equal(h[:5], x[:5]) and torch.equal(h[5:T], want[5:T])
    finally:
        sv.close()


def test_a_captured_step_of_whole_layers(q):
    """plan and step captured once and replayed while the sequences grow equal the uncaptured calls."""
    geo, n, page, width, n_pages, cap = SMALL, 3, 16, 3, 9, 3
    s = torch.cuda.Stream()
    a, b = Server(q, geo, n, page, width, n_pages, cap, s.cuda_stream), Server(q, geo, n, page, width, n_pages, cap, s.cuda_stream)
    try:
        new = torch.ones(n, dtype=torch.int32, device="cuda")
        ha, hb = torch.zeros(cap, geo["H"], device="cuda"), torch.zeros(cap, geo["H"], device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            a.plan(new)
            a.step(ha, cap, 1)
        for i in range(20):
            x = torch.from_numpy(synth.prefill_input(dict(geo, input_seed=i), cap)).cuda()
            ha.copy_(x)
            hb.copy_(x)
            torch.cuda.synchronize()
            g.replay()
            with torch.cuda.stream(s):
                b.plan(new)
                b.step(hb, cap, 1)
            torch.cuda.synchronize()
            assert torch.equal(ha, hb)
        a.ok()
        b.ok()
        assert a.len.tolist() == [20] * 3
    finally:
        a.close()
        b.close()


def test_step_refuses(q):
    geo = SMALL
    sv = Server(q, geo, 2, 16, 2, 4, 8)
    L = q.lib
    other = q.qmoe_kv4_create(q.make_kv4_config(8, 2, 64, 16, 4, 2, 8, 2, 0))
    elsewhere = q.qmoe_kv4_create(q.make_kv4_config(4, 2, 64, 16, 4, 2, 8, 2, torch.cuda.Stream().cuda_stream))
    plain = q.qmoe_create(q.make_config(geo["H"], geo["E"], geo["K"], geo["F"], 8, 1, 0))
    try:
        h = torch.zeros(9, geo["H"], device="cuda")

        def call(**c):
            a = dict(ctx=sv.ctx, kv=sv.kv, layers=sv.layers, caches=sv.caches, nl=2, n=2, t=4, mx=2, cu=sv.cu, len=sv.len,
                     table=sv.table, pos=sv.pos, slots=sv.slots, h=h)
            a.update(c)
            return L.qmoe_step_kv4(a["ctx"], a["kv"], a["layers"], a["caches"], a["nl"], a["n"], a["t"], a["mx"],
                                   *[q._ptr(a[k]) for k in ("cu", "len", "table", "pos", "slots", "h")], None)

        assert call(ctx=None) == 1 and call(ctx=plain) == 1 and call(kv=None) == 1 and call(layers=None) == 1
        assert call(caches=None) == 1 and call(nl=0) == 1
        for k in ("cu", "len", "table", "pos", "slots", "h"):
            assert call(**{k: None}) == 1
        assert call(kv=other) == 4 and call(kv=elsewhere) == 1
        assert call(n=0) == 4 and call(n=3) == 4 and call(t=0) == 4 and call(t=9) == 4 and call(mx=0) == 4 and call(mx=5) == 4
        assert call(h=h.data_ptr() + 4) == 2 and call(slots=sv.slots.data_ptr() + 4) == 2 and call(pos=sv.pos.data_ptr() + 2) == 2
        assert call(layers=(q.qmoe_layer_weights * 2)(sv.structs[0])) == 1            # the second layer is empty
        assert call(caches=(q.qmoe_kv4_cache * 2)(sv.caches[0])) == 1
        assert "layer 1" in q.qmoe_last_error(sv.ctx)
        torch.cuda.synchronize()
        sv.ok()
    finally:
        q.qmoe_destroy(plain)
        q.qmoe_kv4_destroy(other)
        q.qmoe_kv4_destroy(elsewhere)
        sv.close()
