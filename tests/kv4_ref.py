"""Plain numpy forms of the paged 4-bit KV cache's operators, values in 64 bits."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
EPS32 = 2.0 ** -24                                   # half a step, relative


def e4m3_values() -> np.ndarray:
    """Values of the codes 0 .. 126 (code 127 is NaN)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m / 8 * 2.0 ** -6)


def _nearest_even(x, grid):
    """Index of the nearest grid value, ties to the even index (grid ascending)."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    a, b = x - grid[lo], grid[hi] - x
    return np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def quantise(x, g):
    """x [..., n_kv, hd] (any float type), g [n_kv] -> codes, scales, values; each quotient
    and product that decides is rounded to fp32."""
    f = np.float32
    b = x.astype(f).reshape(*x.shape[:-1], -1, 16)
    g = g.astype(f)[:, None]
    pos = g > 0
    amax = np.abs(b).max(-1)
    den = np.where(pos, f(6) * g, f(1)).astype(f)
    ratio = np.minimum((amax / den).astype(f), f(448)).astype(np.float64)
    s = np.where(pos, _nearest_even(ratio, e4m3_values()), 0)
    sv = e4m3_values()[s]
    d = (sv.astype(f) * g).astype(f)[..., None]
    v = np.where(d > 0, b / np.where(d > 0, d, f(1)), f(0)).astype(f)
    c = _nearest_even(np.minimum(np.abs(v.astype(np.float64)), 6.0), E2M1) + 8 * np.signbit(v)
    c = np.where(d > 0, c, 0)
    val = values_of(c.reshape(*x.shape), s, g[:, 0])
    c = c.reshape(*x.shape)
    return (c[..., 0::2] + 16 * c[..., 1::2]).astype(np.uint8), s.astype(np.uint8), val


def values_of(c, s, g):
    """Values of unpacked codes c [..., n_kv, hd] and scale codes s [..., n_kv, hd/16]."""
    m = E2M1[c & 7] * np.where(c >= 8, -1.0, 1.0)
    sv = np.append(e4m3_values(), np.nan)[s & 127]
    return (m.reshape(*m.shape[:-1], -1, 16) * sv[..., None]).reshape(m.shape) * g.astype(np.float64)[:, None]


def unpack(codes):
    return np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)


def plan(seq_len, new_len, table, free, n_free, page, n_pages, cap):
    """One step, request by request.  Returns a dict, or the status that refuses it."""
    width = table.shape[1]
    n = len(seq_len)
    table, free = table.copy(), free.copy()
    tok = need = back = 0
    shape = False
    for L, N in zip(seq_len.tolist(), new_len.tolist()):
        if L < 0 or L > width * page:
            return 8
        have, want = -(-L // page), -(-(L + max(N, 0)) // page)
        shape |= want > width
        tok += max(N, 0)
        need += 0 if N < 0 else want - have
        back += have if N < 0 else 0
    if n_free < 0 or n_free > n_pages or n_free + back - need > n_pages:
        return 8
    if shape or tok > cap:
        return 4
    if n_free + back - need < 0:
        return 5
    stack = free[:n_free].tolist()
    for s in range(n):
        if new_len[s] < 0:
            stack += table[s, :-(-int(seq_len[s]) // page)].tolist()
    out_len = np.zeros(n, np.int32)
    cu = np.zeros(n + 1, np.int32)
    pos, slots = np.full(cap, -1, np.int32), np.full(cap, -1, np.int64)
    t = 0
    for s in range(n):
        L, N = int(seq_len[s]), int(new_len[s])
        if N >= 0:
            for c in range(-(-L // page), -(-(L + N) // page)):
                table[s, c] = stack.pop()
            for p in range(L, L + N):
                pos[t] = p
                slots[t] = int(table[s, p // page]) * page + p % page
                t += 1
            out_len[s] = L + N
        cu[s + 1] = t
    return dict(seq_len=out_len, n_free=len(stack), cu=cu, pos=pos, slots=slots, table=table,
                stack=np.array(stack, np.int32))


def attention(q, cache, cu, seq_len, table, scale, page):
    """q [t, nq, hd] in 64 bits; cache: values k, v [pages, nkv, page, hd].  Returns out, lse and, for
    the tolerance, per row the largest |v|, the largest sum |q k| scale and the visible positions."""
    t, nq, hd = q.shape
    k, v = cache
    n_pages, nkv = k.shape[:2]
    out, lse = np.zeros((t, nq, hd)), np.full((t, nq), -np.inf)
    vmax, zabs, seen = np.zeros((t, nq)), np.zeros((t, nq)), np.zeros(t, int)
    for s in range(len(seq_len)):
        L, q0, q1 = int(seq_len[s]), int(cu[s]), int(cu[s + 1])
        if L == 0 or q1 == q0:
            continue
        cols = table[s, :-(-L // page)].astype(np.int64)
        ok = np.repeat((cols >= 0) & (cols < n_pages), page)[:L]
        cols = np.clip(cols, 0, n_pages - 1)
        for h in range(nq):
            g = h // (nq // nkv)
            ks, vs = k[cols, g].reshape(-1, hd)[:L], v[cols, g].reshape(-1, hd)[:L]
            for i in range(q1 - q0):
                p = np.arange(L)
                vis = (p <= L - (q1 - q0) + i) & ok
                if not vis.any():
                    continue
                z = scale * (ks[vis] @ q[q0 + i, h])
                m = z.max()
                e = np.exp(z - m)
                out[q0 + i, h] = e @ vs[vis] / e.sum()
                lse[q0 + i, h] = m + np.log(e.sum())
                vmax[q0 + i, h] = np.abs(vs[vis]).max()
                zabs[q0 + i, h] = (np.abs(ks[vis]) @ np.abs(q[q0 + i, h])).max() * abs(scale)
                seen[q0 + i] = vis.sum()
    return out, lse, vmax, zabs, seen


def attention_bound(out, vmax, zabs, seen, hd, q_16, out_half):
    """How far out [t, nq, hd] and lse [t, nq] may be from the 64-bit result.

    z is a sum of hd products in fp32 (two fp16 terms of a q value leave 2^-22 of it; a
    16-bit value is one term, exact above 2^-14 of the row's largest and 2^-25 of that below),
    then scaled and shifted: |dz| <= (hd + 8) eps zabs + 2^-22 zabs + a rounding of the
    exponent's argument, at most 4 eps |z|.  exp2 on the device has a relative error below
    2^-22.  The numerator and the sum run over `seen` positions in fp32: (seen + 8) eps each.
    One fp16 term of a 16-bit row's weight adds 2^-11 (and 2^-25 where it is subnormal).
    A weighted mean of v moves by at most 2 (the relative error of its weights) max|v|.
    The result's own type adds half a step."""
    dz = (hd + 12) * EPS32 * zabs + 2.0 ** -22 * (zabs + 1)
    w = dz + 2.0 ** -22 + (seen[:, None] + 8) * EPS32
    lse = w + 4 * EPS32 * zabs
    if q_16:
        w = w + 2.0 ** -11 + seen[:, None] * 2.0 ** -25
    return (2 * w * vmax)[..., None] + out_half * np.abs(out) + 1e-30, lse + 1e-6
