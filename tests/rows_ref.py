"""Plain numpy forms of the 8-bit path's row operators, values in 64 bits."""
from __future__ import annotations

import math

import numpy as np

from tests.kv4_ref import _nearest_even, e4m3_values

U = 2.0 ** -24                                       # half a step of fp32, relative
HALF = {"F32": U, "F16": 2.0 ** -11, "BF16": 2.0 ** -8}
GRID = e4m3_values()
F = np.float32


def _blocks(y):
    """y [rows, cols] as [rows, ceil(cols/128), 128], zeros behind the last column."""
    rows, cols = y.shape
    nb = -(-cols // 128)
    return np.pad(y, ((0, 0), (0, nb * 128 - cols))).reshape(rows, nb, 128)


def e4m3_decode(c):
    c = np.asarray(c).astype(np.int64)
    v = np.append(GRID, np.nan)[c & 127]
    return np.where(c >= 128, -v, v)


def quantise8(y):
    """y [rows, cols] in fp32 -> (codes, scales), each quotient rounded to fp32 once."""
    b = _blocks(y.astype(F))
    s = (np.abs(b).max(-1) / F(448)).astype(F)
    d = s[..., None]
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        q = np.where(d > 0, b / np.where(d > 0, d, F(1)), F(0)).astype(F)
    c = _nearest_even(np.minimum(np.abs(q).astype(np.float64), 448.0), GRID) + 128 * np.signbit(q)
    return np.where(d > 0, c, 0).reshape(len(y), -1)[:, :y.shape[1]].astype(np.uint8), s


def values8(codes, scale):
    v = e4m3_decode(codes)
    return v * np.repeat(scale.astype(np.float64), 128, axis=1)[:, :v.shape[1]]


def rmsnorm(x, res, w, eps):
    """(h, y) in 64 bits."""
    h = x.astype(np.float64) + (0 if res is None else res.astype(np.float64))
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + np.float64(F(eps)))
    return h, y if w is None else y * w.astype(np.float64)


def activate(z, act):
    if act == "RELU":
        return np.maximum(z, 0)
    if act == "SILU":
        return z / (1 + np.exp(-np.clip(z, -700, None)))
    if act == "GELU":
        return z * 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-z / math.sqrt(2))
    return z


def linear(xc, xs, wc, ws, bias, act, res):
    """(out, the sum of the products' sizes) in 64 bits."""
    x = values8(xc, xs)
    w = e4m3_decode(wc) * np.repeat(np.repeat(ws.astype(np.float64), 128, 0), 128, 1)[:wc.shape[0], :wc.shape[1]]
    z = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    if bias is not None:
        z = z + bias
        size = size + np.abs(bias)
    z = activate(z, act)
    return (z if res is None else z + res.astype(np.float64)), size


def rope_freq(rot, base, scaling="plain", factor=1.0, orig_ctx=0.0, beta_fast=32.0, beta_slow=1.0, mscale=0.0):
    j = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2 * j / rot)
    m = mscale or 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        lo, hi = (rot * math.log(orig_ctx / (2 * math.pi * t)) / (2 * math.log(base)) for t in (beta_fast, beta_slow))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        r = np.clip((j - lo) / max(hi - lo, 0.001), 0, 1)
        f = f * (1 - r) + f / factor * r
        m = mscale or (0.1 * math.log(factor) + 1 if factor > 1 else 1.0)
    return f, m


def rope_heads(x, hd, norm, eps):
    """Rows as [tokens, heads, hd] in fp32, each head normalised on demand, every step rounded once."""
    x = x.astype(F).reshape(len(x), -1, hd)
    if norm is None:
        return x
    d = x.astype(np.float64)
    r = (1 / np.sqrt((d * d).mean(-1, keepdims=True) + np.float64(F(eps)))).astype(F)
    return (x * r).astype(F) * norm.astype(F)


def rope(x, cs, rot, layout):
    """x [tokens, heads, hd] fp32 turned by cs [tokens, 2, rot/2] fp32, every step rounded once."""
    x = x.copy()
    c, s = cs[:, None, 0], cs[:, None, 1]
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    p, q = x[..., a].copy(), x[..., b].copy()
    x[..., a] = p * c - q * s
    x[..., b] = q * c + p * s
    return x
