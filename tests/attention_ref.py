"""Attention and dense layers with approximate products in 64 bits, element by
element from the definitions of include/approx_mul.h, on the oracle's products
(oracle.amsim; lut None: the native multiplier's exact ones). What the
definitions round to FP32 is rounded; every other step is float64.

One sequence and one head at a time: q [n, D], k and v [m, D].
"""
import math

import numpy as np

import oracle

LOG2E = 1.4426950408889634
TINY = 2.0 ** -64


def products(a, b, lut, M, E=8):
    """T(a, b) of two broadcast FP32 arrays, as float64."""
    a, b = np.broadcast_arrays(np.asarray(a, np.float32), np.asarray(b, np.float32))
    if lut is None:
        with np.errstate(invalid="ignore", over="ignore"):
            return a.astype(np.float64) * b.astype(np.float64)
    return oracle.amsim(np.ascontiguousarray(a), np.ascontiguousarray(b), lut, M, E).astype(np.float64).reshape(a.shape)


def dots32(a, b, lut, M, E=8):
    """FP32 sums, ascending, of T(a_id, b_jd): [n, m]. The sum of an FP32 number
    and a product rounds to FP32 the same from float64 (table products have 16
    significant bits; for the native multiplier this is the fused
    multiply-add but for a double rounding)."""
    s = np.zeros((a.shape[0], b.shape[0]), np.float32)
    for d in range(a.shape[1]):
        with np.errstate(invalid="ignore", over="ignore"):
            s = (s.astype(np.float64) + products(a[:, None, d], b[None, :, d], lut, M, E)).astype(np.float32)
    return s


def weighted(w, x, seen, lut, M, E=8, weight_first=True):
    """sum over j (where seen) of T(w_ij, x_jd), and of the magnitudes."""
    out = np.zeros((w.shape[0], x.shape[1]))
    mag = np.zeros_like(out)
    for d in range(x.shape[1]):
        t = products(w, x[None, :, d], lut, M, E) if weight_first else products(x[None, :, d], w, lut, M, E)
        t = np.where(seen, t, 0.0)
        with np.errstate(invalid="ignore"):
            out[:, d] = t.sum(1)
            mag[:, d] = np.abs(t).sum(1)
    return out, mag


def causal_mask(n, m, causal=True):
    i, j = np.arange(n)[:, None], np.arange(m)[None]
    return (j <= i + m - n) if causal else np.ones((n, m), bool)


def attention(q, k, v, seen, scale, lut, M, E=8):
    """(o, lse, magnitudes of o's sums)."""
    s = dots32(q, k, lut, M, E)
    bad = (seen & ~(s < np.inf)).any(1)
    with np.errstate(invalid="ignore"):
        t = np.where(seen & (s < np.inf), s.astype(np.float64) * (scale * LOG2E), -np.inf)
    top = np.ceil(t.max(1, initial=-np.inf, keepdims=True))
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.exp2(t - top)
    e = np.where(e >= TINY, e, 0.0).astype(np.float32)
    total = e.astype(np.float64).sum(1)
    o, mag = weighted(e, v, seen, lut, M, E)
    div = np.where(total > 0, total, 1.0)[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        o, mag = np.where(total[:, None] > 0, o / div, 0.0), mag / div
        lse = (top[:, 0] + np.log2(total)) * math.log(2)
    o[bad], lse[bad] = np.nan, np.nan
    return o, lse, mag


def attention_grad(q, k, v, o, lse, dout, seen, scale, lut, M, E=8):
    """(dq, dk, dv) and their magnitudes; o and lse: what the forward pass left (FP32)."""
    delta = (dout.astype(np.float64) * o.astype(np.float64)).sum(1).astype(np.float32).astype(np.float64)
    with np.errstate(invalid="ignore"):
        x = dots32(q, k, lut, M, E).astype(np.float64) * (scale * LOG2E) - lse.astype(np.float64)[:, None] * LOG2E
    p = np.where(seen, np.exp2(np.where(seen, x, -np.inf)), 0.0)
    p = np.where(p >= TINY, p, 0.0).astype(np.float32)
    with np.errstate(invalid="ignore"):
        ds = (p.astype(np.float64) * (dots32(dout, v, lut, M, E).astype(np.float64) - delta[:, None]))
    ds = np.where(seen, ds, 0.0).astype(np.float32)
    ds = np.where(np.abs(ds) >= TINY, ds, np.float32(0))
    dq, mq = weighted(ds, k, seen, lut, M, E)
    dk, mk = weighted(np.ascontiguousarray(ds.T), q, seen.T, lut, M, E, weight_first=False)
    dv, mv = weighted(np.ascontiguousarray(p.T), dout, seen.T, lut, M, E, weight_first=False)
    return (dq * scale, dk * scale, dv), (mq * scale, mk * scale, mv)


def packed(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def attention_packed(q, k, v, cu_q, cu_k, causal, scale, lut, M, E=8):
    """The packed call: (o, lse, mag); rows of no sequence hold NaN in mag."""
    T, H, D = q.shape
    G = H // k.shape[1]
    o, lse, mag = np.zeros((T, H, D)), np.zeros((T, H)), np.full((T, H, D), np.nan)
    for b in range(len(cu_q) - 1):
        a, z, c, y = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        seen = causal_mask(z - a, y - c, causal)
        for h in range(H):
            o[a:z, h], lse[a:z, h], mag[a:z, h] = attention(q[a:z, h], k[c:y, h // G], v[c:y, h // G], seen, scale, lut, M, E)
    return o, lse, mag


def attention_packed_grad(q, k, v, o, lse, dout, cu_q, cu_k, causal, scale, lut, M, E=8):
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    grads = [np.zeros(x.shape) for x in (q, k, v)]
    mags = [np.zeros(x.shape) for x in (q, k, v)]
    for b in range(len(cu_q) - 1):
        a, z, c, y = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        seen = causal_mask(z - a, y - c, causal)
        for h in range(H):
            g = h // G
            one, mag = attention_grad(q[a:z, h], k[c:y, g], v[c:y, g], o[a:z, h], lse[a:z, h], dout[a:z, h], seen, scale, lut, M, E)
            grads[0][a:z, h], mags[0][a:z, h] = one[0], mag[0]
            for i in (1, 2):
                grads[i][c:y, g] += one[i]
                mags[i][c:y, g] += mag[i]
    return grads, mags


def near(got, want, mag, terms, what="", extra=0.0):
    """|got - want| <= (terms + 40) 2^-24 mag: an FP32 sum of `terms` exact
    products errs by at most one rounding (2^-24 of the magnitudes' sum) per
    addition; 32 more for joined chunks, the rest for the final scaling.
    extra: a further relative error of every term. Non-finite values match."""
    got, want, mag = (np.asarray(x, np.float64) for x in (got, want, mag))
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and not np.isinf(got[~inf]).any(), f"{what}: infinities differ"
    ok = np.isfinite(want)
    bound = ((terms + 40) * 2.0 ** -24 + extra) * mag[ok]
    err = np.abs(got[ok] - want[ok])
    assert (err <= bound + 2.0 ** -140).all(), f"{what}: {float((err / np.maximum(bound, 1e-300)).max()):.3g} times the bound"
