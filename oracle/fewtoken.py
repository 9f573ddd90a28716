"""Float64 oracle of the few-token operators: products of BF16 rows with MXFP4
weights, the mixture-of-experts router and the experts' SwiGLU MLPs.

TEST INFRASTRUCTURE, as the rest of this package: NumPy only, no code shared
with the HIP path. Each function returns the exact value (up to float64) and
how far an FP32 evaluation of the same sums may be from it:

  * a sum of K products, each exact in FP32: a product passes at most the 32
    additions of one matrix instruction, one per following instruction (K /
    32) and those of the partial sums' reduction (at most 32), each at most
    half a unit in the last place of a partial sum, which S = sum |products|
    bounds: |y - y_exact| <= (K / 32 + 64) 2^-24 S; and where only n products
    are not zero only n additions round, so n in place of K / 32 + 64 if less;
  * silu(g) u from inexact g, u: |silu'| <= 1.1, so |a - a_exact| <= 1.1 dg
    (|u| + du) + |silu(g)| du + eval, where eval covers the FP32 evaluation
    (rounded exponent argument, exp, add, divide, product): (2 |g| + 16)
    2^-24 |a|, and |a| itself where exp(-g) passes FP32's range (g < -87);
  * the activation is FP32 between the two products, also where three BF16
    values hold it (3 x 8 bits of significand): then it is three sums, of
    which the two of the rests hardly count, and the two additions of them.
"""

import numpy as np

from .mxfp4_ref import bf16_bits_to_f64, dequantize

U = 2.0 ** -24
TINY = 2.0 ** -126      # products below FP32's normal range may count as zero


def _sum_tol(K, x, w, pieces=1):
    """How far an FP32 x @ w^T over K may be off, x of so many pieces."""
    x, w = np.abs(x), np.abs(w).T
    S, n = x @ w, (x > 0).astype(np.float64) @ (w > 0)
    return np.minimum(K / 32 + 63 + pieces, pieces * n) * U * S + pieces * K * TINY


def gemv(x_bits, codes, scales):
    """(y, tol) float64 [M, N]: y = x dq(W)^T and the FP32 tolerance."""
    x = bf16_bits_to_f64(np.asarray(x_bits, dtype=np.uint16))
    w = dequantize(codes, scales)
    return x @ w.T, _sum_tol(x.shape[1], x, w)


def route(x_bits, router_bits, top_k, renormalize):
    """(ids int32, weights, tol) [T, top_k]."""
    x = bf16_bits_to_f64(np.asarray(x_bits, dtype=np.uint16))
    r = bf16_bits_to_f64(np.asarray(router_bits, dtype=np.uint16))
    logits = x @ r.T
    order = np.argsort(-logits, axis=1, kind="stable")[:, :top_k].astype(np.int32)
    away = logits - logits.max(axis=1, keepdims=True)
    p = np.exp(away)
    p /= p.sum(axis=1, keepdims=True)
    w = np.take_along_axis(p, order, axis=1)
    # exp of an argument rounded to FP32, 2 units of exp, the sum over E, the
    # quotient; the same again for the chosen ones' sum when renormalized.
    far = np.abs(np.take_along_axis(away, order, axis=1))
    # (the spread matters where the weight does: terms of the sum are weighted by p)
    mean_far = (p * np.abs(away)).sum(axis=1, keepdims=True)
    rel = (far + mean_far + r.shape[0] + 16) * U
    if renormalize:
        w = w / w.sum(axis=1, keepdims=True)
        rel = rel + (far.max(axis=1, keepdims=True) + mean_far + r.shape[0] + 32) * U
    return order, w, rel * w + 2.0 ** -126


def moe(x_bits, ids, weights, w13_codes, w13_scales, w2_codes, w2_scales):
    """(y, tol) float64 [T, H]."""
    x = bf16_bits_to_f64(np.asarray(x_bits, dtype=np.uint16))
    ids = np.asarray(ids)
    weights = np.asarray(weights, dtype=np.float64)
    T, top_k = ids.shape
    E, two_i = np.asarray(w13_codes).shape[:2]
    I = two_i // 2
    H = x.shape[1]
    y = np.zeros((T, H))
    tol = np.zeros((T, H))
    size = np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if t.size == 0:
            continue
        w13 = dequantize(w13_codes[e], w13_scales[e])
        w2 = dequantize(w2_codes[e], w2_scales[e])
        gu = x[t] @ w13.T
        dgu = _sum_tol(H, x[t], w13)
        g, u, dg, du = gu[:, :I], gu[:, I:], dgu[:, :I], dgu[:, I:]
        with np.errstate(over="ignore"):
            silu = g / (1.0 + np.exp(-g))
        a = silu * u
        da = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du
        da += (2 * np.abs(g) + 16) * U * np.abs(a) + np.where(g < -87, np.abs(a), 0.0)
        part = a @ w2.T
        dpart = da @ np.abs(w2).T + _sum_tol(I, np.abs(a) + da, w2, pieces=3)
        wj = weights[t, j][:, None]
        np.add.at(y, t, wj * part)
        np.add.at(tol, t, np.abs(wj) * dpart)
        np.add.at(size, t, np.abs(wj) * (np.abs(part) + dpart))
    # The weighted sum: a product and at most top_k additions each.
    return y, tol + (top_k + 1) * U * size


def outside(got, want, tol, bf16):
    """Mask of results further off than tol, and, for BF16 results, half a
    step (2^-8 of the value) more."""
    got = np.asarray(got, dtype=np.float64)
    allowed = tol + (2.0 ** -8 * (np.abs(want) + tol) if bf16 else 0.0)
    return ~(np.abs(got - want) <= allowed)
