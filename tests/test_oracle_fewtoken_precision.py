"""The few-token oracle's tolerances tell a lost part of a value from a rounding
(CPU): the experts' activation held in two BF16 values instead of FP32."""

import numpy as np
import torch

import oracle
from fewtoken_cases import one_product_experts
from oracle import fewtoken


def bf16_pieces(a, n):
    """The sum of a's first n BF16 pieces, each nearest to what is left."""
    rest, total = torch.from_numpy(a.astype(np.float32)), 0.0
    for _ in range(n):
        piece = rest.bfloat16().float()
        rest, total = rest - piece, total + piece.double().numpy()
    return total


def evaluate(x, ids, w, ex, pieces):
    """The experts in FP32, the activation in so many BF16 pieces (0: FP32)."""
    c1, s1, c2, s2 = ex
    T, k = ids.shape
    y = np.zeros((T, c2.shape[1]), np.float32)
    xf = torch.from_numpy(oracle.bf16_bits_to_f64(x)).float()
    inter = c1.shape[1] // 2
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            gu = torch.from_numpy(oracle.dequantize(c1[e], s1[e])).float() @ xf[t]
            g, u = gu[:inter], gu[inter:]
            a = (g / (1 + torch.exp(-g)) * u).numpy()
            held = bf16_pieces(a, pieces) if pieces else a.astype(np.float64)
            part = (oracle.dequantize(c2[e], s2[e]) @ held).astype(np.float32)
            y[t] += (w[t, j].astype(np.float64) * part).astype(np.float32)
    return y


def test_two_pieces_of_an_activation_are_outside_and_three_inside():
    x, ids, w, ex = one_product_experts(9, 96, 160, 4, 3, 1)
    y, tol = fewtoken.moe(x, ids, w, *ex)
    for pieces in (0, 3):
        assert not fewtoken.outside(evaluate(x, ids, w, ex, pieces), y, tol, False).any()
    off = fewtoken.outside(evaluate(x, ids, w, ex, 2), y, tol, False)
    assert off.mean() > 0.1, off.mean()


def test_sums_of_few_products_have_tolerances_of_few_roundings():
    """n products that are not zero round n times at most, whatever K is."""
    K = 4096
    x = np.zeros((2, K))
    x[0, 7], x[1, [5, 900, 4000]] = 3.0, [1.0, 2.0, -4.0]
    codes = np.full((1, K // 2), 0x22, np.uint8)               # 1.0
    scales = np.full((1, K // 32), 127, np.uint8)
    bits = oracle.bf16_bits_of(oracle.round_to_bf16(x))
    y, tol = fewtoken.gemv(bits, codes, scales)
    assert y.tolist() == [[3.0], [-1.0]]
    assert np.allclose(tol[:, 0], [3.0 * 2.0 ** -24, 3 * 7.0 * 2.0 ** -24], rtol=1e-6)
    _, dense = fewtoken.gemv(np.full((1, K), 0x3F80, np.uint16), codes, scales)
    assert np.allclose(dense, (K / 32 + 64) * 2.0 ** -24 * K, rtol=1e-6)
