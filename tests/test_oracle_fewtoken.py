"""Pins of the few-token oracle: hand-worked values, closed forms and an FP32
evaluation inside its tolerances (CPU)."""

import numpy as np
import torch

import oracle
from oracle import fewtoken
from synth import bf16_matrix, f32_to_bf16_bits


def _bits(a):
    return f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


def test_gemv_hand_worked():
    # Row 0: code 1 (0.5) under scale 2^1 -> 1.0 everywhere; row 1: code 0xF
    # (-6) under 2^-1 -> -3. x = 2 in every place: 32 * 2 and 32 * -6.
    codes = np.array([[0x11] * 16, [0xFF] * 16], dtype=np.uint8)
    scales = np.array([[128], [126]], dtype=np.uint8)
    y, tol = fewtoken.gemv(_bits(np.full((1, 32), 2.0)), codes, scales)
    assert y.tolist() == [[64.0, -192.0]]
    assert np.all(tol < 1e-3) and np.all(tol > 0)


def test_route_orders_by_logit_then_index():
    # Logits 1, 3, 3, -2: the two equal ones come in index order.
    x = np.zeros((1, 8))
    x[0, 0] = 1.0
    r = np.zeros((4, 8))
    r[:, 0] = [1.0, 3.0, 3.0, -2.0]
    ids, w, tol = fewtoken.route(_bits(x), _bits(r), 3, False)
    assert ids.tolist() == [[1, 2, 0]]
    e = np.exp(np.array([1.0, 3.0, 3.0, -2.0]))
    assert np.allclose(w[0], (e / e.sum())[[1, 2, 0]], rtol=1e-12)
    ids, w, tol = fewtoken.route(_bits(x), _bits(r), 3, True)
    assert abs(w.sum() - 1.0) < 1e-12 and np.all(tol < 1e-5)


def test_moe_closed_form_and_absent_experts():
    # H = I = 32, one expert: Wg = Wu = 1 / 32 everywhere, W2 = 1 in column 0.
    codes1 = np.full((1, 64, 16), 0x22, np.uint8)          # 1.0
    scales1 = np.full((1, 64, 1), 127 - 5, np.uint8)       # 2^-5
    codes2 = np.zeros((1, 32, 16), np.uint8)
    codes2[:, :, 0] = 0x02
    scales2 = np.full((1, 32, 1), 127, np.uint8)
    x = _bits(np.full((3, 32), 3.0))                       # g = u = 3
    ids = np.array([[0, 0], [-1, 0], [1, -7]])
    w = np.array([[0.5, 0.25], [np.nan, 2.0], [1.0, 1.0]], np.float32)
    y, tol = fewtoken.moe(x, ids, w, codes1, scales1, codes2, scales2)
    a = 9.0 / (1.0 + np.exp(-3.0))
    assert np.allclose(y[0], 0.75 * a, rtol=1e-12)
    assert np.allclose(y[1], 2.0 * a, rtol=1e-12)
    assert np.all(y[2] == 0.0) and np.all(tol[2] == 0.0)


def test_fp32_evaluations_stay_inside_the_tolerances():
    rng = np.random.default_rng(5)
    T, H, I, E, k = 5, 288, 96, 6, 3
    x = bf16_matrix((T, H), ("normal", 1.0, 0.01, 20.0), 1)
    c1, s1 = oracle.quantize(bf16_matrix((E * 2 * I, H), ("normal", 0.05, 0.0, 1.0), 2))
    c2, s2 = oracle.quantize(bf16_matrix((E * H, I), ("normal", 0.05, 0.0, 1.0), 3))
    xt = torch.from_numpy(oracle.bf16_bits_to_f64(x)).float()
    w1 = torch.from_numpy(oracle.dequantize(c1, s1)).float()
    y, tol = fewtoken.gemv(x, c1, s1)
    assert not fewtoken.outside((xt @ w1.T).numpy(), y, tol, False).any()
    assert not fewtoken.outside((xt @ w1.T).bfloat16().float().numpy(), y, tol, True).any()
    # A mistake of one part in 2^12 of S is far outside.
    assert fewtoken.outside((xt @ w1.T).numpy() * (1 + 2.0 ** -8), y, tol, False).mean() > 0.5

    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[2, 1] = -1
    w = rng.random((T, k)).astype(np.float32)
    c1, s1 = c1.reshape(E, 2 * I, -1), s1.reshape(E, 2 * I, -1)
    c2, s2 = c2.reshape(E, H, -1), s2.reshape(E, H, -1)
    y, tol = fewtoken.moe(x, ids, w, c1, s1, c2, s2)
    got = np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            gu = torch.from_numpy(oracle.dequantize(c1[e], s1[e])).float() @ xt[t]
            a = torch.nn.functional.silu(gu[:I]) * gu[I:]
            got[t] += w[t, j] * (torch.from_numpy(oracle.dequantize(c2[e], s2[e])).float()
                                 @ a).double().numpy()
    assert not fewtoken.outside(got, y, tol, False).any()

    r = bf16_matrix((16, H), ("normal", 0.06, 0.0, 1.0), 9)
    ids, wr, tol = fewtoken.route(x, r, 4, True)
    p = torch.softmax(xt @ torch.from_numpy(oracle.bf16_bits_to_f64(r)).float().T, dim=1)
    top = p.topk(4, dim=1)
    assert np.array_equal(top.indices.numpy(), ids)
    got = (top.values / top.values.sum(dim=1, keepdim=True)).double().numpy()
    # (torch's logits are FP32 here: only their order of magnitude is checked)
    assert np.all(np.abs(got - wr) <= 64 * tol)
