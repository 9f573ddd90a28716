"""Inputs of the few-token operators that several tests share."""

import numpy as np

from synth import f32_to_bf16_bits, random_codes, random_scales


def one_product_experts(T, H, I, E, k, seed):
    """(x, ids, weights, expert weights) whose every sum has one product that
    is not zero: a token has one activation, an expert's row of W2 one weight,
    so that a result shows the experts' activation to its last bit."""
    rng = np.random.default_rng(seed)
    x = np.zeros((T, H), np.float32)
    x[np.arange(T), rng.integers(0, H, T)] = rng.choice([-1.0, 1.0], T) * rng.uniform(0.5, 2.0, T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.uniform(0.5, 1.0, (T, k)).astype(np.float32)
    c1 = random_codes(E * 2 * I, H, seed + 1)
    s1 = random_scales(E * 2 * I, H, seed + 2, 126, 128)
    c2 = np.zeros((E * H, I // 2), np.uint8)
    place = rng.integers(0, I, E * H)
    c2[np.arange(E * H), place // 2] = rng.integers(1, 8, E * H) << (4 * (place % 2))
    s2 = random_scales(E * H, I, seed + 3, 126, 128)
    return f32_to_bf16_bits(x), ids, w, (c1.reshape(E, 2 * I, -1), s1.reshape(E, 2 * I, -1),
                                         c2.reshape(E, H, -1), s2.reshape(E, H, -1))
