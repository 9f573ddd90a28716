"""Inputs and checks shared by the FP8 GPU tests."""

import numpy as np
import torch

from gpu_helpers import DEV
from oracle import fp8

TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def bf16_of(x):
    """float64 array -> (BF16 tensor on the GPU, its values in 64 bits)."""
    t = torch.from_numpy(np.asarray(x, np.float32)).bfloat16()
    return t.to(DEV), t.double().numpy()


def codes_to_dev(codes, kind):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(TORCH[kind]).to(DEV)


def to_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def operand(rows, K, block, kind, scales, seed, std=1.0):
    """(codes tensor, scales tensor, values in 64 bits) of an operand: a few
    values far out, scales of the quantizer's or, FP32, of amax / largest."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, K)) * std * np.where(rng.random((rows, K)) < 0.01, 50, 1)
    codes, s = fp8.quantize(x, block, kind)
    if scales == "fp32":
        s = (fp8.scale_values(s) * rng.uniform(0.5, 1.0, s.shape)).astype(np.float32)
    return codes_to_dev(codes, kind), to_dev(s), fp8.values(codes, s, block, kind)


def check_product(got, a, b, K, fp8_path, what=""):
    """A GEMM's result against the product of the operands' values. fp8_path:
    BF16 results may have come from the FP8 matrix instructions."""
    C, S = fp8.product(a, b)
    tol = fp8.exact_tolerance(C, S, K)
    if got.dtype == torch.bfloat16:
        if fp8_path:
            tol = tol + fp8.grouped_tolerance(a, b)
        tol = tol + fp8.BF16_HALF_STEP * (np.abs(C) + tol)
    off = np.abs(got.double().cpu().numpy() - C)
    bad = np.argwhere(~(off <= tol))
    assert bad.size == 0, f"{what}: {len(bad)} of {C.size} outside, first {bad[:4].tolist()}"
