"""What the few-token operators promise beyond a case's values: how a result's
type, the batch beside a token, streams, threads and addresses may not change
it (GPU)."""

import pytest
import torch

from gpu_helpers import DEV, announce, bf16_to_dev, u8_to_dev
from synth import bf16_matrix
from test_gpu_fewtoken import choices, experts, run_moe

import block_scaled_microscaling_amd as mx

pytestmark = pytest.mark.gpu

# Sizes that reach each way through the experts: T, H, I, E, top k.
BY_PAIRS = [(1, 512, 288, 8, 4), (6, 1024, 96, 20, 3)]
BY_EXPERTS = [
    (24, 256, 96, 4, 2),            # K split over a workgroup's waves
    (128, 1024, 512, 64, 8),        # a tile a wave, more than 8 pairs an expert
    (64, 288, 2048, 24, 2),         # a tile a wave in the first product alone
    (32, 736, 352, 8, 8),           # waves that share the activations
    (128, 2080, 160, 4, 4),
]


# ---------------------------------------------------------------- precision
@pytest.mark.parametrize("T,H,I,E,k", BY_PAIRS + BY_EXPERTS)
def test_moe_bf16_result_is_the_fp32_result_rounded(T, H, I, E, k):
    """The type of the result says how y is rounded and nothing else: sums and
    activations are the same, so BF16 results are FP32 results rounded once."""
    announce(f"moe BF16 against FP32, T{T} H{H} I{I} E{E} k{k}")
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), T + H)
    ids, w = choices(T, E, k, I, 0.1)
    ex = experts(E, H, I, E + k)
    wide = run_moe(x, ids, w, ex, out_dtype=torch.float32)
    got = run_moe(x, ids, w, ex, out_dtype=torch.bfloat16)
    differ = int((got != wide.bfloat16()).sum())
    assert differ == 0, f"{differ} of {got.numel()}"
