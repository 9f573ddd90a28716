"""The tensor helpers of quantize and GEMM on a given stream: whose memory
their outputs are (GPU)."""

import pytest
import torch

from gpu_helpers import announce, bf16_to_dev
from synth import bf16_matrix

import block_scaled_microscaling_amd as mx

pytestmark = pytest.mark.gpu

M, N, K = 32, 256, 512
CALLS = ["quantize", "quantize_2d", "quantize_sr", "quantize_2d_sr", "gemm", "gemm_tile",
         "gemm_swiglu", "shuffle_b", "gemm_bshuffled", "quantize_frag", "to_frag", "gemm_frag"]


def call_of(name, s):
    """A call of a stream (None: the current one) that returns a tuple of
    tensors, on inputs that are ready on s."""
    with torch.cuda.stream(s):
        x = bf16_to_dev(bf16_matrix((M, K), ("normal", 1.0, 0.0, 1.0), 1))
        w = bf16_to_dev(bf16_matrix((N, K), ("normal", 0.05, 0.0, 1.0), 2))
        a, b = mx.quantize(x), mx.quantize(w)
        shuffled = mx.shuffle_b(*b)
        fa, fb = mx.quantize_frag(x), mx.to_frag(*b)
    torch.cuda.synchronize()
    calls = {
        "quantize": lambda st: mx.quantize(x, stream=st),
        "quantize_2d": lambda st: mx.quantize_2d(x, stream=st),
        "quantize_sr": lambda st: mx.quantize_sr(x, 7, stream=st),
        "quantize_2d_sr": lambda st: mx.quantize_2d_sr(x, 7, stream=st),
        "gemm": lambda st: mx.gemm(*a, *b, stream=st),
        "gemm_tile": lambda st: mx.gemm_tile(*a, *b, stream=st),
        "gemm_swiglu": lambda st: mx.gemm_swiglu(*a, *b, stream=st),
        "shuffle_b": lambda st: mx.shuffle_b(*b, stream=st),
        "gemm_bshuffled": lambda st: mx.gemm_bshuffled(*a, *shuffled, N, stream=st),
        "quantize_frag": lambda st: mx.quantize_frag(x, stream=st),
        "to_frag": lambda st: mx.to_frag(*b, stream=st),
        "gemm_frag": lambda st: mx.gemm_frag(*fa, *fb, M, N, K, stream=st),
    }

    def call(st):
        r = calls[name](st)
        return tuple(t for t in r if t is not None) if isinstance(r, tuple) else (r,)
    return call


@pytest.mark.parametrize("name", CALLS)
def test_outputs_on_a_given_stream(name):
    """A block that the current stream has freed may still be used by what it
    has queued: a call on another stream never gets it, and its results stand
    beside that work."""
    announce(f"{name}: outputs on a given stream")
    s = torch.cuda.Stream()
    call = call_of(name, s)
    want = call(None)
    torch.cuda.synchronize()
    freed = [torch.empty_like(t) for t in want for _ in range(4)]
    at = {t.data_ptr() for t in freed}
    del freed
    got = call(s)
    torch.cuda.synchronize()
    assert not at & {t.data_ptr() for t in got}
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for i in range(3):
        torch.cuda._sleep(1_000_000)
        for t in want:
            for _ in range(3):
                torch.empty_like(t).fill_(3)
        got = call(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"round {i}"
