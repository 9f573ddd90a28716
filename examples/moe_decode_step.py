"""One decode step of a mixture-of-experts MLP block on MXFP4 weights.

    python examples/moe_decode_step.py [--tokens 1] [--hidden 2048]
        [--inter 768] [--experts 128] [--top-k 8] [--steps 200]

A few tokens' BF16 activations go through an output projection (gemv), the
router (moe_route) and the experts (moe); the residual is added by torch. The
weights are random (synthetic), quantized once with quantize. The step runs
eagerly and as a HIP graph; the program prints both times and checks the
last result against a float64 evaluation on the CPU.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_microscaling_amd as mx  # noqa: E402


class MoeBlock:
    """h = x + x Wo^T; y = h + sum over the chosen experts, weights in MXFP4."""

    def __init__(self, hidden, inter, experts, top_k, seed=0, device="cuda:0"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=gen, device=device) * cols ** -0.5
            return w.bfloat16()

        def expert_weights(rows, cols):
            codes, scales = mx.quantize(weight(experts * rows, cols))
            return codes.view(experts, rows, -1), scales.view(experts, rows, -1)

        self.top_k = top_k
        self.proj = mx.quantize(weight(hidden, hidden))
        self.router = weight(experts, hidden)
        self.w13 = expert_weights(2 * inter, hidden)      # per expert [W_gate; W_up]
        self.w2 = expert_weights(hidden, inter)

    def __call__(self, x):
        h = x + mx.gemv(x, *self.proj)
        ids, weights = mx.moe_route(h, self.router, self.top_k)
        return h + mx.moe(h, ids, weights, *self.w13, *self.w2)

    def reference(self, x):
        """The same in float64 on the CPU, with the step's own BF16 roundings
        (of the projection, of h, and of the experts' sum)."""
        import oracle
        bits = oracle.bf16_bits_of
        to64 = lambda t: torch.from_numpy(                     # noqa: E731
            oracle.bf16_bits_to_f64(t.view(torch.int16).cpu().numpy().view("uint16")))
        dq = lambda c, s: torch.from_numpy(                    # noqa: E731
            oracle.dequantize(c.cpu().numpy(), s.cpu().numpy()))
        rounded = lambda t: torch.from_numpy(                  # noqa: E731
            oracle.bf16_bits_to_f64(bits(oracle.round_to_bf16(t.numpy()))))
        x = to64(x)
        h = rounded(x + rounded(x @ dq(*self.proj).T))
        p = torch.softmax(h @ to64(self.router).T, dim=1)
        w, ids = p.topk(self.top_k, dim=1)
        w = w / w.sum(dim=1, keepdim=True)
        y = torch.zeros_like(h)
        inter = self.w2[0].shape[2] * 2
        for e in ids.unique().tolist():
            t, j = torch.nonzero(ids == e, as_tuple=True)
            gu = h[t] @ dq(self.w13[0][e], self.w13[1][e]).T
            act = torch.nn.functional.silu(gu[:, :inter]) * gu[:, inter:]
            y.index_add_(0, t, act @ dq(self.w2[0][e], self.w2[1][e]).T * w[t, j][:, None])
        return h + rounded(y)


def timed(fn, steps):
    """Microseconds a call, among others."""
    fn()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(steps):
        fn()
    torch.cuda.synchronize()
    return (time.perf_counter() - start) / steps * 1e6


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=1)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inter", type=int, default=768)
    p.add_argument("--experts", type=int, default=128)
    p.add_argument("--top-k", type=int, default=8)
    p.add_argument("--steps", type=int, default=200)
    a = p.parse_args(argv)

    block = MoeBlock(a.hidden, a.inter, a.experts, a.top_k)
    x = torch.randn((a.tokens, a.hidden), device="cuda:0").bfloat16()
    eager = timed(lambda: block(x), a.steps)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x)                                  # warm-up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x)
    replay = timed(graph.replay, a.steps)

    want = block.reference(x)
    # A BF16 result is off by half a step, 2^-8 of it, and by what h's own
    # rounding to the other neighbour (2^-8 of h) moves through the experts.
    error = ((y.double().cpu() - want).abs() / (want.abs() + want.abs().max())).max().item()
    print(f"{a.tokens} token(s), hidden {a.hidden}, {a.experts} experts of {a.inter}, "
          f"top {a.top_k}: {eager:.1f} us a step eagerly, {replay:.1f} us as a graph; "
          f"largest error {error:.1e} of the output's range", flush=True)
    return error


if __name__ == "__main__":
    sys.exit(0 if main() < 3 * 2.0 ** -8 else 1)
