"""The few-token operators' larger paths where the small ones are tested
elsewhere: captured into graphs, on a side stream, past 4 GiB of weights and
past one grid's extent (GPU). Each size says which kernels it reaches."""

import numpy as np
import pytest
import torch

from gpu_helpers import DEV, announce, bf16_to_dev, u8_to_dev
from oracle import fewtoken
from synth import bf16_matrix, device_normal_bf16, device_random_bytes
from test_gpu_fewtoken import check, experts

import block_scaled_microscaling_amd as mx

pytestmark = pytest.mark.gpu

# T, K, H, I, E, top k of projection, router and experts one after the other.
LAYERS = [
    # One row group; the router in one launch; experts with K split over waves.
    (24, 512, 256, 96, 4, 2),
    # gemv with 70 KiB of LDS; the router in two launches; a tile a wave.
    (128, 2048, 1024, 96, 160, 8),
    # gemv whose waves share x; two launches by T; experts of shared activations.
    (257, 512, 1024, 96, 8, 3),
]


class Layer:
    def __init__(self, K, H, I, E, k, seed):
        self.k = k
        self.w = mx.quantize(bf16_to_dev(bf16_matrix((H, K), ("normal", 0.07, 0.0, 1.0), seed)))
        self.router = bf16_to_dev(bf16_matrix((E, H), ("normal", 0.1, 0.0, 1.0), seed + 1))
        self.ex = tuple(u8_to_dev(a) for a in experts(E, H, I, seed + 2))

    def __call__(self, x, stream=None):
        """Every result of the three, in order."""
        h = mx.gemv(x, *self.w, stream=stream)
        ids, p = mx.moe_route(h, self.router, self.k, stream=stream)
        return h, ids, p, mx.moe(h, ids, p, *self.ex, stream=stream)


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def inputs_of(T, K, n):
    return [bf16_to_dev(bf16_matrix((T, K), ("normal", 1.0, 0.0, 1.0), 30 + i)) for i in range(n)]


@pytest.mark.parametrize("T,K,H,I,E,k", LAYERS)
def test_larger_layer_captured_replays_equal_eager(T, K, H, I, E, k):
    announce(f"layer captured, {T} tokens, {E} experts")
    layer = Layer(K, H, I, E, k, 21)
    inputs = inputs_of(T, K, 4)
    x = inputs[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(x)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x)
    torch.cuda.synchronize()
    for i, inp in enumerate(inputs):
        x.copy_(inp)
        want = layer(x)
        torch.cuda.synchronize()
        for _ in range(2):
            for t in got:
                t.fill_(77)
            graph.replay()
            torch.cuda.synchronize()
            assert equal(got, want), f"replay {i}"
            _ = (inp.float() * 2).sum().item()


@pytest.mark.parametrize("T,K,H,I,E,k", LAYERS)
def test_larger_layer_on_a_side_stream(T, K, H, I, E, k):
    """All of a layer on a stream that is not the current one, whose own work
    goes on beside it; every result of every round."""
    announce(f"layer on a side stream, {T} tokens, {E} experts")
    layer = Layer(K, H, I, E, k, 11)
    inputs = inputs_of(T, K, 3)
    want = [layer(x) for x in inputs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for i in range(9):
        torch.cuda._sleep(500_000)
        for t in want[0]:
            torch.empty_like(t).fill_(3)
        got = layer(inputs[i % 3], stream=s)
        for t in want[0]:
            torch.empty_like(t).fill_(5)
        torch.cuda.synchronize()
        assert equal(got, want[i % 3]), f"round {i}"
        del got


def test_moe_by_experts_past_2_32_bytes():
    """W13 codes of 8.5 GiB and W2 codes of 4.3 GiB, twice as many pairs as
    experts, all on the experts at the marks."""
    announce("moe by experts, weights past 2^32 bytes")
    T, H, I, E, k = 128, 4096, 4352, 512, 8
    c1 = device_random_bytes((E, 2 * I, H // 2), 1)
    s1 = device_random_bytes((E, 2 * I, H // 32), 2, lo=116, hi=119)
    c2 = device_random_bytes((E, H, I // 2), 3)
    s2 = device_random_bytes((E, H, I // 32), 4, lo=116, hi=119)
    used = [0, (1 << 32) // (I * H), 2 * (1 << 32) // (I * H), E - 1]
    rng = np.random.default_rng(5)
    small = rng.integers(0, 4, (T, k))
    w = rng.random((T, k)).astype(np.float32)
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), 5)
    ids = torch.tensor(used, dtype=torch.int32)[torch.from_numpy(small)].to(DEV)
    got = mx.moe(bf16_to_dev(x), ids, torch.from_numpy(w).to(DEV), c1, s1, c2, s2,
                 out_dtype=torch.float32)
    at = torch.tensor(used, device=DEV)
    rows = [0, 1, 63, 127]
    want, tol = fewtoken.moe(x[rows], small[rows], w[rows],
                             *(t[at].cpu().numpy() for t in (c1, s1, c2, s2)))
    check(got[rows], want, tol)


@pytest.mark.parametrize("M,N,K,rows", [
    (1, 300_000_001, 32, 64),       # short rows
    (1, 4_300_003, 2080, 4),        # one row of x, a workgroup for four rows
    (2, 16_900_003, 32, 16),        # a tile a workgroup
    (6, 33_700_003, 32, 32),        # two tiles
    (5, 67_200_003, 256, 64),       # waves that share x
])
def test_gemv_of_more_workgroups_than_a_grids_row(M, N, K, rows):
    """2^20 workgroups of so many weight rows make a row of the grid: weight
    rows on both sides of each such mark, and the last ones."""
    announce(f"gemv of stacked workgroups, {M} x {N} x {K}")
    mark = rows << 20
    marks = list(range(mark, N, mark))
    assert marks
    codes = device_random_bytes((N, K // 2), 8)
    scales = device_random_bytes((N, K // 32), 9, lo=117, hi=137)
    x = device_normal_bf16((M, K), 10)
    got = mx.gemv(x, codes, scales)
    at = torch.tensor([0, 1] + [m + d for m in marks for d in (-2, -1, 0, 1)] + [N - 2, N - 1],
                      device=DEV)
    want, tol = fewtoken.gemv(x.view(torch.int16).cpu().numpy().view(np.uint16),
                              codes[at].cpu().numpy(), scales[at].cpu().numpy())
    check(got[:, at], want, tol)


def test_layer_captured_on_a_forked_stream():
    """Calls of a given stream inside a capture, joined before its end; what
    they allocate belongs to the graph."""
    announce("layer captured on a forked stream")
    T, K, H, I, E, k = LAYERS[0]
    layer = Layer(K, H, I, E, k, 41)
    inputs = inputs_of(T, K, 3)
    x = inputs[0].clone()
    s = torch.cuda.Stream()
    layer(x, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = layer(x, stream=s)
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for i, inp in enumerate(inputs):
        x.copy_(inp)
        want = layer(x)
        torch.cuda.synchronize()
        for _ in range(2):
            for t in got:
                t.fill_(77)
            graph.replay()
            torch.cuda.synchronize()
            assert equal(got, want), f"replay {i}"
            _ = (inp.float() * 2).sum().item()
