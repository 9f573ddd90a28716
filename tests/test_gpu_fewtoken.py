"""Few-token operators against the float64 oracle on the GPU: gemv, the
mixture-of-experts router and the experts.

Tolerances are the oracle's (oracle/fewtoken.py): the roundings that FP32
sums of exact products can take, and half a step of a BF16 result.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

import block_scaled_microscaling_amd as mx
import oracle
from gpu_helpers import DEV, announce, bf16_to_dev, u8_to_dev
from oracle import fewtoken
from synth import (bf16_matrix, device_normal_bf16, device_random_bytes, random_codes,
                   random_scales)

pytestmark = pytest.mark.gpu

N01 = ("normal", 1.0, 0.01, 20.0)


def host(t):
    return t.double().cpu().numpy()


def check(got, want, tol, what=""):
    bad = fewtoken.outside(host(got), want, tol, got.dtype == torch.bfloat16)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, first "
                           f"{np.argwhere(bad)[:5].tolist()}")


# ------------------------------------------------------------------- gemv
@pytest.mark.parametrize("M", [1, 2])
def test_gemv_decodes_every_code_and_scale_exactly(M):
    """One column of ones picks each weight: codes 0..15 in each place of a
    block under scale bytes 0..252, each result the exact value."""
    announce(f"gemv decode of every code under every scale, {M} rows")
    K, N = 32, 16 * 253
    codes = np.zeros((N, 16), np.uint8)
    scales = np.repeat(np.arange(253, dtype=np.uint8), 16)[:, None]
    for place in (0, 1, 7, 8, 18, 31):
        codes[:] = 0
        code = np.tile(np.arange(16, dtype=np.uint8), 253)
        codes[:, place // 2] = code << (4 * (place % 2))
        x = np.zeros((M, K), np.uint16)
        x[M - 1, place] = 0x3F80                # 1.0
        y = mx.gemv(bf16_to_dev(x), u8_to_dev(codes), u8_to_dev(scales),
                    out_dtype=torch.float32)
        want = oracle.dequantize(codes, scales)[:, place]
        got = host(y)[M - 1]
        normal = np.abs(want) >= 2.0 ** -126
        assert np.array_equal(got[normal], want[normal]), place
        # Below the normal range: the value or zero.
        low = ~normal
        assert np.all((got[low] == want[low]) | (got[low] == 0.0)), place


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 16, 256), (1, 17, 32), (2, 15, 64), (3, 33, 96), (1, 1000, 224),
    (5, 48, 288), (8, 257, 2048), (15, 31, 4128), (16, 16, 512), (17, 40, 1056), (33, 65, 736),
    (48, 64, 1024), (64, 96, 544), (65, 19, 320), (130, 35, 96), (1, 4096, 8192), (7, 512, 14336),
    # Enough tiles for two a workgroup; one row over many rounds of K.
    (3, 5000, 352), (5, 6177, 736), (16, 6200, 544), (40, 4001, 96), (2, 24, 32), (1, 9, 33024),
    (6, 40, 33024),
    # One row of up to 16, 32 and 64 blocks, and tails.
    (1, 1000, 512), (1, 77, 544), (1, 333, 1024), (1, 1029, 1056), (1, 30, 2048), (1, 31, 2080),
    # Enough workgroups for their waves to share x: one unit of K, odd ones.
    (6, 14400, 256), (5, 14341, 800), (16, 14337, 4128), (50, 3600, 288), (9, 20000, 544),
])
def test_gemv_matches_the_oracle(M, N, K, out):
    announce(f"gemv {M}x{N}x{K} {out}")
    x = bf16_matrix((M, K), N01, M + N)
    codes, scales = random_codes(N, K, N + K), random_scales(N, K, K + 1)
    got = mx.gemv(bf16_to_dev(x), u8_to_dev(codes), u8_to_dev(scales), out_dtype=out)
    assert got.shape == (M, N) and got.dtype == out
    check(got, *fewtoken.gemv(x, codes, scales))


def test_gemv_on_quantized_weights_of_every_magnitude():
    """Weights as quantize writes them over the whole BF16 range."""
    announce("gemv on quantized weights of every magnitude")
    M, N, K = 3, 130, 640
    w = (bf16_matrix((N, K), ("normal", 1.0, 0.0, 1.0), 3).astype(np.uint32))
    exps = np.random.default_rng(4).integers(-100, 100, size=(N, 1))
    w64 = np.ldexp(oracle.bf16_bits_to_f64(w.astype(np.uint16)), exps)
    bits = oracle.bf16_bits_of(oracle.round_to_bf16(w64))
    codes, scales = mx.quantize(bf16_to_dev(bits))
    x = bf16_matrix((M, K), ("normal", 0.01, 0.0, 1.0), 5)
    got = mx.gemv(bf16_to_dev(x), codes, scales, out_dtype=torch.float32)
    check(got, *fewtoken.gemv(x, codes.cpu().numpy(), scales.cpu().numpy()))


@pytest.mark.parametrize("M", [1, 2, 20])
def test_gemv_subnormal_activations(M):
    """BF16 subnormals of x against weights of up to 2^127: nothing counts as
    zero before the product."""
    announce(f"gemv subnormal x, {M} rows")
    N, K = 48, 288
    x = np.random.default_rng(M).integers(1, 128, size=(M, K)).astype(np.uint16)
    codes, scales = random_codes(N, K, 1), np.full((N, K // 32), 252, np.uint8)
    got = mx.gemv(bf16_to_dev(x), u8_to_dev(codes), u8_to_dev(scales), out_dtype=torch.float32)
    check(got, *fewtoken.gemv(x, codes, scales))


def test_gemv_strided_rows_canaries_and_unaligned_scales():
    """x is every third row of a larger buffer whose other rows hold NaN, the
    scales start at an odd address, and nothing around y is written."""
    announce("gemv strided rows")
    for M, N, K, dt in [(5, 37, 288, torch.bfloat16), (18, 16, 96, torch.float32)]:
        x = bf16_matrix((M, K), N01, 7)
        big = torch.full((3 * M, K + 40), float("nan"), dtype=torch.bfloat16, device=DEV)
        xs = big[::3, 16:16 + K]
        xs.copy_(bf16_to_dev(x))
        codes, scales = random_codes(N, K, 8), random_scales(N, K, 9)
        flat = torch.full((N * K // 32 + 2,), 255, dtype=torch.uint8, device=DEV)
        flat[1:-1] = u8_to_dev(scales).flatten()
        buf = torch.full((M * N + 64,), 7.0, dtype=dt, device=DEV)
        out = buf[32:32 + M * N].view(M, N)
        mx.gemv(xs, u8_to_dev(codes), flat[1:-1].view(N, K // 32), out=out)
        check(out, *fewtoken.gemv(x, codes, scales))
        assert torch.all(buf[:32] == 7.0) and torch.all(buf[32 + M * N:] == 7.0)


def test_gemv_non_finite_inputs_stay_in_their_row():
    announce("gemv with NaN and Inf rows, NaN scales")
    M, N, K = 6, 50, 352
    x = bf16_matrix((M, K), N01, 1)
    codes, scales = random_codes(N, K, 2), random_scales(N, K, 3)
    want, tol = fewtoken.gemv(x, codes, scales)
    bad = x.copy()
    bad[1, 350] = 0x7FC0                       # NaN in the last block
    bad[4, 3] = 0x7F80                         # Inf
    scales_nan = scales.copy()
    scales_nan[7, 10] = 255                    # a weight row's last scale
    got = mx.gemv(bf16_to_dev(bad), u8_to_dev(codes), u8_to_dev(scales_nan),
                  out_dtype=torch.float32)
    rows = [0, 2, 3, 5]
    cols = [n for n in range(N) if n != 7]
    check(got[rows][:, cols], want[np.ix_(rows, cols)], tol[np.ix_(rows, cols)])
    assert torch.isnan(got[1]).all() and torch.isnan(got[:, 7]).all()
    assert not torch.isfinite(got[4, cols]).any()


def test_gemv_of_shared_rows_strided_and_not_finite():
    """Many weight rows, so that waves share x: rows of a larger buffer of NaN,
    two rows and one weight row not finite, nothing around y written."""
    announce("gemv with shared x, strided, NaN and Inf")
    M, N, K = 19, 6001, 864
    x = bf16_matrix((M, K), N01, 1)
    codes, scales = random_codes(N, K, 2), random_scales(N, K, 3)
    want, tol = fewtoken.gemv(x, codes, scales)
    bad = x.copy()
    bad[1, 863] = 0x7FC0                       # NaN in the last block
    bad[18, 3] = 0x7F80                        # Inf
    scales_nan = scales.copy()
    scales_nan[6000, 26] = 255                 # the last weight row's last scale
    big = torch.full((2 * M, K + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    xs = big[::2, 8:8 + K]
    xs.copy_(bf16_to_dev(bad))
    buf = torch.full((M * N + 64,), 7.0, device=DEV)
    out = buf[32:32 + M * N].view(M, N)
    got = mx.gemv(xs, u8_to_dev(codes), u8_to_dev(scales_nan), out=out)
    rows = [m for m in range(M) if m not in (1, 18)]
    check(got[rows][:, :N - 1], want[rows][:, :N - 1], tol[rows][:, :N - 1])
    assert torch.isnan(got[1]).all() and torch.isnan(got[:, N - 1]).all()
    assert not torch.isfinite(got[18]).any()
    assert torch.all(buf[:32] == 7.0) and torch.all(buf[32 + M * N:] == 7.0)


@pytest.mark.parametrize("M,N", [(8, 300), (16, 700), (9, 10241)])
def test_gemv_decodes_codes_and_scales_in_every_kernel(M, N):
    """x of ones in one block each: each result is a sum of 32 exact values."""
    announce(f"gemv of ones, {M} rows x {N}")
    K = 32 * 24
    codes, scales = random_codes(N, K, N), random_scales(N, K, M)
    x = np.zeros((M, K), np.uint16)
    for m in range(M):
        b = (m * 5 + 3) % 24
        x[m, 32 * b:32 * b + 32] = 0x3F80      # 1.0
    got = mx.gemv(bf16_to_dev(x), u8_to_dev(codes), u8_to_dev(scales), out_dtype=torch.float32)
    want = oracle.dequantize(codes, scales).reshape(N, 24, 32).sum(2)
    want = np.stack([want[:, (m * 5 + 3) % 24] for m in range(M)])
    # 32 values of at most 12 half-steps of one scale add exactly.
    assert np.array_equal(host(got), want)


@pytest.mark.parametrize("M,N", [(1, 2000), (6, 2000), (30, 2000), (30, 6000)])
def test_gemv_gives_the_same_bits_every_time(M, N):
    announce(f"gemv repeated, {M} rows x {N}")
    K = 4128
    x = bf16_to_dev(bf16_matrix((M, K), N01, 1))
    w = u8_to_dev(random_codes(N, K, 2)), u8_to_dev(random_scales(N, K, 3))
    first = mx.gemv(x, *w, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(mx.gemv(x, *w, out_dtype=torch.float32), first)


def test_gemv_past_2_32_bytes():
    """Codes of 4.6 GiB: rows on both sides of the 2 and 4 GiB marks."""
    announce("gemv codes past 2^32 bytes")
    N, K, M = 1_200_003, 8192, 2
    codes = device_random_bytes((N, K // 2), 5)
    scales = device_random_bytes((N, K // 32), 6, lo=117, hi=137)
    x = device_normal_bf16((M, K), 7)
    got = mx.gemv(x, codes, scales, out_dtype=torch.float32)
    mark = (1 << 31) // (K // 2)
    rows = torch.tensor([0, 1, mark - 1, mark, mark + 1, 2 * mark - 1, 2 * mark, 2 * mark + 1,
                         N - 2, N - 1], device=DEV)
    want, tol = fewtoken.gemv(x.view(torch.int16).cpu().numpy().view(np.uint16),
                              codes[rows].cpu().numpy(), scales[rows].cpu().numpy())
    check(got[:, rows], want, tol)


def test_gemv_with_more_rows_than_a_grid_has_threads():
    """300 million weight rows: more than 2^32 threads."""
    announce("gemv of 3e8 rows")
    N, K = 300_000_001, 32
    codes = device_random_bytes((N, K // 2), 8)
    scales = device_random_bytes((N, 1), 9, lo=117, hi=137)
    x = device_normal_bf16((1, K), 10)
    got = mx.gemv(x, codes, scales)
    block = 4 << 20                            # rows of a grid's x extent
    rows = torch.tensor([0, 3, block - 1, block, 7 * block + 5, 71 * block - 1, 71 * block, N - 2,
                         N - 1], device=DEV)
    want, tol = fewtoken.gemv(x.view(torch.int16).cpu().numpy().view(np.uint16),
                              codes[rows].cpu().numpy(), scales[rows].cpu().numpy())
    check(got[:, rows], want, tol)


# ------------------------------------------------------------------ router
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,H,E,k", [
    (1, 8, 1, 1), (1, 4096, 8, 2), (3, 24, 5, 5), (7, 520, 61, 4), (9, 2856, 64, 8),
    (17, 1000, 65, 1), (33, 64, 200, 32), (3, 296, 127, 9), (5, 512, 128, 4),
    (4, 72, 129, 3), (64, 2048, 128, 8), (2, 512, 1024, 32), (100, 72, 256, 6),
])
def test_route_matches_the_oracle(T, H, E, k, renorm):
    announce(f"route {T}x{H} {E} top {k} renorm {renorm}")
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), T)
    r = bf16_matrix((E, H), ("normal", 2.0 / np.sqrt(H), 0.0, 1.0), E)
    ids, w = mx.moe_route(bf16_to_dev(x), bf16_to_dev(r), k, renormalize=renorm)
    want_ids, want, tol = fewtoken.route(x, r, k, renorm)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), want_ids)
    check(w, want, tol)


def test_route_ties_and_extreme_logits():
    """Copied experts tie exactly and come in index order; logits far apart
    underflow to zero weights; x of zeros ties every expert."""
    announce("route ties")
    H, E, k = 136, 70, 9
    x = bf16_matrix((5, H), ("normal", 1.0, 0.0, 1.0), 1)
    x[3] = 0
    x[4, 1:] = 0
    x[4, 0] = 0x4900                           # 2^19: logits far apart
    r = bf16_matrix((E, H), ("normal", 0.1, 0.0, 1.0), 2)
    for e in range(E):
        r[e] = r[e % 7]                        # ten copies of each of seven
    for renorm in (False, True):
        ids, w = mx.moe_route(bf16_to_dev(x), bf16_to_dev(r), k, renormalize=renorm)
        want_ids, want, tol = fewtoken.route(x, r, k, renorm)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        check(w, want, tol)
    assert ids.cpu().numpy()[3].tolist() == list(range(k))


def test_route_nan_rows_and_strides():
    """A NaN token has distinct ids below E and NaN weights; its neighbours,
    rows of a strided buffer, are as ever. Canaries stay."""
    announce("route NaN and strides")
    T, H, E, k = 6, 264, 19, 4
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), 3)
    r = bf16_matrix((E, H), ("normal", 0.1, 0.0, 1.0), 4)
    want_ids, want, tol = fewtoken.route(x, r, k, True)
    big = torch.full((2 * T, H + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    xs = big[::2, 8:8 + H]
    xs.copy_(bf16_to_dev(x))
    xs[2, 5] = float("nan")
    ib = torch.full((T * k + 32,), 77, dtype=torch.int32, device=DEV)
    wb = torch.full((T * k + 32,), 77.0, device=DEV)
    ids, w = ib[16:-16].view(T, k), wb[16:-16].view(T, k)
    mx.moe_route(xs, bf16_to_dev(r), k, ids=ids, weights=w,
                 workspace=mx.moe_route_workspace(T, H, E))
    rows = [0, 1, 3, 4, 5]
    assert np.array_equal(ids.cpu().numpy()[rows], want_ids[rows])
    check(w[rows], want[rows], tol[rows])
    nan_ids = ids.cpu().numpy()[2]
    assert len(set(nan_ids.tolist())) == k and nan_ids.min() >= 0 and nan_ids.max() < E
    assert torch.isnan(w[2]).all()
    assert torch.all(ib[:16] == 77) and torch.all(ib[-16:] == 77)
    assert torch.all(wb[:16] == 77) and torch.all(wb[-16:] == 77)
    # One expert that is NaN for every token is never among the first E - 1.
    r2 = r.copy()
    r2[7, 0] = 0x7FC0
    ids, _ = mx.moe_route(bf16_to_dev(x), bf16_to_dev(r2), E - 1)
    assert not (ids == 7).any()


# ----------------------------------------------------------------- experts
def experts(E, H, I, seed):
    c1, s1 = random_codes(E * 2 * I, H, seed), random_scales(E * 2 * I, H, seed + 1, 116, 121)
    c2, s2 = random_codes(E * H, I, seed + 2), random_scales(E * H, I, seed + 3, 116, 121)
    return (c1.reshape(E, 2 * I, -1), s1.reshape(E, 2 * I, -1), c2.reshape(E, H, -1),
            s2.reshape(E, H, -1))


def choices(T, E, k, seed, absent=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < absent] = -1
    return ids, rng.random((T, k)).astype(np.float32)


def run_moe(x, ids, w, ex, **kw):
    return mx.moe(bf16_to_dev(x), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV),
                  *(u8_to_dev(a) for a in ex), **kw)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,I,E,k,absent", [
    (1, 32, 32, 1, 1, 0.0), (1, 64, 96, 4, 2, 0.0), (1, 2048, 768, 16, 8, 0.0),
    (2, 288, 224, 3, 3, 0.0), (5, 1056, 544, 10, 3, 0.33), (9, 96, 64, 2, 2, 0.0),
    (16, 256, 512, 40, 6, 0.5), (17, 160, 288, 1, 1, 0.0), (33, 64, 32, 6, 4, 0.1),
    (64, 128, 96, 128, 8, 0.0), (32, 96, 128, 1024, 32, 0.0), (1024, 32, 64, 3, 1, 0.2),
    (1, 512, 4096, 2, 2, 0.0), (3, 4096, 32, 5, 2, 0.0),
    # Enough tiles for one a wave: many pairs an expert; fewer pairs than
    # experts, and tiles that fill no workgroup.
    (128, 1024, 512, 64, 8, 0.1), (16, 288, 288, 1000, 16, 0.2), (2, 160, 1056, 9, 9, 0.3),
    (1, 96, 224, 40, 32, 0.5),
    # Fewer pairs than experts with many bytes; by experts: up to two pairs an
    # expert (K split over waves, and a tile a wave), and more.
    (6, 1024, 1152, 20, 3, 0.1), (6, 3680, 1856, 20, 3, 0.0), (20, 1024, 1152, 20, 3, 0.1),
    (5, 1696, 4640, 6, 2, 0.0), (14, 1120, 1760, 24, 3, 0.1), (9, 3648, 2240, 14, 2, 0.0),
    (40, 1024, 512, 64, 4, 0.0), (28, 1024, 512, 64, 4, 0.1), (64, 288, 544, 64, 5, 0.0),
    (40, 160, 288, 3, 2, 0.1),
    (64, 128, 96, 16, 8, 0.0), (100, 32, 32, 2, 1, 0.5),
    # By pairs: up to 16, 32 and 64 blocks of H.
    (3, 512, 96, 20, 4, 0.1), (2, 544, 32, 12, 3, 0.0), (1, 1024, 64, 6, 5, 0.2),
    (2, 1056, 32, 16, 4, 0.0), (1, 2048, 96, 8, 4, 0.0), (1, 2080, 64, 8, 4, 0.3),
    # Many pairs an expert: waves that share the activations, one unit of K or
    # less and several; H that leaves half a workgroup; rounds of workgroups.
    (32, 736, 352, 8, 8, 0.0), (64, 992, 96, 8, 6, 0.3), (40, 1056, 800, 8, 5, 0.0),
    (128, 2080, 160, 4, 4, 0.1), (32, 512, 512, 16, 8, 0.0),
])
def test_moe_matches_the_oracle(T, H, I, E, k, absent, out):
    announce(f"moe T{T} H{H} I{I} E{E} k{k} absent {absent} {out}")
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), T + H)
    ids, w = choices(T, E, k, I, absent)
    ex = experts(E, H, I, E + k)
    got = run_moe(x, ids, w, ex, out_dtype=out)
    assert got.shape == (T, H) and got.dtype == out
    check(got, *fewtoken.moe(x, ids, w, *ex))


@pytest.mark.parametrize("T", [4, 20])
def test_moe_absent_repeated_and_out_of_range_experts(T):
    """Tokens with no expert here give zeros (NaN weights beside them are
    not read into the sum), every pair may name the same expert, an expert
    may be named twice by a token, and ids far outside count as absent."""
    announce(f"moe unusual choices, {T} tokens")
    H, I, E, k = 96, 160, 5, 4
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), 1)
    ex = experts(E, H, I, 3)
    ids, w = choices(T, E, k, 2)
    ids[0] = [-1, 5, 2**31 - 1, -2**31]
    w[0] = np.nan
    ids[1] = 3
    ids[2] = [4, -1, 4, 1000]
    w[2, 1] = np.inf
    got = run_moe(x, ids, w, ex, out_dtype=torch.float32)
    assert torch.all(got[0] == 0.0)
    check(got, *fewtoken.moe(x, ids, w, *ex))
    none = run_moe(x, np.full((T, k), E, np.int32), w, ex)
    assert torch.all(none == 0.0)
    one = np.full((T, k), 2, np.int32)
    check(run_moe(x, one, w[3:4].repeat(T, 0), ex), *fewtoken.moe(x, one, w[3:4].repeat(T, 0), *ex))


@pytest.mark.parametrize("T", [8, 24])
def test_moe_non_finite_tokens_stay_alone(T):
    announce(f"moe NaN and overflowing tokens among {T}")
    H, I, E, k = 64, 96, 4, 2
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), 1)
    ex = experts(E, H, I, 5)
    ids, w = choices(T, E, k, 6)
    want, tol = fewtoken.moe(x, ids, w, *ex)
    bad = x.copy()
    bad[3, 10] = 0x7FC0                        # NaN
    bad[5, :] = 0x7F00                         # 2^127: the activation overflows
    got = run_moe(bad, ids, w, ex, out_dtype=torch.float32)
    rows = [t for t in range(T) if t not in (3, 5)]
    check(got[rows], want[rows], tol[rows])
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[5]).any()


def test_moe_many_pairs_an_expert_with_tokens_not_finite():
    """Non-finite tokens, an expert whose pairs are one token's many times, one
    that is every token's, one of none; equal bits each time."""
    announce("moe of many pairs, NaN and Inf tokens")
    T, H, I, E, k = 48, 1120, 288, 8, 6
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), 1)
    ex = experts(E, H, I, 5)
    ids, w = choices(T, E, k, 6)
    ids[:, 0] = 2
    ids[ids == 7] = 2
    ids[9] = 5
    want, tol = fewtoken.moe(x, ids, w, *ex)
    bad = x.copy()
    bad[3, 10] = 0x7FC0                        # NaN
    bad[40, :] = 0x7F00                        # 2^127: the activation overflows
    rows = [t for t in range(T) if t not in (3, 40)]
    for dt in (torch.float32, torch.bfloat16):
        got = run_moe(bad, ids, w, ex, out_dtype=dt)
        check(got[rows], want[rows], tol[rows])
        assert torch.isnan(got[3]).all() and not torch.isfinite(got[40]).any()
        for _ in range(3):
            assert torch.equal(run_moe(bad, ids, w, ex, out_dtype=dt)[rows], got[rows])


@pytest.mark.parametrize("T", [5, 11])
def test_moe_strides_canaries_and_bits(T):
    """x rows strided among NaN, unaligned scales, canaries around y and the
    workspace, and the same bits from every run."""
    announce(f"moe strides and canaries, {T} tokens")
    H, I, E, k = 160, 96, 7, 3
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), 1)
    c1, s1, c2, s2 = experts(E, H, I, 7)
    ids, w = choices(T, E, k, 8, 0.2)
    big = torch.full((2 * T, H + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    big[::2, :H] = bf16_to_dev(x)
    off = lambda s: torch.cat([torch.full((1,), 255, dtype=torch.uint8, device=DEV),  # noqa: E731
                               u8_to_dev(s).flatten()])[1:].view(s.shape)
    need = mx.moe_workspace(T, H, I, k).numel()
    wsb = torch.full((need + 256,), 99, dtype=torch.uint8, device=DEV)
    args = (big[::2, :H], torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV),
            u8_to_dev(c1), off(s1), u8_to_dev(c2), off(s2))
    for dt in (torch.float32, torch.bfloat16):
        buf = torch.full((T * H + 64,), 7.0, dtype=dt, device=DEV)
        out = buf[32:-32].view(T, H)
        mx.moe(*args, out=out, workspace=wsb[128:128 + need])
        check(out, *fewtoken.moe(x, ids, w, c1, s1, c2, s2))
        assert torch.all(buf[:32] == 7.0) and torch.all(buf[-32:] == 7.0)
        assert torch.all(wsb[:128] == 99) and torch.all(wsb[128 + need:] == 99)
        for _ in range(3):
            assert torch.equal(mx.moe(*args, out_dtype=dt), out)


@pytest.mark.parametrize("T,k,E", [(1, 6, 48), (3, 4, 48), (64, 6, 48), (64, 6, 8), (100, 8, 10)])
def test_moe_workspace_may_hold_anything(T, k, E):
    """A workspace of NaN, and absent experts whose part of it nothing writes."""
    announce(f"moe with a workspace of NaN, {T} tokens, {E} experts")
    H, I = 512, 288
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), 1)
    ids, w = choices(T, E, k, 2, 0.4)
    ex = experts(E, H, I, 3)
    ws = torch.full((mx.moe_workspace(T, H, I, k).numel(),), 255, dtype=torch.uint8, device=DEV)
    for dt in (torch.float32, torch.bfloat16):
        check(run_moe(x, ids, w, ex, out_dtype=dt, workspace=ws), *fewtoken.moe(x, ids, w, *ex))


def test_moe_expert_weights_past_2_32_bytes():
    """W13 codes of 4.5 GiB and W2 codes of 2.3 GiB: the last experts."""
    announce("moe weights past 2^32 bytes")
    T, H, I, E, k = 3, 2048, 2304, 1024, 2
    c1 = device_random_bytes((E, 2 * I, H // 2), 1)
    s1 = device_random_bytes((E, 2 * I, H // 32), 2, lo=116, hi=119)
    c2 = device_random_bytes((E, H, I // 2), 3)
    s2 = device_random_bytes((E, H, I // 32), 4, lo=116, hi=119)
    ids = np.array([[1023, 455], [911, 0], [456, 910]], np.int32)
    w = np.array([[0.5, 0.25], [1.0, 0.125], [0.75, 0.3]], np.float32)
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), 5)
    got = mx.moe(bf16_to_dev(x), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), c1,
                 s1, c2, s2, out_dtype=torch.float32)
    used = sorted(set(ids.flatten().tolist()))
    at = torch.tensor(used, device=DEV)
    small = np.array([[used.index(e) for e in row] for row in ids])
    want, tol = fewtoken.moe(x, small, w, *(t[at].cpu().numpy() for t in (c1, s1, c2, s2)))
    check(got, want, tol)


# ------------------------------------------------- together, streams, graphs
def layer(x, w, ex, top_k, router):
    """Projection, router and experts, as a decode step runs them."""
    h = mx.gemv(x, *w)
    ids, p = mx.moe_route(h, router, top_k)
    return mx.moe(h, ids, p, *ex)


def layer_parts(seed):
    K, H, I, E = 192, 256, 96, 12
    w = mx.quantize(bf16_to_dev(bf16_matrix((H, K), ("normal", 0.07, 0.0, 1.0), seed)))
    router = bf16_to_dev(bf16_matrix((E, H), ("normal", 0.1, 0.0, 1.0), seed + 1))
    ex = tuple(u8_to_dev(a) for a in experts(E, H, I, seed + 2))
    return K, w, router, ex


def test_layer_on_a_side_stream():
    """Inputs written and outputs read on a stream that is not the current
    one, workspaces freed at once: the same bits."""
    announce("layer on a side stream")
    K, w, router, ex = layer_parts(11)
    x = bf16_to_dev(bf16_matrix((4, K), ("normal", 1.0, 0.0, 1.0), 2))
    want = layer(x, w, ex, 3, router)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = torch.empty_like(want)
    h = mx.gemv(x, *w)
    torch.cuda.synchronize()
    for _ in range(20):
        ids, p = mx.moe_route(h, router, 3, stream=s)
        mx.moe(h, ids, p, *ex, out=y, stream=s)
        # Memory that torch hands out next must not be the workspaces'.
        _ = torch.full((1 << 16,), 3.0, device=DEV)
    s.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("T", [1, 9])
def test_layer_captured_replays_equal_eager(T):
    announce(f"layer captured, {T} tokens")
    K, w, router, ex = layer_parts(21)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    inputs = [bf16_to_dev(bf16_matrix((T, K), ("normal", 1.0, 0.0, 1.0), 30 + i))
              for i in range(4)]
    x.copy_(inputs[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(x, w, ex, 3, router)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, w, ex, 3, router)
    torch.cuda.synchronize()
    for i, inp in enumerate(inputs):
        x.copy_(inp)
        want = layer(x, w, ex, 3, router)
        torch.cuda.synchronize()
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {i}"
        _ = (inp.float() * 2).sum().item()


@pytest.mark.parametrize("tokens", [1, 5])
def test_example_of_a_decode_step(tokens):
    """examples/moe_decode_step.py: projection, router and experts together,
    eagerly and as a graph. Its result is BF16 and passes three roundings of
    2^-8, each of a value no larger than the output's range."""
    announce(f"example of a decode step, {tokens} tokens")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "moe_decode_step.py")
    spec = importlib.util.spec_from_file_location("moe_decode_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    error = example.main(["--tokens", str(tokens), "--hidden", "256", "--inter", "96",
                          "--experts", "12", "--top-k", "3", "--steps", "5"])
    assert error < 3 * 2.0 ** -8


def test_refusals_of_the_tensor_layer():
    announce("refusals")
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    c = torch.zeros((8, 32), dtype=torch.uint8, device=DEV)
    s = torch.zeros((8, 2), dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        mx.gemv(x, c, s[:, :1].contiguous())
    with pytest.raises(ValueError):
        mx.gemv(x.t(), c, s)                       # rows not contiguous
    with pytest.raises(ValueError):
        mx.gemv(x, c, s, out=torch.zeros((4, 9), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        mx.gemv(x, c, s, out_dtype=torch.float16)
    with pytest.raises(mx.Mxfp4Error):
        mx.gemv(x[:0], c, s)                       # no tokens
    with pytest.raises(mx.Mxfp4Error):
        mx.gemv(x[:1].expand(4, 64), c, s)         # rows on top of each other
    with pytest.raises(mx.Mxfp4Error):
        mx.moe_route(x, x, 5)                      # more than there are
    with pytest.raises(mx.Mxfp4Error):
        mx.moe_route(x, x, 0)
    many = torch.zeros((300, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        mx.moe_route(x, many, 2, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(TypeError):
        mx.moe_route(x, many, 2, workspace=torch.empty(1 << 20, device=DEV))
    with pytest.raises(TypeError):
        mx.gemv(x, c, s, stream=0)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    ex = (torch.zeros((2, 64, 32), dtype=torch.uint8, device=DEV),
          torch.zeros((2, 64, 2), dtype=torch.uint8, device=DEV),
          torch.zeros((2, 64, 16), dtype=torch.uint8, device=DEV),
          torch.zeros((2, 64, 1), dtype=torch.uint8, device=DEV))
    assert mx.moe(x, ids, ids.float(), *ex).shape == (4, 64)
    with pytest.raises(TypeError):
        mx.moe(x, ids.long(), ids.float(), *ex)
    with pytest.raises(ValueError):
        mx.moe(x, ids, ids.float()[:2], *ex)
    with pytest.raises(ValueError):
        mx.moe(x, ids, ids.float(), ex[0][:, :32].contiguous(), *ex[1:])
    with pytest.raises(ValueError):
        mx.moe(x, ids, ids.float(), *ex, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
