"""What the few-token operators promise beyond a case's values: how a result's
type, the batch beside a token, streams, threads and addresses may not change
it (GPU)."""

import threading

import numpy as np
import pytest
import torch

from fewtoken_cases import one_product_experts
from gpu_helpers import DEV, announce, bf16_to_dev, u8_to_dev
from oracle import fewtoken
from synth import bf16_matrix, f32_to_bf16_bits, random_codes, random_scales
from test_gpu_fewtoken import N01, check, choices, experts, run_moe

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


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,I,E,k", BY_PAIRS + BY_EXPERTS)
def test_moe_activation_to_its_last_bit(T, H, I, E, k, out):
    """Sums of one product each, so that the tolerance is a few roundings and
    a lost third part of an activation would show in FP32 results."""
    announce(f"moe of single products, T{T} H{H} I{I} E{E} k{k} {out}")
    x, ids, w, ex = one_product_experts(T, H, I, E, k, T + I)
    check(run_moe(x, ids, w, ex, out_dtype=out), *fewtoken.moe(x, ids, w, *ex))


@pytest.mark.parametrize("T,H,I,E,k", BY_PAIRS + BY_EXPERTS)
def test_moe_activation_next_to_fp32s_largest(T, H, I, E, k):
    """g = u = 2^64 (1 - 2^-12) exactly, so a = 2^128 (1 - 2^-11 + 2^-24) is
    finite in FP32 and above BF16's largest value; W2 takes 2^-11 of it."""
    announce(f"moe of the largest activations, T{T} H{H} I{I} E{E} k{k}")
    x = np.zeros((T, H), np.float32)
    x[:, 0], x[:, 1] = 2.0 ** 64 * (255 / 256), 15 * 2.0 ** 52
    c1 = np.zeros((E, 2 * I, H // 2), np.uint8)
    c1[:, :, 0] = 0x22                         # 1.0 and 1.0
    c2 = np.zeros((E, H, I // 2), np.uint8)
    c2[:, :, 0] = 0x01                         # 0.5
    ex = (c1, np.full((E, 2 * I, H // 32), 127, np.uint8), c2,
          np.full((E, H, I // 32), 117, np.uint8))
    ids = np.full((T, k), -1, np.int32)
    ids[:, 0] = np.arange(T) % E
    want = 2.0 ** 117 * (1 - 2.0 ** -11 + 2.0 ** -24)
    for out in (torch.float32, torch.bfloat16):
        got = run_moe(f32_to_bf16_bits(x), ids, np.ones((T, k), np.float32), ex, out_dtype=out)
        exact = torch.full((T, H), want, dtype=torch.float64).to(out).to(DEV)
        assert torch.equal(got, exact), got.flatten()[:4].tolist()


# ------------------------------------------------------------------ streams
def side_calls(s):
    """The three operators on inputs that are ready on s: name, call of a
    stream (None: the current one) that returns a tuple."""
    K, H, I, E, T = 512, 256, 96, 4, 24
    with torch.cuda.stream(s):
        x = bf16_to_dev(bf16_matrix((T, K), ("normal", 1.0, 0.0, 1.0), 1))
        w = mx.quantize(bf16_to_dev(bf16_matrix((H, K), ("normal", 0.05, 0.0, 1.0), 2)))
        h = bf16_to_dev(bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), 3))
        router = bf16_to_dev(bf16_matrix((E, H), ("normal", 0.1, 0.0, 1.0), 4))
        ids, p = choices(T, E, 2, 5)
        ids, p = torch.from_numpy(ids).to(DEV), torch.from_numpy(p).to(DEV)
        ex = tuple(u8_to_dev(a) for a in experts(E, H, I, 6))
    torch.cuda.synchronize()
    return [("gemv", lambda st: (mx.gemv(x, *w, stream=st),)),
            ("moe_route", lambda st: mx.moe_route(h, router, 2, stream=st)),
            ("moe", lambda st: (mx.moe(h, ids, p, *ex, stream=st),))]


def test_outputs_on_a_given_stream_are_that_streams_memory():
    """A block that the current stream has freed may still be used by what it
    has queued: a call on another stream never gets it."""
    announce("outputs on a given stream: whose memory")
    s = torch.cuda.Stream()
    for name, call in side_calls(s):
        want = call(None)
        torch.cuda.synchronize()
        freed = [torch.empty_like(t) for t in want for _ in range(4)]
        at = {t.data_ptr() for t in freed}
        del freed
        got = call(s)
        torch.cuda.synchronize()
        assert not at & {t.data_ptr() for t in got}, name
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_outputs_on_a_given_stream_beside_queued_work():
    """The current stream still has writes of freed blocks queued when the call
    on another stream is made and when it runs."""
    announce("outputs on a given stream beside queued work")
    s = torch.cuda.Stream()
    for name, call in side_calls(s):
        want = call(None)
        torch.cuda.synchronize()
        for i in range(6):
            torch.cuda._sleep(1_000_000)
            for t in want:
                for _ in range(3):
                    torch.empty_like(t).fill_(3)
            got = call(s)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), f"{name}, round {i}"
            del got


def test_stream_of_another_device_is_refused():
    """Before its handle is asked for: no other device need be there."""
    announce("stream of another device")
    other = torch.cuda.Stream(stream_id=0, device_index=1, device_type=1)
    assert other.device.index == 1
    for name, call in side_calls(torch.cuda.Stream()):
        with pytest.raises(ValueError, match="stream must be of the current device"):
            call(other)


# ------------------------------------------------------------------ threads
def test_calls_from_several_threads():
    """Products whose kernel takes LDS by K, from threads of their own streams
    at once: short K beside long ones."""
    announce("gemv from four threads")
    M, N = 16, 6200
    cases = []
    for i, K in enumerate((256, 8192, 1024, 4128)):
        x = bf16_matrix((M, K), N01, i)
        codes, scales = random_codes(N, K, i), random_scales(N, K, i)
        cases.append((bf16_to_dev(x), u8_to_dev(codes), u8_to_dev(scales)))
    want = [mx.gemv(*c, out_dtype=torch.float32) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(50):
                y = mx.gemv(*cases[i], out_dtype=torch.float32, stream=s)
                s.synchronize()
                if not torch.equal(y, want[i]):
                    wrong.append(i)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001  (reported by the test's own thread)
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


# ---------------------------------------------------------------- addresses
@pytest.mark.parametrize("T,H,I,E,k", BY_PAIRS + BY_EXPERTS)
def test_moe_result_at_any_four_byte_address(T, H, I, E, k):
    """y, ids and weights one element past a 16-byte boundary, nothing around y
    written."""
    announce(f"moe at 4-byte addresses, T{T} H{H} I{I} E{E} k{k}")
    x = bf16_matrix((T, H), ("normal", 1.0, 0.0, 1.0), T + H)
    ids, w = choices(T, E, k, I, 0.1)
    ex = tuple(u8_to_dev(a) for a in experts(E, H, I, E + k))
    def off(a):
        return torch.cat([torch.zeros(1, dtype=a.dtype), a.flatten()]).to(DEV)[1:].view(a.shape)

    ids, w = torch.from_numpy(ids), torch.from_numpy(w)
    want = mx.moe(bf16_to_dev(x), ids.to(DEV), w.to(DEV), *ex, out_dtype=torch.float32)
    for dt, lead in ((torch.float32, 1), (torch.bfloat16, 2)):
        buf = torch.full((T * H + 2 * lead,), 7.0, dtype=dt, device=DEV)
        out = buf[lead:-lead].view(T, H)
        assert out.data_ptr() % 16 == 4
        mx.moe(bf16_to_dev(x), off(ids), off(w), *ex, out=out)
        assert torch.equal(out, want.to(dt))
        assert torch.all(buf[:lead] == 7.0) and torch.all(buf[-lead:] == 7.0)


@pytest.mark.parametrize("M,N,K", [(1, 333, 512), (1, 333, 4128), (3, 333, 512), (16, 333, 512),
                                   (16, 6200, 512), (16, 14337, 512)])
def test_gemv_result_at_any_four_byte_address(M, N, K):
    announce(f"gemv at 4-byte addresses, {M} x {N} x {K}")
    x = bf16_to_dev(bf16_matrix((M, K), N01, M))
    w = u8_to_dev(random_codes(N, K, N)), u8_to_dev(random_scales(N, K, K))
    for dt, lead in ((torch.float32, 1), (torch.bfloat16, 2)):
        want = mx.gemv(x, *w, out_dtype=dt)
        buf = torch.full((M * N + 2 * lead,), 7.0, dtype=dt, device=DEV)
        out = buf[lead:-lead].view(M, N)
        assert out.data_ptr() % 16 == 4
        mx.gemv(x, *w, out=out)
        assert torch.equal(out, want)
        assert torch.all(buf[:lead] == 7.0) and torch.all(buf[-lead:] == 7.0)


# ------------------------------------------------------------------- router
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,H,E,k,spread", [
    (1, 4096, 8, 2, 1.0), (7, 296, 120, 8, 1.0), (13, 2856, 61, 4, 1.0), (64, 4096, 128, 8, 1.0),
    (5, 1024, 256, 8, 1.0), (3, 256, 1000, 32, 1.0),
    (9, 512, 48, 32, 12.0), (9, 512, 300, 32, 12.0),   # weights down to 2^-100
])
def test_route_weights_are_rounded_once(T, H, E, k, spread, renorm):
    """64-bit logits, exponentials and sums: a weight is FP32's nearest, or next
    to it where 64 bits are at a border (H 2^-53 of a logit's products)."""
    announce(f"route weights {T} x {H}, {E} top {k}, spread {spread}, renorm {renorm}")
    x = bf16_matrix((T, H), ("normal", spread, 0.0, 1.0), T)
    r = bf16_matrix((E, H), ("normal", 1.0 / np.sqrt(H), 0.0, 1.0), E)
    ids, w = mx.moe_route(bf16_to_dev(x), bf16_to_dev(r), k, renormalize=renorm)
    want_ids, want, _ = fewtoken.route(x, r, k, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    off = np.abs(w.double().cpu().numpy() - want) / np.maximum(want, 2.0 ** -126)
    assert off.max() <= 2.0 ** -24 * (1 + 2.0 ** -10), off.max() * 2.0 ** 24
