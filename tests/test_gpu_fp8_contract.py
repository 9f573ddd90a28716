"""The FP8 operators as a program calls them (GPU): captured and replayed, on
other streams beside queued work, from several threads, past 2^31 and 2^32
bytes, and what the tensor layer refuses."""

import threading

import numpy as np
import pytest
import torch

import block_scaled_microscaling_amd as mx
from fp8_cases import bf16_of
from gpu_helpers import DEV, announce

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def raw(t):
    """Bits, so that NaN codes compare too."""
    return t.view(torch.uint8) if t.dtype != torch.uint8 else t


def layer(M, H, I, seed, out=torch.bfloat16):
    """Inputs and weights of a gated MLP, and its training step on them."""
    rng = np.random.default_rng(seed)
    x, dy = (bf16_of(rng.normal(size=(M, H)))[0] for _ in range(2))
    w13 = bf16_of(rng.normal(size=(2 * I, H)) / np.sqrt(H))[0]
    w2 = bf16_of(rng.normal(size=(H, I)) / np.sqrt(I))[0]
    weights = [mx.quantize_fp8_2d(w, block_rows=128) for w in (w13, w2)]

    def step(stream=None):
        s = dict(stream=stream)
        (wq, ws, wt, wts), (vq, vs, vt, vts) = weights
        xq, xs, xt, xts = mx.quantize_fp8_2d(x, **s)
        aq, as_, act, gu = mx.gemm_fp8_swiglu(xq, xs, wq, ws, want_act=True, want_gu=True, **s)
        y = mx.gemm_fp8(aq, as_, vq, vs, **s)
        dq, ds = mx.quantize_fp8(dy, **s)
        dact = mx.gemm_fp8(dq, ds, vt, vts, **s)
        gq, gs, gt, gts = mx.swiglu_fp8_backward(dact, gu, **s)
        dx = mx.gemm_fp8(gq, gs, wt, wts, **s)
        dw = mx.gemm_fp8(gt, gts, xt, xts, out_dtype=out, **s)
        return y, dx, dw, aq, as_, gu, gt, gts
    return x, dy, step


SIZES = [(1, 256, 128), (48, 272, 256), (200, 384, 384), (2900, 512, 1536)]


@pytest.mark.parametrize("M,H,I", SIZES)
def test_training_step_captured_and_replayed(M, H, I):
    announce(f"FP8 MLP step in a graph {M}x{H}x{I}")
    x, dy, step = layer(M, H, I, 1, torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        torch.manual_seed(i)
        x.copy_(torch.randn(x.shape, device=DEV))
        dy.copy_(torch.randn(x.shape, device=DEV))
        want = [raw(t).clone() for t in step()]
        torch.cuda.synchronize()
        for t in held:
            raw(t).fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(raw(t), w) for t, w in zip(held, want)), f"replay {i}"
        assert held[0].isfinite().all() and held[2].isfinite().all()
        _ = (x.float() * 2).sum().item()


def test_two_graphs_of_the_same_weights():
    """Each graph has workspaces of its own: replays of two, one behind the
    other and on two streams, give what eager runs give."""
    announce("two FP8 graphs")
    made, kept = [], []
    for seed in (1, 2):
        x, dy, step = layer(40, 256, 256, seed)
        want = [raw(t).clone() for t in step()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step()
        made.append((g, held, want, torch.cuda.Stream()))
        kept.append(step)                     # what the graph reads
    for i in range(4):
        for g, held, want, s in made:
            for t in held:
                raw(t).zero_()
        torch.cuda.synchronize()
        for g, held, want, s in made:
            if i % 2:
                with torch.cuda.stream(s):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        for g, held, want, s in made:
            assert all(torch.equal(raw(t), w) for t, w in zip(held, want)), i


@pytest.mark.parametrize("M,H,I", SIZES)
def test_outputs_on_a_given_stream(M, H, I):
    """Outputs of a call on a given stream are that stream's memory, and stand
    beside what other streams have queued."""
    announce(f"FP8 MLP step on a given stream {M}x{H}x{I}")
    x, dy, step = layer(M, H, I, 3)
    s = torch.cuda.Stream()
    want = [raw(t).clone() for t in step()]
    torch.cuda.synchronize()
    for i in range(3):
        freed = [torch.empty_like(t) for t in want for _ in range(3)]
        at = {t.data_ptr() for t in freed}
        torch.cuda._sleep(1_000_000)
        for t in freed:
            t.fill_(7)
        del freed, t
        got = step(s)
        torch.cuda.synchronize()
        assert not at & {t.data_ptr() for t in got}
        assert all(torch.equal(raw(a), b) for a, b in zip(got, want)), i


def test_calls_from_several_threads():
    announce("FP8 calls from four threads")
    steps = [layer(*size, 5)[2] for size in SIZES]
    wants = [[raw(t).clone() for t in step()] for step in steps]
    torch.cuda.synchronize()
    wrong = []

    def work(step, want):
        s = torch.cuda.Stream()
        for _ in range(8):
            got = step(s)
            s.synchronize()
            if not all(torch.equal(raw(a), b) for a, b in zip(got, want)):
                wrong.append(1)
    threads = [threading.Thread(target=work, args=a) for a in zip(steps, wants)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not wrong


def test_given_outputs_and_workspace():
    announce("FP8 given outputs")
    x = bf16_of(np.random.default_rng(0).normal(size=(70, 272)))[0]
    codes = torch.empty((70, 272), dtype=F8, device=DEV)
    scales = torch.empty((70, 3), dtype=torch.uint8, device=DEV)
    r = mx.quantize_fp8(x, codes=codes, scales=scales)
    assert r[0] is codes and r[1] is scales
    w, ws = mx.quantize_fp8(x, block_rows=128)
    out = torch.empty((70, 70), dtype=torch.float32, device=DEV)
    assert mx.gemm_fp8(codes, scales, w, ws, out=out) is out
    assert torch.equal(out, mx.gemm_fp8(codes, scales, w, ws, out_dtype=torch.float32))
    a, sa = mx.quantize_fp8(x[:, :256].contiguous())
    w, ws = mx.quantize_fp8(torch.randn(256, 256, device=DEV).bfloat16(), block_rows=128)
    space = mx.gemm_fp8_swiglu_workspace(70, 128, 256)
    space.fill_(255)
    got = mx.gemm_fp8_swiglu(a, sa, w, ws, workspace=space)
    want = mx.gemm_fp8_swiglu(a, sa, w, ws)
    assert all(torch.equal(raw(p), raw(q)) for p, q in zip(got, want))
    with pytest.raises(ValueError, match="workspace must hold"):
        mx.gemm_fp8_swiglu(a, sa, w, ws, workspace=space[:-1])


def test_refusals_of_the_tensor_layer():
    announce("FP8 refusals")
    x = torch.randn(32, 256, device=DEV).bfloat16()
    a, sa = mx.quantize_fp8(x)
    b, sb = mx.quantize_fp8(x, block_rows=128)
    bf, sbf = mx.quantize_fp8(x, block_rows=128, scale_dtype=torch.float32)
    rows, srows = mx.quantize_fp8(x, scale_dtype=torch.float32)
    for bad, kind in [
            (lambda: mx.quantize_fp8(x[:, :250]), ValueError),
            (lambda: mx.quantize_fp8(x.t()), ValueError),
            (lambda: mx.quantize_fp8(x[:0]), ValueError),
            (lambda: mx.quantize_fp8(x, block_rows=32), ValueError),
            (lambda: mx.quantize_fp8(x, dtype=torch.bfloat16), TypeError),
            (lambda: mx.quantize_fp8(x, scale_dtype=torch.bfloat16), TypeError),
            (lambda: mx.quantize_fp8(x, codes=a[:, :128]), ValueError),
            (lambda: mx.quantize_fp8(x[:, 4:132]), mx.Mxfp4Error),
            (lambda: mx.gemm_fp8(a, sa, b, sbf), TypeError),
            (lambda: mx.gemm_fp8(rows, srows, rows, srows), ValueError),
            (lambda: mx.gemm_fp8(a, sa, b.view(torch.float8_e5m2), sb), TypeError),
            (lambda: mx.gemm_fp8(a, sa[:, :1], b, sb), ValueError),
            (lambda: mx.gemm_fp8(a, sa, b[:, :128], sb), ValueError),
            (lambda: mx.gemm_fp8(a, sa, b, sb, out_dtype=torch.float16), TypeError),
            (lambda: mx.gemm_fp8(a[:0], sa[:0], b, sb), mx.Mxfp4Error),
            (lambda: mx.gemm_fp8(a, sa, b, sb, stream=3), TypeError),
            (lambda: mx.gemm_fp8_swiglu(a, sa, b, sb), ValueError),
            (lambda: mx.swiglu_fp8_backward(x[:, :128], x), ValueError),
            (lambda: mx.swiglu_fp8_backward(x, x), ValueError),
            (lambda: mx.swiglu_fp8_backward(x, torch.cat([x, x], 1), dtype=torch.uint8), TypeError)]:
        with pytest.raises(kind):
            bad()
    torch.cuda.synchronize()
    assert mx.gemm_fp8(a, sa, b, sb).isfinite().all()


# ------------------------------------------------- past 2^31 and 2^32 bytes
def values(c, s, block, rows):
    """Values of some rows, in 64 bits."""
    s = torch.exp2(s[rows // block].double() - 127).repeat_interleave(128, 1)[:, : c.shape[1]]
    return c[rows].double() * s


def codes_of(R, K, seed, block=1):
    """Random E4M3 codes without NaN, and scales near 1."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = torch.randint(0, 0x70, (R, K), dtype=torch.uint8, generator=g, device=DEV)
    s = torch.randint(118, 122, (-(-R // block), -(-K // 128)), dtype=torch.uint8, generator=g,
                      device=DEV)
    return c.view(F8), s


def sampled(n, seed):
    """Some rows, the first and the last, and those around 2^31 and 2^32 bytes
    are among any even spread."""
    g = torch.Generator().manual_seed(seed)
    r = torch.cat([torch.tensor([0, n - 1]), torch.randint(0, n, (40,), generator=g),
                   torch.linspace(0, n - 1, 23).long()])
    return r.unique().to(DEV)


@pytest.mark.parametrize("M,N,K,out", [
    (70001, 512, 65536, torch.bfloat16),     # A past 2^32 bytes, large tiles
    (70001, 130, 65536, torch.float32),      # tiles of 128 rows
    (3, 70001, 65536, torch.bfloat16),       # B past 2^32 bytes, few rows
    (600, 70001, 65536, torch.bfloat16),
    (66000, 36000, 128, torch.bfloat16),     # C past 2^32 bytes
    (36000, 33001, 32, torch.float32)])
def test_gemm_past_32_bits(M, N, K, out):
    announce(f"gemm_fp8 {M}x{N}x{K} {out}")
    a, sa = codes_of(M, K, 1)
    b, sb = codes_of(N, K, 2, 128)
    got = mx.gemm_fp8(a, sa, b, sb, out_dtype=out)
    m, n = sampled(M, 1), sampled(N, 2)
    va, vb = values(a, sa, 1, m), values(b, sb, 128, n)
    want = va @ vb.t().contiguous()          # all values are positive: C is S
    g = got[m][:, n].double()
    # BF16: its half step, 2^-9 of S for the FP8 instructions' groups of eight.
    tol = ((K + 8) * 2.0 ** -24 + (2.0 ** -8 + 2.0 ** -9 if out == torch.bfloat16 else 0)) * want
    assert ((g - want).abs() <= tol).all()


@pytest.mark.parametrize("M", [1, 2, 17, 100, 300, 9000])
@pytest.mark.parametrize("N,K", [(1, 16), (16, 128), (100, 272), (128, 384), (129, 128)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gemm_with_few_scales(M, N, K, out):
    """Scale arrays of one byte to a few, at the end of an allocation's page."""
    announce(f"gemm_fp8 few scales {M}x{N}x{K} {out}")
    a, sa = codes_of(M, K, 1)
    b, sb = codes_of(N, K, 2, 128)
    got = mx.gemm_fp8(a, sa, b, sb, out_dtype=out).double()
    rows = torch.arange(M, device=DEV), torch.arange(N, device=DEV)
    want = values(a, sa, 1, rows[0]) @ values(b, sb, 128, rows[1]).t().contiguous()
    tol = ((K + 8) * 2.0 ** -24 + (2.0 ** -8 + 2.0 ** -9 if out == torch.bfloat16 else 0)) * want
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("I", [32512, 32768])
def test_swiglu_of_few_rows_and_large_weights(I):
    """Weights whose half ends just below and just above 2^32 bytes."""
    M, K = 5, 131072
    announce(f"gemm_fp8_swiglu {M}x{K}x{I}")
    a, sa = codes_of(M, K, 1)
    w, sw = codes_of(2 * I, K, 2, 128)
    sw = (sw - 30).contiguous()
    codes, scales, act, gu = mx.gemm_fp8_swiglu(a, sa, w, sw, want_act=True, want_gu=True)
    m, n = torch.arange(M, device=DEV), sampled(2 * I, 4)
    want = values(a, sa, 1, m) @ values(w, sw, 128, n).t().contiguous()
    tol = (K + 8) * 2.0 ** -24 + 2.0 ** -8 + 2.0 ** -9
    assert ((gu[:, n].double() - want).abs() <= tol * want).all()
    again = mx.quantize_fp8(act)
    assert torch.equal(raw(codes), raw(again[0])) and torch.equal(scales, again[1])


def test_swiglu_and_backward_past_32_bits():
    M, H, I = 70001, 128, 32768
    announce(f"gemm_fp8_swiglu and backward {M}x{H}x{I}")
    a, sa = codes_of(M, H, 1)
    w, sw = codes_of(2 * I, H, 2, 128)
    sw = (sw - 20).contiguous()
    codes, scales, act, gu = mx.gemm_fp8_swiglu(a, sa, w, sw, want_act=True, want_gu=True)
    m, n = sampled(M, 3), sampled(2 * I, 4)
    want = values(a, sa, 1, m) @ values(w, sw, 128, n).t().contiguous()
    assert ((gu[m][:, n].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -16) * want).all()
    again = mx.quantize_fp8(act[m].contiguous())
    assert torch.equal(raw(codes)[m], raw(again[0])) and torch.equal(scales[m], again[1])
    del codes, scales
    d, ds, dt, dts = mx.swiglu_fp8_backward(act, gu)
    # A part of the rows alone gives the same rows, and its whole blocks of
    # columns the same parts of the transposed form.
    r0 = 69888                                # 546 blocks of 128
    part = mx.swiglu_fp8_backward(act[r0:].contiguous(), gu[r0:].contiguous())
    assert torch.equal(raw(d)[r0:], raw(part[0])) and torch.equal(ds[r0:], part[1])
    assert torch.equal(raw(dt)[:, r0:], raw(part[2])) and torch.equal(dts[:, 546:], part[3])


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_past_32_bits(rows):
    M, K = 40001, 65536
    announce(f"quantize_fp8_2d {M}x{K} rows={rows}")
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.empty((M, K), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    codes, scales, codes_t, scales_t = mx.quantize_fp8_2d(x, block_rows=rows)
    alone = mx.quantize_fp8(x, block_rows=rows)
    assert torch.equal(raw(codes), raw(alone[0])) and torch.equal(scales, alone[1])
    del alone
    r0, c0 = 39936, 65408                     # the last blocks of rows and of columns
    part = mx.quantize_fp8_2d(x[r0:, c0:], block_rows=rows)
    s0 = r0 if rows == 1 else r0 // 128
    assert torch.equal(raw(codes)[r0:, c0:], raw(part[0]))
    assert torch.equal(scales[s0:, c0 // 128:], part[1])
    assert torch.equal(raw(codes_t)[c0:, r0:], raw(part[2]))
    t0 = c0 if rows == 1 else c0 // 128
    assert torch.equal(scales_t[t0:, r0 // 128:], part[3])
