"""The FP8 operators against the oracle (GPU): quantize bit for bit, products
within the roundings they may take, the gated MLP forward and backward."""

import numpy as np
import pytest
import torch

import block_scaled_microscaling_amd as mx
from fp8_cases import TORCH, bf16_of, bytes_of, check_product, codes_to_dev, operand, to_dev
from gpu_helpers import DEV, announce
from oracle import fp8

pytestmark = pytest.mark.gpu

KINDS = ["e4m3", "e5m2"]
SCALE = {"ue8m0": torch.uint8, "fp32": torch.float32}


def scale_array(s, scales):
    return s if scales == "ue8m0" else (2.0 ** (s.astype(np.float64) - 127)).astype(np.float32)


def check_quantize(x, values, rows, kind, scales="ue8m0", both=False):
    args = dict(block_rows=rows, dtype=TORCH[kind], scale_dtype=SCALE[scales])
    got = mx.quantize_fp8_2d(x, **args) if both else mx.quantize_fp8(x, **args)
    want = list(fp8.quantize(values, rows, kind))
    if both:
        want += list(fp8.quantize(fp8.transposed(values), rows, kind))
    assert len(got) == len(want)
    for i in range(0, len(got), 2):
        assert got[i].dtype == TORCH[kind] and got[i + 1].dtype == SCALE[scales]
        assert np.array_equal(got[i + 1].cpu().numpy(), scale_array(want[i + 1], scales)), i
        c, w = bytes_of(got[i]), want[i]
        nan = np.isnan(fp8.TABLES[kind][w])
        assert np.array_equal(np.isnan(fp8.TABLES[kind][c]), nan), i
        assert np.array_equal(c[~nan], w[~nan]), i


# ---------------------------------------------------------------- quantize
SHAPES = [(1, 16), (1, 4096), (2, 128), (3, 144), (17, 2064), (127, 256), (128, 128), (129, 272),
          (300, 1040), (1000, 80)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_quantize(M, K, rows, both, kind):
    announce(f"quantize_fp8 {M}x{K} rows={rows} both={both} {kind}")
    rng = np.random.default_rng(M * 7 + K)
    x = rng.normal(size=(M, K)) * np.where(rng.random((M, K)) < 0.01, 200, 1)
    x *= 2.0 ** rng.integers(-20, 20, (M, 1))
    x[:, : min(K, 16)] *= rng.random((M, 1)) < 0.7        # rows and blocks with zeros
    check_quantize(*bf16_of(x), rows, kind, "ue8m0" if (M + rows) % 2 else "fp32", both)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,both", [(1, False), (1, True), (128, True)])
def test_quantize_every_bf16_value(kind, rows, both):
    """Each pattern, subnormals, infinities and NaN among them, beside others of
    its sign and exponent, and once more under a scale 2^6 larger."""
    announce(f"quantize_fp8 of every BF16 pattern rows={rows} both={both} {kind}")
    bits = np.arange(65536, dtype=np.uint16).reshape(512, 128)
    v = (bits.astype(np.uint32) << 16).view(np.float32)
    beside = v.copy()
    with np.errstate(over="ignore", invalid="ignore"):
        beside[:, 0] = np.where(np.isfinite(v[:, -1]), np.abs(v[:, -1]) * 64, 1.0)
    both_v = np.concatenate([v, beside])
    t = torch.from_numpy(both_v).bfloat16()
    check_quantize(t.to(DEV), t.double().numpy(), rows, kind, both=both)


@pytest.mark.parametrize("rows,both", [(1, False), (1, True), (128, False), (128, True)])
def test_quantize_rows_of_a_wider_tensor(rows, both):
    announce(f"quantize_fp8 of a slice rows={rows} both={both}")
    rng = np.random.default_rng(5)
    wide, values = bf16_of(rng.normal(size=(70, 640)))
    check_quantize(wide[3:60, 128:416], values[3:60, 128:416], rows, "e4m3", both=both)


def test_quantize_writes_nothing_else():
    """Outputs inside larger buffers: what lies around them stays."""
    announce("quantize_fp8: around the outputs")
    M, K = 130, 272
    rng = np.random.default_rng(6)
    x, values = bf16_of(rng.normal(size=(M, K)))
    Mp, KB, MB = 144, 3, 2
    for rows, both in ((1, False), (1, True), (128, True)):
        sizes = [M * K, M * KB if rows == 1 else MB * KB]
        if both:
            sizes += [K * Mp, K * MB if rows == 1 else KB * MB]
        bufs = [torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV) for n in sizes]
        ptrs = [b.data_ptr() + 256 for b in bufs]
        s = torch.cuda.current_stream().cuda_stream
        if both:
            rc = mx.mxfp4_quantize_fp8_2d(x.data_ptr(), K, M, K, rows, mx.FP8_E4M3,
                                          mx.SCALE_UE8M0, *ptrs, s)
        else:
            rc = mx.mxfp4_quantize_fp8(x.data_ptr(), K, M, K, rows, mx.FP8_E4M3, mx.SCALE_UE8M0,
                                       *ptrs, s)
        assert rc == 0
        want = list(fp8.quantize(values, rows, "e4m3"))
        if both:
            want += list(fp8.quantize(fp8.transposed(values), rows, "e4m3"))
        for b, n, w in zip(bufs, sizes, want):
            got = b.cpu().numpy()
            assert (got[:256] == 0xA5).all() and (got[256 + n:] == 0xA5).all()
            assert np.array_equal(got[256:256 + n], w.ravel())


# -------------------------------------------------------------------- gemm
GEMMS = [(1, 1, 16), (1, 16, 128), (1, 333, 2064), (3, 130, 80), (16, 64, 1024), (17, 33, 144),
         (32, 257, 4096), (33, 96, 384), (64, 129, 528), (65, 127, 16), (65, 257, 1040),
         (128, 128, 128), (130, 384, 640), (200, 8, 2048), (257, 1001, 272), (300, 513, 1152)]


@pytest.mark.parametrize("M,N,K", GEMMS)
@pytest.mark.parametrize("scales,block", [("ue8m0", 128), ("ue8m0", 1), ("fp32", 128)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gemm(M, N, K, scales, block, out):
    kind = KINDS[(M + N + block) % 2]
    announce(f"gemm_fp8 {M}x{N}x{K} {kind} {scales}/{block} {out}")
    a, sa, va = operand(M, K, 1, kind, scales, M + K)
    b, sb, vb = operand(N, K, block, "e4m3", scales, N + K + 1, std=0.02)
    got = mx.gemm_fp8(a, sa, b, sb, out_dtype=out)
    assert got.shape == (M, N) and got.dtype == out
    check_product(got, va, vb, K, True, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N", [(1, 40), (20, 40), (70, 40), (150, 300)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gemm_of_exact_sums(M, N, out):
    """Small whole numbers under power-of-two scales: every sum is exact, so the
    result is (BF16: its rounding), and one-hot rows pick single elements."""
    announce(f"gemm_fp8 exact {M}x{N} {out}")
    K = 400
    rng = np.random.default_rng(M)
    a = rng.integers(-4, 5, (M, K)).astype(np.float64)
    a[0] = 0
    a[0, 399] = 1
    b = rng.integers(-4, 5, (N, K)).astype(np.float64)
    ea, eb = rng.integers(-3, 4, (M, 4)), rng.integers(-3, 4, (N, 4))
    A = codes_to_dev(fp8.encode(a, "e5m2"), "e5m2")
    B = codes_to_dev(fp8.encode(b, "e4m3"), "e4m3")
    assert np.array_equal(fp8.TABLES["e5m2"][fp8.encode(a, "e5m2")], a)
    sa, sb = (ea + 127).astype(np.uint8), (eb + 127).astype(np.uint8)
    want = (a * fp8.spread(2.0 ** ea, 1, M, K)) @ (b * fp8.spread(2.0 ** eb, 1, N, K)).T
    got = mx.gemm_fp8(A, to_dev(sa), B, to_dev(sb), out_dtype=out)
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(out))


@pytest.mark.parametrize("M", [2, 40, 100])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gemm_nan_and_infinity_stay_in_their_rows(M, out):
    """A NaN or an infinity in a row of A reaches that row alone; the padding of
    a short last block is not read from the next row."""
    announce(f"gemm_fp8 non-finite M={M} {out}")
    N, K = 48, 144
    a, sa, va = operand(M, K, 1, "e5m2", "ue8m0", 1)
    b, sb, vb = operand(N, K, 128, "e4m3", "ue8m0", 2)
    raw = a.view(torch.uint8)
    raw[1, 0] = 0x7F          # NaN at the beginning of row 1, behind row 0's short block
    got = mx.gemm_fp8(a, sa, b, sb, out_dtype=out)
    assert got[1].isnan().all()
    keep = np.arange(M) != 1
    check_product(got[torch.from_numpy(keep).to(DEV)], va[keep], vb, K, True)
    raw[1, 0] = 0x7C          # infinity
    got = mx.gemm_fp8(a, sa, b, sb, out_dtype=out)
    assert not got[1].isfinite().any()
    raw[1, 0] = 0
    sa[M - 1, 1] = 255        # a NaN scale
    got = mx.gemm_fp8(a, sa, b, sb, out_dtype=out)
    assert got[M - 1].isnan().all() and got[: M - 1].isfinite().all()


@pytest.mark.parametrize("M,N", [(5, 33), (70, 200), (129, 130)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gemm_writes_nothing_else(M, N, out):
    announce(f"gemm_fp8 around C {M}x{N} {out}")
    K = 272
    a, sa, va = operand(M, K, 1, "e4m3", "ue8m0", 1)
    b, sb, vb = operand(N, K, 128, "e4m3", "ue8m0", 2)
    size = M * N * out.itemsize
    buf = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    rc = mx.mxfp4_gemm_fp8(a.data_ptr(), mx.FP8_E4M3, sa.data_ptr(), b.data_ptr(), sb.data_ptr(),
                           mx.SCALE_UE8M0, 128, M, N, K,
                           mx.OUT_FP32 if out == torch.float32 else mx.OUT_BF16,
                           buf.data_ptr() + 256, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert (buf[:256] == 0xA5).all() and (buf[256 + size:] == 0xA5).all()
    check_product(buf[256:256 + size].view(out).view(M, N), va, vb, K, True)


# --------------------------------------------------------------- gated MLP
MLPS = [(1, 16, 128), (1, 528, 384), (5, 256, 128), (33, 144, 256), (64, 272, 128),
        (65, 128, 128), (130, 400, 256), (257, 1040, 384), (300, 256, 640)]


@pytest.mark.parametrize("M,H,I", MLPS)
def test_swiglu(M, H, I):
    announce(f"gemm_fp8_swiglu {M}x{H}x{I}")
    a, sa, va = operand(M, H, 1, "e4m3", "ue8m0", M + H)
    w, sw, vw = operand(2 * I, H, 128, "e4m3", "ue8m0", I, std=2.0 / np.sqrt(H))
    codes, scales, act, gu = mx.gemm_fp8_swiglu(a, sa, w, sw, want_act=True, want_gu=True)
    C, S = fp8.product(va, vw)
    off = fp8.exact_tolerance(C, S, H) + fp8.grouped_tolerance(va, vw)
    check_product(gu, va, vw, H, True, "gu")
    g, u, dg, du = C[:, :I], C[:, I:], off[:, :I], off[:, I:]
    ref = fp8.swiglu(g, u)
    tol = fp8.swiglu_tolerance(g, u, dg, du)
    tol = tol + fp8.BF16_HALF_STEP * (np.abs(ref) + tol)
    got = act.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol).all()
    # The codes are the quantize of the kernel's own act, and the same without
    # the other outputs.
    want = fp8.quantize(got, 1, "e4m3")
    for again in ((codes, scales), mx.gemm_fp8_swiglu(a, sa, w, sw),
                  mx.gemm_fp8_swiglu(a, sa, w, sw, want_gu=True)):
        assert np.array_equal(bytes_of(again[0]), want[0])
        assert np.array_equal(again[1].cpu().numpy(), want[1])


@pytest.mark.parametrize("M,I", [(1, 128), (5, 384), (127, 128), (128, 256), (129, 128), (333, 640)])
@pytest.mark.parametrize("kind", KINDS)
def test_swiglu_backward(M, I, kind):
    announce(f"swiglu_fp8_backward {M}x{I} {kind}")
    rng = np.random.default_rng(M + I)
    gu, vgu = bf16_of(rng.normal(size=(M, 2 * I)) * np.where(rng.random((M, 2 * I)) < 0.02, 30, 2))
    d, vd = bf16_of(rng.normal(size=(M, I)) * 1e-3 * 2.0 ** rng.integers(-12, 12, (M, 1)))
    g, u = vgu[:, :I], vgu[:, I:]
    ref, tol = fp8.swiglu_backward(vd, g, u), fp8.swiglu_backward_tolerance(vd, g, u)
    codes, scales, codes_t, scales_t = mx.swiglu_fp8_backward(d, gu, dtype=TORCH[kind])
    assert codes.shape == (M, 2 * I) and codes_t.shape == (2 * I, (M + 15) // 16 * 16)
    ok, oks = fp8.check_quantized(bytes_of(codes), scales.cpu().numpy(), ref, tol, kind)
    assert ok.all() and oks.all()
    ok, oks = fp8.check_quantized(bytes_of(codes_t), scales_t.cpu().numpy(), fp8.transposed(ref),
                                  fp8.transposed(tol), kind)
    assert ok.all() and oks.all()
    assert not bytes_of(codes_t)[:, M:].any()


def test_swiglu_backward_extremes():
    """Infinities, NaN and overflow stay in their own elements; gates far out
    saturate; zeros give zeros."""
    announce("swiglu_fp8_backward extremes")
    M, I = 20, 128
    rng = np.random.default_rng(3)
    v = rng.normal(size=(M, 2 * I))
    v[0, :I], v[1, :I] = -200.0, 200.0
    d = rng.normal(size=(M, I))
    d[2, 7], d[3, 9], d[4] = np.inf, np.nan, 0.0
    d[5], v[5, I:] = 3e38, 3e38                      # dg overflows
    gu, vgu = bf16_of(v)
    dt, vd = bf16_of(d)
    codes, scales, codes_t, _ = mx.swiglu_fp8_backward(dt, gu)
    got = codes.float().cpu().numpy()
    # NaN exactly where the gradient is not finite in FP32: dg overflows in all
    # of row 5, du where |g s| > 1.13 there.
    with np.errstate(all="ignore"):
        ref = fp8.swiglu_backward(vd, vgu[:, :I], vgu[:, I:])
        bad = ~np.isfinite(ref.astype(np.float32))
    assert bad[2].sum() == 2 and bad[3].sum() == 2 and bad[5, :I].all() and not bad[5, I:].all()
    assert np.array_equal(np.isnan(got), bad)
    assert np.array_equal(np.isnan(codes_t.float().cpu().numpy())[:, :M], bad.T)
    assert not got[0].any() and not got[4].any()
    rows = [1] + list(range(6, M))
    ref = ref[rows]
    tol = fp8.swiglu_backward_tolerance(vd, vgu[:, :I], vgu[:, I:])[rows]
    ok, oks = fp8.check_quantized(bytes_of(codes)[rows], scales.cpu().numpy()[rows], ref, tol, "e4m3")
    assert ok.all() and oks.all()


@pytest.mark.parametrize("M,H,I", [(1, 144, 128), (48, 256, 128), (200, 272, 256)])
def test_mlp_forward_and_backward(M, H, I):
    """The layer as it is used: y = W2 (silu(Wg x) u), and the gradients of x and
    all three weights, every step's operands from the step before. Each product
    is checked against its own operands, and the whole against the unquantized
    layer's gradient by autograd in 64 bits within the quantization's error."""
    announce(f"FP8 MLP {M}x{H}x{I}")
    rng = np.random.default_rng(M)
    x, vx = bf16_of(rng.normal(size=(M, H)))
    w13, v13 = bf16_of(rng.normal(size=(2 * I, H)) / np.sqrt(H))
    w2, v2 = bf16_of(rng.normal(size=(H, I)) / np.sqrt(I))
    dy, vdy = bf16_of(rng.normal(size=(M, H)))
    xq, xs, xt, xts = mx.quantize_fp8_2d(x)
    wq, ws, wt, wts = mx.quantize_fp8_2d(w13, block_rows=128)
    w2q, w2s, w2t, w2ts = mx.quantize_fp8_2d(w2, block_rows=128)
    # forward
    aq, as_, act, gu = mx.gemm_fp8_swiglu(xq, xs, wq, ws, want_act=True, want_gu=True)
    y = mx.gemm_fp8(aq, as_, w2q, w2s)
    # backward
    dq, ds, dt, dts = mx.quantize_fp8_2d(dy)
    dact = mx.gemm_fp8(dq, ds, w2t, w2ts)
    gq, gs, gt, gts = mx.swiglu_fp8_backward(dact, gu)
    dx = mx.gemm_fp8(gq, gs, wt, wts)
    dw13 = mx.gemm_fp8(gt, gts, xt, xts, out_dtype=torch.float32)
    _, _, at, ats = mx.quantize_fp8_2d(act)
    dw2 = mx.gemm_fp8(dt, dts, at, ats, out_dtype=torch.float32)

    def held(c, s, rows=1):
        return fp8.values(bytes_of(c), s.cpu().numpy(), rows, "e4m3")
    check_product(y, held(aq, as_), held(w2q, w2s, 128), I, True, "y")
    check_product(dact, held(dq, ds), held(w2t, w2ts, 128), H, True, "dact")
    check_product(dx, held(gq, gs), held(wt, wts, 128), 2 * I, True, "dx")
    check_product(dw13, held(gt, gts), held(xt, xts), gt.shape[1], False, "dw13")
    check_product(dw2, held(dt, dts), held(at, ats), dt.shape[1], False, "dw2")

    # Every operand is off by at most 2^-4 of itself: fifteen elements in a
    # hundred of the sums' magnitude covers a product of two such.
    t = [torch.from_numpy(v).requires_grad_() for v in (vx, v13, v2)]
    gu64 = t[0] @ t[1].T
    (torch.nn.functional.silu(gu64[:, :I]) * gu64[:, I:] @ t[2].T).backward(torch.from_numpy(vdy))
    for got, want in zip((dx, dw13, dw2), (t[0].grad, t[1].grad, t[2].grad)):
        got, want = got.double().cpu(), want
        assert got.shape == want.shape
        assert torch.linalg.norm(got - want) <= 0.15 * torch.linalg.norm(want)


# ------------------------------------------------------------- large tiles
def check_product_on_gpu(got, a, sa, b, sb, block, fp8_path):
    """check_product in 64 bits on the GPU, for sizes that take large tiles."""
    def vals(c, s, rows):
        s = s.double() if s.dtype == torch.float32 else torch.exp2(s.double() - 127)
        s = s.repeat_interleave(rows, 0)[: c.shape[0]].repeat_interleave(128, 1)[:, : c.shape[1]]
        return c.double() * s
    K = a.shape[1]
    va, vb = vals(a, sa, 1), vals(b, sb, block)
    C, S = va @ vb.t().contiguous(), va.abs() @ vb.abs().t().contiguous()
    tol = (K + 8) * 2.0 ** -24 * S
    if got.dtype == torch.bfloat16:
        if fp8_path:
            def tops(v):
                pad = -v.shape[1] % 8
                return torch.nn.functional.pad(v.abs(), (0, pad)).view(v.shape[0], -1, 8).amax(2)
            tol = tol + 8 * 2.0 ** -13 * (tops(va) @ tops(vb).t().contiguous())
        tol = tol + fp8.BF16_HALF_STEP * (C.abs() + tol)
    bad = ((got.double() - C).abs() > tol) | got.isnan()
    assert not bad.any(), f"{int(bad.sum())} outside, first {bad.nonzero()[:4].tolist()}"
    return C, va, vb


BIG = [(3200, 2900, 16), (2817, 3333, 128), (3201, 3137, 400), (4096, 2304, 512),
       (2900, 3211, 640), (2818, 3000, 784), (2817, 2944, 1168)]


@pytest.mark.parametrize("M,N,K", BIG)
@pytest.mark.parametrize("scales,block", [("ue8m0", 128), ("ue8m0", 1), ("fp32", 128)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gemm_of_many_tiles(M, N, K, scales, block, out):
    kind = KINDS[(M + N + block) % 2]
    announce(f"gemm_fp8 {M}x{N}x{K} {kind} {scales}/{block} {out}")
    a, sa, _ = operand(M, K, 1, kind, scales, M + K)
    b, sb, _ = operand(N, K, block, "e4m3", scales, N + K + 1, std=0.02)
    got = mx.gemm_fp8(a, sa, b, sb, out_dtype=out)
    check_product_on_gpu(got, a, sa, b, sb, block, True)


@pytest.mark.parametrize("M,H,I", [(2900, 16, 1536), (4096, 512, 1152), (2817, 656, 1664)])
def test_swiglu_of_many_tiles(M, H, I):
    announce(f"gemm_fp8_swiglu {M}x{H}x{I}")
    a, sa, _ = operand(M, H, 1, "e4m3", "ue8m0", M + H)
    w, sw, _ = operand(2 * I, H, 128, "e4m3", "ue8m0", I, std=2.0 / np.sqrt(H))
    codes, scales, act, gu = mx.gemm_fp8_swiglu(a, sa, w, sw, want_act=True, want_gu=True)
    C, va, vw = check_product_on_gpu(gu, a, sa, w, sw, 128, True)
    off = fp8.exact_tolerance(*fp8.product(va.cpu().numpy(), vw.cpu().numpy()), H)
    off = off + fp8.grouped_tolerance(va.cpu().numpy(), vw.cpu().numpy())
    C = C.cpu().numpy()
    ref = fp8.swiglu(C[:, :I], C[:, I:])
    tol = fp8.swiglu_tolerance(C[:, :I], C[:, I:], off[:, :I], off[:, I:])
    tol = tol + fp8.BF16_HALF_STEP * (np.abs(ref) + tol)
    got = act.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol).all()
    want = fp8.quantize(got, 1, "e4m3")
    for again in ((codes, scales), mx.gemm_fp8_swiglu(a, sa, w, sw)):
        assert np.array_equal(bytes_of(again[0]), want[0])
        assert np.array_equal(again[1].cpu().numpy(), want[1])
