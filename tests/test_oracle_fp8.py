"""Pins of the FP8 oracle: types and rounding against torch's on the CPU, the
scale rule by brute force, quantize's layouts by hand, the product and the
gated MLP's gradient against closed forms and differences."""

import numpy as np
import pytest
import torch

from oracle import fp8

TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_values_are_torchs(kind):
    want = torch.arange(256, dtype=torch.uint8).view(TORCH[kind]).double().numpy()
    assert np.array_equal(fp8.TABLES[kind], want, equal_nan=True)
    assert np.nanmax(np.where(np.isfinite(want), want, 0)) == fp8.LARGEST[kind]


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_rounding_is_torchs_within_the_type(kind):
    """Every BF16 value up to the largest, and FP32 values at and beside every
    tie: torch's conversion on the CPU rounds to nearest even."""
    bits = np.arange(0, 65536, dtype=np.uint32)
    v = (bits << 16).view(np.float32)
    pos = fp8.TABLES[kind][:127 if kind == "e4m3" else 124]
    ties = ((pos[1:] + pos[:-1]) / 2).astype(np.float32)
    v = np.concatenate([v, ties, np.nextafter(ties, np.float32(0)),
                        np.nextafter(ties, np.float32(1e9)), -ties])
    v = v[np.isfinite(v) & (np.abs(v) <= fp8.LARGEST[kind])]
    want = torch.from_numpy(v).to(TORCH[kind]).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(v, kind), want)


def test_non_finite_codes():
    v = np.array([np.inf, -np.inf, np.nan])
    assert fp8.encode(v, "e4m3").tolist()[:2] == [0x7F, 0xFF]
    assert np.isnan(fp8.TABLES["e4m3"][fp8.encode(v, "e4m3")]).all()
    assert fp8.encode(v, "e5m2").tolist()[:2] == [0x7C, 0xFC]
    assert np.isnan(fp8.TABLES["e5m2"][fp8.encode(v, "e5m2")[2]])


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_scale_rule_by_trial(kind):
    """Every positive finite BF16 amax: 2^e brings it within the type and
    2^(e - 1) does not."""
    amax = (np.arange(1, 0x7F80, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)
    e = fp8.exponents(amax, kind)
    top = fp8.LARGEST[kind]
    free = (e > -126) & (e < 127)
    assert (amax <= top * 2.0 ** e.astype(np.float64)).all()
    assert (amax[free] > top * 2.0 ** (e[free] - 1.0)).all()
    assert fp8.exponents(np.array([0.0]), kind)[0] == -126
    assert fp8.exponents(np.array([top, np.nextafter(top, 1e9)]), kind).tolist() == [0, 1]


def test_blocks_by_hand():
    """Ends of blocks: 3 x 144 has scales [3, 2], in blocks [1, 2]; a block's
    scale follows its own largest element, non-finite ones left out."""
    x = np.zeros((3, 144))
    x[0, 5], x[1, 127], x[2, 128], x[2, 143] = 448.0, 449.0, 1.75, np.inf
    codes, s = fp8.quantize(x, 1, "e4m3")
    assert s.tolist() == [[127, 1], [128, 1], [1, 119]]
    assert codes[0, 5] == 0x7E and codes[2, 128] == 0x7E and codes[2, 143] == 0x7F
    codes, s = fp8.quantize(x, 128, "e4m3")
    assert s.tolist() == [[128, 119]]
    assert fp8.values(codes, s, 128, "e4m3")[0, 5] == 448.0
    t = fp8.transposed(x)
    assert t.shape == (144, 16) and t[5, 0] == 448.0 and not t[:, 3:].any()


def test_product_of_one_hot_operands():
    """C[m, n] picks b[n, k] where row m of a is one element: block scales reach
    the right elements."""
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 0x78, (40, 272)).astype(np.uint8)
    scales = rng.integers(120, 135, (40, 3)).astype(np.uint8)
    b = fp8.values(codes, scales, 1, "e4m3")
    a = np.zeros((3, 272))
    a[0, 0] = a[1, 130] = a[2, 271] = 2.0
    C, S = fp8.product(a, b)
    for m, k in enumerate([0, 130, 271]):
        want = 2.0 * fp8.TABLES["e4m3"][codes[:, k]] * 2.0 ** (scales[:, k // 128] - 127.0)
        assert np.array_equal(C[m], want) and np.array_equal(S[m], np.abs(want))


def test_gradient_against_differences():
    rng = np.random.default_rng(1)
    g, u, d = rng.normal(size=(3, 40, 24)) * 2
    got = fp8.swiglu_backward(d, g, u)
    h = 1e-6
    dg = d * (fp8.swiglu(g + h, u) - fp8.swiglu(g - h, u)) / (2 * h)
    du = d * (fp8.swiglu(g, u + h) - fp8.swiglu(g, u - h)) / (2 * h)
    assert np.allclose(got, np.concatenate([dg, du], 1), rtol=1e-8, atol=1e-8)
    tg, tu = (torch.from_numpy(v).requires_grad_() for v in (g, u))
    (torch.nn.functional.silu(tg) * tu).backward(torch.from_numpy(d))
    want = np.concatenate([tg.grad.numpy(), tu.grad.numpy()], 1)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-13)


def test_tolerances_hold_for_fp32_and_reject_slips():
    """torch's FP32 evaluation lies within them; a slip does not."""
    rng = np.random.default_rng(2)
    g, u, d = (rng.normal(size=(64, 256)) * s for s in (4, 1, 1e-3))
    g32, u32, d32 = (v.astype(np.float32) for v in (g, u, d))
    g, u, d = (v.astype(np.float64) for v in (g32, u32, d32))
    t = lambda v: torch.from_numpy(v)  # noqa: E731
    s = torch.sigmoid(t(g32))
    act = (t(g32) * s * t(u32)).double().numpy()
    zero = np.zeros_like(g)
    assert (np.abs(act - fp8.swiglu(g, u)) <= fp8.swiglu_tolerance(g, u, zero, zero)).all()
    dg = (t(d32) * t(u32) * s * (1 + t(g32) * (1 - s))).double().numpy()
    du = (t(d32) * t(g32) * s).double().numpy()
    tol = fp8.swiglu_backward_tolerance(d, g, u)
    off = np.abs(np.concatenate([dg, du], 1) - fp8.swiglu_backward(d, g, u))
    assert (off <= tol).all()
    swapped = fp8.swiglu_backward(d, u, g)
    assert (np.abs(swapped - fp8.swiglu_backward(d, g, u)) > tol).mean() > 0.9
    x = np.concatenate([dg, du], 1)
    codes, scales = fp8.quantize(x, 1, "e4m3")
    ok, oks = fp8.check_quantized(codes, scales, fp8.swiglu_backward(d, g, u), tol, "e4m3")
    assert ok.all() and oks.all()
    ok, _ = fp8.check_quantized(codes ^ 1, scales, fp8.swiglu_backward(d, g, u), tol, "e4m3")
    assert ok.mean() < 0.01
    _, oks = fp8.check_quantized(codes, scales + np.uint8(1), fp8.swiglu_backward(d, g, u), tol, "e4m3")
    assert not oks.any()
