"""The FP8 operators' definitions in NumPy and 64 bits: the two types, the
scale rule, quantize, the product and the gated MLP's activation, forward and
backward, with the tolerances that follow from how they may be computed.

Types (OCP 8-bit floating point): sign, exponent field e, mantissa m of b bits.
E4M3: b = 3, bias 7, no infinities, e = 15 with m = 7 is NaN, largest 448.
E5M2: b = 2, bias 15, e = 31 is infinity (m = 0) or NaN, largest 57344.
"""

import numpy as np

BLOCK = 128
TYPES = {"e4m3": (3, 7), "e5m2": (2, 15)}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


def table(kind):
    """The 256 values of a type, by its definition."""
    bits, bias = TYPES[kind]
    out = np.empty(256)
    for code in range(256):
        e, m = (code & 0x7F) >> bits, code & ((1 << bits) - 1)
        v = m * 2.0 ** (1 - bias - bits) if e == 0 else (1 + m * 2.0 ** -bits) * 2.0 ** (e - bias)
        if kind == "e4m3" and (code & 0x7F) == 0x7F:
            v = np.nan
        if kind == "e5m2" and e == 31:
            v = np.inf if m == 0 else np.nan
        out[code] = -v if code & 0x80 else v
    return out


TABLES = {kind: table(kind) for kind in TYPES}


def exponents(amax, kind):
    """The smallest integer e with amax <= largest * 2^e, in [-126, 127]; -126
    where amax is 0. (Found by trial around the logarithm.)"""
    amax = np.asarray(amax, np.float64)
    e = np.floor(np.log2(np.where(amax > 0, amax, 1.0) / LARGEST[kind])).astype(np.int64) - 1
    for _ in range(4):
        e = np.where(amax > LARGEST[kind] * 2.0 ** e.astype(np.float64), e + 1, e)
    return np.where(amax > 0, np.clip(e, -126, 127), -126)


def encode(v, kind):
    """Codes of the values nearest to v, ties to the even code; the sign is kept.
    Infinities and NaN: E4M3 has NaN for both."""
    v = np.asarray(v, np.float64)
    pos = TABLES[kind][:0x7F if kind == "e4m3" else 0x7C]     # finite, ascending
    mag = np.abs(v)
    hi = np.clip(np.searchsorted(pos, np.where(np.isfinite(mag), mag, 0.0)), 0, len(pos) - 1)
    lo = np.maximum(hi - 1, 0)
    with np.errstate(invalid="ignore"):
        d_hi, d_lo = np.abs(pos[hi] - mag), np.abs(mag - pos[lo])
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isinf(v), 0x7F if kind == "e4m3" else 0x7C, code)
    code = np.where(np.isnan(v), 0x7F, code)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def _cut(n, rows):
    return -(-n // rows)


def quantize(x, rows, kind):
    """(codes [M, K], scale bytes [ceil(M / rows), ceil(K / 128)]) of x [M, K]
    in 64 bits."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    finite = np.where(np.isfinite(x), np.abs(x), 0.0)
    pad = np.zeros((_cut(M, rows) * rows, _cut(K, BLOCK) * BLOCK))
    pad[:M, :K] = finite
    amax = pad.reshape(_cut(M, rows), rows, _cut(K, BLOCK), BLOCK).max(axis=(1, 3))
    e = exponents(amax, kind)
    return encode(x / spread(2.0 ** e.astype(np.float64), rows, M, K), kind), (e + 127).astype(np.uint8)


def transposed(x):
    """x^T with zeros to a multiple of 16 columns."""
    M, K = x.shape
    out = np.zeros((K, _cut(M, 16) * 16))
    out[:, :M] = x.T
    return out


def spread(scales, rows, M, K):
    """A scale for every element of [M, K]."""
    return np.repeat(np.repeat(scales, rows, axis=0)[:M], BLOCK, axis=1)[:, :K]


def scale_values(scales):
    """Scales as values: bytes are UE8M0."""
    if scales.dtype == np.uint8:
        return 2.0 ** (scales.astype(np.float64) - 127)
    return scales.astype(np.float64)


def values(codes, scales, rows, kind):
    return TABLES[kind][codes] * spread(scale_values(scales), rows, *codes.shape)


def product(a, b):
    """(C, S): a b^T and the sums of magnitudes."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def exact_tolerance(C, S, K):
    """FP32 sums of exact products, in any order: fewer than K + 8 roundings,
    each at most 2^-24 of a running sum that S bounds (8: waves' and blocks'
    sums, a scale of a block's sum, the scales' product)."""
    return (K + 8) * 2.0 ** -24 * S


def grouped_tolerance(a, b):
    """What the FP8 matrix instructions may lose besides: of every 8 neighbours
    in K, each product less than 2^-13 of the largest one's power of two. The
    sum over groups of 8 2^-13 max |a| max |b| bounds it."""
    def tops(x):
        pad = np.zeros((x.shape[0], _cut(x.shape[1], 8) * 8))
        pad[:, :x.shape[1]] = np.abs(x)
        return pad.reshape(x.shape[0], -1, 8).max(axis=2)
    return 8 * 2.0 ** -13 * (tops(a) @ tops(b).T)


BF16_HALF_STEP = 2.0 ** -8      # of the value: at most half of 2^-7


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_tolerance(g, u, dg, du):
    """Of act in FP32 from g, u that are off by dg, du: silu's slope is at most
    1.1; the evaluation in FP32 rounds exp's argument (|g| 2^-24 relative) and
    takes fewer than 16 half steps more; below -87 exp overflows and act is 0."""
    act = np.abs(swiglu(g, u))
    silu = np.abs(g * sigmoid(g))
    return (1.1 * dg * (np.abs(u) + du) + silu * du + (2 * np.abs(g) + 16) * 2.0 ** -24 * act
            + np.where(g < -87, act, 0.0))


def swiglu_backward(dact, g, u):
    """[dg, du] of act = silu(g) u from dact."""
    s = sigmoid(g)
    return np.concatenate([dact * u * s * (1 + g * (1 - s)), dact * g * s], axis=1)


def swiglu_backward_tolerance(dact, g, u):
    """Of [dg, du] evaluated in FP32: s is off by (|g| + 3) 2^-23 relative
    (exp's argument and value, the addition, the reciprocal), 1 - s by s's error
    and one half step of at most 1, g times it likewise, then fewer than 6 half
    steps; below -87 exp overflows and s is 0."""
    s = sigmoid(g)
    eps = 2.0 ** -24
    ds = 2 * (np.abs(g) + 3) * eps * s
    inner = np.abs(1 + g * (1 - s))
    d_inner = np.abs(g) * (ds + 2 * eps) + 3 * eps * (1 + np.abs(g) * (1 - s))
    dg = np.abs(dact * u) * (ds * inner + s * d_inner + 6 * eps * s * inner)
    du = np.abs(dact * g) * (ds + 6 * eps * s)
    low = np.where(g < -87, 1.0, 0.0)
    ref = np.abs(swiglu_backward(dact, g, u))
    tiny = 2.0 ** -140                # FP32's own spacing near 0, with room
    return np.concatenate([dg, du], axis=1) + np.concatenate([low, low], axis=1) * ref + tiny


def check_quantized(codes, scales, x, off, kind):
    """Whether (codes, scale bytes) [1 x 128 blocks] are a quantize of some
    values within `off` of x: the scale is one that such an amax may have, and
    every code is within half a step of such a value. Returns a bool array of
    the codes and one of the scales."""
    M, K = x.shape
    e = scales.astype(np.int64) - 127

    def tops(v):
        pad = np.zeros((M, _cut(K, BLOCK) * BLOCK))
        pad[:, :K] = v
        return pad.reshape(M, -1, BLOCK).max(axis=2)
    least = exponents(tops(np.maximum(np.abs(x) - off, 0.0)), kind)
    most = exponents(tops(np.abs(x) + off), kind)
    ok_scales = (e >= least) & (e <= most)
    s = spread(2.0 ** e.astype(np.float64), 1, M, K)
    lo, hi = encode((x - off) / s, kind), encode((x + off) / s, kind)
    got = TABLES[kind][codes]
    ok = (got >= TABLES[kind][lo]) & (got <= TABLES[kind][hi])
    return ok, ok_scales
