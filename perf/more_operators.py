"""The FP8 operators with a scale for each block of 128: their cases, plain forms and work.

An MLP whose operands are 8-bit floating point, beside the 4-bit ones: codes
are E4M3 (or, for gradients, E5M2), and each block of 128 elements of a row,
or each 128 x 128 block of a weight, has a scale, UE8M0 (a power of two's
biased exponent) or FP32.

  quantize  BF16 rows -> codes and scales; the scale is the smallest power of
            two that brings the block's largest magnitude within the type;
            of x alone, or of x and of x^T in one pass
  gemm      C[m, n] = sum_k dq(A[m, k]) dq(B[n, k])
  swiglu    the gate+up product of a gated MLP against [W_gate; W_up] with
            act = silu(g) * u, rounded to BF16 and quantized, in its epilogue;
            for training also g and u
  grad      its backward pass: the gradients of g and u from act's, quantized
            in both directions, then dx = dgu W13 and dW13 = dgu^T x

`run` computes a case in its plain form (elementary torch operations in 32
bits), or, where `own` is true, through the framework's entry points.
"""

import math

import torch

own = False

DEV = "cuda:0"
BLOCK = 128
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
OUT = {"bf16": torch.bfloat16, "fp32": torch.float32}

if own:
    import block_scaled_microscaling_amd  # noqa: F401


# ------------------------------------------------------------------- cases
def _quantize(name, M, K, block, both, type, scales):
    return {"name": name, "op": "quantize", "M": M, "K": K, "block": block, "both": both,
            "type": type, "scales": scales}


def _gemm(name, M, N, K, type, scales, block, out):
    return {"name": name, "op": "gemm", "M": M, "N": N, "K": K, "type": type, "scales": scales,
            "block": block, "out": out}


def _swiglu(name, M, H, I, train):
    return {"name": name, "op": "swiglu", "M": M, "H": H, "I": I, "train": train}


def _grad(name, M, H, I, type):
    return {"name": name, "op": "grad", "M": M, "H": H, "I": I, "type": type}


def listed():
    return [
        # One token's activation in a decode step: launch latency is all of it.
        _quantize("quantize_1x4096", 1, 4096, 1, False, "e4m3", "ue8m0"),
        # A training activation, for the forward product and the weight gradient.
        _quantize("quantize_both_8192x8192", 8192, 8192, 1, True, "e4m3", "ue8m0"),
        # An MLP's gate+up weight, for the forward product and dx.
        _quantize("quantize_weight_28672x4096", 28672, 4096, 128, True, "e4m3", "ue8m0"),
        # One token of a decode loop against a weight with FP32 scales.
        _gemm("gemm_1x8192x8192_fp32s", 1, 8192, 8192, "e4m3", "fp32", 128, "bf16"),
        # The skinny decode shape, and the square one.
        _gemm("gemm_32x8192x8192", 32, 8192, 8192, "e4m3", "ue8m0", 128, "bf16"),
        _gemm("gemm_8192x8192x8192", 8192, 8192, 8192, "e4m3", "ue8m0", 128, "bf16"),
        # An MLP's down projection of a prompt, with FP32 scales.
        _gemm("gemm_16384x4096x14336_fp32s", 16384, 4096, 14336, "e4m3", "fp32", 128, "bf16"),
        # Odd sizes: rows that fill no tile, odd columns, K that ends inside a block.
        _gemm("gemm_333x6177x7952", 333, 6177, 7952, "e4m3", "ue8m0", 128, "fp32"),
        # Gate+up of one token, and of a training batch that keeps g and u.
        _swiglu("swiglu_1x4096x14336", 1, 4096, 14336, False),
        _swiglu("swiglu_16384x4096x14336_train", 16384, 4096, 14336, True),
        # The backward pass of that layer, and one of odd sizes with E5M2 gradients.
        _grad("grad_16384x4096x14336", 16384, 4096, 14336, "e4m3"),
        _grad("grad_1001x2064x1408_e5m2", 1001, 2064, 1408, "e5m2"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "swiglu", "grad"])
    type = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op == "quantize":
        while True:
            M, K = _log_int(rng, 1, 65536), 16 * _log_int(rng, 1, 2048)
            if M * K <= 28672 * 4096:
                break
        case = _quantize("", M, K, rng.choice([1, 1, 128]), rng.random() < 0.5, type,
                         rng.choice(["ue8m0", "fp32"]))
    elif op == "gemm":
        while True:
            M, N, K = _log_int(rng, 1, 16384), _log_int(rng, 16, 28672), 16 * _log_int(rng, 4, 896)
            if rng.random() < 0.5:
                N, K = max(16, N // 64 * 64), max(128, K // 128 * 128)
            if M * N * K <= 16384 * 4096 * 14336:
                break
        scales = rng.choice(["ue8m0", "ue8m0", "fp32"])
        block = 128 if scales == "fp32" else rng.choice([128, 1])
        case = _gemm("", M, N, K, type, scales, block, rng.choice(["bf16", "fp32"]))
    else:
        most = 16384 * 4096 * 14336
        while True:
            M, H, I = _log_int(rng, 1, 16384), 16 * _log_int(rng, 16, 512), 128 * _log_int(rng, 2, 128)
            if rng.random() < 0.5:
                H = max(128, H // 128 * 128)
            if M * H * I <= most // (2 if op == "grad" else 1):
                break
        case = _swiglu("", M, H, I, rng.random() < 0.5) if op == "swiglu" else _grad("", M, H, I, type)
    del case["name"]
    return case


def _ceil(n, d):
    return -(-n // d)


# ----------------------------------------------------- the plain quantizer
def _blocks(x, rows):
    """[R, rows, C, 128] of x [M, K], with zeros past its ends."""
    M, K = x.shape
    R, C = _ceil(M, rows), _ceil(K, BLOCK)
    if (R * rows, C * BLOCK) != (M, K):
        x = torch.nn.functional.pad(x, (0, C * BLOCK - K, 0, R * rows - M))
    return x.view(R, rows, C, BLOCK)


def _exponents(amax, largest):
    """The smallest e with amax <= largest * 2^e, at least -126."""
    m, e = torch.frexp(amax)        # amax = m 2^e, m in [0.5, 1)
    m0, e0 = math.frexp(largest)
    e = torch.where(m > m0, e + 1 - e0, e - e0)
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(-126, 127)


def _plain_quantize(x, rows, type, scales):
    """Codes [M, K] and scales [ceil(M / rows), ceil(K / 128)] of x."""
    M, K = x.shape
    b = _blocks(x.float(), rows)
    e = _exponents(b.abs().amax(dim=(1, 3)), LARGEST[type])
    s = ((e + 127) << 23).view(torch.float32)
    codes = (b / s[:, None, :, None]).to(CODES[type])
    codes = codes.view(b.shape[0] * rows, b.shape[2] * BLOCK)[:M, :K].contiguous()
    return codes, s if scales == "fp32" else (e + 127).to(torch.uint8)


def _plain_quantize_t(x, rows, type, scales):
    """The same of x^T, whose rows are filled with zeros to a multiple of 16."""
    M = x.shape[0]
    xt = torch.nn.functional.pad(x, (0, 0, 0, _ceil(M, 16) * 16 - M)).t().contiguous()
    return _plain_quantize(xt, rows, type, scales)


def _scale(scales):
    return scales if scales.dtype == torch.float32 else (scales.int() << 23).view(torch.float32)


def _values(codes, scales, rows, dtype=torch.float32):
    """dq(codes) of shape [M, K]."""
    M, K = codes.shape
    s = _scale(scales).to(dtype).repeat_interleave(rows, dim=0)[:M]
    b = _blocks(codes.to(dtype), 1).squeeze(1) * s[:, :, None]
    return b.view(M, -1)[:, :K]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    state = dict(case)

    def held(rows, K, std, block, type, scales, t=False):
        """A quantized N(0, std) matrix (t: the form of its transpose)."""
        x = (normal(rows, K) * std).bfloat16()
        if scales == "fp32":
            # As a checkpoint holds it: a scale of the block's own, amax / 448.
            b = _blocks(x.float(), block)
            s = (b.abs().amax(dim=(1, 3)) / LARGEST[type]).clamp_min(2.0 ** -126)
            codes = (b / s[:, None, :, None]).clamp(-LARGEST[type], LARGEST[type]).to(CODES[type])
            return codes.view(-1, b.shape[2] * BLOCK)[:rows, :K].contiguous(), s
        return (_plain_quantize_t if t else _plain_quantize)(x, block, type, scales)

    if case["op"] == "quantize":
        x = normal(case["M"], case["K"])
        # Some values far out, as activations have them.
        far = torch.rand(x.shape, generator=gen, device=DEV) < 0.001
        state["x"] = torch.where(far, 100 * x, x).bfloat16()
    elif case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        state["a"], state["a_scales"] = held(M, K, 1.0, 1, case["type"], case["scales"])
        state["b"], state["b_scales"] = held(N, K, 0.02, case["block"], "e4m3", case["scales"])
    elif case["op"] == "swiglu":
        M, H, I = case["M"], case["H"], case["I"]
        state["a"], state["a_scales"] = held(M, H, 1.0, 1, "e4m3", "ue8m0")
        state["w"], state["w_scales"] = held(2 * I, H, 0.02, 128, "e4m3", "ue8m0")
    else:
        M, H, I = case["M"], case["H"], case["I"]
        state["dact"] = (normal(M, I) * 1e-3).bfloat16()
        state["gu"] = normal(M, 2 * I).bfloat16()
        state["x_t"], state["x_t_scales"] = held(M, H, 1.0, 1, "e4m3", "ue8m0", t=True)
        state["w_t"], state["w_t_scales"] = held(H, 2 * I, 0.02, 128, "e4m3", "ue8m0")
    return state


# ------------------------------------------------------------- plain forms
def _plain_swiglu(s):
    gu = torch.matmul(_values(s["a"], s["a_scales"], 1), _values(s["w"], s["w_scales"], 128).t())
    g, u = gu[:, :s["I"]], gu[:, s["I"]:]
    act = (g * torch.sigmoid(g) * u).bfloat16()
    codes, scales = _plain_quantize(act, 1, "e4m3", "ue8m0")
    out = [codes, scales.view(torch.float8_e8m0fnu)]
    return out + [gu.bfloat16()] if s["train"] else out


def _plain_grad(s):
    g, u, d = s["gu"][:, :s["I"]].float(), s["gu"][:, s["I"]:].float(), s["dact"].float()
    sig = torch.sigmoid(g)
    dgu = torch.cat([d * u * sig * (1 + g * (1 - sig)), d * g * sig], dim=1)
    rows = _values(*_plain_quantize(dgu, 1, s["type"], "ue8m0"), 1)
    dx = torch.matmul(rows, _values(s["w_t"], s["w_t_scales"], 128).t()).bfloat16()
    cols = _values(*_plain_quantize_t(dgu, 1, s["type"], "ue8m0"), 1)
    dw = torch.matmul(cols, _values(s["x_t"], s["x_t_scales"], 1).t()).bfloat16()
    return dx, dw


def run(state):
    s = state
    if own:
        import block_scaled_microscaling_amd as mx
        if s["op"] == "quantize":
            f = mx.quantize_fp8_2d if s["both"] else mx.quantize_fp8
            return f(s["x"], block_rows=s["block"], dtype=CODES[s["type"]],
                     scale_dtype=torch.float32 if s["scales"] == "fp32" else torch.uint8)
        if s["op"] == "gemm":
            return mx.gemm_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"],
                               out_dtype=OUT[s["out"]])
        if s["op"] == "swiglu":
            out = mx.gemm_fp8_swiglu(s["a"], s["a_scales"], s["w"], s["w_scales"],
                                     want_gu=s["train"])
            return [out[0], out[1].view(torch.float8_e8m0fnu), *out[2:]]
        d, d_scales, d_t, d_t_scales = mx.swiglu_fp8_backward(s["dact"], s["gu"],
                                                              dtype=CODES[s["type"]])
        return (mx.gemm_fp8(d, d_scales, s["w_t"], s["w_t_scales"]),
                mx.gemm_fp8(d_t, d_t_scales, s["x_t"], s["x_t_scales"]))
    if s["op"] == "quantize":
        out = _plain_quantize(s["x"], s["block"], s["type"], s["scales"])
        return out + _plain_quantize_t(s["x"], s["block"], s["type"], s["scales"]) if s["both"] else out
    if s["op"] == "gemm":
        return torch.matmul(_values(s["a"], s["a_scales"], 1),
                            _values(s["b"], s["b_scales"], s["block"]).t()).to(OUT[s["out"]])
    return _plain_swiglu(s) if s["op"] == "swiglu" else _plain_grad(s)


# -------------------------------------------------------------------- work
def _held_bytes(rows, K, block=1, scale=1):
    """Codes and scales of a [rows, K] operand."""
    return rows * K + scale * _ceil(rows, block) * _ceil(K, BLOCK)


def work(case):
    M = case["M"]
    if case["op"] == "quantize":
        K, scale = case["K"], 4 if case["scales"] == "fp32" else 1
        n = 2 * M * K + _held_bytes(M, K, case["block"], scale)
        if case["both"]:
            n += _held_bytes(K, _ceil(M, 16) * 16, case["block"], scale)
        return {"bytes": n, "flops": 0}
    if case["op"] == "gemm":
        N, K, scale = case["N"], case["K"], 4 if case["scales"] == "fp32" else 1
        return {"bytes": _held_bytes(M, K, 1, scale) + _held_bytes(N, K, case["block"], scale)
                + (4 if case["out"] == "fp32" else 2) * M * N, "flops": 2 * M * N * K}
    H, I = case["H"], case["I"]
    if case["op"] == "swiglu":
        return {"bytes": _held_bytes(M, H) + _held_bytes(2 * I, H, 128) + _held_bytes(M, I)
                + (4 * M * I if case["train"] else 0), "flops": 4 * M * H * I}
    # Inputs and results; the quantized gradients of g and u lie between.
    Mp = _ceil(M, 16) * 16
    return {"bytes": 6 * M * I + _held_bytes(H, Mp) + _held_bytes(H, 2 * I, 128) + 2 * M * H
            + 4 * I * H, "flops": 8 * M * H * I}


# ------------------------------------------------------- 64-bit definition
def _two_to(e):
    """2^e in float64, from its bits (a power function may be a bit off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(v, type):
    """The representable value nearest to float64 v, ties to the even one: the
    spacing is 2^(floor(log2 |v|) - mantissa bits), that of the smallest
    normal's binade below it."""
    bits, least = (3, -6) if type == "e4m3" else (2, -14)
    e = (torch.frexp(v).exponent - 1).clamp_min(least)
    step = _two_to(e - bits)
    return torch.round(v / step) * step


def _exact_quantize(x, rows, type):
    """float64 code values [M, K] and exponents per block, block by block of rows."""
    M, K = x.shape
    values, exps = torch.empty((M, K), dtype=torch.float64, device=DEV), []
    step = max(rows, (1 << 26) // K // rows * rows)
    for r in range(0, M, step):
        b = _blocks(x[r:r + step].double(), rows)
        amax = b.abs().amax(dim=(1, 3))
        e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / LARGEST[type]))
        # The logarithm may be off by one at a power of two.
        e = e.clamp(-1000, 1000)
        e = torch.where(amax <= LARGEST[type] * _two_to(e - 1), e - 1, e)
        e = torch.where(amax > LARGEST[type] * _two_to(e), e + 1, e).clamp(-126, 127)
        v = _nearest(b / _two_to(e)[:, None, :, None], type)
        n = min(step, M - r)
        values[r:r + n] = v.view(-1, b.shape[2] * BLOCK)[:n, :K]
        exps.append(e)
    return values, torch.cat(exps)


def _exact_transpose(x):
    return torch.cat([x, x.new_zeros((-x.shape[0] % 16, x.shape[1]))]).t().contiguous()


def _exact_values(values, exps, rows):
    s = _two_to(exps).repeat_interleave(rows, 0)[:values.shape[0]]
    return values * s.repeat_interleave(BLOCK, 1)[:, :values.shape[1]]


def _held64(codes, scales, rows):
    s = scales.double() if scales.dtype == torch.float32 else _two_to(scales.int() - 127)
    s = s.repeat_interleave(rows, 0)[:codes.shape[0]]
    return codes.double() * s.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _product64(a, b):
    """a b^T in pieces of b's rows."""
    step = max(1, (1 << 27) // b.shape[1])
    return torch.cat([a @ b[r:r + step].t().contiguous() for r in range(0, b.shape[0], step)], dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        out = []
        for x in [s["x"], _exact_transpose(s["x"])] if case["both"] else [s["x"]]:
            v, e = _exact_quantize(x, case["block"], case["type"])
            out += [v, _two_to(e) if case["scales"] == "fp32" else (e + 127).to(torch.uint8)]
        return out
    if case["op"] == "gemm":
        return _product64(_held64(s["a"], s["a_scales"], 1),
                          _held64(s["b"], s["b_scales"], case["block"]))
    I = case["I"]
    if case["op"] == "swiglu":
        gu = _product64(_held64(s["a"], s["a_scales"], 1), _held64(s["w"], s["w_scales"], 128))
        g, u = gu[:, :I], gu[:, I:]
        # act is BF16 by definition: the quantizer sees it rounded.
        v, e = _exact_quantize((g / (1 + torch.exp(-g)) * u).bfloat16(), 1, "e4m3")
        return [v, _two_to(e)] + ([gu] if case["train"] else [])
    g, u, d = s["gu"][:, :I].double(), s["gu"][:, I:].double(), s["dact"].double()
    sig = 1 / (1 + torch.exp(-g))
    dgu = torch.cat([d * u * (sig + g * sig * (1 - sig)), d * g * sig], dim=1)
    del g, u, d, sig
    dx = _product64(_exact_values(*_exact_quantize(dgu, 1, case["type"]), 1),
                    _held64(s["w_t"], s["w_t_scales"], 128))
    cols = _exact_values(*_exact_quantize(_exact_transpose(dgu), 1, case["type"]), 1)
    return dx, _product64(cols, _held64(s["x_t"], s["x_t_scales"], 1))
