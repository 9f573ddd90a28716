"""The few-token operators on MXFP4 weights: their cases, plain forms and work.

Three operators of a decode step, whose activations stay BF16 (a token or a
few, too few for the 32-row blocks of the a4w4 GEMM) while the weights are
MXFP4 (two E2M1 codes a byte, one UE8M0 scale per 32 elements of a row):

  gemv       y[M, N] = x[M, K] dq(W[N, K])^T
  moe_route  the router of a mixture of experts: logits x R^T, softmax over
             the experts, the top k of them (ties to the lowest index) and
             their weights, as they are or divided by their sum
  moe        the experts' SwiGLU MLPs of routed tokens and their weighted sum,
             y[t] = sum_j w[t, j] W2_e (silu(Wg_e x[t]) * (Wu_e x[t])) with
             e = ids[t, j]; an id outside the experts adds nothing (an expert
             that another device holds)

`run` computes a case in its plain form (elementary torch operations in 32
bits, the router's logits in 64), or, where `own` is true, through the
framework's entry points.
"""

import math

import torch

own = False

DEV = "cuda:0"
BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

if own:
    import block_scaled_microscaling_amd  # noqa: F401


# ------------------------------------------------------------------- cases
def _gemv(name, M, N, K, out):
    return {"name": name, "op": "gemv", "M": M, "N": N, "K": K, "out": out}


def _route(name, T, H, E, k, renorm):
    return {"name": name, "op": "route", "T": T, "H": H, "E": E, "k": k, "renorm": renorm}


def _moe(name, T, H, I, E, k, out, absent):
    return {"name": name, "op": "moe", "T": T, "H": H, "I": I, "E": E, "k": k, "out": out,
            "absent": absent}


def listed():
    return [
        # A small projection of one token: launch latency is all of it.
        _gemv("gemv_1x256x256", 1, 256, 256, "fp32"),
        # One token of a decode loop against the 8192 x 8192 decode weight.
        _gemv("gemv_1x8192x8192", 1, 8192, 8192, "bf16"),
        # Eight sequences through an MLP's down projection.
        _gemv("gemv_8x4096x14336", 8, 4096, 14336, "bf16"),
        # Sixteen sequences through the gate+up projection.
        _gemv("gemv_16x28672x4096", 16, 28672, 4096, "bf16"),
        # Odd sizes: five tokens, rows that fill no tile, K past whole lines.
        _gemv("gemv_5x6177x7968", 5, 6177, 7968, "fp32"),
        # The router of one token with few experts, and with many.
        _route("route_1x4096_8top2", 1, 4096, 8, 2, True),
        _route("route_64x4096_128top8", 64, 4096, 128, 8, True),
        # Odd sizes, and the softmax's own weights.
        _route("route_13x2856_61top4", 13, 2856, 61, 4, False),
        # One token through two of eight large experts (the MLP shapes above).
        _moe("moe_1x4096x14336_8top2", 1, 4096, 14336, 8, 2, "bf16", 0.0),
        # One token, and a batch, through many small experts.
        _moe("moe_1x2048x768_128top8", 1, 2048, 768, 128, 8, "bf16", 0.0),
        _moe("moe_32x2048x768_128top8", 32, 2048, 768, 128, 8, "bf16", 0.0),
        # Odd sizes, with a third of the chosen experts on other devices.
        _moe("moe_7x1056x544_10top3", 7, 1056, 544, 10, 3, "fp32", 0.33),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemv", "route", "moe"])
    if op == "gemv":
        while True:
            M, N, K = _log_int(rng, 1, 64), _log_int(rng, 32, 28672), BLOCK * _log_int(rng, 8, 448)
            if rng.random() < 0.5:
                N = max(32, N // 64 * 64)
            if N * K <= 28672 * 4096 and M * N * K <= 16 * 28672 * 4096:
                case = _gemv("", M, N, K, rng.choice(["bf16", "fp32"]))
                break
    elif op == "route":
        E = _log_int(rng, 4, 256)
        case = _route("", _log_int(rng, 1, 64), 8 * _log_int(rng, 8, 1024), E,
                      rng.randint(1, min(8, E)), rng.random() < 0.5)
    else:
        while True:
            E = _log_int(rng, 4, 128)
            T, k = _log_int(rng, 1, 32), rng.randint(1, min(8, E))
            H, I = BLOCK * _log_int(rng, 8, 128), BLOCK * _log_int(rng, 8, 448)
            if E * H * I <= 8 * 4096 * 14336 and T * k * H * I <= 256 * 2048 * 768:
                case = _moe("", T, H, I, E, k, rng.choice(["bf16", "fp32"]),
                            rng.choice([0.0, 0.0, 0.5]))
                break
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
def _quantized(rows, K, std, gen):
    """MXFP4 codes and scales of a N(0, std) weight [rows, K]: the scale's
    exponent is floor(log2 of the block's largest) - 2, codes are nearest."""
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, K // BLOCK), dtype=torch.uint8, device=DEV)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        w = torch.randn((n, K // BLOCK, BLOCK), generator=gen, device=DEV) * std
        top = w.abs().amax(dim=2).clamp_min(2.0 ** -100)
        e = torch.frexp(top).exponent - 3
        v = w / torch.ldexp(torch.ones_like(top), e)[..., None]
        c = torch.bucketize(v.abs(), borders, out_int32=True).to(torch.uint8)
        c |= torch.signbit(v).to(torch.uint8) << 3
        c = c.reshape(n, K)
        codes[r:r + n] = c[:, 0::2] | (c[:, 1::2] << 4)
        scales[r:r + n] = (e + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    state = dict(case)
    if case["op"] == "gemv":
        state["x"] = normal(case["M"], case["K"]).bfloat16()
        state["codes"], state["scales"] = _quantized(case["N"], case["K"], 0.02, gen)
    elif case["op"] == "route":
        state["x"] = normal(case["T"], case["H"]).bfloat16()
        state["router"] = (normal(case["E"], case["H"]) / math.sqrt(case["H"])).bfloat16()
    else:
        T, H, I, E, k = (case[n] for n in "THIEk")
        state["x"] = normal(T, H).bfloat16()
        score = normal(T, E)
        top = score.topk(k, dim=1)
        ids = top.indices.int()
        if case["absent"] > 0:
            away = torch.rand((T, k), generator=gen, device=DEV) < case["absent"]
            ids = torch.where(away, torch.full_like(ids, -1), ids)
        state["ids"] = ids.contiguous()
        state["weights"] = torch.softmax(top.values, dim=1).contiguous()
        c, s = _quantized(E * 2 * I, H, 0.02, gen)
        state["w13_codes"], state["w13_scales"] = c.view(E, 2 * I, H // 2), s.view(E, 2 * I, -1)
        c, s = _quantized(E * H, I, 0.02, gen)
        state["w2_codes"], state["w2_scales"] = c.view(E, H, I // 2), s.view(E, H, -1)
    # What the plain form decodes a byte with: its two elements, low nibble first.
    signed = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    byte = torch.arange(256, device=DEV)
    state["pairs"] = torch.stack([signed[byte & 15], signed[byte >> 4]], dim=1)
    return state


# ------------------------------------------------------------- plain forms
def _out_type(state):
    return torch.float32 if state["out"] == "fp32" else torch.bfloat16


def _dequantize(codes, scales, pairs):
    """float32 [..., K] of codes [..., K/2] and scales [..., K/32]."""
    v = pairs.index_select(0, codes.reshape(-1).int()).view(*scales.shape, BLOCK)
    return (v * (scales.int() << 23).view(torch.float32)[..., None]).flatten(-2)


def _plain_gemv(s):
    w = _dequantize(s["codes"], s["scales"], s["pairs"])
    return torch.matmul(s["x"].float(), w.t()).to(_out_type(s))


def _plain_route(s):
    # 64 bits: which of two close experts is chosen hangs on a logit's last bits.
    logits = torch.matmul(s["x"].double(), s["router"].double().t())
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    weights = torch.softmax(logits, dim=1).gather(1, order)
    if s["renorm"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    return order.int(), weights.float()


def _plain_moe(s):
    ids = s["ids"].long()
    here = (ids >= 0) & (ids < s["E"])
    e = torch.where(here, ids, torch.zeros_like(ids))
    w13 = _dequantize(s["w13_codes"][e], s["w13_scales"][e], s["pairs"])      # [T, k, 2I, H]
    h = torch.matmul(w13, s["x"].float()[:, None, :, None]).squeeze(3)
    del w13
    g, u = h[..., :s["I"]], h[..., s["I"]:]
    act = g * torch.sigmoid(g) * u
    w2 = _dequantize(s["w2_codes"][e], s["w2_scales"][e], s["pairs"])         # [T, k, H, I]
    y = torch.matmul(w2, act[..., None]).squeeze(3)
    weight = torch.where(here, s["weights"], torch.zeros_like(s["weights"]))
    return (y * weight[..., None]).sum(dim=1).to(_out_type(s))


def run(state):
    if own:
        import block_scaled_microscaling_amd as mx
        if state["op"] == "gemv":
            return mx.gemv(state["x"], state["codes"], state["scales"],
                           out_dtype=_out_type(state))
        if state["op"] == "route":
            return mx.moe_route(state["x"], state["router"], state["k"],
                                renormalize=state["renorm"])
        return mx.moe(state["x"], state["ids"], state["weights"], state["w13_codes"],
                      state["w13_scales"], state["w2_codes"], state["w2_scales"],
                      out_dtype=_out_type(state))
    return {"gemv": _plain_gemv, "route": _plain_route, "moe": _plain_moe}[state["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    out = {"bf16": 2, "fp32": 4}
    if case["op"] == "gemv":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K // 2 + N * K // BLOCK + 2 * M * K + out[case["out"]] * M * N,
                "flops": 2 * M * N * K}
    if case["op"] == "route":
        T, H, E, k = (case[n] for n in "THEk")
        return {"bytes": 2 * T * H + 2 * E * H + 8 * T * k, "flops": 2 * T * H * E}
    T, H, I, E, k = (case[n] for n in "THIEk")
    # Experts that any token chose, in the mean over uniform choices.
    held = (1.0 - case["absent"]) * k
    active = E * (1.0 - (1.0 - held / E) ** T)
    weight = 3 * H * I
    return {"bytes": int(active * (weight // 2 + weight // BLOCK)) + 2 * T * H + 8 * T * k
            + out[case["out"]] * T * H,
            "flops": int(2 * weight * T * held)}


# ------------------------------------------------------- 64-bit definition
def _value64(codes, scales):
    """float64 [rows, K] by the format's definition: the element with exponent
    field e and mantissa bit m is (-1)^s 2^(e - 1) (1 + m / 2), or m / 2 for
    e = 0, times 2^(scale - 127)."""
    nibbles = torch.stack([codes & 15, codes >> 4], dim=2).flatten(1).to(torch.int16)
    e, m = (nibbles >> 1) & 3, (nibbles & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    v = torch.where(nibbles >= 8, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, dim=1)


def _product64(x, codes, scales):
    """x [M, K] times the rows' values, in pieces of rows."""
    step = max(1, (1 << 26) // x.shape[1])
    return torch.cat([x @ _value64(codes[r:r + step], scales[r:r + step]).t().contiguous()
                      for r in range(0, codes.shape[0], step)], dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "gemv":
        return _product64(x, s["codes"], s["scales"])
    if case["op"] == "route":
        logits = (x[:, None, :] * s["router"].double()[None]).sum(dim=2)
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        # An expert's place: how many are larger, or equal with a lower index.
        before = torch.ones_like(logits[0][:, None] * logits[0][None]).tril(-1) > 0
        larger = (logits[:, None, :] > logits[:, :, None])
        same = (logits[:, None, :] == logits[:, :, None]) & before
        place = (larger | same).sum(dim=2)
        ids = torch.argsort(place, dim=1)[:, :case["k"]]
        w = p.gather(1, ids)
        return ids.int(), w / w.sum(dim=1, keepdim=True) if case["renorm"] else w
    y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        gu = _product64(x[t], s["w13_codes"][e], s["w13_scales"][e])
        g, u = gu[:, :case["I"]], gu[:, case["I"]:]
        part = _product64(g / (1 + torch.exp(-g)) * u, s["w2_codes"][e], s["w2_scales"][e])
        y.index_add_(0, t, part * s["weights"][t, j].double()[:, None])
    return y
