"""Cases of the microscaled 4-bit (MX4) operators: quantisation of activation
rows, their product with MX4 weights and with packed ternary weights, and the
whole linear layer of either.

MX4: blocks of 32 consecutive k share one power of two 2^e (a byte e + 127),
and each value is a 4-bit float of 1 sign, 2 exponent and 1 mantissa bits:
magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.  A block of largest magnitude a has
e = floor(log2 a) - 2, at least -127, and each value is x * 2^-e rounded half
to even, at most 6 in magnitude.

``own`` False computes the operators from elementary torch operations in 32
bits; True calls the library.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# The largest listed product, and the largest matrices of it.
MOST_MNK = 8192 * 13824 * 5120
MOST_NK = 55296 * 5120
MOST_MN = 8192 * 13824


def listed():
    return [
        # One token's hidden state: two launches, all latency.
        {"name": "quant decode", "op": "quant", "m": 1, "k": 2560, "type": "bf16"},
        # A prefill batch of 32-bit rows whose length is no multiple of a block.
        {"name": "quant prefill ragged", "op": "quant", "m": 2045, "k": 6907, "type": "fp32"},
        # One token against a small projection, and against the widest matrix.
        {"name": "w4 decode small", "op": "w4", "m": 1, "n": 2560, "k": 2560, "out": "fp32"},
        {"name": "w4 decode large", "op": "w4", "m": 1, "n": 55296, "k": 5120, "out": "bf16"},
        # A few sequences decoded together, a count that fills no tile.
        {"name": "w4 short batch", "op": "w4", "m": 19, "n": 13824, "k": 2560, "out": "fp32"},
        # A prompt, and a large prefill batch.
        {"name": "w4 prefill", "op": "w4", "m": 512, "n": 13824, "k": 2560, "out": "bf16"},
        {"name": "w4 prefill large", "op": "w4", "m": 8192, "n": 13824, "k": 5120, "out": "bf16"},
        # The same range with ternary weights: decode over a long k, a prompt
        # through a down projection, a large prefill batch of odd length.
        {"name": "w2 decode large", "op": "w2", "m": 1, "n": 5120, "k": 27648, "out": "fp32"},
        {"name": "w2 prefill", "op": "w2", "m": 512, "n": 2560, "k": 6912, "out": "bf16"},
        {"name": "w2 prefill ragged", "op": "w2", "m": 4001, "n": 13824, "k": 2560, "out": "fp32"},
        # The whole layer for one token, float row in, float row out.
        {"name": "layer w4 decode", "op": "layer w4", "m": 1, "n": 13824, "k": 2560, "type": "bf16", "out": "bf16"},
        {"name": "layer w2 decode", "op": "layer w2", "m": 1, "n": 6912, "k": 5120, "type": "bf16", "out": "fp32"},
    ]


def _size(rng, low, high):
    """A whole number spread over the logarithm of low..high, odd or even."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quant", "w4", "w2", "w4", "w2", "layer w4", "layer w2"])
    if op == "quant":
        k = _size(rng, 32, 27648)
        return {"op": op, "m": _size(rng, 1, max(1, min(8192, 2045 * 6907 // k))), "k": k,
                "type": rng.choice(sorted(TYPES))}
    k = _size(rng, 32, 27648)
    n = _size(rng, 16, min(55296, MOST_NK // k))
    m = rng.choice([1, _size(rng, 2, 32), _size(rng, 33, max(33, min(8192, MOST_MNK // (n * k), MOST_MN // n)))])
    case = {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["fp32", "bf16"])}
    if op.startswith("layer"):
        case["type"] = rng.choice(sorted(TYPES))
    return case


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _blocks(x):
    """x [R, K] in 32 bits, padded with zeros to whole tiles of 128, as [R, blocks, 32]."""
    r, k = x.shape
    return torch.nn.functional.pad(x.float(), (0, -k % 128)).view(r, -1, 32)


def _power(e):
    """2^e in 32 bits for whole e in -127..127."""
    bits = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22))
    return bits.to(torch.int32).view(torch.float32)


def _round(x):
    """x [R, K] -> the block exponents [R, B] and the values times 2^-e, rounded, [R, B, 32]."""
    b = _blocks(x)
    a = b.abs().amax(2)
    e = torch.where(a > 0, torch.frexp(a.double())[1] - 3, -127).clamp(-127, 127).to(torch.int32)
    y = b * _power(-e).unsqueeze(2)
    g = y.abs()
    step = torch.where(g < 2, 0.5, torch.where(g < 4, 1.0, 2.0))
    return e, torch.copysign(((g / step).round() * step).clamp(max=6.0), y)


def _rounded(x):
    """The 32-bit values [R, K] that x stands for after quantisation."""
    e, q = _round(x)
    return (q * _power(e).unsqueeze(2)).flatten(1)[:, :x.shape[1]]


def _values(codes, scales, k):
    """Two codes a byte, the lower k in the lower half, and a scale byte a block -> 32-bit values."""
    table = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], 2).flatten(1).int()]
    return (v.view(v.shape[0], -1, 32) * _power(scales.int() - 127).unsqueeze(2)).flatten(1)[:, :k]


def _plain(state):
    case, op = state["case"], state["case"]["op"]
    k = case["k"]
    if op == "quant":
        return {"values": _rounded(state["x"]).to(state["x"].dtype)}
    x = _rounded(state["x"]) if op.startswith("layer") else _values(state["x_codes"], state["x_scales"], k)
    if op.endswith("w4"):
        y = x @ _values(state["w_codes"], state["w_scales"], k).t()
    else:
        y = (x @ state["w"].float().t()) * state["s_w"]
    return {"y": y.to(TYPES[case["out"]])}


def _own(state):
    import w2a8_gemv_amd as w2a8
    case, op = state["case"], state["case"]["op"]
    n, k = case.get("n"), case["k"]
    if op == "quant":
        x_q, x_s = w2a8.quant_act_mx4(state["x"])
        return {"values": w2a8.dequant_act_mx4(x_q, x_s, k, dtype=state["x"].dtype)}
    out = TYPES[case["out"]]
    if op == "w4":
        return {"y": w2a8.gemm_w4mx4(state["w_packed"], state["x_q"], state["x_s"], n, k, out_dtype=out)}
    if op == "w2":
        return {"y": w2a8.gemm_w2mx4(state["w_packed"], state["x_q"], state["x_s"], state["s_w"], n, k, out_dtype=out)}
    if op == "layer w4":
        return {"y": w2a8.linear_w4mx4(state["x"], state["w_packed"], n, k, out_dtype=out)}
    return {"y": w2a8.linear_w2mx4(state["x"], state["w_packed"], state["s_w"], n, k, out_dtype=out)}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _codes(x):
    """x [R, K] -> its 4-bit codes [R, padded K], one a byte, and the scale bytes [R, blocks]."""
    e, q = _round(x)
    g = q.abs()
    c = torch.where(g < 2, g * 2, torch.where(g < 4, g + 2, g / 2 + 4)).to(torch.uint8)
    return (c + 8 * (q < 0)).to(torch.uint8).flatten(1), (e + 127).to(torch.uint8)


def _pairs(c):
    """Codes two a byte, the lower k in the lower half: the form they are exchanged in."""
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _interleaved(c):
    """Codes two a byte as the library's rows hold them: byte j of a chunk of
    16 holds values j and 8 + j, byte 4 + j values 4 + j and 12 + j."""
    c = c.view(c.shape[0], -1, 2, 2, 4)
    return (c[:, :, 0] | (c[:, :, 1] << 4)).reshape(c.shape[0], -1)


def _four_tiles(s):
    """Scale bytes [R, 4 a tile] -> [R, groups of four tiles, 4 blocks, 4 tiles]."""
    s = torch.nn.functional.pad(s, (0, -s.shape[1] % 16))
    return s.view(s.shape[0], -1, 4, 4).transpose(2, 3).contiguous()


def _tiled(c, s):
    """The packed form of MX4 weights: 16 x 128 tiles of codes, then of scales."""
    rows = -c.shape[0] % 16
    c = torch.nn.functional.pad(_interleaved(c), (0, 0, 0, rows))
    s = torch.nn.functional.pad(s, (0, 0, 0, rows))
    tiles = c.view(c.shape[0] // 16, 16, -1, 4, 16).permute(0, 2, 3, 1, 4)
    scales = _four_tiles(s)
    scales = scales.view(s.shape[0] // 16, 16, -1, 4, 4).permute(0, 2, 3, 1, 4)
    return torch.cat([tiles.flatten(), scales.flatten()])


def _ternary_packed(w):
    """The packed form of ternary weights (32 x 128 tiles, code w + 1)."""
    n, k = w.shape
    c = torch.nn.functional.pad((w + 1).to(torch.uint8), (0, -k % 128, 0, -n % 32), value=1)
    c = c.view((n + 31) // 32, 8, 4, (k + 127) // 128, 8, 4, 4)
    b = c[..., 0, :] | (c[..., 1, :] << 2) | (c[..., 2, :] << 4) | (c[..., 3, :] << 6)
    return b.permute(0, 3, 1, 4, 2, 5).flatten()


def _float_rows(gen, m, k):
    """Hidden states: normal, with one channel in 128 some twenty times larger."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    loud = torch.rand(k, generator=gen, device="cuda") < 1 / 128
    return x * torch.where(loud, 20.0, 1.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    state = {"case": case}
    x = _float_rows(gen, m, k)
    if op == "quant" or op.startswith("layer"):
        state["x"] = x.to(TYPES[case["type"]])
    else:
        c, s = _codes(x)
        state["x_codes"], state["x_scales"] = _pairs(c), s
        state["x_q"], state["x_s"] = _interleaved(c), _four_tiles(s).flatten(1)
    if op.endswith("w4"):
        c, s = _codes(torch.randn(case["n"], k, generator=gen, device="cuda") * 0.02)
        state["w_codes"], state["w_scales"] = _pairs(c), s
        state["w_packed"] = _tiled(c, s)
    elif op.endswith("w2"):
        w = torch.randint(-1, 2, (case["n"], k), generator=gen, device="cuda", dtype=torch.int8)
        state["w"], state["w_packed"] = w, _ternary_packed(w)
        state["s_w"] = float(torch.rand(1, generator=gen, device="cuda").float()) / 32 + 1 / 64
    return state


def work(case):
    m, k = case["m"], case["k"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    mx = k / 2 + k / 32                       # bytes of a row of k values
    if case["op"] == "quant":
        return {"bytes": m * (2 * k * size[case["type"]] + mx), "flops": 4 * m * k}
    n = case["n"]
    weights = n * (mx if case["op"].endswith("w4") else k / 4)
    rows = m * (k * size[case["type"]] if case["op"].startswith("layer") else mx)
    return {"bytes": weights + rows + m * n * size[case["out"]], "flops": 2 * m * n * k}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_rounded(x):
    """x [R, K] in 64 bits -> the values that its MX4 codes stand for: the
    magnitude's place among the seven borders between neighbours, where a tie
    goes to the even code."""
    r, k = x.shape
    b = torch.zeros(r, -(-k // 32) * 32, dtype=torch.float64, device=x.device)
    b[:, :k] = x.double()
    b = b.view(r, -1, 32)
    a = b.abs().max(2, keepdim=True).values
    e = (torch.floor(torch.log2(a)) - 2).clamp(min=-127)
    e = torch.where(torch.ldexp(torch.ones_like(a), e + 3) <= a, e + 1, e)       # a logarithm next to a whole number
    e = torch.where((torch.ldexp(torch.ones_like(a), e + 2) > a) & (e > -127), e - 1, e)
    unit = torch.pow(2.0, e)
    g = b.abs() / unit
    v = torch.zeros_like(g)
    for border, closed, gap in ((0.25, False, 0.5), (0.75, True, 0.5), (1.25, False, 0.5), (1.75, True, 0.5),
                                (2.5, False, 1.0), (3.5, True, 1.0), (5.0, False, 2.0)):
        v += gap * ((g >= border) if closed else (g > border))
    return (torch.sign(b) * v * unit).flatten(1)[:, :k]


def _exact_values(codes, scales, k):
    c = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = (codes % 16).double(), (codes // 16).double()
    sign, c = 1 - 2 * (c >= 8), c % 8
    expo, half = torch.floor(c / 2), c % 2
    v = sign * torch.where(expo > 0, (1 + half / 2) * torch.pow(2.0, expo - 1), half / 2)
    unit = torch.pow(2.0, scales.double() - 127)
    return (v * unit.repeat_interleave(32, 1))[:, :k]


def exact(case, seed):
    state = prepare(case, seed)
    op, k = case["op"], case["k"]
    if op == "quant":
        return {"values": _exact_rounded(state["x"])}
    x = _exact_rounded(state["x"]) if op.startswith("layer") else _exact_values(state["x_codes"], state["x_scales"], k)
    if op.endswith("w4"):
        w = _exact_values(state["w_codes"], state["w_scales"], k)
        return {"y": x @ w.t()}
    return {"y": (x @ state["w"].double().t()) * state["s_w"]}
