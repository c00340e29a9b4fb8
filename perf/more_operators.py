"""Cases of the operators around the ternary layers that take and make int8 rows:
root-mean-square normalisation with the residual's addition into int8 rows,
products of int8 rows with 4-bit weights and group scales, and a
mixture-of-experts layer with ternary experts for a few tokens.

norm: h = x + residual, rounded to their type; v = h * weight in 32 bits;
a = max |v| of the row; codes = v * (127 / a) rounded half to even, each step in
32 bits; scale = a / 127 / sqrt(mean(h^2) + eps).

w4: y[m][n] = s_a[m] * sum_g s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) * x[m][k],
q and z in 0..15 (z = 8 without zero points), groups of consecutive k.

moe: every token takes the top_k experts of its router logits (ties: the lower
index), weighted by a softmax over them or over all.  For each, int8 rows times
ternary weights:
  g = ((x w_gate^T) s_a) s_gate,  u = ((x w_up^T) s_a) s_up,
  h = silu(g) u  or  relu(g)^2 u,  h to int8 by its largest magnitude (s_h),
  y += p ((q w_down^T) s_h) s_down.

``own`` False computes the operators from elementary torch operations; True
calls the library.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
FLT_MAX = torch.finfo(torch.float32).max

# The largest listed matrices: a 4-bit one, all experts' ones, the norm's rows.
MOST_NK = 55296 * 5120
MOST_EXPERTS = 16 * 5120 * 6912
MOST_MK = 8192 * 5120


def listed():
    return [
        # One token's hidden state behind a block, added to the residual.
        {"name": "norm decode", "op": "norm", "m": 1, "k": 2560, "type": "bf16", "residual": True, "weight": True},
        # A large prefill batch of a wide model.
        {"name": "norm prefill", "op": "norm", "m": 8192, "k": 5120, "type": "bf16", "residual": True, "weight": True},
        # The inner norm of a feed-forward block: no residual, rows of odd length in 32 bits.
        {"name": "norm ragged", "op": "norm", "m": 2045, "k": 6907, "type": "fp32", "residual": False, "weight": True},
        # One token through a small projection kept in 4 bits.
        {"name": "w4 decode small", "op": "w4", "m": 1, "n": 2560, "k": 2560, "group": 128, "scale": "fp16", "zeros": False, "out": "fp32"},
        # One token against the widest matrix: an output head.
        {"name": "w4 decode large", "op": "w4", "m": 1, "n": 55296, "k": 5120, "group": 128, "scale": "bf16", "zeros": False, "out": "bf16"},
        # A few sequences decoded together, the finest groups, zero points, a k that ends inside a group.
        {"name": "w4 batch ragged", "op": "w4", "m": 19, "n": 13824, "k": 2570, "group": 32, "scale": "fp16", "zeros": True, "out": "fp32"},
        # Many sequences decoded together through a down projection.
        {"name": "w4 batch", "op": "w4", "m": 64, "n": 5120, "k": 27648, "group": 64, "scale": "fp16", "zeros": False, "out": "bf16"},
        # One token through a few large experts.
        {"name": "moe decode large", "op": "moe", "m": 1, "h": 2560, "i": 6912, "e": 8, "top_k": 2, "act": "relu2", "renormalize": True},
        # One token through many small experts.
        {"name": "moe decode small", "op": "moe", "m": 1, "h": 2560, "i": 640, "e": 64, "top_k": 8, "act": "silu", "renormalize": False},
        # A few sequences decoded together, rows of odd length.
        {"name": "moe batch ragged", "op": "moe", "m": 13, "h": 2565, "i": 1283, "e": 32, "top_k": 4, "act": "silu", "renormalize": True},
        # Many sequences decoded together: every expert has tokens.
        {"name": "moe batch", "op": "moe", "m": 64, "h": 5120, "i": 6912, "e": 16, "top_k": 2, "act": "relu2", "renormalize": True},
    ]


def _size(rng, low, high):
    """A whole number spread over the logarithm of low..high, odd or even."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "w4", "moe", "w4", "moe"])
    if op == "norm":
        k = _size(rng, 32, 27648)
        return {"op": op, "m": _size(rng, 1, max(1, min(8192, MOST_MK // (2 * k)))), "k": k, "type": rng.choice(sorted(TYPES)),
                "residual": rng.random() < 0.7, "weight": rng.random() < 0.8}
    if op == "w4":
        k = _size(rng, 32, 27648)
        return {"op": op, "m": rng.choice([1, _size(rng, 2, 64)]), "n": _size(rng, 16, min(55296, MOST_NK // k)), "k": k,
                "group": rng.choice([32, 64, 128]), "scale": rng.choice(["bf16", "fp16"]), "zeros": rng.random() < 0.5,
                "out": rng.choice(["fp32", "bf16"])}
    h, i = _size(rng, 256, 5120), _size(rng, 128, 6912)
    e = _size(rng, 4, min(128, MOST_EXPERTS // (h * i)))
    return {"op": op, "m": rng.choice([1, _size(rng, 2, 64)]), "h": h, "i": i, "e": e, "top_k": rng.randint(1, min(8, e)),
            "act": rng.choice(["relu2", "silu"]), "renormalize": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _codes8(v):
    """Rows in 32 bits -> int8 codes (as 32-bit values) and each row's largest magnitude / 127."""
    a = v.abs().amax(-1, keepdim=True)
    inv = torch.where(a > 0, (127.0 / a.double()).float().clamp(max=FLT_MAX), 0.0)   # the 32-bit quotient, at a border too
    return (v * inv).round().clamp(-127, 127), a / 127.0


def _plain_norm(state):
    x, r = state["x"], state["residual"]
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    v = h.float()
    scale = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    q, s = _codes8(v if state["weight"] is None else v * state["weight"].float())
    return {"values": q * (s * scale)} if r is None else {"values": q * (s * scale), "h": h}


def _plain_w4(state):
    case = state["case"]
    k = case["k"]
    q = torch.stack([state["codes"] & 15, state["codes"] >> 4], 2).flatten(1)[:, :k].float()
    of = torch.arange(k, device=q.device) // case["group"]
    z = state["zeros"].float()[:, of] if case["zeros"] else 8.0
    w = (q - z) * state["scales"].float()[:, of]
    return {"y": ((state["x"].float() @ w.t()) * state["s_a"][:, None]).to(TYPES[case["out"]])}


def _act(name, g, u):
    return g / (1.0 + torch.exp(-g)) * u if name == "silu" else (g.clamp(min=0) * g.clamp(min=0)) * u


def _choose(state, logits):
    """The experts of each token, [M, top_k], and their weights."""
    case = state["case"]
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    best, ids = best[:, :case["top_k"]], ids[:, :case["top_k"]]
    e = torch.exp(best - best[:, :1])
    whole = e if case["renormalize"] else torch.exp(logits - best[:, :1])
    return ids, e / whole.sum(1, keepdim=True)


def _plain_moe(state):
    case = state["case"]
    m, e, top = case["m"], case["e"], case["top_k"]
    ids, p = _choose(state, state["logits"].float())
    x, sa = state["x"].float(), state["s_a"][:, None, None]
    few = m * top <= e
    if few:
        rows = x.repeat_interleave(top, 0).unsqueeze(2)
        first = lambda w: torch.bmm(w[ids.flatten()].float(), rows).view(m, top, -1)  # noqa: E731
    else:
        of = ids.unsqueeze(2).expand(-1, -1, case["i"])
        first = lambda w: (x @ w.float().flatten(0, 1).t()).view(m, e, -1).gather(1, of)  # noqa: E731
    g = (first(state["w_gate"]) * sa) * state["s_gate"][ids].unsqueeze(2)
    u = (first(state["w_up"]) * sa) * state["s_up"][ids].unsqueeze(2)
    q, s = _codes8(_act(case["act"], g, u))
    if few:
        d = torch.bmm(state["w_down"][ids.flatten()].float(), q.flatten(0, 1).unsqueeze(2)).view(m, top, -1)
    else:
        every = torch.zeros(m, e, case["i"], device=q.device).scatter(1, of, q)
        d = torch.bmm(every.transpose(0, 1).contiguous(), state["w_down"].float().transpose(1, 2).contiguous())
        d = d.transpose(0, 1).gather(1, ids.unsqueeze(2).expand(-1, -1, case["h"]))
    y = ((d * s) * state["s_down"][ids].unsqueeze(2) * p.unsqueeze(2)).sum(1)
    return {"y": y.to(torch.bfloat16)}


def _plain(state):
    return {"norm": _plain_norm, "w4": _plain_w4, "moe": _plain_moe}[state["case"]["op"]](state)


def _own(state):
    import w2a8_gemv_amd as w2a8
    case = state["case"]
    if case["op"] == "norm":
        x_q, s_a, h = w2a8.rmsnorm_quant_int8(state["x"], state["weight"], residual=state["residual"], eps=EPS)
        values = torch.mul(x_q, s_a.unsqueeze(1))
        return {"values": values} if state["residual"] is None else {"values": values, "h": h}
    if case["op"] == "w4":
        return {"y": w2a8.gemm_w4a8(state["w_packed"], state["x"], state["s_a"], case["n"], case["k"], case["group"],
                                    scale_dtype=TYPES[case["scale"]], zeros=case["zeros"], out_dtype=TYPES[case["out"]])}
    return {"y": w2a8.moe(state["x"], state["s_a"], state["logits"], state["p_gate"], state["p_up"], state["p_down"],
                          state["s_gate"], state["s_up"], state["s_down"], case["h"], case["i"], case["top_k"],
                          activation=case["act"], renormalize=case["renormalize"], out_dtype=torch.bfloat16)}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _float_rows(gen, m, k):
    """Hidden states: normal, with one channel in 128 some twenty times larger."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    loud = torch.rand(k, generator=gen, device="cuda") < 1 / 128
    return x * torch.where(loud, 20.0, 1.0)


def _int8_rows(gen, m, k):
    q, s = _codes8(_float_rows(gen, m, k))
    return q.to(torch.int8), s.flatten()


def _w4_packed(q, scales, zeros, group):
    """The packed form of 4-bit weights: q int [N, K] with 8 subtracted, and so zeros.
    Tiles of 16 rows x 128 k, a lane's 32 values in 128 / group pieces (one at least),
    two values a byte; then the scales and the zeros, 16 rows x 4 groups at a time."""
    n, k = q.shape
    parts = max(1, 128 // group)
    q = torch.nn.functional.pad(q, (0, -k % 128, 0, -n % 16))
    strips = q.shape[0] // 16
    v = q.view(strips, 16, -1, parts, 4, 32 // parts).permute(0, 2, 4, 1, 3, 5).reshape(-1, 4, 2, 4)
    codes = ((v[:, :, 0] & 15) | ((v[:, :, 1] & 15) << 4)).to(torch.uint8).flatten()
    per_group = lambda t: torch.nn.functional.pad(t, (0, -t.shape[1] % 4, 0, -n % 16)).view(strips, 16, -1, 4) \
        .transpose(1, 2).contiguous().view(torch.uint8).flatten()  # noqa: E731
    parts = [codes, per_group(scales)]
    return torch.cat(parts if zeros is None else parts + [per_group(zeros.to(torch.int8))])


def _ternary_packed(w):
    """The packed form of ternary weights [E, N, K], one expert a row (32 x 128 tiles, code w + 1)."""
    e, n, k = w.shape
    c = torch.nn.functional.pad((w + 1).to(torch.uint8), (0, -k % 128, 0, -n % 32), value=1)
    c = c.view(e, (n + 31) // 32, 8, 4, (k + 127) // 128, 8, 4, 4)
    b = c[..., 0, :] | (c[..., 1, :] << 2) | (c[..., 2, :] << 4) | (c[..., 3, :] << 6)
    return b.permute(0, 1, 4, 2, 5, 3, 6).flatten(1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.rand(*shape, generator=gen, device="cuda")  # noqa: E731
    state = {"case": case}
    if case["op"] == "norm":
        m, k, dtype = case["m"], case["k"], TYPES[case["type"]]
        state["x"] = (torch.randn(m, k, generator=gen, device="cuda") * 0.5).to(dtype)
        state["residual"] = _float_rows(gen, m, k).to(dtype) if case["residual"] else None
        state["weight"] = (1 + 0.1 * torch.randn(k, generator=gen, device="cuda")).to(dtype) if case["weight"] else None
        return state
    if case["op"] == "w4":
        n, k, groups = case["n"], case["k"], -(-case["k"] // case["group"])
        state["x"], state["s_a"] = _int8_rows(gen, case["m"], k)
        q = torch.randint(0, 16, (n, k), generator=gen, device="cuda", dtype=torch.int8)
        state["scales"] = (0.002 + 0.008 * rand(n, groups)).to(TYPES[case["scale"]])
        state["zeros"] = torch.randint(5, 11, (n, groups), generator=gen, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        c = torch.nn.functional.pad(q, (0, k % 2)).to(torch.uint8)
        state["codes"] = c[:, 0::2] | (c[:, 1::2] << 4)
        state["w_packed"] = _w4_packed(q - 8, state["scales"], state["zeros"].to(torch.int8) - 8 if case["zeros"] else None, case["group"])
        return state
    m, h, i, e = case["m"], case["h"], case["i"], case["e"]
    state["x"], state["s_a"] = _int8_rows(gen, m, h)
    state["logits"] = 2 * torch.randn(m, e, generator=gen, device="cuda")
    for name, n, k in (("gate", i, h), ("up", i, h), ("down", h, i)):
        w = torch.randint(-1, 2, (e, n, k), generator=gen, device="cuda", dtype=torch.int8)
        state["w_" + name], state["p_" + name] = w, _ternary_packed(w)
        state["s_" + name] = rand(e) / 32 + 1 / 64
    return state


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    m = case["m"]
    if case["op"] == "norm":
        k, t = case["k"], size[case["type"]]
        moved = t * (3 if case["residual"] else 1) + 1
        return {"bytes": m * (k * moved + 4) + (k * t if case["weight"] else 0), "flops": 8 * m * k}
    if case["op"] == "w4":
        n, k, groups = case["n"], case["k"], -(-case["k"] // case["group"])
        weights = n * (k / 2 + groups * (3 if case["zeros"] else 2))
        return {"bytes": weights + m * (k + 4) + m * n * size[case["out"]], "flops": 2 * m * n * k}
    h, i, e, top = case["h"], case["i"], case["e"], case["top_k"]
    taken = e * (1 - (1 - top / e) ** m)          # experts that some token takes, on average
    return {"bytes": taken * 3 * h * i / 4 + m * (h + 4 + 4 * e + 2 * h), "flops": m * top * 6 * h * i}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _to32(v):
    """64-bit values rounded to 32 bits, where the definition rounds."""
    return v.float().double()


def _exact_norm(state):
    x, r, w = state["x"], state["residual"], state["weight"]
    h = x.double() if r is None else (x.double() + r.double()).to(x.dtype).double()
    v = h if w is None else _to32(h * w.double())
    a = v.abs().max(1, keepdim=True).values
    q = torch.clamp(torch.round(_to32(v * _to32(127.0 / a).clamp(max=FLT_MAX))), -127, 127)
    q = torch.where(a == 0, torch.zeros_like(q), q)
    values = q * (a / 127.0) / torch.sqrt((h ** 2).sum(1, keepdim=True) / h.shape[1] + EPS)
    return {"values": values} if r is None else {"values": values, "h": h}


def _exact_w4(state):
    case = state["case"]
    n, k, group = case["n"], case["k"], case["group"]
    c = state["codes"]
    q = torch.empty(n, 2 * c.shape[1], dtype=torch.float64, device=c.device)
    q[:, 0::2], q[:, 1::2] = (c % 16).double(), (c // 16).double()
    q = q[:, :k]
    if case["zeros"]:
        q -= state["zeros"].double().repeat_interleave(group, 1)[:, :k]
    else:
        q -= 8
    q *= state["scales"].double().repeat_interleave(group, 1)[:, :k]
    x = state["x"].double() * state["s_a"].double().unsqueeze(1)
    return {"y": x @ q.t()}


def _exact_moe(state):
    case = state["case"]
    x = state["x"].double() * state["s_a"].double().unsqueeze(1)
    logits = state["logits"].double()
    y = torch.zeros(case["m"], case["h"], dtype=torch.float64, device=x.device)
    place = torch.arange(case["e"], device=x.device)
    for e in range(case["e"]):
        mine = logits[:, e:e + 1]
        before = (logits > mine) | ((logits == mine) & (place < e))
        rows = (before.sum(1) < case["top_k"]).nonzero().flatten()
        if not rows.numel():
            continue
        g = (x[rows] @ state["w_gate"][e].double().t()) * state["s_gate"][e].double()
        u = (x[rows] @ state["w_up"][e].double().t()) * state["s_up"][e].double()
        h = u * (g * torch.sigmoid(g) if case["act"] == "silu" else torch.relu(g) ** 2)
        s = h.abs().max(1, keepdim=True).values / 127
        q = torch.round(h / torch.where(s > 0, s, 1.0)) * s
        # The softmax over all experts, or over those that this token takes.
        rank = ((logits.unsqueeze(2) < logits.unsqueeze(1)) | ((logits.unsqueeze(2) == logits.unsqueeze(1)) & (place.unsqueeze(0) < place.unsqueeze(1)))).sum(2)
        taken = logits if not case["renormalize"] else logits.masked_fill(rank >= case["top_k"], -math.inf)
        p = torch.softmax(taken, 1)[rows, e].unsqueeze(1)
        y[rows] += p * (q @ state["w_down"][e].double().t()) * state["s_down"][e].double()
    return {"y": y}


def exact(case, seed):
    state = prepare(case, seed)
    return {"norm": _exact_norm, "w4": _exact_w4, "moe": _exact_moe}[case["op"]](state)
