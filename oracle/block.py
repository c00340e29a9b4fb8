"""Plain numpy reference of the operators around the ternary layers: the norm
into int8 rows, products with group-scaled 4-bit weights, and the mixture of
ternary experts.

Steps that ``include/w2a8_block.h`` states in fp32 are rounded to fp32 here, each
from its value in 64 bits; the others stay in 64 bits.  The layout follows the
header and is written out index by index, with none of the library's code.
"""
from __future__ import annotations

import numpy as np

FLT_MAX = np.float64(np.finfo(np.float32).max)


def f32(v):
    """Values in 64 bits rounded to fp32 (still held in 64 bits)."""
    with np.errstate(over="ignore"):
        return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


def codes8(v):
    """fp32 rows -> (codes as float64, largest magnitudes [R, 1]); a row that is not finite
    has codes 0 and an infinite or NaN magnitude."""
    a = np.abs(v).max(-1, keepdims=True)
    fine = np.isfinite(a)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.minimum(f32(127.0 / np.where(a > 0, a, np.inf)), FLT_MAX)
    inv = np.where(fine & (a > 0), inv, 0.0)
    q = np.clip(np.rint(f32(np.where(fine, v, 0.0) * inv)), -127, 127)
    return q, a


def rmsnorm_quant(h, weight, eps):
    """h: the rounded sums [M, K] in 64 bits, weight [K] or None -> (codes, s_a in 64 bits)."""
    with np.errstate(over="ignore", invalid="ignore"):
        v = h if weight is None else f32(h * weight)
    q, a = codes8(v)
    with np.errstate(divide="ignore", invalid="ignore"):
        s = np.where(a == 0, 0.0, a / 127 / np.sqrt((h ** 2).mean(1, keepdims=True) + eps))
    bad = ~(np.isfinite(a) & np.isfinite(h).all(1, keepdims=True))
    return np.where(bad, 0.0, q), np.where(bad, np.nan, s)[:, 0]


# ---------------------------------------------------------------------------
# 4-bit weights with group scales
# ---------------------------------------------------------------------------
def w4_interchange(q):
    """q uint8 [N, K] -> [N, ceil(K/2)], the lower k in the lower half."""
    n, k = q.shape
    p = np.zeros((n, k + k % 2), np.uint8)
    p[:, :k] = q
    return p[:, 0::2] | (p[:, 1::2] << 4)


def w4_packed(q, scale_bits, zeros, group):
    """q uint8 [N, K], scale bits uint16 and zeros uint8 (or None) [N, groups] -> W4T16x128."""
    n, k = q.shape
    ns, kt, p = -(-n // 16), -(-k // 128), 128 // group
    gq = -(-scale_bits.shape[1] // 4)
    codes = np.zeros((ns, kt, 64, 16), np.uint8)
    for s in range(ns):
        for t in range(kt):
            for c in range(4):
                for r in range(16):
                    for v in range(32):
                        i, o = v // (32 // p), v % (32 // p)
                        kk, row = 128 * t + (128 // p) * i + (32 // p) * c + o, 16 * s + r
                        if kk < k and row < n:
                            j, b = v // 8, v % 8
                            codes[s, t, 16 * c + r, 4 * j + b % 4] |= (((int(q[row, kk]) - 8) & 15) << (4 * (b // 4)))
    sc = np.zeros((ns, gq, 16, 4), np.uint16)
    zs = np.zeros((ns, gq, 16, 4), np.int8)
    for row in range(n):
        for g in range(scale_bits.shape[1]):
            sc[row // 16, g // 4, row % 16, g % 4] = scale_bits[row, g]
            if zeros is not None:
                zs[row // 16, g // 4, row % 16, g % 4] = int(zeros[row, g]) - 8
    parts = [codes.reshape(-1), sc.reshape(-1).view(np.uint8)]
    return np.concatenate(parts if zeros is None else parts + [zs.reshape(-1).view(np.uint8)])


def w4_product(x, s_a, q, scales, zeros, group):
    """In 64 bits: (y [M, N], the sum over groups of the magnitudes of their terms [M, N])."""
    x = x.astype(np.float64)
    n, k = q.shape
    y = np.zeros((x.shape[0], n))
    size = np.zeros_like(y)
    for g in range(-(-k // group)):
        z = 8.0 if zeros is None else zeros[:, g:g + 1].astype(np.float64)
        w = (q[:, g * group:(g + 1) * group].astype(np.float64) - z) * scales[:, g:g + 1].astype(np.float64)
        term = x[:, g * group:(g + 1) * group] @ w.T
        y += term
        size += np.abs(term)
    s = s_a.astype(np.float64)[:, None]
    return y * s, size * np.abs(s)


# ---------------------------------------------------------------------------
# Mixture of experts
# ---------------------------------------------------------------------------
def moe_route(logits, top_k, renormalize):
    """logits float64 [M, E] -> per token the list of (expert, weight), None where a logit is a
    NaN or +infinity."""
    out = []
    for row in logits:
        if np.isnan(row).any() or (row == np.inf).any():
            out.append(None)
            continue
        order = sorted(range(len(row)), key=lambda e: (-row[e], e))[:top_k]
        order = [e for e in order if row[e] != -np.inf]
        if not order:
            out.append([])
            continue
        top = row[order[0]]
        total = sum(np.exp(row[e] - top) for e in (order if renormalize else range(len(row))))
        out.append([(e, np.exp(row[e] - top) / total) for e in order])
    return out


def moe(x, s_a, logits, w_gate, w_up, w_down, s_gate, s_up, s_down, top_k, act, renormalize):
    """x int8 [M, H], weights int8 [E, ., .]: (y [M, H] in 64 bits, bound [M, H]).

    bound: how far y may be off because silu's exponential is not correctly rounded.  h is then
    off by at most 12 units 2^-24 of itself (the exponential 2 units of 2^-24 as the result of a
    correctly reduced argument plus its own rounding, the sum, the quotient and the product one
    each, with room), its largest magnitude too, and v * 127 / a by at most 127 * 26 units: a
    code within that of a border may be its neighbour, and the scale is off by 14 units."""
    M, H = x.shape
    I = w_gate.shape[1]
    y, bound = np.zeros((M, H)), np.zeros((M, H))
    unit = 2.0 ** -24
    for m, chosen in enumerate(moe_route(np.asarray(logits, np.float64), top_k, renormalize)):
        if chosen is None:
            y[m] = np.nan
            continue
        for e, p in chosen:
            xi = x[m].astype(np.int64)
            sa = np.float64(s_a[m])
            g = f32(f32(f32(w_gate[e].astype(np.int64) @ xi) * sa) * np.float64(s_gate[e]))
            u = f32(f32(f32(w_up[e].astype(np.int64) @ xi) * sa) * np.float64(s_up[e]))
            with np.errstate(over="ignore", invalid="ignore"):
                if act == "relu2":
                    r = np.maximum(g, 0.0) + 0 * g
                    h = f32(f32(r * r) * u)
                else:
                    h = f32(f32(g / f32(1 + f32(np.exp(-g)))) * u)
            if not np.isfinite(h).all():
                y[m] = np.nan
                continue
            q, a = codes8(h[None])
            a = float(a[0, 0])
            sh, wd = float(f32(a / 127)), w_down[e].astype(np.float64)
            part = f32(f32(f32(wd @ q[0]) * sh) * np.float64(s_down[e]))
            y[m] += p * part
            if act == "silu" and a > 0:
                v = np.abs(h) * (127 / a)
                near = np.abs(v - np.floor(v) - 0.5) <= 127 * 26 * unit
                bound[m] += p * abs(float(s_down[e])) * (np.abs(wd) @ near) * sh + 14 * unit * p * np.abs(part)
    return y, bound
