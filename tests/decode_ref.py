"""Plain references of head norms with rotation and of token log probabilities, from the definitions in
include/moe_decode.h, in 64 bits (angles exactly, as fractions), with the bounds that the error analysis gives."""
import fractions
import functools
import math

import numpy as np

PI = fractions.Fraction("3.14159265358979323846264338327950288419716939937510")
ULP = 2.0 ** -24  # half an ulp of fp32, relative


@functools.lru_cache(maxsize=1 << 18)
def _angle(position, f):
    """position * f in radians, less whole turns, to 64 bits."""
    turn = position * fractions.Fraction(f) / (2 * PI)
    return float((turn - round(turn)) * 2 * PI)


def rope(x, positions, weight, freq, factor, start, inter, eps=1e-6):
    """x: float64 [N, H, D]; weight: [D] or None; freq: [rot / 2] floats (empty: no rotation). Returns y, and the error that
    fp32 arithmetic may leave, before y is rounded to its type."""
    # a norm: the sum of squares to 14 roundings (chains of 8, and 6 additions; positive terms), of which the root keeps half, the mean, its sum with
    # eps and the root's own 4 half ulps, and two products
    y, off = np.array(x), np.zeros_like(x)
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
        off = np.abs(y) * (14 / 2 + 2 + 4 + 2) * ULP
    h = len(freq)
    if not h:
        return y, off
    angle = np.array([[_angle(int(p), float(f)) for f in freq] for p in positions])
    c, s = (factor * t(angle)[:, None] for t in (np.cos, np.sin))
    i = np.arange(h)
    a, b = (start + 2 * i, start + 2 * i + 1) if inter else (start + i, start + h + i)
    u, v, du, dv = y[..., a], y[..., b], off[..., a], off[..., b]
    # cos and sin: half turns rounded to fp32 (3.2 half ulps), their own error (2), the factor (1 and its own rounding 1); a product and a fused one (2)
    size = abs(factor) * (np.abs(u) + np.abs(v)) * (3.2 + 2 + 2 + 2) * ULP + abs(factor) * (du + dv)
    out, bound = np.array(y), off
    out[..., a], out[..., b] = u * c - v * s, u * s + v * c
    bound[..., a] = bound[..., b] = size
    return out, bound


def logprobs(x, ids, top, scale, tile):
    """x: float64 [R, V]. Returns logprobs, top_logprobs, top_ids, entropy, lse, and the bounds of their fp32 errors (of log s,
    and of the entropy). tile: logits that a thread's maximum moves by, at least."""
    R, V = x.shape
    lp, tl, ti = np.full((R, ids.shape[1]), -np.inf), np.full((R, top), -np.inf), np.zeros((R, top), np.int64)
    ent, lse, off, eoff = np.zeros(R), np.full(R, -np.inf), np.zeros(R), np.zeros(R)
    for r in range(R):
        order = np.lexsort((np.arange(V), -x[r]))
        ti[r] = order[:top]
        m = x[r].max()
        if m == -np.inf:
            continue
        t = (x[r] - m) * scale
        e = np.exp(t)
        s, some = e.sum(), e > 0
        p = e / s
        logp = t - math.log(s)
        ok = (ids[r] >= 0) & (ids[r] < V)
        lp[r, ok] = logp[ids[r][ok]]
        tl[r] = logp[ti[r]]
        ent[r] = -(p[some] * logp[some]).sum()
        lse[r] = m * scale + math.log(s)
        # an exponent: difference, product and its factor (4 half ulps of t); its power (2^-22: 4); additions: 16 of a tile, one and
        # three products a tile, 8 + 3 + 3 joinings of 4
        n = 4 + 16 + 4 * (V // tile + 2) + 4 * 14
        et, et2 = (p[some] * -t[some]).sum(), (p[some] * t[some] ** 2).sum()
        off[r] = ULP * (4 * et + n)
        eoff[r] = off[r] + ULP * (et * (n + 4) + 4 * et2 + 2 * (et + math.log(s)))
    return lp, tl, ti, ent, lse, off, eoff
