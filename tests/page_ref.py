"""Definitions in 64 bits, with error bounds, of the calls over a cache in pages
and of the norms and rotation in front of it.

Bounds: a rounding to bf16 is off by at most 2^-8 of the value (half a step), an
fp32 operation by 2^-24 of its result.
"""
import math

import numpy as np
import torch

D = 128
U32, BF = 2.0 ** -24, 2.0 ** -8
E4M3_MAX = np.float32(448)
TINY = np.float32(2.0 ** -126)


def quantise(x):
    """x [..., d] fp64 holding bf16 values: the e4m3 values and fp32 scales of the
    definition, to the bit (fp32 operations as it names them)."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        scale = np.maximum(np.abs(x).max(-1) / E4M3_MAX, TINY)     # a NaN stays
        y = x * (np.float32(1) / scale)[..., None]
    y = np.clip(y, -E4M3_MAX, E4M3_MAX)
    v = torch.from_numpy(np.ascontiguousarray(y)).to(torch.float8_e4m3fn)
    return v, scale


def norm_rope(x, w, pos, inv_freq, eps, interleaved, scale):
    """One head x [d] (w None: not normed): the result and its bound, without the
    rounding to bf16."""
    y = np.array(x, dtype=np.float64)
    mag = 1.0
    if w is not None:
        y = y / math.sqrt((y * y).mean() + eps) * w
        mag = 24.0          # sum of squares (8 + 4 adds and squares), root, quotient, two products
    out, bound = y.copy(), mag * U32 * np.abs(y)
    h = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        # the angle modulo a turn from integers: position times the frequency's turns
        turn = math.fmod(int(pos) * float(f), 2 * math.pi) if abs(pos) < 2 ** 20 else None
        if turn is None:
            from fractions import Fraction
            two_pi = Fraction("6.283185307179586476925286766559005768394338798750211641949889")
            q = Fraction(float(f)) * int(pos) / two_pi
            turn = float((q - math.floor(q)) * two_pi)
        c, s = math.cos(turn) * scale, math.sin(turn) * scale
        out[a], out[b] = y[a] * c - y[b] * s, y[b] * c + y[a] * s
        # angle: f / 2 pi to 53 bits times the position, one rounding to fp32 of at most half a
        # turn (pi 2^-24), sine and cosine to 2 ulp, a product with the scale, two products, a sum
        e = abs(scale) * (math.pi * U32 + abs(pos) * abs(f) * 2.0 ** -52 + 4 * U32) + 4 * U32 * abs(scale)
        bound[a] = bound[b] = (abs(y[a]) + abs(y[b])) * (e + mag * U32 * abs(scale))
    return out, bound


def attend(q, k, v):
    """q [G][d], k, v [n][d] as they are held: o, lse and their bounds (o with the
    rounding to bf16)."""
    G, n = q.shape[0], k.shape[0]
    if n == 0:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, D)), np.zeros(G)
    x = q @ k.T / math.sqrt(D)
    top = x.max(1, keepdims=True)
    p = np.exp(x - top)
    z = p.sum(1, keepdims=True)
    p /= z
    o, lse = p @ v, (np.log(z) + top)[:, 0]
    # a logit: 128 products added in fp32 (each sum may be cut off instead of rounded: 2^-23), the
    # scales, the exponent's argument (|x| and the maximum, both a few roundings)
    ex = 130 * 2 * U32 * (np.abs(q) @ np.abs(k).T) / math.sqrt(D) + 8 * U32 * (np.abs(x) + np.abs(top))
    # a weight: its logit's and the maximum's error, the exponential, rescaling, two 16-bit terms
    ew = np.expm1(2 * ex.max(1, keepdims=True)) + 16 * U32 + 2.0 ** -16
    # sums of n terms in parts: tiles of 16 added in fp32
    es = (n / 16 + 64) * 2 * U32
    bo = (p @ np.abs(v)) * (2 * ew + 2 * es) + BF * np.abs(o) + 1e-37
    bl = ex.max(1) + ew[:, 0] + es + 4 * U32 * np.abs(lse)
    return o, lse, bo, bl
