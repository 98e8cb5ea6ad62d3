"""Plain 64-bit forms of rotation, rotated append, chunk attention and decode with sinks."""
from __future__ import annotations

import math

import numpy as np
import torch

from _cache_ops import Layout  # noqa: F401

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


# ------------------------------------------------------------------ rotation
def rates(rot, base, scaling=None, factor=1.0, original=0):
    """(radians per position of every pair, magnitude)."""
    got, magnitude = [], 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    for j in range(rot // 2):
        r = base ** (-2.0 * j / rot)
        if scaling == "linear":
            r /= factor
        if scaling == "yarn":
            edge = [rot * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            slow = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            r = r * (1 - slow) + r / factor * slow
            magnitude = 0.1 * math.log(factor) + 1
        got.append(r)
    return np.array(got), magnitude


def turn(x, at, rate, magnitude, weight=None, eps=1e-6, interleaved=False):
    """x [N, H, D] float64, at [N] -> (rotated, length of every element's pair)."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    half = len(rate)
    y, size = x.copy(), np.abs(x)
    if half:
        angle = np.asarray(at, dtype=np.float64)[:, None] * rate
        c, s = magnitude * np.cos(angle)[:, None], magnitude * np.sin(angle)[:, None]
        i = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
        a, b = x[..., i[0]], x[..., i[1]]
        y[..., i[0]], y[..., i[1]] = a * c - b * s, a * s + b * c
        size[..., i[0]] = size[..., i[1]] = abs(magnitude) * np.hypot(a, b)
    return y, size


def turn_tolerance(y, size, dtype):
    """One rounding to `dtype`; before it 32-bit arithmetic: the mean of up to 256 squares in a
    chain of 16 and 4 more sums (20 half steps), its reciprocal root (2 steps), two products, an
    angle off by 2^-25 half turns and sines off by 2 steps, a product and a sum: under 16 steps
    of 2^-23, relative to the pair's length.  A rounding may fall on either side of its tie."""
    return HALF[dtype] * np.abs(y) * (1 + 2.0 ** -7) + 2.0 ** -19 * size + TINY[dtype]


# ------------------------------------------------------------------ attention
def attend_rows(q, at, k, v, scale, window, sink, hkv):
    """q [n, Hq, D] at positions at [n] over k, v [Hkv, L, D], float64 -> (out, sum p |v|)."""
    n, hq, d = q.shape
    g = hq // hkv
    out, size = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i in range(n):
        p = int(at[i])
        if p < 0:
            continue
        t = np.arange(p + 1)
        if window > 0:
            t = t[(t > p - window) | (t < sink)]
        for h in range(hkv):
            s = (q[i, h * g:(h + 1) * g] @ k[h][t].T) * scale
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[i, h * g:(h + 1) * g] = w @ v[h][t]
            size[i, h * g:(h + 1) * g] = w @ np.abs(v[h][t])
    return out, size


def attend_tolerance(size, keys, vmax):
    """fp16 output of fp16 weights: a rounding of each weight (2^-11 of it, or 2^-25 where it is
    that small beside the largest) and one of the sum (2^-11); scores in 32 bits, off by under
    2^-17, and 32-bit sums besides."""
    return (2.0 ** -10 + 2.0 ** -15) * size + keys * 2.0 ** -25 * vmax + 2.0 ** -25


def f64(t):
    return t.detach().cpu().double().numpy()
