"""CPU oracle of the full-attention layer's operators -- TEST INFRASTRUCTURE.

Only ``tests/`` and ``__graft_entry__.smoke()`` may import this module; the
product library never loads it.  Everything is numpy in float64, from the
operators' definitions (include/moe.h):

    rope     y = x * weight / sqrt(mean(x^2) + eps), columns i and i + R / 2 of the
             first R turned by position * inv_freq[i]
    attend   o_i = sum_j softmax_j(scale q_i . k_j) v_j, j <= i + Lk - Lq
    quantise per 64 columns: bias = bf16(min), scale = bf16((max - min) / 15),
             code = round((x - bias) / scale) in 0 .. 15, value = scale * code + bias

mutation plants a mistake for the pin tests: 1 turns the other way, 2 pairs
neighbouring columns, 3 sees one key too many, 4 aligns queries with the first
keys, 5 maps query head h to key head h % H_kv, 6 gives the odd column the low
half of a byte.
"""
from __future__ import annotations

import numpy as np


def norm_rope(x, weight, positions, inv_freq, eps, mutation: int = 0):
    """x [N][H][D] -> (rotated, normed) in float64."""
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    d = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = np.where(d == 0, 0, x / np.where(d == 0, 1, d)) * w
    if inv_freq is None or len(inv_freq) == 0:
        return y, y
    half = len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    s, c = np.sin(a) * (-1 if mutation == 1 else 1), np.cos(a)
    out = y.copy()
    lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if mutation == 2 else (slice(0, half), slice(half, 2 * half))
    out[..., lo] = y[..., lo] * c - y[..., hi] * s
    out[..., hi] = y[..., hi] * c + y[..., lo] * s
    return out, y


def attend(q, k, v, scale, offsets=None, k_offsets=None, mutation: int = 0, late=None):
    """q [N][Hq][D], k, v [M][Hkv][D]: (o, sum_j softmax_j |v_j|, reach), reach
    [N][Hq] the largest sum_d |q_d k_jd| that a query meets; offsets None: one
    sequence.  late: keys further than that ahead are seen, too."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    (N, Hq, D), (M, Hk) = q.shape, k.shape[:2]
    offsets = [0, N] if offsets is None else [int(x) for x in offsets]
    k_offsets = ([0, M] if len(offsets) == 2 else offsets) if k_offsets is None else [int(x) for x in k_offsets]
    o, mag, reach = np.zeros_like(q), np.zeros_like(q), np.zeros((N, Hq))
    for i in range(len(offsets) - 1):
        a, b, c, d = offsets[i], offsets[i + 1], k_offsets[i], k_offsets[i + 1]
        ahead = np.arange(d - c)[None, :] - np.arange(b - a)[:, None]
        shift = 0 if mutation == 4 else (d - c) - (b - a)
        seen = ahead <= shift + (1 if mutation == 3 else 0)
        for h in range(Hq):
            g = h % Hk if mutation == 5 else h // (Hq // Hk)
            if b == a or d == c:
                continue
            x = np.where(seen, (q[a:b, h] @ k[c:d, g].T) * scale, -np.inf)
            top = x.max(1, keepdims=True)
            p = np.exp(x - np.where(np.isfinite(top), top, 0))
            total = p.sum(1, keepdims=True)
            p = p / np.where(total == 0, 1, total)
            o[a:b, h], mag[a:b, h] = p @ v[c:d, g], p @ np.abs(v[c:d, g])
            reach[a:b, h] = np.where(seen, np.abs(q[a:b, h]) @ np.abs(k[c:d, g]).T, 0).max(1)
    return o, mag, reach


def bf16(x):
    """float64 rounded to the nearest bfloat16, ties to even (finite values in
    range)."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e, -125) - 8)
    return np.round(x / step) * step


def quantise(x):
    """x [..., D]: (codes [..., D] uint8, scale, bias [..., D / 64])"""
    g = np.asarray(x, np.float64)
    g = g.reshape(*g.shape[:-1], g.shape[-1] // 64, 64)
    bias = bf16(g.min(-1))
    scale = bf16((g.max(-1) - g.min(-1)) / 15)
    s = np.where(scale == 0, 1, scale)[..., None]
    c = np.where(scale[..., None] == 0, 0, np.clip(np.round((g - bias[..., None]) / s), 0, 15))
    return c.reshape(*x.shape).astype(np.uint8), scale, bias


def values(codes, scale, bias):
    """float64 values of codes [..., D] with scale, bias [..., D / 64]"""
    g = np.asarray(codes, np.float64).reshape(*scale.shape, 64)
    return (np.asarray(scale)[..., None] * g + np.asarray(bias)[..., None]).reshape(codes.shape)


def unpack(codes, mutation: int = 0):
    """codes [..., D / 2] bytes -> [..., D], the even column in the low half"""
    c = np.asarray(codes, np.uint8)
    pair = (c >> 4, c & 15) if mutation == 6 else (c & 15, c >> 4)
    return np.stack(pair, -1).reshape(*c.shape[:-1], 2 * c.shape[-1])
