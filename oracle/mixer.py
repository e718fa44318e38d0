"""CPU oracle of the mixer's operators -- TEST INFRASTRUCTURE.

Only ``tests/`` and ``__graft_entry__.smoke()`` may import this module; the
product library never loads it.  Everything is numpy in float64, from the
operators' definitions (include/moe.h, include/gdn.h):

    norm    s = x + residual,  y = s * weight / sqrt(mean(s^2) + eps)
            scale = max|y| / 448,  code = the e4m3 value nearest to y / scale
    matmul  out[t][n] = xs[t] * ws[n] * sum_k x[t][k] * w[n][k]
    scan    S <- decay S + v_t k_t^T,  o_t = S q_t   per value head

mutation plants a mistake for the pin tests: 1 divides by max|s| instead of
the root mean square, 2 drops the residual, 3 swaps the two scales' roles, 4
reads the output before the write, 5 decays the new token too, 6 maps value
head h to key head h % H_k, 7 decays once per sequence instead of per token.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def e4m3_values() -> np.ndarray:
    """float64 value of each of the 256 codes: 1 sign, 4 exponent (bias 7) and 3
    mantissa bits, no infinities, 0x7f and 0xff NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    mag[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -mag, mag)


def rmsnorm(x, weight, eps, residual=None, mutation: int = 0):
    """(y, s) in float64 for rows x [rows][d]."""
    s = np.asarray(x, np.float64)
    if residual is not None and mutation != 2:
        s = s + np.asarray(residual, np.float64)
    ms = np.abs(s).max(1, keepdims=True) ** 2 if mutation == 1 else (s * s).mean(1, keepdims=True)
    return s / np.sqrt(ms + eps) * np.asarray(weight, np.float64), s


def matmul(x, xs, w, ws, mutation: int = 0):
    """xs[t] ws[n] sum_k x[t][k] w[n][k] of code values x [T][K], w [N][K]."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    xs, ws = np.asarray(xs, np.float64), np.asarray(ws, np.float64)
    if mutation == 3:
        return (x @ w.T) * xs[None, :] * ws[:, None]  # (meaningful only when T == N)
    return (x @ w.T) * xs[:, None] * ws[None, :]


def decay_scan(q, k, v, decay, state=None, offsets=None, mutation: int = 0):
    """q, k [N][H_k][d_k], v [N][H_v][d_v], offsets [n + 1] (None: one
    sequence): (o [N][H_v][d_v], states [n][H_v][d_v][d_k])."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    lam = np.asarray(decay, np.float64)[:, None, None]
    N, Hk, dk = k.shape
    Hv, dv = v.shape[1:]
    offsets = [0, N] if offsets is None else [int(x) for x in offsets]
    n = len(offsets) - 1
    heads = np.arange(Hv) % Hk if mutation == 6 else np.arange(Hv) // (Hv // Hk)
    S = np.zeros((n, Hv, dv, dk)) if state is None else np.array(state, np.float64)
    o = np.zeros((N, Hv, dv))
    for i in range(n):
        for t in range(offsets[i], offsets[i + 1]):
            new = v[t][:, :, None] * k[t][heads][:, None, :]
            if mutation == 4:
                o[t] = np.einsum("hji,hi->hj", S[i], q[t][heads])
            if mutation == 5:
                S[i] = lam * (S[i] + new)
            elif mutation == 7:
                S[i] = (lam if t == offsets[i] else 1.0) * S[i] + new
            else:
                S[i] = lam * S[i] + new
            if mutation != 4:
                o[t] = np.einsum("hji,hi->hj", S[i], q[t][heads])
    return o, S
