"""fp64 oracle of the cached-history operators: per-head norm and rotation with its backward pass, the e4m3
rows of the cache, and attention over a cached history. Plain numpy, one sequence and head at a time; test
infrastructure only."""
from __future__ import annotations

import math

import numpy as np

HALVES, ADJACENT = 0, 1
E_LO, E_HI = -100, 119


def pair_columns(rotary_dim: int, layout: int):
    """(first, second) column of every pair."""
    i = np.arange(rotary_dim // 2)
    return (i, i + rotary_dim // 2) if layout == HALVES else (2 * i, 2 * i + 1)


def _turn(n, positions, rotary_dim, base, layout, sign):
    out = np.array(n, dtype=np.float64)
    if rotary_dim == 0:
        return out
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    t = np.asarray(positions, np.float64)[:, None, None] * base ** (-2.0 * i / rotary_dim)
    u, v = pair_columns(rotary_dim, layout)
    c, s = np.cos(t), sign * np.sin(t)
    out[..., u] = n[..., u] * c - n[..., v] * s
    out[..., v] = n[..., u] * s + n[..., v] * c
    return out


def norm_rotate(x, gain, positions, rotary_dim, base, layout, eps):
    """x [rows, heads, d_head] -> the normalised and rotated rows."""
    x = np.asarray(x, np.float64)
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    return _turn(n, positions, rotary_dim, base, layout, 1.0)


def norm_rotate_backward(x, gain, positions, rotary_dim, base, layout, eps, dy):
    """(dx, d_gain) for the upstream gradient dy."""
    x, g = np.asarray(x, np.float64), np.asarray(gain, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    dn = _turn(np.asarray(dy, np.float64), positions, rotary_dim, base, layout, -1.0)
    dx = r * dn * g - x * r ** 3 * np.mean(dn * g * x, -1, keepdims=True)
    return dx, np.sum(dn * x * r, axis=(0, 1))


def e4m3_round(v):
    """Numbers of magnitude at most 448 rounded to e4m3 (4 significant bits down to 2^-6, steps of 2^-9 below),
    ties to even."""
    v = np.asarray(v, np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.round(v / step) * step


def quantise(x):
    """Rows x [..., d_head] -> (e4m3 numbers, exponents): x ~ number * 2^exponent."""
    x = np.asarray(x, np.float64)
    amax = np.abs(x).max(-1)
    e = np.zeros(amax.shape, np.int64)
    for i in np.ndindex(amax.shape):
        if amax[i] > 0:
            k = math.floor(math.log2(amax[i])) - 9
            while amax[i] > 448.0 * 2.0 ** k:
                k += 1
            e[i] = min(max(k, E_LO), E_HI)
    return e4m3_round(np.clip(x / 2.0 ** e[..., None], -448.0, 448.0)), e


def attention(q, k, v, causal, first_position):
    """q [n, heads, d_head] against k, v [length, kv_heads, d_head]: (a, sum_j p_j |v_j|), zeros where a row sees
    nothing. Row i is at position first_position + i (causal)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, heads, dh = q.shape
    group = heads // k.shape[1]
    a, mag = np.zeros_like(q), np.zeros_like(q)
    for i in range(n):
        end = min(len(k), first_position + i + 1) if causal else len(k)
        if end <= 0:
            continue
        for h in range(heads):
            s = k[:end, h // group] @ q[i, h] / math.sqrt(dh)
            p = np.exp(s - s.max())
            p /= p.sum()
            a[i, h] = p @ v[:end, h // group]
            mag[i, h] = p @ np.abs(v[:end, h // group])
    return a, mag
