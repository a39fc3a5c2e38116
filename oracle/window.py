"""Layers with a window — TEST INFRASTRUCTURE (CPU oracle, float64).

Norm and rotation of heads, attention through a sliding window with sinks, and the
stretched angles of the rotation. Arrays are widened exactly.
"""
from __future__ import annotations

import math

import numpy as np


def norm(x, weight, eps):
    """Heads [..., D] over their root mean square, times a weight a channel (None: as they are)."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(x, cs, interleaved):
    """x [T, H, D], cs [T, r / 2, 2]: the pairs of the first r values turned, and the
    largest |a cos| + |b sin| that each result is the difference or sum of."""
    y, size = np.array(x, dtype=np.float64), np.abs(np.asarray(x, dtype=np.float64))
    cs = np.asarray(cs, dtype=np.float64)[:, None]
    half = cs.shape[2]
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b, c, s = x[..., ia], x[..., ib], cs[..., i, 0], cs[..., i, 1]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia], size[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, size


def visible(n, L, window, sinks):
    """[n, L]: which keys the last n rows of a sequence of L keys see."""
    p = (L - n + np.arange(n))[:, None]
    j = np.arange(L)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def attend(q, k, v, scale, window, sinks):
    """q [n, Hq, D] over a sequence's keys and values [L, Hkv, D]: out, lse, and for the
    error bounds sum_j |w_j v_j| and the largest scale * sum_d |q_d k_d| of each row.
    What no row sees is not read."""
    q = np.asarray(q, dtype=np.float64)
    n, Hq, _ = q.shape
    L, Hkv, _ = k.shape
    seen = visible(n, L, window, sinks)
    used = np.flatnonzero(seen.any(0))
    seen = seen[:, used]
    group = np.arange(Hq) // (Hq // Hkv)
    kk = np.asarray(k[used], dtype=np.float64)[:, group].transpose(1, 0, 2)
    vv = np.asarray(v[used], dtype=np.float64)[:, group].transpose(1, 0, 2)
    qq = q.transpose(1, 0, 2)
    x = np.where(seen, scale * (qq @ kk.transpose(0, 2, 1)), -np.inf)
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    total = e.sum(-1, keepdims=True)
    w = e / total
    dot = np.where(seen, scale * (np.abs(qq) @ np.abs(kk).transpose(0, 2, 1)), 0.0).max(-1)
    return ((w @ vv).transpose(1, 0, 2), (m + np.log(total))[..., 0].T, (w @ np.abs(vv)).transpose(1, 0, 2), dot.T)


def angles(base, r, kind, factor, low, high, original, attention):
    """Angle of each pair at position 1 and the factor on cos and sin, pair by pair from
    the definitions."""
    out = []
    for i in range(r // 2):
        f = base ** (-2.0 * i / r)
        if kind == "linear":
            f = f / factor
        elif kind == "base":
            f = (base * factor ** (r / (r - 2))) ** (-2.0 * i / r)
        elif kind == "bands":
            wave = 2 * math.pi / f
            if wave > original / low:
                f = f / factor
            elif wave >= original / high:
                s = (original / wave - low) / (high - low)
                f = (1 - s) * f / factor + s * f
        elif kind == "ramp":
            c = lambda n: r * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))
            first, last = max(math.floor(c(high)), 0), min(math.ceil(c(low)), r - 1)
            share = min(max((i - first) / ((last - first) if last > first else 0.001), 0.0), 1.0)
            f = f * (1 - share) + f / factor * share
        out.append(f)
    if attention == 0.0:
        attention = 0.1 * math.log(factor) + 1.0 if kind == "ramp" else 1.0
    return np.array(out), attention
