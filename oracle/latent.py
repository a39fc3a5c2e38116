"""Latent attention — TEST INFRASTRUCTURE (CPU oracle, float64).

A latent cache row of a token is [c, r]: a latent part and a rotary key part,
shared by every head. Arrays are widened exactly; index work is in Python.
"""
from __future__ import annotations

import numpy as np

from .rope import apply_rope

ROPE = 64


def append(cache, c_kv, k_rope, positions, slots, base):
    """The cache after the append: rows [c, rotated r] at their slots (negative: skipped)."""
    out = np.array(cache, dtype=np.float64)
    rows = out.reshape(-1, out.shape[-1])
    kr = apply_rope(np.asarray(k_rope)[:, None], positions, base)[:, 0]
    for t, s in enumerate(slots):
        if s >= 0:
            rows[s] = np.concatenate([np.asarray(c_kv[t], dtype=np.float64), kr[t]])
    return out


def gather_sequence(cache, table, n):
    """The first n cached rows of a sequence, through its page table."""
    P = cache.shape[1]
    return np.array([cache[table[j // P], j % P] for j in range(n)], dtype=np.float64).reshape(n, cache.shape[-1])


def _softmax_rows(scores, visible):
    x = np.where(visible, scores, -np.inf)
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    total = e.sum(-1, keepdims=True)
    return e / total, (m + np.log(total))[..., 0]


def _visible(n, L):
    return np.arange(L)[None, :] <= (L - n + np.arange(n))[:, None]


def _spread(q, k, w, v, scale):
    """What the error bounds need of each row: sum_j |w_j v_j|, and the largest
    scale * sum_d |q_d k_d| over its keys."""
    return (np.einsum("hnl,hld->nhd", w, np.abs(v)), scale * (np.abs(q) @ np.abs(k).transpose(0, 2, 1)).max(-1).T)


def attend_absorbed(q, rows, scale):
    """q [n, H, ld + 64] over a sequence's rows [L, ld + 64]: out, lse, and the
    spread figures of _spread."""
    q = np.asarray(q, dtype=np.float64).transpose(1, 0, 2)
    k, v = rows[None], rows[None, :, :-ROPE]
    w, lse = _softmax_rows(scale * (q @ k.transpose(0, 2, 1)), _visible(q.shape[1], rows.shape[0]))
    vv = np.broadcast_to(v, (q.shape[0],) + v.shape[1:])
    return (w @ v).transpose(1, 0, 2), lse.T, _spread(q, k, w, vv, scale)


def attend_expanded(q, k_nope, v, k_rope, scale):
    """q [n, H, 192], k_nope and v [L, H, 128], k_rope [L, 64] of one sequence."""
    f = np.float64
    L, H = np.asarray(k_nope).shape[:2]
    k = np.concatenate([np.asarray(k_nope, dtype=f), np.broadcast_to(np.asarray(k_rope, dtype=f)[:, None], (L, H, ROPE))], -1)
    k, vv = k.transpose(1, 0, 2), np.asarray(v, dtype=f).transpose(1, 0, 2)
    q = np.asarray(q, dtype=f).transpose(1, 0, 2)
    w, lse = _softmax_rows(scale * (q @ k.transpose(0, 2, 1)), _visible(q.shape[1], L))
    return (w @ vv).transpose(1, 0, 2), lse.T, _spread(q, k, w, vv, scale)
