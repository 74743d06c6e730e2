"""Linear attention with one decay per head, the state cache and the add-norm — TEST INFRASTRUCTURE ONLY.

Plain fp64 restatements, written from the formulas in ``include/kda.h``: the
token recurrence, the per-row int8 rounding and the residual/RMS-norm row. Each
recurrence also returns the size of its terms (the same sums over magnitudes),
which the tests' error bounds are made of.
"""
from __future__ import annotations

import numpy as np


def recurrence(q, k, v, g, lens, state, scale):
    """q, k [T, Hk, K], v [T, H, V], g [T, H] or [H], lens: tokens of each sequence, state [N, H, K, V] or None.
    Returns o [T, H, V], its terms' size, the final states and their terms' size (T may exceed sum(lens))."""
    q, k, v, g = (np.asarray(x, dtype=np.float64) for x in (q, k, v, g))
    T, H, V = v.shape
    K, rep, N = q.shape[2], H // q.shape[1], len(lens)
    q, k = np.repeat(q, rep, axis=1), np.repeat(k, rep, axis=1)
    d = np.exp(np.broadcast_to(g, (T, H)))
    o, size = np.zeros((T, H, V)), np.zeros((T, H, V))
    S = np.zeros((N, H, K, V)) if state is None else np.array(state, dtype=np.float64)
    A = np.abs(S)
    t = 0
    for n, length in enumerate(lens):
        for t in range(t, t + length):
            S[n] = d[t][:, None, None] * S[n] + k[t][:, :, None] * v[t][:, None, :]
            A[n] = d[t][:, None, None] * A[n] + np.abs(k[t][:, :, None] * v[t][:, None, :])
            o[t] = scale * np.einsum("hkv,hk->hv", S[n], q[t])
            size[t] = abs(scale) * np.einsum("hkv,hk->hv", A[n], np.abs(q[t]))
        t = t + 1 if length else t
    return o, size, S, A


def quantise_rows(state):
    """Codes (float64 integers) and scales of fp32 states [..., K, V], one scale per row of V."""
    x = np.asarray(state, dtype=np.float32)
    amax = np.abs(x).max(-1, keepdims=True)
    inv = np.where(amax > 0, np.float32(127) / np.where(amax > 0, amax, 1), np.float32(0)).astype(np.float32)
    return np.rint((x * inv).astype(np.float32)).astype(np.float64), (amax / np.float32(127))[..., 0].astype(np.float64)


def add_rms_norm(x, residual, weight, eps):
    """h = x + residual and n = h / sqrt(mean(h^2) + eps) * weight, by rows."""
    h = np.asarray(x, dtype=np.float64) + np.asarray(residual, dtype=np.float64)
    return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
