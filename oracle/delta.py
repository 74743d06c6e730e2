"""Delta rule with one decay per head, the gated norm to e4m3 and the scaled product — TEST INFRASTRUCTURE ONLY.

Plain fp64 restatements, written from the formulas in ``include/kda.h``. The recurrence also returns how far a result may be
off, from the roundings of the form that computes it:

A token's map of the state, S -> e^g (I - beta k k^T) S + beta k v^T, makes no difference between two states longer (2-norm, by
value columns) as long as g <= 0 and 0 <= beta |k|^2 <= 2. So what a token's arithmetic is off by, E_t, is in the final state at
most E_t times the decays after it, and errors add up: e_t = e^g_t e_{t-1} + |E_t|. With s = |S| before the token (a column's
length) and f = 2^-24:

  recurrence, fp32   the products of 128 terms are off by at most 130 f |k| s, the decay by 4 f, each of the update's two roundings
                     by f of its terms: |E| <= f (8 s + 150 beta |k|^2 s + 8 beta |k| |v|).
  chunks             operands of the tensor cores are two bf16 terms: off by at most w = 2^-16 of themselves. In a chunk, z_t = v_t -
                     e^G_t S^T k_t of its entry state (|z| <= |v| + |k| s) and x = T z with |T_ts| <= beta_t beta_s |k_t| |k_s| (s < t),
                     |T_tt| = beta_t: the response of x_t to v_s. The entry state, z, T (and the product of the second terms, left
                     out) are off by w each, x by w again, and fp32 sums of 128 terms twice by 130 f, together taken as 2^-15:
                     |E_t| <= |k_t| 2^-15 (|x_t| + beta_t (|k| s + 4 |z_t| + 4 |k_t| sum_{s<t} beta_s |k_s| |z_s|)) + 8 f s.

The output adds its own products (the same counts). In chunks it has two: q_t with the entry state, in two bf16 terms (w of it, |q_t| w s),
and P T with z, in two terms too (w). P T, the response of o_t to z_s, at most |q_t| beta_s |k_s|, is the one operand that is rounded once to
bf16 (2^-8); before that P's and T's terms and the product of their second ones, left out, are w each (T's own error is in x's, and so in E).
Sums of 128 to 256 terms in fp32, truncated, are 2^-15. Together 2^-8 and at most 8 w of the response, here 1.02 x 2^-8 + 4 w (9 w), and 3
w of the entry state's part, here 4 w: w = 2^-16, 4 w = 2^-14.
"""
from __future__ import annotations

import numpy as np

from .gates import sigmoid

F = 2.0 ** -24


def recurrence(q, k, v, g, beta, lens, state, scale, chunk=0):
    """q, k [T, Hk, K], v [T, H, V], g, beta [T, H], lens: tokens of each sequence, state [N, H, K, V] or None; chunk: tokens of
    a chunk, 0 for the recurrence. Returns o [T, H, V], what it may be off before its own rounding, the final states and what a
    column of them may be off (its length) [N, H, V]. T may exceed sum(lens)."""
    q, k, v, g, beta = (np.asarray(x, dtype=np.float64) for x in (q, k, v, g, beta))
    T, H, V = v.shape
    K, rep, N = q.shape[2], H // q.shape[1], len(lens)
    q, k = np.repeat(q, rep, axis=1), np.repeat(k, rep, axis=1)
    d = np.exp(g)
    o, off = np.zeros((T, H, V)), np.zeros((T, H, V))
    S = np.zeros((N, H, K, V)) if state is None else np.array(state, dtype=np.float64)
    E = np.zeros((N, H, V))
    qn, kn = np.linalg.norm(q, axis=2), np.linalg.norm(k, axis=2)
    t = 0
    for n, length in enumerate(lens):
        entry, resp = np.linalg.norm(S[n], axis=1), np.zeros((H, V))
        for i in range(length):
            s = np.linalg.norm(S[n], axis=1)
            b, kk, qq = np.abs(beta[t])[:, None], kn[t][:, None], qn[t][:, None]
            if chunk and i % chunk == 0:
                entry, resp = s, np.zeros((H, V))
            S[n] *= d[t][:, None, None]
            x = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S[n], k[t]))
            S[n] += k[t][:, :, None] * x[:, None, :]
            o[t] = scale * np.einsum("hkv,hk->hv", S[n], q[t])
            if chunk:
                z = np.abs(v[t]) + kk * entry
                local = kk * 2.0 ** -15 * (np.abs(x) + b * (kk * entry + 4 * z + 4 * kk * resp)) + 8 * F * s
                resp = resp + b * kk * z
                more = (2.0 ** -8 * 1.02) * resp + 2.0 ** -14 * (entry + resp)
            else:
                local = F * (8 * s + 150 * b * kk * kk * s + 8 * b * kk * np.abs(v[t]))
                more = 160 * F * (s + kk * np.abs(x))
            E[n] = d[t][:, None] * E[n] + local
            off[t] = abs(scale) * qq * (2 * E[n] + more)
            t += 1
    return o, off, S, E


def gated_norm(x, gate, weight, eps, silu):
    """n = x / sqrt(mean(x^2) + eps) * weight * act(gate) over the last axis."""
    x, gate = np.asarray(x, dtype=np.float64), np.asarray(gate, dtype=np.float64)
    act = sigmoid(gate) * (gate if silu else 1.0)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64) * act


def scaled_matmul(x, x_scale, w, w_scale):
    """y [T, N] and the same sums over magnitudes; x [T, K], x_scale [T] or [T, KB], w [N, K], w_scale [NB, KB]."""
    x, w, xs, ws = (np.asarray(a, dtype=np.float64) for a in (x, w, x_scale, w_scale))
    K = x.shape[1]
    ws = np.repeat(np.repeat(ws, 128, 0)[:w.shape[0]], 128, 1)[:, :K]
    xs = xs[:, None] if xs.ndim == 1 else np.repeat(xs, 128, 1)[:, :K]
    a, b = x * xs, w * ws
    return a @ b.T, np.abs(a) @ np.abs(b).T
