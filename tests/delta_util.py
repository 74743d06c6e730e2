"""The delta rule in chunks with the roundings of a kernel on bf16 tensor cores, on the host: what a bound on its outputs has to let through, and
what it has to reject. (Sums in 64 bits; operands in one or two bf16 terms.)"""
import numpy as np
import torch

U = 2.0 ** -8  # half a step of bf16, at most, of the value


def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).float().to(torch.bfloat16).double().numpy()


def terms(x, n):
    """x in n bf16 terms."""
    hi = bf16(x)
    return hi if n == 1 else hi + bf16(x - hi)


def one_head(q, k, v, g, beta, s0, scale, q_state=2, z_out=2, chunk=64):
    """One head of one sequence: o, rounded to bf16, the final state, and the 2-norm that o's rounded operands say its error has: each
    product's term is off by a rounding of its own, U / 2.3 of it on average over values. q_state, z_out: terms of the state that q multiplies,
    of the z that P T multiplies."""
    S, o, var = np.array(s0, dtype=np.float64), np.zeros(v.shape), np.zeros(v.shape)
    for a in range(0, len(q), chunk):
        Q, K, V, G, b = q[a:a + chunk], k[a:a + chunk], v[a:a + chunk], np.cumsum(g[a:a + chunk]), beta[a:a + chunk]
        low = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0)))
        T = np.linalg.inv(np.eye(len(G)) + np.tril(b[:, None] * (K @ K.T) * low, -1)) * b[None]
        PT = (scale * (Q @ K.T) * low) @ T
        d = np.exp(G)[:, None]
        z = V - d * (K @ terms(S, 2))
        x = terms(T, 2) @ terms(z, 2)
        out = scale * d * (Q @ terms(S, q_state)) + bf16(PT) @ terms(z, z_out)
        o[a:a + chunk] = bf16(out)
        var[a:a + chunk] = out ** 2 + PT ** 2 @ z ** 2
        S = np.exp(G[-1]) * S + K.T @ terms(np.exp(G[-1] - G)[:, None] * x, 2)
    return o, S, U / 2.3 * np.sqrt(var.sum())


def sharp_cases():
    """Inputs for which one more rounding of an operand shows: the output is the decayed state alone (nothing is written); a chunk of one token
    that reads what it wrote; tokens that do so each by itself (orthogonal keys); and all of it in an ordinary prompt."""
    D, H = 128, 2
    rng = np.random.default_rng(12)
    unit = lambda x: bf16(x / np.linalg.norm(x, axis=-1, keepdims=True))
    make = lambda T: dict(q=unit(rng.standard_normal((T, H, D))), k=unit(rng.standard_normal((T, H, D))), v=bf16(rng.standard_normal((T, H, D))),
                          g=np.float32(-0.02 * rng.random((T, H))).astype(np.float64), beta=np.float32(rng.random((T, H))).astype(np.float64))
    state = make(192)
    state["beta"][:] = 0
    single = make(64)
    single["q"] = single["k"]
    own = make(128)
    own["k"][:] = own["q"][:] = np.eye(D)[rng.permutation(D)][:, None]
    ordinary = make(300)
    s0 = lambda n, size: np.float32(rng.standard_normal((n, H, D, D)) * size).astype(np.float64)
    return {"state": (state, [128, 64], s0(2, 1.0)), "single": (single, [1] * 64, s0(64, 0.02)), "own": (own, [64, 64], s0(2, 0.02)),
            "ordinary": (ordinary, [200, 100], s0(2, 0.3))}


def emulate(x, lens, s0, scale, **kw):
    o, S, var, a = np.zeros(x["v"].shape), np.zeros(s0.shape), 0.0, 0
    for n, c in enumerate(lens):
        for h in range(o.shape[1]):
            o[a:a + c, h], S[n, h], e = one_head(*(x[i][a:a + c, h] for i in ("q", "k", "v", "g", "beta")), s0[n, h], scale, **kw)
            var += e ** 2
        a += c
    return o, S, np.sqrt(var)
