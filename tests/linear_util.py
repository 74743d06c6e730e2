"""Inputs that the linear-attention tests share."""
import numpy as np
import torch

D = 128


def linear_inputs(lens, H, Hk, seed):
    rng = np.random.default_rng(seed)
    T = sum(lens)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    q, k = (torch.from_numpy(unit(rng.standard_normal((T, Hk, D)))).to(torch.bfloat16) for _ in range(2))
    v = torch.from_numpy(rng.standard_normal((T, H, D))).to(torch.bfloat16)
    g = torch.from_numpy(-np.log1p(np.exp(rng.standard_normal((T, H)))) * np.exp(-4 * rng.random(H))).float()
    return {"q": q, "k": k, "v": v, "g": g}
