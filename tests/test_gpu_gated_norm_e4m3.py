"""GPU tests of the gated RMS norm of the heads' outputs to e4m3 against fp64.

Bounds: the scale by fp32 sums of 128 terms, a root, a sigmoid (exp, sum, reciprocal: 8 units in the last place), products and two
divisions: 1e-5 relative covers them (168 f). y by half an e4m3 step (2^-4 relative, 2^-10 in the subnormal range) after the same."""
import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from oracle import delta as ref

pytestmark = pytest.mark.gpu
D = 128


def make(T, H, seed, fp32=False, size=1.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H, D)) * np.exp(rng.standard_normal((T, H, 1))) * size)
    gate = torch.from_numpy(rng.standard_normal((T, H, D)) * 2).to(torch.bfloat16)
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).float()
    return x.to(torch.float32 if fp32 else torch.bfloat16), gate, w


def check(x, gate, w, eps, silu, y, scale):
    T, H, _ = x.shape
    n = ref.gated_norm(x.double().numpy(), gate.double().numpy(), w.double().numpy(), eps, silu)
    want = np.abs(n).max(-1) / 448
    got = scale.double().cpu().numpy()
    assert got.shape == (T, H) and (np.abs(got - want) <= 1e-5 * want).all()
    val = y.cpu().float().double().numpy().reshape(T, H, D)
    z = n / np.where(got == 0, 1, got)[..., None]
    assert (np.abs(val - z) <= np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10) + 1e-5 * np.abs(z)).all()
    assert np.abs(val).max() <= 448


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (7, 96), (33, 1), (31, 4), (65, 16), (1000, 3)])
def test_rows(T, H, fp32, silu):
    x, g, w = make(T, H, T + H, fp32)
    y, scale = kda.gated_rms_norm(x.cuda(), g.cuda(), w.cuda(), 1e-5, activation="silu" if silu else "sigmoid")
    assert y.dtype is torch.float8_e4m3fn and y.shape == (T, H * D)
    check(x, g, w, 1e-5, silu, y, scale)


def test_gate_is_a_slice_and_another_stream():
    x, g, w = make(20, 3, 4)
    wide = torch.full((20, 5 * D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    gate = wide[:, D:4 * D].view(20, 3, D)
    gate.copy_(g)
    xc, wc, s = x.cuda(), w.cuda(), torch.cuda.Stream()
    torch.cuda.synchronize()
    y, scale = kda.gated_rms_norm(xc, gate, wc, stream=s)
    s.synchronize()
    check(x, g, w, 1e-5, False, y, scale)


@pytest.mark.parametrize("size,eps", [(1e-18, 1e-5), (1e-18, 1e-40), (1e15, 1e-5), (2.0 ** -60, 1e-36)])
def test_sizes(size, eps):
    x, g, w = make(9, 2, 8, fp32=True, size=size)
    y, scale = kda.gated_rms_norm(x.cuda(), g.cuda(), w.cuda(), eps)
    check(x, g, w, eps, False, y, scale)


@pytest.mark.parametrize("size,weight,eps", [(1e17, 1e21, 1e-5), (1e-18, 1e-21, 1e-40), (1e-5, 1e38, 1e-5), (1e-15, 1e25, 1e-5)])
def test_products_out_of_range(size, weight, eps):
    """x * weight overflows or underflows fp32 where n does not; or 448 / n may."""
    x, g, w = make(9, 2, 10, fp32=True, size=size)
    w = w * weight
    y, scale = kda.gated_rms_norm(x.cuda(), g.cuda(), w.cuda(), eps)
    check(x, g, w, eps, False, y, scale)


def test_zero_rows_closed_gates_and_what_is_not_finite():
    x, g, w = make(8, 2, 9)
    x[0, 0] = 0
    g[1, 1] = -200.0              # sigmoid below 2^-100
    x[2, 0, 5] = float("nan")
    x[3, 1, 7] = float("inf")
    g[4, 0, 9] = float("nan")
    g[5, 1] = -1e30               # exp overflows: closed, not NaN
    g[6, 0] = 1e30
    for name, silu in (("sigmoid", False), ("silu", True)):
        y, scale = kda.gated_rms_norm(x.cuda(), g.cuda(), w.cuda(), activation=name)
        y, scale = y.cpu().float().view(8, 2, D), scale.cpu()
        for t, h in ((0, 0), (5, 1)) + (((1, 1),) if not silu else ()):
            assert scale[t, h] == 0 and bool((y[t, h] == 0).all())
        for t, h in ((2, 0), (3, 1), (4, 0)):
            assert bool(torch.isnan(scale[t, h])) and bool(torch.isnan(y[t, h]).all())
        keep = torch.ones(8, 2, dtype=torch.bool)
        for t, h in ((0, 0), (1, 1), (2, 0), (3, 1), (4, 0), (5, 1)):
            keep[t, h] = False
        n = ref.gated_norm(x.double().numpy(), g.double().numpy(), w.double().numpy(), 1e-5, silu)[keep.numpy()]
        got = (y * scale[..., None]).double()[keep].numpy()
        assert (np.abs(got - n) <= 2.0 ** -4 * np.abs(n) * 1.001 + 2.0 ** -10 * np.abs(n).max(-1, keepdims=True) / 448 * 1.001).all()
