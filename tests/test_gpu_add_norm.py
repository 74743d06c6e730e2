"""GPU tests of the residual addition + RMS norm + e4m3 output against fp64.

Bounds: the residual is off by half a bf16 step (2^-8 relative) and the fp32 addition (2^-24 of each term); the scale by fp32
sums (a relative 1e-5 covers 32768 terms in a tree, a root, two divisions); y by half an e4m3 step (2^-4 relative, 2^-10 in the
subnormal range) after a relative fp32 error of 1e-5."""
import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from oracle import linear as ref

pytestmark = pytest.mark.gpu


def make(T, d, seed, fp32=False):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, d)) * np.exp(rng.standard_normal((T, 1)))).to(torch.bfloat16)
    r = torch.from_numpy(rng.standard_normal((T, d)) * 3).to(torch.float32 if fp32 else torch.bfloat16)
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(d)).float()
    return x, r, w


def check(x, r, w, eps, y, scale, res):
    h, n = ref.add_rms_norm(x.double().numpy(), r.double().numpy(), w.double().numpy(), eps)
    ulp = 2.0 ** -24 if r.dtype == torch.float32 else 2.0 ** -8 * 1.001
    size = np.abs(x.double().numpy()) + np.abs(r.double().numpy())
    assert (np.abs(res.double().cpu().numpy() - h) <= ulp * np.abs(h) + 2.0 ** -24 * size).all()
    want = np.abs(n).max(-1) / 448
    got = scale.double().cpu().numpy()
    assert (np.abs(got - want) <= 1e-5 * want).all()
    val = y.cpu().float().double().numpy()
    z = n / got[:, None]
    tol = np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10) + 1e-5 * (np.abs(z) + size / np.maximum(np.abs(h), 1e-30) * np.abs(z) * 0.01)
    assert (np.abs(val - z) <= tol).all()
    assert np.abs(val).max() <= 448


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (2, 8), (5, 9), (4, 64), (3, 256), (7, 257), (9, 1000), (33, 1024), (3, 1031),
                                 (5, 2048), (2, 2049), (3, 4096), (2, 4097), (2, 8192), (3, 8193), (7, 12288), (2, 12755),
                                 (2, 16384), (2, 16385), (1, 32768), (2, 32767)])
def test_rows(T, d, fp32):
    x, r, w = make(T, d, T + d, fp32)
    y, scale, res = kda.add_rms_norm(x.cuda(), r.cuda(), w.cuda(), 1e-5)
    assert res.dtype == r.dtype
    check(x, r, w, 1e-5, y, scale, res)


def test_shapes_in_place_and_streams():
    x, r, w = make(24, 384, 5)
    xc, wc = x.view(2, 3, 4, 384).cuda(), w.cuda()
    rc = r.view(2, 3, 4, 384).cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, scale, res = kda.add_rms_norm(xc, rc, wc, in_place=True, stream=s)
    s.synchronize()
    assert res is rc and y.shape == xc.shape and scale.shape == (2, 3, 4)
    check(x, r, w, 1e-6, y.view(24, 384), scale.view(-1), res.view(24, 384))


def test_no_rows():
    y, scale, res = kda.add_rms_norm(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                                     torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda"))
    assert y.shape == (0, 64) and scale.shape == (0,)


def test_neighbours_of_an_odd_row_stay():
    """Rows of 13 elements share groups of 8: each writes its own elements only."""
    x, r, w = make(65, 13, 6)
    whole = kda.add_rms_norm(x.cuda(), r.cuda(), w.cuda())
    y = torch.full((66, 13), 1.5, device="cuda").to(torch.float8_e4m3fn)
    res = torch.full((66, 13), 7.0, dtype=torch.bfloat16, device="cuda")
    scale = torch.full((66,), 5.0, device="cuda")
    kda.kda_add_rms_norm(x.cuda(), r.cuda(), w.cuda(), 1e-6, res[:65], y[:65], scale[:65])
    assert torch.equal(y[:65].float(), whole[0].float()) and torch.equal(scale[:65], whole[1]) and torch.equal(res[:65], whole[2])
    assert bool((y[65].float() == 1.5).all()) and bool((res[65] == 7).all()) and float(scale[65]) == 5


@pytest.mark.parametrize("size", [2.0 ** -119, 1.2 * 2.0 ** -120, 2.0 ** -126])
@pytest.mark.parametrize("d", [64, 1031])
def test_small_rows_with_a_small_eps(d, size):
    """n = h / sqrt(eps) * w is of ordinary size where the factor that takes h * w to the codes, 448 / max|h w|, overflows."""
    x, r, w = make(3, d, 7, fp32=True)
    x = torch.zeros_like(x)
    r[:, ::5] = 0
    r = r / r.abs().amax(1, keepdim=True) * size
    w = torch.ones_like(w)
    y, scale, res = kda.add_rms_norm(x.cuda(), r.cuda(), w.cuda(), 1e-16)
    assert bool((scale > 2.0 ** -109).all())
    check(x, r, w, float(np.float32(1e-16)), y, scale, res)


@pytest.mark.parametrize("d", [64, 1031, 4096])
def test_zero_tiny_and_no_number_rows(d):
    x = torch.zeros(6, d, dtype=torch.bfloat16)
    r = torch.zeros(6, d, dtype=torch.bfloat16)
    x[1, 3], x[2, d - 1], x[3, 5] = float("nan"), float("inf"), 1e30
    x[4], r[4] = 2.0, -2.0
    x[5] = 1.0
    y, scale, res = (t.cpu().float() for t in kda.add_rms_norm(x.cuda(), r.cuda(), torch.ones(d, device="cuda"), 1e-6))
    assert float(scale[0]) == 0 and bool((y[0] == 0).all()) and float(scale[4]) == 0 and bool((y[4] == 0).all())
    assert bool(scale[1:4].isnan().all()) and bool(y[1:4].isnan().all())
    assert bool((y[5] == 448).all())
