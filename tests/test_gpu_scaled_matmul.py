"""GPU tests of the e4m3 product with scales against fp64.

Bound: y is rounded once (2^-8 of it). With A the same sum over magnitudes and f = 2^-24: a block's 128 products are exact and added in
fp32, truncating (2 f) at most 128 times over four instructions, its scale is one rounding, and so is each block's addition:
(256 + blocks + 8) f A.
"""
import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from oracle import delta as ref

pytestmark = pytest.mark.gpu
F = 2.0 ** -24


def make(T, N, K, per_block, seed):
    rng = np.random.default_rng(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    x = torch.from_numpy(rng.standard_normal((T, K)) * 60).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    w = torch.from_numpy(rng.standard_normal((N, K)) * 60).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    xs = torch.from_numpy(np.exp(rng.standard_normal((T, kb) if per_block else T)) * 0.01).float()
    ws = torch.from_numpy(np.exp(rng.standard_normal((nb, kb))) * 1e-3).float()
    return x, xs, w, ws


def check(x, xs, w, ws, y):
    want, size = ref.scaled_matmul(x.float(), xs, w.float(), ws)
    got = y.double().cpu().numpy().reshape(want.shape)
    tol = 2.0 ** -8 * 1.001 * np.abs(want) + (264 + ws.shape[1]) * F * size + 1e-38
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{np.max(err / tol):.3g} of the bound"


@pytest.mark.parametrize("per_block", [False, True])
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 128, 128), (2, 129, 144), (3, 7, 4096), (16, 256, 256), (17, 300, 272),
                                   (32, 96, 2048), (33, 1000, 400), (64, 128, 1024), (64, 4100, 128), (65, 128, 128),
                                   (100, 200, 384), (128, 640, 2048), (129, 136, 2064), (200, 33, 512), (257, 257, 640),
                                   (300, 6176, 256), (1000, 1031, 272), (1024, 2048, 512), (2100, 300, 128), (2500, 2304, 1152)])
def test_products(T, N, K, per_block):
    x, xs, w, ws = make(T, N, K, per_block, T + N + K)
    y = kda.scaled_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), check=True)
    assert y.dtype is torch.bfloat16 and y.shape == (T, N)
    check(x, xs, w, ws, y)


def test_leading_dimensions_stream_and_no_rows():
    x, xs, w, ws = make(24, 256, 384, True, 5)
    d = [t.cuda() for t in (x.view(2, 3, 4, 384), xs.view(2, 3, 4, 3), w, ws)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = kda.scaled_matmul(*d, stream=s, check=True)
    assert y.shape == (2, 3, 4, 256)
    check(x, xs, w, ws, y)
    assert kda.scaled_matmul(d[0][:0], d[1][:0], d[2], d[3]).shape == (0, 3, 4, 256)


@pytest.mark.parametrize("T", [5, 90, 700])
def test_what_is_not_finite_stays_in_its_row(T):
    x, xs, w, ws = make(T, 200, 256, False, 6)
    clean = kda.scaled_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda()).cpu()
    x[1, 130] = float("nan")
    xs[3] = float("nan")
    y = kda.scaled_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda()).cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    rest = [t for t in range(T) if t not in (1, 3)]
    assert torch.equal(y[rest], clean[rest])


def test_rows_behind_y_stay_as_they_were():
    """y is a part of a larger buffer: nothing is written around it."""
    for T, N in ((5, 130), (70, 136), (70, 131), (300, 264)):
        x, xs, w, ws = make(T, N, 256, True, 7)
        buf = torch.full((T + 200, N), 7.0, dtype=torch.bfloat16, device="cuda")
        y = buf[:T]
        kda.kda_scaled_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), y)
        check(x, xs, w, ws, y)
        assert bool((buf[T:] == 7.0).all())


def test_replayed_in_a_graph():
    x, xs, w, ws = make(40, 2048, 2048, False, 8)
    d = [t.cuda() for t in (x, xs, w, ws)]
    first = kda.scaled_matmul(*d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = kda.scaled_matmul(*d)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first)
    check(x, xs, w, ws, first)


def test_two_at_once():
    """Wide, narrow and clustered tiles beside one another on two streams: each holds tensor memory of the SMs that it shares."""
    cases = [make(2500, 2304, 640, True, 11), make(40, 2048, 2048, False, 12), make(300, 640, 640, True, 13)]
    d = [[t.cuda() for t in c] for c in cases]
    want = [kda.scaled_matmul(*c, check=True) for c in d]
    streams = [torch.cuda.Stream() for _ in d]
    torch.cuda.synchronize()
    got = [[kda.scaled_matmul(*d[(i + j) % 3], stream=s) for i in range(6)] for j, s in enumerate(streams)]
    torch.cuda.synchronize()
    for j in range(3):
        for i in range(6):
            assert torch.equal(got[j][i], want[(i + j) % 3])
