"""GPU tests of the e4m3 product's pairs of CTAs (256 x 256 tiles) where tiles end beyond the operands, against fp64.

Every size here is one for which the tile rule takes pairs on 152 SMs. Bound as for the other tiles: y is rounded once (2^-8 of it); with A
the same sum over magnitudes and f = 2^-24, products are exact, sums of 128 in fp32 truncate (2 f) at most 128 times, a block's scale is one rounding
and so is its addition: (256 + blocks + 8) f A.
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
    x, w = (torch.from_numpy(rng.standard_normal((n, K)) * 60).float().clamp(-448, 448).to(torch.float8_e4m3fn) for n in (T, N))
    xs = torch.from_numpy(np.exp(rng.standard_normal((T, kb) if per_block else T)) * 0.01).float()
    # (neighbouring groups of outputs far apart: a scale of the wrong group shows)
    ws = torch.from_numpy(np.exp(rng.standard_normal((nb, kb))) * 1e-3 * np.where(np.arange(nb) % 2, 16.0, 1.0)[:, None]).float()
    return x, xs, w, ws


@pytest.mark.parametrize("per_block", [False, True])
@pytest.mark.parametrize("T,N,K", [
    (2404, 2057, 1168),  # 9 columns in the last tile: its second group of outputs is none; odd outputs; 100 rows for the last pair: one CTA's
    (2300, 2056, 1136),  # the same columns by tiled stores; the last block of channels 112 wide
    (2404, 2312, 1168),  # 8 columns in the last tile, in the first half's first CTA
    (2350, 2431, 272),   # 127 columns in it: to the end of a half's part but one
    (4500, 1161, 144),   # 137: one group and 9 columns of the next; 148 rows for the last pair; a block of 16 channels
    (2310, 2177, 400),   # 129; 6 rows for the last pair
    (4500, 1176, 128),   # 152, tiled; one block
])
def test_ragged_tiles_of_pairs(T, N, K, per_block):
    x, xs, w, ws = make(T, N, K, per_block, T + N + K)
    buf = torch.full((T + 300, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y, status = buf[:T], torch.ones(1, dtype=torch.int32, device="cuda")
    kda.kda_scaled_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), y, status)
    assert int(status) == 0 and bool((buf[T:] == 7.0).all())
    want, size = ref.scaled_matmul(x.float(), xs, w.float(), ws)
    got = y.double().cpu().numpy()
    tol = 2.0 ** -8 * 1.001 * np.abs(want) + (264 + ws.shape[1]) * F * size + 1e-38
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{np.max(err / tol):.3g} of the bound"


def test_the_last_tile_gets_its_own_scale_group():
    """Codes of 1 and distinct scales of powers of two: sums are exact, so every output names the scales that it got."""
    T, N, K = 2404, 2057, 256
    one = lambda n: torch.ones(n, K).to(torch.float8_e4m3fn).cuda()
    ws = 2.0 ** torch.arange(-17, 17).reshape(17, 2).float()
    y = kda.scaled_matmul(one(T), torch.ones(T, device="cuda"), one(N), ws.cuda(), check=True).double().cpu()
    want = (128.0 * ws.double().sum(1)).repeat_interleave(128)[:N]
    assert torch.equal(y, want[None].expand(T, N).to(torch.bfloat16).double())
