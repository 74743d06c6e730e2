"""GPU tests of the int8 state cache: its codes are whole numbers and equal the restated rounding; what it reads back is off by
at most half a step of the row's scale; and a serving run load -> prefill -> decode -> store."""
import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from kda_chunked_prefill_gb300 import inputs as kin
from oracle import linear as ref

pytestmark = pytest.mark.gpu
D = 128


def states(M, H, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal((M, H, D, D)) * np.exp(2 * rng.standard_normal((M, H, D, 1)))).float()


def cache(S, H):
    return (torch.full((S, H, D, D), 99, dtype=torch.int8, device="cuda"), torch.full((S, H, D), 3.0, device="cuda"))


@pytest.mark.parametrize("M,H,S", [(1, 1, 1), (3, 5, 7), (17, 2, 40), (2, 96, 3)])
def test_store_and_load(M, H, S):
    x = states(M, H, M + H)
    slots = torch.from_numpy(np.random.default_rng(S).permutation(S)[:M].astype(np.int32))
    codes, scales = cache(S, H)
    kda.state_store(x.cuda(), slots.cuda(), codes, scales, check=True)
    want, ws = ref.quantise_rows(x.numpy())
    at = slots.long()
    assert np.array_equal(codes.cpu()[at].double().numpy(), want)
    assert np.array_equal(scales.cpu()[at].double().numpy(), ws)
    rest = torch.ones(S, dtype=torch.bool)
    rest[at] = False
    assert bool((codes.cpu()[rest] == 99).all()) and bool((scales.cpu()[rest] == 3.0).all())
    back = kda.state_load(codes, scales, slots.cuda(), check=True).cpu()
    assert torch.equal(back, codes.cpu()[at].float() * scales.cpu()[at][..., None])
    amax = x.abs().amax(-1, keepdim=True).double()
    # half a step, and four fp32 roundings of values up to amax
    assert bool(((back.double() - x.double()).abs() <= amax / 254 * (1 + 1e-6) + amax * 2.0 ** -21).all())


def test_rows_without_a_slot_and_equal_slots():
    x = states(5, 2, 8)
    codes, scales = cache(4, 2)
    slots = torch.tensor([2, -1, 0, 2, -1], dtype=torch.int32)
    kda.state_store(x.cuda(), slots.cuda(), codes, scales, check=True)
    want, _ = ref.quantise_rows(x.numpy())
    got = codes.cpu().double().numpy()
    assert np.array_equal(got[0], want[2]) and np.array_equal(got[2], want[3])  # the last row of a slot stays
    assert (got[[1, 3]] == 99).all()
    back = kda.state_load(codes, scales, slots.cuda(), check=True)
    assert bool((back[[1, 4]] == 0).all()) and torch.equal(back[0], back[3])


def test_many_rows_of_one_slot():
    x = states(700, 1, 9)
    codes, scales = cache(2, 1)
    kda.state_store(x.cuda(), torch.ones(700, dtype=torch.int32, device="cuda"), codes, scales, check=True)
    assert np.array_equal(codes.cpu().double().numpy()[1], ref.quantise_rows(x[-1].numpy())[0])


@pytest.mark.parametrize("slot", [4, -2, 2 ** 31 - 1, -2 ** 31])
def test_bad_slots_are_skipped_and_reported(slot):
    x = states(2, 1, 10).cuda()
    codes, scales = cache(4, 1)
    slots = torch.tensor([slot, 1], dtype=torch.int32, device="cuda")
    for call in (lambda: kda.state_store(x, slots, codes, scales, check=True),
                 lambda: kda.state_load(codes, scales, slots, check=True)):
        with pytest.raises(kda.KdaError) as e:
            call()
        assert e.value.code == kda.KDA_ERR_BAD_SLOT
    assert bool((codes[[0, 2, 3]] == 99).all()) and bool((codes[1] != 99).any())
    assert bool((kda.state_load(codes, scales, slots)[0] == 0).all())


def test_rows_of_zeros_tiny_values_and_no_numbers():
    x = torch.zeros(1, 1, D, D)
    x[0, 0, 1] = 1e-38
    x[0, 0, 2, 5] = float("nan")
    x[0, 0, 3, 7] = float("-inf")
    x[0, 0, 4, 3] = -3.0e38
    x[0, 0, 5, 0] = 2.0 ** -99
    x[0, 0, 6, 0], x[0, 0, 6, 1:] = 127.0, 0.5  # ties: 0.5 and 1.5 go to even
    x[0, 0, 6, 64:] = 1.5
    codes, scales = cache(1, 1)
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.state_store(x.cuda(), slots, codes, scales, check=True)
    back = kda.state_load(codes, scales, slots).cpu()[0, 0]
    assert bool((back[:2] == 0).all()) and bool(back[2:4].isnan().all())
    assert back[4, 3] == pytest.approx(-3.0e38, rel=1e-6) and bool((back[4, :3] == 0).all())
    assert back[5, 0] == pytest.approx(2.0 ** -99, rel=1e-6)
    assert back[6, 0] == 127 and bool((back[6, 1:64] == 0).all()) and bool((back[6, 64:] == 2).all())


def test_offsets_past_32_bits():
    """A cache whose last slots lie behind 2^32 code bytes (2^30 elements a slot row of 16 heads x 128 x 128 is 256 KB)."""
    S, H = 17000, 16
    codes = torch.empty((S, H, D, D), dtype=torch.int8, device="cuda")
    scales = torch.empty((S, H, D), device="cuda")
    x = states(2, H, 12)
    slots = torch.tensor([S - 1, 16400], dtype=torch.int32, device="cuda")
    kda.state_store(x.cuda(), slots, codes, scales, check=True)
    want, _ = ref.quantise_rows(x.numpy())
    assert np.array_equal(codes[[S - 1, 16400]].cpu().double().numpy(), want)
    back = kda.state_load(codes, scales, slots, check=True)
    assert torch.equal(back, codes[slots.long()].float() * scales[slots.long()][..., None])


def test_serving_run():
    """Cached prefixes in, prompt, two tokens, states back into the cache: the linear layer and the KDA layer on the same cache."""
    from linear_util import linear_inputs
    H, lens = 4, [150, 64, 201]
    prefix = states(3, H, 40) * 0.05
    codes, scales = cache(8, H)
    slots = torch.tensor([6, -1, 2], dtype=torch.int32, device="cuda")
    kda.state_store(prefix.cuda(), slots, codes, scales, check=True)
    s0 = kda.state_load(codes, scales, slots, check=True)
    host = s0.cpu()
    assert bool((host[1] == 0).all())
    # KDA layer: same result as from the host copy of the loaded states
    inp = kin.make_inputs(lens, H, seed=3, state_std=0.02)
    args = [inp[k].cuda() for k in ("q", "k", "v", "g", "beta", "cu_seqlens")]
    a = kda.chunk_fwd(*args, s0, scale=inp["scale"], lower_bound=inp["lower_bound"], check=True)
    b = kda.chunk_fwd(*args, host.cuda(), scale=inp["scale"], lower_bound=inp["lower_bound"], check=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # linear layer: prompt, then two tokens, against the recurrence over all tokens
    x = linear_inputs([n + 2 for n in lens], H, 2, seed=4)
    first = np.concatenate([[0], np.cumsum([n + 2 for n in lens])])
    pick = lambda t, last: torch.cat([t[f + n:f + n + 2] if last else t[f:f + n] for f, n in zip(first, lens)]).cuda()
    names = ("q", "k", "v", "g")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    o1, s1 = kda.linear_chunk_fwd(*[pick(x[k], False) for k in names], cu, s0, check=True)
    o2, s2 = kda.linear_decode_fwd(*[pick(x[k], True) for k in names], 3, s1, in_place=True, check=True)
    ro, size, rs, rsize = ref.recurrence(*[x[k].double().numpy() for k in names], [n + 2 for n in lens],
                                         host.double().numpy(), D ** -0.5)
    cuts = np.concatenate([[0], np.cumsum(lens)])
    for i, n in enumerate(lens):
        got = torch.cat([o1[cuts[i]:cuts[i + 1]], o2[2 * i:2 * i + 2]]).double().cpu().numpy()
        want, sz = ro[first[i]:first[i + 1]], size[first[i]:first[i + 1]]
        assert (np.abs(got - want) <= 2.0 ** -8 * (1.01 * np.abs(want) + 1.1 * sz) + 1e-30).all()
    # 3.03 u^2, u = 2^-8: the two-term operands of the state's update (derived in test_gpu_linear.py)
    assert (np.abs(s2.double().cpu().numpy() - rs) <= (3.03 * 2.0 ** -16 + 1200 * 2.0 ** -24) * rsize).all()
    kda.state_store(s2, torch.tensor([6, 0, 2], dtype=torch.int32, device="cuda"), codes, scales, check=True)
    again = kda.state_load(codes, scales, torch.tensor([6, 0, 2], dtype=torch.int32, device="cuda"))
    amax = s2.abs().amax(-1, keepdim=True)
    assert bool(((again - s2).abs() <= amax / 254 + amax * 2.0 ** -20).all())


def test_layer_run_in_a_graph():
    """Norm, projection, load, prompt, store, captured once and replayed on new inputs: as the same calls made one by one, and the
    prompt as the recurrence over what the projection made."""
    H, Hk, width, lens = 4, 2, 256, [300, 20, 129]
    T = sum(lens)
    gen = torch.Generator().manual_seed(50)
    rand = lambda *shape: torch.randn(*shape, generator=gen)
    x, residual, weight = rand(T, width).bfloat16().cuda(), rand(T, width).cuda(), (1 + 0.1 * rand(width)).cuda()
    w_qkv = (rand(width, (2 * Hk + H) * D) * 0.01).bfloat16().cuda()
    g = (-torch.rand(H, generator=gen) * 0.2).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    codes, scales = cache(6, H)
    kda.state_store(states(3, H, 51).cuda() * 0.1, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), codes, scales)
    slots_in, slots_out = (torch.tensor(i, dtype=torch.int32, device="cuda") for i in ([2, -1, 0], [3, 4, 5]))

    def layer():
        y, y_scale, res = kda.add_rms_norm(x, residual, weight, 1e-6)
        qkv = (y.float() * y_scale[:, None]).bfloat16() @ w_qkv
        q, k, v = (t.view(T, -1, D) for t in qkv.split([Hk * D, Hk * D, H * D], dim=1))
        s0 = kda.state_load(codes, scales, slots_in)
        o, state = kda.linear_chunk_fwd(q, k, v, g, cu, s0)
        kda.state_store(state, slots_out, codes, scales)
        return q, k, v, s0, o, state, res

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for _ in range(2):
        x.copy_(rand(T, width).bfloat16())
        residual.copy_(rand(T, width))
        graph.replay()
        torch.cuda.synchronize()
        got, stored = [t.clone() for t in out], (codes.clone(), scales.clone())
        codes[3:], scales[3:] = 0, 0
        want = layer()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(codes, stored[0]) and torch.equal(scales, stored[1])
        q, k, v, s0, o, state, res = (t.double().cpu().numpy() for t in got)
        assert np.array_equal(res, (x.float() + residual).double().cpu().numpy())
        ro, size, rs, rsize = ref.recurrence(q, k, v, np.broadcast_to(g.double().cpu().numpy(), (T, H)), lens, s0, D ** -0.5)
        # as in test_gpu_linear.py: one rounding of o, one of each score and of the state's copy, fp32 sums
        assert (np.abs(o - ro) <= 2.0 ** -8 * (1.01 * np.abs(ro) + 1.05 * size) + 1200 * 2.0 ** -24 * size + 1e-30).all()
        assert (np.abs(state - rs) <= (3.03 * 2.0 ** -16 + 1200 * 2.0 ** -24) * rsize).all()
