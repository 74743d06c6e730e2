"""GPU tests of the delta rule with one decay per head (chunked and recurrent forms) against the fp64 recurrence.

Bounds element by element: oracle/delta.py derives them; o adds its own rounding, 2^-8 of itself. Over all elements (2-norms):
errors of many roundings add up like independent ones. o: bf16 of itself (half a step is 2^-8 at most, 2^-8 / sqrt(3) on average over
a step and less, 2^-8 / 2.3, over values), of the chunk's responses, of Z and of the state that q multiplies: sqrt(4) / 2.3 = 0.87 of 2^-8
at most: below 2^-8. Final state: five operands of two bf16 terms, each at most
2^-16 and on average a fifth of it off: below 2^-16; the recurrence is fp32: below 2^-20.
"""
import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from oracle import delta as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
D = 128
CHUNK = 64


def make(lens, H, Hk, seed, state=True, extra=0, rate=1.0, common=0.3):
    """`common`: the part that all keys share (0: random directions)."""
    rng = np.random.default_rng(seed)
    T = sum(lens) + extra
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    q, k = (torch.from_numpy(unit(rng.standard_normal((T, Hk, D)) + common * rng.standard_normal(D))).to(torch.bfloat16)
            for _ in range(2))
    v = torch.from_numpy(rng.standard_normal((T, H, D))).to(torch.bfloat16)
    g = -rate * np.log1p(np.exp(rng.standard_normal((T, H)))) * np.exp(-4 * rng.random(H))
    return {"q": q, "k": k, "v": v, "g": torch.from_numpy(g).float(),
            "beta": torch.from_numpy(1 / (1 + np.exp(-rng.standard_normal((T, H))))).float(), "lens": lens,
            "cu": torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32), "scale": D ** -0.5,
            "s0": torch.from_numpy(rng.standard_normal((len(lens), H, D, D)) * 0.3).float() if state else None}


def oracle_of(x, chunk=CHUNK):
    f = lambda t: None if t is None else t.double().numpy()
    return ref.recurrence(*(f(x[n]) for n in ("q", "k", "v", "g", "beta")), x["lens"], f(x["s0"]), x["scale"], chunk)


def rel(a, b):
    return np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-300)


def check(x, o, fs, want=None, chunk=CHUNK, norms=True):
    ro, off, rs, soff = oracle_of(x, chunk) if want is None else want
    n = sum(x["lens"])
    if n:
        o = o[:n].double().cpu().numpy()
        err, tol = np.abs(o - ro[:n]), U * 1.001 * np.abs(ro[:n]) + off[:n] + 1e-30
        assert np.isfinite(o).all() and (err <= tol).all(), f"o: {np.max(err / tol):.3g} of the bound"
        assert not norms or rel(o, ro[:n]) <= U
    if fs is not None and rs.size:
        s = fs.double().cpu().numpy()
        err, tol = np.abs(s - rs), soff[:, :, None, :] + 2 * ref.F * np.abs(rs) + 1e-30
        assert np.isfinite(s).all() and (err <= tol).all(), f"final state: {np.max(err / tol):.3g} of the bound"
        # (below 2^-126 fp32 holds no relative precision, and below 2^-149 nothing: 5000 tokens of e^-0.0254 leave e^-127)
        assert not norms or np.abs(rs).max() < 2.0 ** -126 or rel(s, rs) <= (2.0 ** -16 if chunk else 2.0 ** -20)


def dev(x):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}


def chunk(x, **kw):
    d = dev(x)
    return kda.gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], d["s0"], scale=x["scale"], check=True, **kw)


def decode(x, **kw):
    d = dev(x)
    return kda.gated_delta_decode_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], len(x["lens"]), d["s0"], scale=x["scale"],
                                      check=True, **kw)


# ------------------------------------------------------------------ the recurrence
@pytest.mark.parametrize("N,Tn,H,Hk,state", [(1, 1, 1, 1, True), (3, 1, 4, 2, True), (2, 4, 6, 6, True), (5, 2, 3, 1, False),
                                             (2, 64, 2, 2, True), (1, 7, 96, 32, True), (4, 0, 2, 2, True), (300, 1, 2, 2, True)])
def test_decode(N, Tn, H, Hk, state):
    x = make([Tn] * N, H, Hk, seed=N + Tn + H, state=state)
    o, fs = decode(x)
    check(x, o, fs, chunk=0)


@pytest.mark.parametrize("g", [0.0, -1e-6, -5.0, -90.0, float("-inf")])
def test_decode_extreme_decays(g):
    x = make([5] * 3, 2, 2, seed=5)
    x["g"].fill_(g)
    o, fs = decode(x)
    check(x, o, fs, chunk=0)


@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0, -0.5])
def test_decode_extreme_strengths(beta):
    x = make([6] * 2, 2, 1, seed=6)
    x["beta"].fill_(beta)
    o, fs = decode(x)
    if beta < 0:  # grows: the bound's premise does not hold; 6 steps of a factor up to 1.5
        ro, off, rs, soff = oracle_of(x, 0)
        check(x, o, fs, (ro, off * 16, rs, soff * 16), chunk=0)
    else:
        check(x, o, fs, chunk=0)


def test_decode_in_place_on_slices_and_another_stream():
    x = make([3] * 4, 4, 2, seed=7)
    d = dev(x)
    T = 12
    qkv = torch.full((T, 8 * D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :2 * D].view(T, 2, D), qkv[:, 2 * D:4 * D].view(T, 2, D), qkv[:, 4 * D:8 * D].view(T, 4, D)
    q.copy_(d["q"]), k.copy_(d["k"]), v.copy_(d["v"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, fs = kda.gated_delta_decode_fwd(q, k, v, d["g"], d["beta"], 4, d["s0"], in_place=True, check=True, stream=s)
    assert fs is d["s0"]
    check(x, o, fs, chunk=0)


def test_decode_many_steps_is_the_prompt():
    """A sequence token by token, the state carried in place, and as one prompt."""
    x = make([40], 3, 3, seed=8)
    d = dev(x)
    s, rows = d["s0"].clone(), []
    for t in range(40):
        o, _ = kda.gated_delta_decode_fwd(*(d[n][t:t + 1] for n in ("q", "k", "v", "g", "beta")), 1, s, in_place=True)
        rows.append(o)
    check(x, torch.cat(rows), s, chunk=0)


def test_decode_flags_gates():
    for bad in (1e-3, float("nan")):
        x = make([2] * 3, 2, 2, seed=9)
        x["g"][3, 1] = bad
        with pytest.raises(kda.KdaError) as e:
            decode(x)
        assert e.value.code == kda.KDA_ERR_GATE_RANGE


# ------------------------------------------------------------------ prompts
PROMPTS = {
    "one_token": ([1], 1, 1, False),
    "one_chunk": ([64], 2, 2, False),
    "one_over": ([65], 2, 1, True),
    "one_short": ([63], 2, 2, True),
    "two_chunks": ([128], 2, 2, True),
    "ragged": ([130, 0, 64, 1, 127, 128, 383, 0, 5], 3, 3, True),
    "ragged_no_state": ([33, 400, 0, 17], 4, 2, False),
    "shared_heads": ([200, 70], 6, 2, True),
    "long": ([1500], 2, 2, True),
    "few_tokens_each": ([1, 2, 3, 0, 4] * 5, 3, 1, True),
    "all_empty": ([0, 0, 0], 2, 2, True),
    "many_heads": ([300, 40], 96, 32, True),
}


@pytest.mark.parametrize("name", list(PROMPTS))
def test_prompts(name):
    lens, H, Hk, state = PROMPTS[name]
    x = make(lens, H, Hk, seed=sum(lens) + H, state=state)
    o, fs = chunk(x)
    check(x, o, fs)


@pytest.mark.parametrize("lens,H", [([4000, 9], 1), ([2600, 1, 0, 3100], 2)])
def test_few_long_chains(lens, H):
    """Few (sequence, head) chains of many chunks, with slow decays: old tokens matter to the end."""
    x = make(lens, H, H, seed=77, rate=0.02)
    o, fs = chunk(x)
    check(x, o, fs)


@pytest.mark.parametrize("g", [0.0, -1e-6, -0.3, -5.0, -60.0, -138.5, float("-inf")])
def test_extreme_decays(g):
    x = make([300, 20], 2, 2, seed=15)
    x["g"].fill_(g)
    o, fs = chunk(x)
    check(x, o, fs)


@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0])
@pytest.mark.parametrize("common", [0.0, 0.3, 3.0, 1e6])
def test_strengths_and_like_keys(beta, common):
    """Keys that share most of their direction, or all of it (beta = 1: each token replaces what the one before wrote; 2: reflects)."""
    x = make([200, 64, 3], 2, 2, seed=16, common=common, rate=0.05)
    # unit keys as bf16 holds them: beta |k|^2 stays below 2
    x["k"] = (x["k"].double() * 0.995).to(torch.bfloat16)
    x["beta"].fill_(beta)
    o, fs = chunk(x)
    # (2 and equal keys: T's entries are 2 in size and alternate, errors of a chunk add up in step)
    check(x, o, fs, norms=not (beta == 2.0 and common >= 3.0))


@pytest.mark.parametrize("total", [-0.6, -5.0, -13.0, -40.0])
@pytest.mark.parametrize("lens,H", [([384, 128, 70], 3), ([5000], 1)])
def test_states_that_only_decay(lens, H, total):
    """No writing: what is left of the initial state, to the end, is its decay alone, to fp32's relative precision: a chunk's
    decay is off by 4 f, and there is one a chunk."""
    x = make(lens, H, H, seed=38)
    x["beta"].fill_(0.0)
    x["g"].fill_(total / 64 if H > 1 else total / 512)
    o, fs = chunk(x)
    want = oracle_of(x)
    check(x, o, fs, want)
    s, rs = fs.double().cpu().numpy(), want[2]
    chunks = max(lens) // 64 + 2
    assert (np.abs(s - rs) <= (8 * chunks + 64) * ref.F * np.abs(rs) + 1e-36).all()


def test_a_state_decays_at_once():
    """One strong decay in the middle of a chunk, among slow ones."""
    for g in (-3.0, -17.0, -100.0, float("-inf")):
        x = make([140, 300], 2, 2, seed=39, rate=0.01)
        x["g"][[60, 250, 400], :] = g
        o, fs = chunk(x)
        check(x, o, fs)


def test_large_and_small_values():
    for size in (2.0 ** 60, 2.0 ** -60):
        x = make([150, 70], 2, 2, seed=32)
        x["v"], x["s0"] = x["v"] * size, x["s0"] * size
        o, fs = chunk(x)
        check(x, o, fs)


@pytest.mark.parametrize("lens", [[1500, 0, 37, 100], [0, 0, 0, 1900], [512, 512, 512, 512]])
def test_padded_batch(lens):
    """2048 rows for four sequences: rows behind the last sequence are neither used nor written."""
    x = make(lens, 4, 2, seed=34, extra=2048 - sum(lens))
    n = sum(lens)
    want = oracle_of(x)
    for key in ("q", "k", "v", "g", "beta"):
        x[key][n:] = float("nan")
    d = dev(x)
    o = torch.full((2048, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fs, status = torch.empty_like(d["s0"]), torch.ones(1, dtype=torch.int32, device="cuda")
    kda.kda_gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], d["s0"], x["scale"], o, fs, status)
    check(x, o, fs, want)
    assert int(status) == 0 and bool((o[n:] == 7.0).all())


def test_prompt_in_place_on_slices_and_another_stream():
    x = make([300, 40, 0, 170], 4, 2, seed=35)
    d = dev(x)
    want = kda.gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], d["s0"], check=True)
    check(x, *want)
    T = 510
    qkv = torch.full((T, 8 * D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :2 * D].view(T, 2, D), qkv[:, 2 * D:4 * D].view(T, 2, D), qkv[:, 4 * D:8 * D].view(T, 4, D)
    q.copy_(d["q"]), k.copy_(d["k"]), v.copy_(d["v"])
    o = torch.empty_like(d["v"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kda.kda_gated_delta_chunk_fwd(q, k, v, d["g"], d["beta"], d["cu"], d["s0"], x["scale"], o, d["s0"], stream=s)
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(d["s0"], want[1])


def test_cut_sequences_with_states_in_place():
    """Long sequences in parts, beside short and empty ones; the state's buffer updated. The last part of a sequence may end before the
    first begins: it must not find the final state."""
    for lens, H in (([3000, 40, 0, 1700], 2), ([64 * 5, 6000], 1), ([9000], 4)):
        x = make(lens, H, H, seed=55, rate=0.1)
        d = dev(x)
        want = kda.gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], d["s0"], check=True)
        check(x, *want)
        o = torch.empty_like(d["v"])
        kda.kda_gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], d["s0"], x["scale"], o, d["s0"])
        assert torch.equal(o, want[0]) and torch.equal(d["s0"], want[1])
    x = make([5000, 30], 2, 2, seed=56, state=False, rate=0.1)
    check(x, *chunk(x))
    o, fs = chunk(x, output_final_state=False)
    assert fs is None
    check(x, o, None)


def test_parts_and_joins_in_rounds():
    """More parts of cut sequences, and more columns to join, than an SM each."""
    x = make([6000, 7000], 8, 4, seed=61, rate=0.1)
    check(x, *chunk(x))


def test_many_sequences():
    """More sequences than the plan holds lengths of, empty ones among them, one long one."""
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(0, 4, 4300)]
    lens[17], lens[4299] = 700, 65
    x = make(lens, 1, 1, seed=57)
    o, fs = chunk(x)
    check(x, o, fs)


@pytest.mark.parametrize("lens,H", [([1] * 255 + [2049], 2), ([0] * 60 + [300, 64, 65, 1] + [2] * 5, 3), ([7] * 30 + [0, 90] + [1] * 3, 2),
                                    ([16] * 20, 2), ([64, 0, 0, 0, 0, 0, 0, 0], 2), ([0] * 7 + [65, 0], 2),
                                    ([0] * 800 + [6000, 1, 900], 1)])
def test_long_sequences_among_short_ones(lens, H):
    """Few tokens a sequence on average, but not in every one: the long ones run as chunks. States in place."""
    x = make(lens, H, H, seed=42, extra=5)
    x["g"][sum(lens):] = float("nan")
    d = dev(x)
    o = torch.full_like(d["v"], 7.0)
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    kda.kda_gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], d["s0"], x["scale"], o, d["s0"], status)
    x["g"][sum(lens):] = 0
    check(x, o, d["s0"])
    assert int(status) == 0 and bool((o[sum(lens):] == 7.0).all())


def test_overlapping_long_sequences_among_short_ones():
    """Bounds that run backwards in a batch of few tokens a sequence: reported, nothing outside the workspace is written."""
    T, N = 600, 200
    x = make([T], 1, 1, seed=60, state=False)
    d = dev(x)
    cu = torch.tensor([0, 100] * (N // 2) + [T], dtype=torch.int32, device="cuda")
    need = kda.gated_delta_workspace_size(N, T, 1)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    o, fs = torch.empty_like(d["v"]), torch.empty(N, 1, D, D, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, None, x["scale"], o, fs, status, workspace=ws[:need])
    assert int(status) == kda.KDA_ERR_BAD_SEQLENS and bool((ws[need:] == 255).all())


@pytest.mark.parametrize("H,Hk", [(1, 1), (5, 1), (32, 4)])
def test_lengths_around_chunks_and_cuts(H, Hk):
    for lens in ([64 * 8 - 1, 64 * 8, 64 * 8 + 1], [1 + 64 * 30], [64 * 31, 2]):
        x = make(lens, H, Hk, seed=H + len(lens), rate=0.3)
        o, fs = chunk(x)
        check(x, o, fs)


def test_workspace_given_and_too_small():
    x = make([300, 65], 2, 2, seed=58)
    d = dev(x)
    need = kda.gated_delta_workspace_size(2, 365, 2)
    o, fs = torch.empty_like(d["v"]), torch.empty_like(d["s0"])
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
    args = (d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], d["s0"], x["scale"], o, fs)
    kda.kda_gated_delta_chunk_fwd(*args, workspace=ws[:need])
    check(x, o, fs)
    assert bool((ws[need:] == 255).all())
    for bad in (ws[:need - 1], ws[16:16 + need]):
        with pytest.raises(kda.KdaError) as e:
            kda.kda_gated_delta_chunk_fwd(*args, workspace=bad)
        assert e.value.code == kda.KDA_ERR_INVALID_ARG


def test_overlapping_lengths_stay_inside_the_workspace():
    """Bounds that are each in range but run backwards hold more tokens than there are: reported, nothing outside is written."""
    T, H = 4000, 1
    x = make([T], H, H, seed=59, state=False)
    d = dev(x)
    cu = torch.tensor([0, T] * 40, dtype=torch.int32, device="cuda")
    N = 79
    need = kda.gated_delta_workspace_size(N, T, H)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    o, fs = torch.empty_like(d["v"]), torch.empty(N, H, D, D, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, None, x["scale"], o, fs, status, workspace=ws[:need])
    assert int(status) == kda.KDA_ERR_BAD_SEQLENS and bool((ws[need:] == 255).all())


def test_bad_lengths_are_skipped():
    """cu_seqlens that run backwards or past the rows: reported, the other sequences are right."""
    x = make([100, 50, 80], 2, 2, seed=36, extra=20)
    want = oracle_of(x)
    d = dev(x)
    for cu, good in (([0, 100, 90, 230], [(0, 0, 100)]), ([0, 100, 150, 1000], [(0, 0, 100), (1, 100, 150)]),
                     ([0, -5, 150, 230], [(2, 150, 230)])):
        o, fs = torch.full_like(d["v"], 7.0), torch.full_like(d["s0"], 7.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kda.kda_gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                      d["s0"], x["scale"], o, fs, status)
        assert int(status) == kda.KDA_ERR_BAD_SEQLENS
        for n, a, b in good:
            assert np.abs(o[a:b].double().cpu().numpy() - want[0][a:b]).max() <= 0.05 * np.abs(want[0][a:b]).max()


def test_prompt_flags_gates():
    for bad in (1e-3, float("nan")):
        x = make([100, 130, 60], 2, 2, seed=9)
        x["g"][150, 1] = bad
        with pytest.raises(kda.KdaError) as e:
            chunk(x)
        assert e.value.code == kda.KDA_ERR_GATE_RANGE


def test_a_nan_stays_in_its_sequence_and_head():
    x = make([150, 130, 60], 2, 2, seed=10)
    want = oracle_of(x)
    x["v"][200, 1] = float("nan")
    o, fs = chunk(x)
    o, fs = o.cpu(), fs.cpu()
    assert torch.isnan(o[200, 1]).all() and torch.isnan(fs[1, 1]).any()
    keep = torch.ones(340, 2, dtype=torch.bool)
    keep[150:280, 1] = False
    assert torch.isfinite(o[keep]).all() and torch.isfinite(fs[[0, 0, 1, 2, 2], [0, 1, 0, 0, 1]]).all()
    err = (o.double() - torch.from_numpy(want[0])).abs()[keep]
    assert bool((err <= U * torch.from_numpy(want[0]).abs()[keep] * 1.001 + torch.from_numpy(want[1])[keep]).all())


def test_calls_in_graphs_and_on_streams_at_once():
    """A captured prompt call, replayed on new inputs, beside an eager one on another stream."""
    a, b = make([200, 90, 31], 3, 3, seed=11), make([31, 200, 90], 3, 3, seed=12)
    da, db = dev(a), dev(b)
    names = ("q", "k", "v", "g", "beta", "cu", "s0")
    held = {n: da[n].clone() for n in names}
    call = lambda d: kda.gated_delta_chunk_fwd(*(d[n] for n in names))
    call(held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, fs = call(held)
    other = torch.cuda.Stream()
    for x, d in ((a, da), (b, db), (a, da)):
        for n in names:
            held[n].copy_(d[n])
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            eo, es = call(db)
        torch.cuda.synchronize()
        check(x, o, fs)
        check(b, eo, es)
