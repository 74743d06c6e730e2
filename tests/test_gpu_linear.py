"""GPU tests of the linear attention with one decay per head (chunked and recurrent forms) against the fp64 recurrence.

Bounds, from the number of roundings (u = 2^-8 for bf16, half a step; 2^-24 for fp32; A = the same sums over magnitudes):
  o (both)       u |o| for its own rounding; the chunked form also rounds each decayed score and the state that q multiplies
                 once to bf16: u A.
  final state    the chunked form's update operands w v are two bf16 terms h + l. With w = a + b + e in bf16, |w - a| <= u w and
                 |e| <= u^2 w; h = bf16(v a), whose remainder r = v a - h has 8 bits and is exact, |r| <= u |v a|; l = bf16(v b + r)
                 is off by u (|v b| + |r|) <= 2 u^2 (1 + u)^2 |w v|. Together 3 u^2 (1 + u)^2 <= 3.03 u^2: 3.03 u^2 A.
                 All fp32 sums: at most 128 terms a chunk and one step a chunk, taken as 600 roundings of 2^-24, truncations
                 counted double: together below 8e-5 A.
"""
import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from kda_chunked_prefill_gb300 import _lib
from oracle import linear as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
FP32 = 1200 * 2.0 ** -24
D = 128


def make(lens, H, Hk, seed, state=True, decay="token", extra=0, rate=1.0):
    rng = np.random.default_rng(seed)
    T = sum(lens) + extra
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    q, k = (torch.from_numpy(unit(rng.standard_normal((T, Hk, D)))).to(torch.bfloat16) for _ in range(2))
    v = torch.from_numpy(rng.standard_normal((T, H, D))).to(torch.bfloat16)
    g = -rate * np.log1p(np.exp(rng.standard_normal((T, H) if decay == "token" else (H,)))) * np.exp(-4 * rng.random(H))
    return {"q": q, "k": k, "v": v, "g": torch.from_numpy(g).float(), "lens": lens,
            "cu": torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32), "scale": D ** -0.5,
            "s0": torch.from_numpy(rng.standard_normal((len(lens), H, D, D)) * 0.3).float() if state else None}


def oracle_of(x):
    f = lambda t: None if t is None else t.double().numpy()
    return ref.recurrence(f(x["q"]), f(x["k"]), f(x["v"]), f(x["g"]), x["lens"], f(x["s0"]), x["scale"])


def check(x, o, fs, want=None, chunked=True):
    ro, size, rs, rsize = oracle_of(x) if want is None else want
    n = sum(x["lens"])
    o = o[:n].double().cpu().numpy()
    err, tol = np.abs(o - ro[:n]), U * np.abs(ro[:n]) * 1.01 + ((U * 1.05 if chunked else 0) + FP32) * size[:n] + 1e-30
    assert np.isfinite(o).all() and (err <= tol).all(), f"o: {np.max(err / tol):.3g} of the bound"
    if fs is not None:
        s = fs.double().cpu().numpy()
        err, tol = np.abs(s - rs), ((3.03 * U * U if chunked else 0) + FP32) * rsize + 1e-30
        assert np.isfinite(s).all() and (err <= tol).all(), f"final state: {np.max(err / tol):.3g} of the bound"


def dev(x):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}


def chunk(x, **kw):
    d = dev(x)
    return kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], scale=x["scale"], check=True, **kw)


CHUNK = {
    "one_token": ([1], 1, 1, False, "token"),
    "one_chunk": ([128], 2, 2, False, "token"),
    "one_over": ([129], 2, 1, True, "token"),
    "two_chunks": ([256], 2, 2, True, "head"),
    "ragged": ([130, 0, 64, 1, 127, 128, 383, 0, 5], 3, 3, True, "token"),
    "ragged_no_state": ([33, 400, 0, 17], 4, 2, False, "token"),
    "shared_heads": ([200, 70], 6, 2, True, "head"),
    "long": ([1500], 2, 2, True, "token"),
    "few_tokens_each": ([1, 2, 3, 0, 4] * 5, 3, 1, True, "token"),
    "all_empty": ([0, 0, 0], 2, 2, True, "token"),
    "many_heads": ([300, 40], 96, 32, True, "head"),
}


@pytest.mark.parametrize("name", list(CHUNK))
def test_chunk(name):
    lens, H, Hk, state, decay = CHUNK[name]
    x = make(lens, H, Hk, seed=sum(lens) + H, state=state, decay=decay)
    o, fs = chunk(x)
    check(x, o, fs)


@pytest.mark.parametrize("lens,H", [([4000, 9], 1), ([2600, 1, 0, 3100], 2)])
def test_chunk_few_long_chains(lens, H):
    """Few (sequence, head) chains of many chunks, with slow decays: old tokens matter to the end."""
    x = make(lens, H, H, seed=77, rate=0.02)
    o, fs = chunk(x)
    check(x, o, fs)


@pytest.mark.parametrize("g", [0.0, -1e-6, -5.0, -60.0, -138.5, float("-inf")])
def test_chunk_extreme_decays(g):
    x = make([300, 20], 2, 2, seed=5)
    x["g"].fill_(g)
    o, fs = chunk(x)
    check(x, o, fs)


@pytest.mark.parametrize("g", [-0.2, -0.25, -0.2598, -0.2602, -0.3, -1.0])
def test_chunk_decay_of_a_whole_chunk(g):
    """A chunk's whole decay on both sides of 2^-48 (128 tokens of -0.26): scores without anchors and with."""
    x = make([300, 128, 70], 2, 1, seed=31)
    x["g"].fill_(g)
    o, fs = chunk(x)
    check(x, o, fs)


@pytest.mark.parametrize("total", [-0.6, -0.75, -5.0, -9.0, -13.0, -20.0, -40.0])
@pytest.mark.parametrize("lens,H", [([384, 128, 70], 3), ([5000], 1)])
@pytest.mark.parametrize("size", [0.0, 1e-7])
def test_states_that_only_decay(lens, H, total, size):
    """Values of (almost) nothing: what is left of the initial state, to the end, is its decay alone. `total`: a chunk's, or, with
    one long sequence (cut into segments of four chunks and more), four chunks'."""
    x = make(lens, H, H, seed=38)
    x["v"] = x["v"] * size
    x["g"].fill_(total / 128 if H > 1 else total / 512)
    o, fs = chunk(x)
    check(x, o, fs)


def test_a_state_decays_at_once():
    """One strong decay in the middle of a chunk, no values: sums of a strong and of slow decays."""
    for g in (-3.0, -12.8, -17.0, -30.0, -100.0):
        x = make([140, 300], 2, 2, seed=39, rate=0.01)
        x["v"] = x["v"] * 0.0
        x["g"][[60, 250, 400], :] = g
        o, fs = chunk(x)
        check(x, o, fs)


def test_chunk_large_values():
    """Scores and outputs of 2^30 and more, with decays close to where chunks stop being computed without anchors."""
    x = make([400, 50], 2, 2, seed=32)
    x["g"].fill_(-0.25)
    for key in ("q", "k", "v"):
        x[key] = x[key] * 4096
    o, fs = chunk(x)
    check(x, o, fs)


def test_chunk_more_sequences_than_are_sorted():
    x = make([20] * 250 + [4000] + [19] * 150, 1, 1, seed=33)
    o, fs = chunk(x)
    check(x, o, fs)


@pytest.mark.parametrize("lens", [[1500, 0, 37, 100], [0, 0, 0, 1900], [512, 512, 512, 512]])
def test_padded_batch_whose_rows_divide_by_its_sequences(lens):
    """2048 rows for four sequences: of equal lengths, or of any and padding behind them."""
    x = make(lens, 16, 4, seed=34, extra=2048 - sum(lens))
    n = sum(lens)
    want = oracle_of(x)
    for key in ("q", "k", "v", "g"):
        x[key][n:] = float("nan")
    d = dev(x)
    o = torch.full((2048, 16, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fs, status = torch.empty_like(d["s0"]), torch.ones(1, dtype=torch.int32, device="cuda")
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], x["scale"], o, fs, status)
    check(x, o, fs, want)
    assert int(status) == 0 and bool((o[n:] == 7.0).all())


def test_cut_sequences_with_states_in_place():
    """Long sequences in segments, shared heads, slices of one projection, the state's buffer updated: the same as apart."""
    x = make([3000, 40, 0, 1700], 4, 2, seed=35, rate=0.1)
    d = dev(x)
    want = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], check=True)
    check(x, *want)
    T = 4740
    qkv = torch.full((T, 8 * D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :2 * D].view(T, 2, D), qkv[:, 2 * D:4 * D].view(T, 2, D), qkv[:, 4 * D:8 * D].view(T, 4, D)
    q.copy_(d["q"]), k.copy_(d["k"]), v.copy_(d["v"])
    o = torch.empty_like(d["v"])
    kda.kda_linear_chunk_fwd(q, k, v, d["g"], d["cu"], d["s0"], x["scale"], o, d["s0"])
    assert torch.equal(o, want[0]) and torch.equal(d["s0"], want[1])


@pytest.mark.parametrize("lens,H", [([1] * 255 + [2049], 2), ([0] * 60 + [300, 64, 65, 1] + [2] * 5, 3), ([7] * 30 + [0, 90] + [1] * 3, 2),
                                    ([9] * 20, 2), ([64, 0, 0, 0, 0, 0, 0, 0], 2), ([0] * 7 + [65, 0], 2),
                                    ([0] * 800 + [6000, 1, 900], 1)])
def test_long_sequences_among_short_ones(lens, H):
    """Few tokens a sequence on average, but not in every one."""
    x = make(lens, H, H, seed=42, extra=5)
    x["g"][sum(lens):] = float("nan")
    d = dev(x)
    o = torch.full_like(d["v"], 7.0)
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], x["scale"], o, d["s0"], status)  # states in place
    x["g"][sum(lens):] = 0
    check(x, o, d["s0"])
    assert int(status) == 0 and bool((o[sum(lens):] == 7.0).all())


def test_a_sequence_decides_its_form_by_its_own_length():
    """A prompt among single tokens gives what it gives alone, and so do they: chunks and the recurrence round differently."""
    x = make([1] * 40 + [300], 2, 2, seed=43)
    d = dev(x)
    cut = lambda a, b: [d[key][a:b] for key in ("q", "k", "v", "g")]
    cu = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
    o, fs = kda.linear_chunk_fwd(*cut(0, 340), d["cu"], d["s0"], check=True)
    a = kda.linear_chunk_fwd(*cut(0, 40), cu(*range(41)), d["s0"][:40].contiguous(), check=True)
    b = kda.linear_chunk_fwd(*cut(40, 340), cu(0, 300), d["s0"][40:].contiguous(), check=True)
    assert torch.equal(o, torch.cat([a[0], b[0]])) and torch.equal(fs, torch.cat([a[1], b[1]]))


@pytest.mark.parametrize("cu", [[0] + [100] * 40 + [90, 200], [0, 150] + [100] * 40, [0] * 40 + [-5, 200], [0] * 40 + [210]])
def test_bad_offsets_of_a_batch_of_few_tokens(cu):
    """Reported, whatever form the valid ones run; rows of no valid sequence are left."""
    x = make([200], 2, 2, seed=44)
    d = dev(x)
    s0 = torch.zeros(len(cu) - 1, 2, D, D, device="cuda")
    o = torch.full_like(d["v"], 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], torch.tensor(cu, dtype=torch.int32, device="cuda"), s0, x["scale"], o,
                             torch.empty_like(s0), status)
    assert int(status) == kda.KDA_ERR_BAD_SEQLENS


@pytest.mark.parametrize("lens,H", [([17] * 1000, 16), ([0] * 300 + [2100, 1, 700] + [12] * 200, 4), ([5000, 4000, 300], 1),
                                    ([4000] + [20] * 500, 1)])
def test_workspace_holds_the_states_of_cut_sequences_alone(lens, H):
    """Its size does not grow by a state for every sequence, and nothing behind it is written."""
    T, N = sum(lens), len(lens)
    need = kda.linear_workspace_size(N, T, H)
    # a sequence is cut where it is longer than 4 chunks at least, into no more than twice its length over theirs
    assert need <= 2 * T // 512 * H * 4 * (D * D + 1) + (N + T // 512) * 64 + 4096
    rep = 4 if H == 16 else 1
    x = make(lens, H // rep, H // rep, seed=41)
    d = dev(x)
    d["g"], d["v"], d["s0"] = (d["g"].repeat(1, rep), d["v"].repeat(1, rep, 1), d["s0"].repeat(1, rep, 1, 1))
    d["q"], d["k"] = (d[key].repeat(1, rep, 1) for key in ("q", "k"))
    ws = torch.full((need + (1 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    o, fs = torch.empty_like(d["v"]), torch.empty_like(d["s0"])
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], x["scale"], o, fs, status, workspace=ws[:need])
    assert int(status) == 0 and bool((ws[need:] == 0x5a).all())
    check(x, o[:, :H // rep], fs[:, :H // rep])


def test_invalid_sequences_by_the_thousand():
    """Most of 70000 offsets out of range: those sequences are skipped and reported, the others computed."""
    N, T = 70000, 640010
    x = make([100, 2500], 1, 1, seed=37)
    d = dev(x)
    wide = lambda t: torch.cat([t, torch.zeros((T - 2600, *t.shape[1:]), dtype=t.dtype, device="cuda")])
    cu = torch.full((N + 1,), -1, dtype=torch.int32, device="cuda")
    cu[:2] = torch.tensor([0, 100])
    cu[-2:] = torch.tensor([100, 2600])
    o = torch.full((T, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_linear_chunk_fwd(wide(d["q"]), wide(d["k"]), wide(d["v"]), wide(d["g"]), cu, None, x["scale"], o, None, status)
    assert int(status) == kda.KDA_ERR_BAD_SEQLENS and bool((o[2600:] == 7.0).all())
    check(dict(x, s0=None), o[:2600], None)


def test_sequences_that_overlap_are_refused():
    """Offsets that go back and cover the rows several times: an error, and nothing is written."""
    x = make([3000], 1, 1, seed=36)
    d = dev(x)
    cu = torch.tensor([0, 3000] * 4, dtype=torch.int32, device="cuda")
    o = torch.full((3000, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    s0, fs = torch.zeros(7, 1, D, D, device="cuda"), torch.full((7, 1, D, D), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu, s0, x["scale"], o, fs, status)
    assert int(status) == kda.KDA_ERR_BAD_SEQLENS and bool((o == 7.0).all()) and bool((fs == 7.0).all())


def test_chunk_resets_inside_a_sequence():
    """-inf at some tokens forgets what was before; the rest decays slowly."""
    x = make([500, 77], 2, 2, seed=6, rate=0.05)
    x["g"][[3, 130, 131, 255, 256, 400, 510], :] = float("-inf")
    o, fs = chunk(x)
    check(x, o, fs)


def test_chunk_strided_projection():
    x = make([190, 33], 4, 2, seed=9)
    d = dev(x)
    qkv = torch.full((223, 2 * 2 * D + 4 * D + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :2 * D].view(223, 2, D), qkv[:, 2 * D:4 * D].view(223, 2, D), qkv[:, 4 * D:8 * D].view(223, 4, D)
    q.copy_(d["q"]), k.copy_(d["k"]), v.copy_(d["v"])
    o, fs = kda.linear_chunk_fwd(q, k, v, d["g"], d["cu"], d["s0"], check=True)
    check(x, o, fs)
    o2, fs2 = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], check=True)
    assert torch.equal(o, o2) and torch.equal(fs, fs2)


@pytest.mark.parametrize("lens", [[130, 20], [3, 1], [2000, 5]])
def test_rows_behind_the_last_sequence(lens):
    """Padding rows hold NaN on the way in and keep their values on the way out."""
    x = make(lens, 2, 2, seed=13, extra=150)
    n = sum(lens)
    want = oracle_of(x)
    for key in ("q", "k", "v", "g"):
        x[key][n:] = float("nan")
    d = dev(x)
    o = torch.full((n + 150, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fs = torch.empty_like(d["s0"])
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], x["scale"], o, fs, status)
    check(x, o, fs, want)
    assert int(status) == 0 and bool((o[n:] == 7.0).all())


def test_sequences_do_not_see_each_other():
    """NaN in one sequence (its last chunk shares rows with the next one's tile) stays in that sequence."""
    x = make([100, 70, 300], 2, 2, seed=14)
    clean = chunk(x)
    bad = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    for key in ("q", "k", "v"):
        bad[key][100:170] = float("nan")
    d = dev(bad)
    o, fs = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], scale=x["scale"])
    for part in (slice(0, 100), slice(170, 470)):
        assert torch.equal(o[part], clean[0][part])
    assert torch.equal(fs[[0, 2]], clean[1][[0, 2]])


def test_chunk_in_place_state_and_no_state_out():
    x = make([150, 0, 90], 2, 2, seed=15)
    d = dev(x)
    o = torch.empty_like(d["v"])
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], x["scale"], o, d["s0"])
    check(x, o, d["s0"])
    o2, none = chunk(x, output_final_state=False)
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("lens,H", [([700, 300], 2), ([5000], 1), ([2, 1, 3], 2)])
def test_chunk_is_deterministic_on_any_stream(lens, H):
    x = make(lens, H, H, seed=16)
    d = dev(x)
    a = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"])
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], stream=s[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for o, fs in got:
        assert torch.equal(o, a[0]) and torch.equal(fs, a[1])


def test_chunk_in_two_captured_graphs():
    """Two captured calls with workspaces of their own, replayed on two streams at once."""
    runs = []
    for seed, lens in ((21, [3000, 40]), (22, [900, 2500])):
        x = make(lens, 2, 2, seed=seed)
        d = dev(x)
        kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"])
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            out = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], scale=x["scale"])
        runs.append((x, d, graph, side, out))
    for _ in range(3):
        for _, _, graph, side, _ in runs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for x, _, _, _, (o, fs) in runs:
        check(x, o, fs)


def test_device_errors():
    x = make([130, 20], 2, 2, seed=17)
    for bad in (1e-3, float("nan"), float("inf")):
        y = dict(x, g=x["g"].clone())
        y["g"][140, 1] = bad
        with pytest.raises(kda.KdaError) as e:
            chunk(y)
        assert e.value.code == kda.KDA_ERR_GATE_RANGE
    for cu in ([0, 151, 150], [0, 130, 151], [1, 130, 150], [0, -5, 150]):
        with pytest.raises(kda.KdaError) as e:
            chunk(dict(x, cu=torch.tensor(cu, dtype=torch.int32)))
        assert e.value.code == kda.KDA_ERR_BAD_SEQLENS


@pytest.mark.parametrize("lens,H", [([300, 128, 70], 2), ([5000], 1)])
@pytest.mark.parametrize("g", [1e-9, 1e-6, 1e-3])
def test_a_gate_a_little_above_zero_is_reported_and_no_more(lens, H, g):
    """States grow by e^g then, as the formula has it: a rounding error in g does not lose them."""
    x = make(lens, H, H, seed=45)
    x["g"].fill_(g)
    d = dev(x)
    o, fs, status = torch.empty_like(d["v"]), torch.empty_like(d["s0"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], x["scale"], o, fs, status)
    assert int(status) == kda.KDA_ERR_GATE_RANGE
    check(x, o, fs)


@pytest.mark.parametrize("lens,at", [([300, 70, 129], 45), ([300, 70, 129], 200), ([300, 70, 129], 359), ([40, 6000], 3000),
                                     ([3, 5, 9], 5)])
def test_a_gate_that_is_no_number_shows(lens, at):
    """From the token of a NaN gate on its sequence and head are NaN, in every form; nothing else is touched by it."""
    x = make(lens, 2, 2, seed=40, rate=0.3)
    clean = chunk(x)
    want = oracle_of(x)
    x["g"][at, 1] = float("nan")
    d = dev(x)
    o, fs = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], scale=x["scale"])
    n = int(np.searchsorted(np.cumsum(lens), at, side="right"))
    end = sum(lens[:n + 1])
    assert bool(o[at:end, 1].isnan().all()) and bool(fs[n, 1].isnan().all())
    same = torch.ones(sum(lens), 2, dtype=torch.bool)
    same[end - lens[n]:end, 1] = False
    assert torch.equal(o[same.cuda()], clean[0][same.cuda()])
    o, fs = o.clone(), fs.clone()
    o[at:end, 1], fs[n, 1] = clean[0][at:end, 1], clean[1][n, 1]
    assert torch.equal(fs, clean[1])
    check(x, o, fs, want)  # its chunk's tokens in front of it, too


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("N,Tn,H,Hk,state,decay", [
    (1, 1, 1, 1, True, "token"), (7, 1, 16, 8, True, "head"), (64, 1, 16, 16, False, "token"), (5, 3, 4, 1, True, "token"),
    (3, 4, 16, 8, True, "head"), (2, 64, 2, 2, True, "token"), (3, 5, 5, 5, False, "head"), (2, 0, 3, 3, True, "token")])
def test_decode(N, Tn, H, Hk, state, decay):
    x = make([Tn] * N, H, Hk, seed=N + 10 * Tn + H, state=state, decay=decay)
    d = dev(x)
    o, fs = kda.linear_decode_fwd(d["q"], d["k"], d["v"], d["g"], N, d["s0"], check=True)
    check(x, o, fs, chunked=False)
    if state:
        o2, fs2 = kda.linear_decode_fwd(d["q"], d["k"], d["v"], d["g"], N, d["s0"], in_place=True)
        assert fs2 is d["s0"] and torch.equal(o, o2) and torch.equal(fs, fs2)


def test_decode_reports_bad_gates():
    x = make([1] * 3, 2, 2, seed=3)
    x["g"][1, 1] = 0.5
    d = dev(x)
    with pytest.raises(kda.KdaError) as e:
        kda.linear_decode_fwd(d["q"], d["k"], d["v"], d["g"], 3, d["s0"], check=True)
    assert e.value.code == kda.KDA_ERR_GATE_RANGE


def test_prompt_then_tokens():
    """Prefill 200 tokens, then decode two steps of two tokens from its state: the recurrence over all of them."""
    x = make([204, 204], 4, 2, seed=31)
    take = lambda t, a, b: torch.cat([t[:204][a:b], t[204:][a:b]]).cuda().contiguous()
    cu = torch.tensor([0, 200, 400], dtype=torch.int32, device="cuda")
    part = lambda a, b: [take(x[k], a, b) for k in ("q", "k", "v", "g")]
    o, s = kda.linear_chunk_fwd(*part(0, 200), cu, x["s0"].cuda(), check=True)
    outs = [o.view(2, 200, 4, D)]
    for a in (200, 202):
        o, s = kda.linear_decode_fwd(*part(a, a + 2), 2, s, in_place=True)
        outs.append(o.view(2, 2, 4, D))
    check(x, torch.cat(outs, 1).reshape(408, 4, D), s)
