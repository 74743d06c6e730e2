"""GPU tests of the chunked delta rule with one decay per head on malformed batches: bounds that run backwards or out of range are reported, the
sequences that they belong to are skipped, and every other one gets its own result, whatever the workspace held before.

Bounds element by element as in the tests of well-formed batches: oracle/delta.py derives them. (A row of two overlapping sequences may hold
either's output.)
"""
import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from oracle import delta as ref

pytestmark = pytest.mark.gpu
D, U, UNTOUCHED = 128, 2.0 ** -8, 7.0


def make(T, N, H, Hk, seed):
    rng = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    q, k = (torch.from_numpy(unit(rng.standard_normal((T, Hk, D)))).to(torch.bfloat16) for _ in range(2))
    return {"q": q, "k": k, "v": torch.from_numpy(rng.standard_normal((T, H, D))).to(torch.bfloat16),
            "g": torch.from_numpy(-0.2 * rng.random((T, H))).float(),
            "beta": torch.from_numpy(rng.random((T, H))).float(),
            "s0": torch.from_numpy(rng.standard_normal((N, H, D, D)) * 0.3).float()}


def bounds(lens, **changed):
    cu = [0] + np.cumsum(lens).tolist()
    for at, value in changed.items():
        cu[int(at[1:])] = value
    return cu, sum(lens)


LONG_AMONG_SHORT = [2] * 40 + [700] + [0, 1, 3] * 50 + [65] + [2] * 60 + [130, 64] + [1] * 40
CASES = {
    # a long sequence, one that runs backwards, and one inside the first's rows
    "inside_another": ([0, 1000, 10, 230], 1000),
    "past_the_rows": bounds([100] * 64, b10=7000),
    "past_the_rows_odd": bounds([100] * 64, b11=10 ** 9),
    "negative": bounds([100] * 64, b32=-1),
    "backwards": bounds([100] * 64, b20=1750),
    "several": bounds([70, 129, 0, 64] * 20, b6=-2 ** 31, b33=2 ** 31 - 1, b34=0, b62=5260),
    "the_last": bounds([100] * 40, b40=4001),
    "a_long_one": bounds([3000, 0, 500, 40], b3=9999),
    "not_from_zero": bounds([100, 200], b0=3),
    "long_among_short": bounds(LONG_AMONG_SHORT, b20=10 ** 6),
    "long_among_short_backwards": bounds(LONG_AMONG_SHORT, b100=0, b261=5),
    "all_overlap": ([0, 600] * 50 + [600], 600),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_what_is_not_malformed_is_right(name, in_place):
    cu, T = CASES[name]
    N, H = len(cu) - 1, 2
    x = make(T, N, H, 1, seed=len(name))
    well = [n for n in range(N) if cu[0] == 0 and 0 <= cu[n] <= cu[n + 1] <= T]
    assert len(well) < N
    d = {n: t.cuda() for n, t in x.items()}
    need = kda.gated_delta_workspace_size(N, T, H)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    o = torch.full_like(d["v"], UNTOUCHED)
    fs = d["s0"] if in_place else torch.full_like(d["s0"], UNTOUCHED)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                  d["s0"], D ** -0.5, o, fs, status, workspace=ws[:need])
    assert int(status) == kda.KDA_ERR_BAD_SEQLENS and bool((ws[need:] == 255).all())

    o, fs = o.double().cpu().numpy(), fs.double().cpu().numpy()
    of = np.zeros(T, dtype=int)  # sequences that a row belongs to
    for n in well:
        of[cu[n]:cu[n + 1]] += 1
    assert (o[of == 0] == UNTOUCHED).all()
    skipped = [n for n in range(N) if n not in well]
    assert (fs[skipped] == (x["s0"].double().numpy()[skipped] if in_place else UNTOUCHED)).all()
    seen = {}
    for n in well:
        a, b = cu[n], cu[n + 1]
        if name == "all_overlap" and n not in well[:3] + well[-3:]:
            continue
        f = lambda t: t[a:b].double().numpy()
        ro, off, rs, soff = ref.recurrence(*(f(x[i]) for i in ("q", "k", "v", "g", "beta")), [b - a],
                                           x["s0"][n:n + 1].double().numpy(), D ** -0.5, 64)
        err, tol = np.abs(fs[n] - rs[0]), soff[0][:, None, :] + 2 * ref.F * np.abs(rs[0]) + 1e-30
        assert np.isfinite(fs[n]).all() and (err <= tol).all(), f"final state of {n}: {np.max(err / tol):.3g} of the bound"
        alone = of[a:b] == 1
        err, tol = np.abs(o[a:b] - ro), U * 1.001 * np.abs(ro) + off + 1e-30
        assert np.isfinite(o[a:b]).all() and (err <= tol)[alone].all(), f"o of {n}: {np.max((err / tol)[alone]):.3g} of the bound"
        seen[n] = a, b
    assert len(seen) >= min(len(well), 6)


def test_the_next_call_is_not_touched():
    """A malformed batch leaves nothing behind for a well-formed one in the same workspace."""
    x = make(2000, 4, 2, 2, seed=1)
    d = {n: t.cuda() for n, t in x.items()}
    need = kda.gated_delta_workspace_size(4, 2000, 2)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    o, fs, status = torch.empty_like(d["v"]), torch.empty_like(d["s0"]), torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(cu):
        kda.kda_gated_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                      d["s0"], D ** -0.5, o, fs, status, workspace=ws)
        return int(status), o.clone(), fs.clone()

    good = [0, 700, 700, 1900, 2000]
    want = call(good)
    assert want[0] == 0 and call([0, 700, 3000, 1900, 2000])[0] == kda.KDA_ERR_BAD_SEQLENS
    got = call(good)
    assert got[0] == 0 and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
