"""GPU tests of the chunked delta rule on batches of thousands of short sequences: long ones among them are found, and finding out that there are
none, or few, costs little beside the sequences themselves."""
import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from oracle import delta as ref

pytestmark = pytest.mark.gpu
D, U = 128, 2.0 ** -8


def make(lens, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, N = sum(lens), len(lens)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    return {"q": unit(rand(T, H, D)), "k": unit(rand(T, H, D)), "v": rand(T, H, D).to(torch.bfloat16),
            "g": -torch.rand(T, H, device="cuda", generator=g), "beta": torch.rand(T, H, device="cuda", generator=g),
            "cu": torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda"), "s0": rand(N, H, D, D) * 0.3}


def call(x, **kw):
    return kda.gated_delta_chunk_fwd(*(x[n] for n in ("q", "k", "v", "g", "beta", "cu", "s0")), **kw)


@pytest.mark.parametrize("lens,H", [
    # more long sequences than the outputs' pass has CTAs for (an SM, four times), so that the last of them are run in rounds
    ([1] * 200 + [65, 128, 70, 100] * 40 + [0, 1, 2] * 300, 8),
    # more of them, and more of their chunks, than the plan holds lengths of
    (([3] * 3 + [0] + [65]) * 4200 + [0] * 3000, 1),
])
def test_many_long_sequences_among_short_ones(lens, H):
    x = make(lens, H, seed=len(lens))
    o, fs = call(x, check=True)
    again = call(x)
    assert torch.equal(again[0], o) and torch.equal(again[1], fs)
    cu = np.concatenate([[0], np.cumsum(lens)])
    rng = np.random.default_rng(0)
    long = [n for n, c in enumerate(lens) if c > 64]
    some = sorted({*rng.choice(long, 60), *rng.choice(len(lens), 60), long[0], long[-1], 0, len(lens) - 1})
    # every sequence against the recurrence's own entry point or the oracle is too slow: all finite, and these against fp64
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(fs).all())
    rows = np.concatenate([np.arange(cu[n], cu[n + 1]) for n in some])
    f = lambda t: t[torch.from_numpy(rows).cuda()].double().cpu().numpy()
    at = torch.tensor(some).cuda()
    ro, off, rs, soff = ref.recurrence(f(x["q"]), f(x["k"]), f(x["v"]), f(x["g"]), f(x["beta"]), [lens[n] for n in some],
                                       x["s0"][at].double().cpu().numpy(), D ** -0.5, 64)
    err, tol = np.abs(f(o) - ro), U * 1.001 * np.abs(ro) + off + 1e-30
    assert (err <= tol).all(), f"o: {np.max(err / tol):.3g} of the bound"
    err, tol = np.abs(fs[at].double().cpu().numpy() - rs), soff[:, :, None, :] + 2 * ref.F * np.abs(rs) + 1e-30
    assert (err <= tol).all(), f"final state: {np.max(err / tol):.3g} of the bound"


def test_every_sequence_of_a_batch_with_many_long_ones():
    """Each sequence alone against its place in the batch: the long ones by the same kernels, uncut; the short ones by the recurrence."""
    lens, H = [1] * 200 + [65, 128, 70, 100] * 40 + [0, 1, 2] * 300, 8
    x = make(lens, H, seed=5)
    o, fs = call(x, check=True)
    cu = np.concatenate([[0], np.cumsum(lens)])
    long = [n for n, c in enumerate(lens) if c > 64]
    rows = torch.from_numpy(np.concatenate([np.arange(cu[n], cu[n + 1]) for n in long])).cuda()
    at = torch.tensor(long).cuda()
    one = {k: x[k][rows] for k in ("q", "k", "v", "g", "beta")}
    one["cu"] = torch.tensor(np.concatenate([[0], np.cumsum([lens[n] for n in long])]), dtype=torch.int32, device="cuda")
    one["s0"] = x["s0"][at]
    po, ps = call(one, check=True)
    # (two forms of the same sums: the state within 2 x 2^-15 of its size, o within two roundings of its own and of what the scores lose)
    assert float((fs[at] - ps).norm() / ps.norm()) <= 2.0 ** -14 and float((o[rows].float() - po.float()).norm() / po.float().norm()) <= 2.0 ** -7


def best_of(f, n=5):
    f()
    times = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


def test_short_sequences_take_the_recurrences_time():
    """20,000 sequences of one token: what the prompt call adds to the recurrence, which reads and writes every state, is a small part. (Where
    each of its CTAs looked through all bounds, it took twice as long.)"""
    N, H = 20000, 2
    x = make([1] * N, H, seed=6)
    o, fs = call(x, check=True)
    do, ds = kda.gated_delta_decode_fwd(*(x[n] for n in ("q", "k", "v", "g", "beta")), N, x["s0"], check=True)
    assert torch.equal(o, do) and torch.equal(fs, ds)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    chunk = best_of(lambda: kda.kda_gated_delta_chunk_fwd(*args, x["cu"], x["s0"], D ** -0.5, o, fs))
    steps = best_of(lambda: kda.kda_gated_delta_decode_fwd(*args, N, x["s0"], D ** -0.5, o, fs))
    assert chunk <= 1.35 * steps, (chunk, steps)


def test_a_captured_call_finds_the_long_ones_anew():
    """The same graph on other bounds: which sequences are long, whether any is, and whether bounds are in order, is found at each replay. Two
    graphs with workspaces of their own, replayed at once on two streams."""
    T, N, H = 1500, 300, 2
    rng = np.random.default_rng(3)
    batch = lambda *long: [*long, *rng.multinomial(T - sum(long), np.full(N - len(long), 1 / (N - len(long)))).tolist()]
    batches = [batch(900, 130, 65), batch(), batch(64, 66, 700), [0] * (N - 1) + [T], batch(65)]
    x = make(batches[0], H, seed=7)
    names = ("q", "k", "v", "g", "beta")
    cu = [torch.tensor(np.concatenate([[0], np.cumsum(b)]), dtype=torch.int32, device="cuda") for b in batches]
    assert all(sum(b) == T and len(b) == N for b in batches)
    want = [kda.gated_delta_chunk_fwd(*(x[n] for n in names), c, x["s0"], check=True) for c in cu]
    held, graphs = [cu[0].clone(), cu[1].clone()], []
    torch.cuda.synchronize()
    for h in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = kda.gated_delta_chunk_fwd(*(x[n] for n in names), h, x["s0"])
        graphs.append((g, out))
    bad = cu[2].clone()
    bad[150] = 10 ** 6
    streams = [torch.cuda.Stream() for _ in graphs]
    for i in range(2 * len(cu)):
        at = [(i + j) % len(cu) for j in range(2)]
        for h, a in zip(held, at):
            h.copy_(bad if i == 3 else cu[a])
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, out), a in zip(graphs, at):
            if i != 3:
                assert torch.equal(out[0], want[a][0]) and torch.equal(out[1], want[a][1])
