"""GPU tests of the chunked delta rule's roundings: o has its own and that of P T, and no operand that depends on the state loses its second
bf16 term. 2-norms against fp64 in parts of what these roundings add up to (tests/delta_util.py; 1.1 as derived in test_host_delta_bound.py,
where dropping a term gives 1.13 to 1.4), element by element against the bound."""
import numpy as np
import pytest
import torch

import delta_util as du
import kda_chunked_prefill_gb300 as kda
from oracle import delta as ref

pytestmark = pytest.mark.gpu
CASES = {n: c for n, c in du.sharp_cases().items() if n != "single"}  # (that batch is run by the recurrence)
SCALE = 128 ** -0.5


@pytest.mark.parametrize("name", list(CASES))
def test_no_term_is_dropped(name):
    x, lens, s0 = CASES[name]
    t = lambda a, kind: torch.from_numpy(np.ascontiguousarray(a)).to(kind).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    o, fs = kda.gated_delta_chunk_fwd(*(t(x[n], torch.bfloat16) for n in ("q", "k", "v")), *(t(x[n], torch.float32) for n in ("g", "beta")),
                                      cu, t(s0, torch.float32), scale=SCALE, check=True)
    ro, off, rs, soff = ref.recurrence(*(x[n] for n in ("q", "k", "v", "g", "beta")), lens, s0, SCALE, 64)
    err = np.abs(o.double().cpu().numpy() - ro)
    assert (err <= du.U * 1.001 * np.abs(ro) + off + 1e-30).all()
    assert np.linalg.norm(err) <= 1.1 * du.emulate(x, lens, s0, SCALE)[2]
    s = np.abs(fs.double().cpu().numpy() - rs)
    assert (s <= soff[:, :, None, :] + 2 * ref.F * np.abs(rs)).all()
    assert np.linalg.norm(s) <= 2.0 ** -16 * np.linalg.norm(rs)


def test_the_same_call_gives_the_same_bits():
    """Cuts and the order in which segments are listed do not change the sums."""
    g = torch.Generator(device="cuda").manual_seed(0)
    lens, H = [3000, 40, 0, 1700, 1, 6000], 3
    T = sum(lens)
    q, k, v = (torch.randn(T, H, 128, device="cuda", generator=g).mul_(0.088).to(torch.bfloat16) for _ in range(3))
    args = (q, k, v, -0.1 * torch.rand(T, H, device="cuda", generator=g), torch.rand(T, H, device="cuda", generator=g),
            torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda"),
            torch.randn(len(lens), H, 128, 128, device="cuda", generator=g))
    want = kda.gated_delta_chunk_fwd(*args, check=True)
    for _ in range(10):
        got = kda.gated_delta_chunk_fwd(*args)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
