"""The bound on the chunked delta rule's outputs lets the kernel's roundings through and no others: a host emulation with operands in two bf16
terms is inside, one that drops the second term of the state that q multiplies, or of the z that P T multiplies, is not (no GPU).

The 2-norm's limit, 1.1: U / 2.3 is a rounding's mean over the values that these sums have, to a few per cent. The fewest values are P T's in chunks of
one token, 128 with one rounding each, whose squares spread by 0.9 of their mean: 8 % of the mean of 128, a third of the variance, 1.3 % of the norm.
"""
import numpy as np
import pytest

import delta_util as du
from oracle import delta as ref

CASES = du.sharp_cases()
SCALE = 128 ** -0.5


def against(name, **kw):
    """The emulation's error: the largest in parts of the bound, element by element; its 2-norm in parts of what the roundings add up to."""
    x, lens, s0 = CASES[name]
    ro, off, rs, soff = ref.recurrence(*(x[n] for n in ("q", "k", "v", "g", "beta")), lens, s0, SCALE, 64)
    o, S, norm = du.emulate(x, lens, s0, SCALE, **kw)
    assert (np.abs(S - rs) <= soff[:, :, None, :] + 2 * ref.F * np.abs(rs)).all()
    err = np.abs(o - ro)
    return np.max(err / (du.U * 1.001 * np.abs(ro) + off + 1e-30)), np.linalg.norm(err) / norm


@pytest.mark.parametrize("name", list(CASES))
def test_two_terms_are_inside(name):
    most, norm = against(name)
    assert most <= 1 and norm <= 1.1


def test_one_term_of_the_state_is_not():
    assert against("state", q_state=1)[0] > 1
    assert against("state", q_state=1)[1] > 1.1


def test_one_term_of_what_a_chunk_adds_is_not():
    assert against("single", z_out=1)[0] > 1
    for name in ("single", "own", "ordinary"):
        assert against(name, z_out=1)[1] > 1.1
