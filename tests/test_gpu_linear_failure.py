"""Failure detection of the chunked linear attention, tested without a GPU fault.

Every wait inside the kernel is bounded, and a role whose wait runs out leaves; the others meet it at no barrier without a limit
but the pass's end, to which all come. Here the decays of some chunk's values are withheld (in the pass over cut sequences' states
or in that over the outputs), so v~, then U, P v and the output, for which the scores' and the state's warps wait, run out after
two seconds at most: the device reports KDA_ERR_TIMEOUT, and the same context, with the same workspace, then runs a normal call that
is right."""
import time

import pytest
import torch

import kda_chunked_prefill_gb300 as kda

from test_gpu_linear import check, dev, make

pytestmark = pytest.mark.gpu

WHOLE, CUT = ([256, 512, 128], 2), ([6000, 40, 1300], 1)


@pytest.mark.parametrize("lens,H,withhold", [
    (*WHOLE, (-1, 0)), (*WHOLE, (-1, 1)),
    ([130, 64, 210], 4, (-1, 1)),                                  # chunks that are not full
    ([256, 130, 384, 256], 96, (-1, 3)), ([256, 130, 384, 256], 96, (-1, 5)),  # tasks in a row
    ([512] * 4, 16, (-1, 2)),                                      # equal lengths
    (*CUT, (0, -1)), (*CUT, (2, -1)), (*CUT, (-1, 0)), (*CUT, (-1, 2))])
def test_withheld_decays_time_out_and_the_context_stays_usable(lens, H, withhold):
    x = make(lens, H, H, seed=60)
    d = dev(x)
    T, N = sum(lens), len(lens)
    ws = torch.empty(max(256, kda.linear_workspace_size(N, T, H)), dtype=torch.uint8, device="cuda")
    o, fs = torch.empty_like(d["v"]), torch.empty_like(d["s0"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.monotonic()
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], x["scale"], o, fs, status, workspace=ws,
                             withhold=withhold)
    torch.cuda.synchronize()
    elapsed = time.monotonic() - t0
    assert int(status) == kda.KDA_ERR_TIMEOUT
    assert elapsed < 20.0, f"the timed-out launch took {elapsed:.1f} s"
    kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], x["scale"], o, fs, status, workspace=ws)
    assert int(status) == kda.KDA_OK
    check(x, o, fs)


def test_nothing_withheld_is_the_ordinary_call():
    x = make([300, 70], 2, 2, seed=61)
    d = dev(x)
    want = kda.linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], check=True)
    for withhold in ((-1, -1), (-1, 1000)):
        o, fs = torch.empty_like(d["v"]), torch.empty_like(d["s0"])
        kda.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["s0"], x["scale"], o, fs, withhold=withhold)
        assert torch.equal(o, want[0]) and torch.equal(fs, want[1])
