"""GPU tests of the failure detection: an operand that is not handed on makes bounded waits run out, the status says so, every block
leaves and the context stays usable."""
import pytest
import torch

import kda_chunked_prefill_gb300 as kda

pytestmark = pytest.mark.gpu


def delta_inputs():
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(700, 2, 128, device="cuda", generator=g).mul_(0.09).to(torch.bfloat16) for _ in range(3))
    gate = -torch.rand(700, 2, device="cuda", generator=g)
    beta = torch.rand(700, 2, device="cuda", generator=g)
    return q, k, v, gate, beta, torch.tensor([0, 200, 700], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("withhold", [0, 2])
def test_delta_chunks_time_out_and_the_next_call_is_right(withhold):
    x = delta_inputs()
    want = kda.gated_delta_chunk_fwd(*x, check=True)
    o, fs = torch.empty_like(x[2]), torch.empty(2, 2, 128, 128, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_gated_delta_chunk_fwd(*x, None, 128 ** -0.5, o, fs, status, withhold=withhold)
    assert int(status) == kda.KDA_ERR_TIMEOUT
    got = kda.gated_delta_chunk_fwd(*x, check=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_delta_states_of_cut_sequences_time_out():
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(6000, 1, 128, device="cuda", generator=g).mul_(0.09).to(torch.bfloat16) for _ in range(3))
    x = (q, k, v, torch.zeros(6000, 1, device="cuda"), torch.rand(6000, 1, device="cuda", generator=g),
         torch.tensor([0, 6000], dtype=torch.int32, device="cuda"))
    want = kda.gated_delta_chunk_fwd(*x, check=True)
    o, fs = torch.empty_like(v), torch.empty(1, 1, 128, 128, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_gated_delta_chunk_fwd(*x, None, 128 ** -0.5, o, fs, status, withhold=1)
    assert int(status) == kda.KDA_ERR_TIMEOUT
    got = kda.gated_delta_chunk_fwd(*x, check=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,N,K", [(7, 2048, 2048), (40, 256, 640), (300, 640, 640), (9000, 2304, 640)])
@pytest.mark.parametrize("withhold", [0, 1])
def test_products_time_out_and_the_next_call_is_right(T, N, K, withhold):
    """(Groups of four blocks; a block of threads with one group only withholds nothing at 1.)"""
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = (torch.randn(n, K, device="cuda", generator=g).to(torch.float8_e4m3fn) for n in (T, N))
    xs, ws = torch.rand(T, device="cuda"), torch.rand(-(-N // 128), K // 128, device="cuda")
    want = kda.scaled_matmul(x, xs, w, ws, check=True)
    y, status = torch.empty_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_scaled_matmul(x, xs, w, ws, y, status, withhold=withhold)
    assert int(status) == kda.KDA_ERR_TIMEOUT or (withhold == 1 and T <= 64 and torch.equal(y, want))
    assert torch.equal(kda.scaled_matmul(x, xs, w, ws, check=True), want)
