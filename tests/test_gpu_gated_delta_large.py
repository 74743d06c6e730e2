"""GPU tests of the gated delta rule, the gated norm and the e4m3 product on tensors of more than 2^31 elements: what lies far behind the start is
the same as in a call of its own. (Bit for bit where the same form computes it; else within both calls' roundings: o and y 2 x 2^-8, states
2 x 2^-16, and as much again.)"""
import pytest
import torch

import kda_chunked_prefill_gb300 as kda

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def bf16(*shape, size=1.0):
    x = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    for part in x.split(1 << 14):
        part.normal_(0, size)
    return x


def test_prompts_far_behind_the_start():
    """The last sequences of 270,000 tokens of 64 heads, 2.2 * 10^9 elements, q and k as slices of one tensor of 3.3 * 10^9."""
    H, Hk, last = 64, 16, [700, 64, 0, 1, 130]
    lens = [1000] * 269 + last
    T = sum(lens)
    torch.manual_seed(0)
    qk = bf16(T, (2 * Hk + 64) * D, size=0.088)
    q, k = (qk[:, i * Hk * D:(i + 1) * Hk * D].view(T, Hk, D) for i in range(2))
    v = bf16(T, H, D)
    g, beta = -0.1 * torch.rand(T, H, device="cuda"), torch.rand(T, H, device="cuda")
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    assert v.numel() > 2 ** 31 and qk.numel() > 2 ** 31
    o, fs = kda.gated_delta_chunk_fwd(q, k, v, g, beta, cu, check=True)
    n, own = sum(last), torch.tensor([0] + torch.tensor(last).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    part = [t[T - n:].contiguous() for t in (q, k, v, g, beta)]
    po, ps = kda.gated_delta_chunk_fwd(*part, own, check=True)
    assert float((o[T - n:].float() - po.float()).norm() / po.float().norm()) <= 2.0 ** -7
    assert float((fs[-len(last):] - ps).norm() / ps.norm()) <= 2.0 ** -14
    assert bool(torch.isfinite(o[T - n:]).all())
    # the same rows token after token
    m = [i for i, c in enumerate(last) if c == 1][0]
    at = T - n + sum(last[:m])
    do, ds = kda.gated_delta_decode_fwd(*(t[at:at + 1].contiguous() for t in (q, k, v, g, beta)), 1)
    assert float((o[at].float() - do[0].float()).abs().max()) <= 2.0 ** -6 * float(do.float().abs().max())
    # the norm of these rows, gated by v
    w = torch.rand(D, device="cuda")
    y, scale = kda.gated_rms_norm(o, v, w, activation="silu")
    py, pscale = kda.gated_rms_norm(o[T - n:].contiguous(), v[T - n:].contiguous(), w, activation="silu")
    assert torch.equal(y[T - n:].view(torch.uint8), py.view(torch.uint8)) and torch.equal(scale[T - n:], pscale)


def test_steps_far_behind_the_start():
    """66,000 sequences of 2 heads: 2.2 * 10^9 elements of states."""
    N, H = 66000, 2
    torch.manual_seed(1)
    q, k, v = (bf16(N, H, D, size=0.1) for _ in range(3))
    g, beta, s = -torch.rand(N, H, device="cuda"), torch.rand(N, H, device="cuda"), torch.empty(N, H, D, D, device="cuda")
    for part in s.split(1000):
        part.normal_()
    assert s.numel() > 2 ** 31
    before = s[-3:].clone()
    o, fs = kda.gated_delta_decode_fwd(q, k, v, g, beta, N, s, in_place=True, check=True)
    po, ps = kda.gated_delta_decode_fwd(*(t[-3:].contiguous() for t in (q, k, v, g, beta)), 3, before)
    assert torch.equal(o[-3:], po) and torch.equal(fs[-3:], ps)


@pytest.mark.parametrize("T,N,K", [(700000, 4096, 128), (40, 12345, 256)])
def test_products_far_behind_the_start(T, N, K):
    """2.9 * 10^9 outputs; and weights of 2.2 * 10^9 codes."""
    K = K if T > 64 else 180224
    torch.manual_seed(2)
    make = lambda r: torch.randint(0, 120, (r, K), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    x, w, xs, ws = make(T), make(N), torch.rand(T, device="cuda"), torch.rand(-(-N // 128), -(-K // 128), device="cuda")
    assert T * N > 2 ** 31 or N * K > 2 ** 31
    y = kda.scaled_matmul(x, xs, w, ws, check=True)
    if T > 64:
        p = kda.scaled_matmul(x[-2560:].contiguous(), xs[-2560:].contiguous(), w, ws, check=True)
        y = y[-2560:]
    else:
        rows = N // 128 * 128 - 256  # whole groups of outputs before the last ones, in other tiles of another call
        p = kda.scaled_matmul(x, xs, w[rows:].contiguous(), ws[rows // 128:].contiguous(), check=True)
        y = y[:, rows:]
    assert float((y.float() - p.float()).abs().max()) <= 2.0 ** -7 * float(p.float().abs().max())
