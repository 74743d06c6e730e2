"""GPU tests that the plain calls (native code, without a stream and a check) are the general ones: the same bits, the same refusals, the
states in place."""
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from kda_chunked_prefill_gb300 import _lib

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def built():
    _lib.load_library(build_if_missing=True)
    if _lib._native is None:
        pytest.skip("the native calls are not built")


def qkv(T, Hk, H, strided):
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    wide = torch.randn(T, (2 * Hk + H) * D + 16, device="cuda", generator=gen).mul_(0.09).to(torch.bfloat16)
    q, k, v = (wide[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, Hk), (Hk, 2 * Hk), (2 * Hk, 2 * Hk + H)))
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return q, k, v, -torch.rand(T, H, device="cuda", generator=gen), torch.rand(T, H, device="cuda", generator=gen)


def both(call, monkeypatch):
    """The call's outputs as native code, which must have taken it, and in general; a refusal by what it raises."""
    seen = []

    class Spy:
        def __getattr__(self, name):
            f = getattr(native, name)
            return lambda *a: seen.append(f(*a)) or seen[-1]

    def run():
        try:
            return call()
        except Exception as e:
            return type(e), getattr(e, "code", None), str(e)

    native = _lib._native
    monkeypatch.setattr(_lib, "_native", Spy())
    a = run()
    monkeypatch.setattr(_lib, "_native", None)
    b = run()
    monkeypatch.setattr(_lib, "_native", native)
    assert len(seen) == 1
    return a, b, seen[0]


def same(a, b):
    if isinstance(a, torch.Tensor):
        return a.dtype is b.dtype and a.shape == b.shape and a.is_contiguous() and torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    if isinstance(a, tuple):
        return len(a) == len(b) and all(same(x, y) for x, y in zip(a, b))
    return a is b or a == b


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("T,Hk,H", [(1, 1, 1), (3, 1, 2), (150, 2, 4)])
def test_same_outputs(T, Hk, H, strided, monkeypatch):
    q, k, v, g, beta = qkv(T, Hk, H, strided)
    cu = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    s0 = torch.randn(2, H, D, D, device="cuda")
    w = torch.rand(D, device="cuda")
    x = torch.randint(0, 120, (T, 4, 2 * D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    m = torch.randint(0, 120, (300, 2 * D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ws = torch.rand(3, 2, device="cuda")
    state = torch.randn(T, H, D, D, device="cuda")
    for call in (lambda: kda.gated_delta_chunk_fwd(q, k, v, g, beta, cu, s0),
                 lambda: kda.gated_delta_chunk_fwd(q, k, v, g, beta, cu, scale=0.3, output_final_state=False),
                 lambda: kda.gated_delta_decode_fwd(q, k, v, g, beta, T, state),
                 lambda: kda.gated_delta_decode_fwd(q, k, v, g, beta, T, scale=0.5),
                 lambda: kda.gated_rms_norm(v.contiguous(), v, w, 1e-6),
                 lambda: kda.gated_rms_norm(v.float().contiguous(), v, w, activation="silu"),
                 lambda: kda.scaled_matmul(x, torch.ones(T, 4, device="cuda"), m, ws),
                 lambda: kda.scaled_matmul(x, torch.ones(T, 4, 2, device="cuda"), m, ws),
                 lambda: kda.scaled_matmul(x[0, 0], torch.ones(2, device="cuda"), m, ws)):
        a, b, native = both(call, monkeypatch)
        assert native is not None and same(a, b)


def test_states_in_place(monkeypatch):
    q, k, v, g, beta = qkv(6, 2, 2, False)
    s0 = torch.randn(3, 2, D, D, device="cuda")
    want = kda.gated_delta_decode_fwd(q, k, v, g, beta, 3, s0.clone())
    o, s = kda.gated_delta_decode_fwd(q, k, v, g, beta, 3, s0, in_place=True)
    assert s is s0 and torch.equal(s, want[1]) and torch.equal(o, want[0])


def test_same_refusals(monkeypatch):
    q, k, v, g, beta = qkv(6, 2, 2, False)
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    w = torch.rand(D, device="cuda")
    x = torch.zeros(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
    ones = torch.ones(4, device="cuda")
    chunk, decode = kda.gated_delta_chunk_fwd, kda.gated_delta_decode_fwd
    for call, refused_by in (
            (lambda: chunk(q.float(), k, v, g, beta, cu), None), (lambda: chunk(q, k[:5], v, g, beta, cu), None),
            (lambda: chunk(q, k, v, g.double(), beta, cu), None), (lambda: chunk(q, k, v, g, beta.t(), cu), None),
            (lambda: chunk(q, k, v, g, beta, cu.long()), None), (lambda: chunk(q, k, v, g, beta, cu.cpu()), None),
            (lambda: chunk(q.cpu(), k, v, g, beta, cu), None), (lambda: chunk(q, k, v[:, :1], g[:, :1], beta[:, :1], cu), None),
            (lambda: chunk(q, k, v, g, beta, cu, w), None), (lambda: chunk(q, k, v, g, beta, cu, scale=float("nan")), int),
            (lambda: chunk(q[..., ::2], k, v, g, beta, cu), None), (lambda: decode(q, k, v, g, beta, 4), None),
            (lambda: decode(q, k, v, g, beta, 6, in_place=True), None), (lambda: decode(q, k, v, g, beta, -1), None),
            (lambda: kda.gated_rms_norm(v, v[:, :1], w), None), (lambda: kda.gated_rms_norm(v, v, w, 0.0), int),
            (lambda: kda.gated_rms_norm(v.half(), v, w), None), (lambda: kda.scaled_matmul(x, ones[:3], x, ones.view(2, 2)), None),
            (lambda: kda.scaled_matmul(x[:, :248].contiguous(), ones, x[:, :248].contiguous(), ones[:2].view(1, 2)), int),
            (lambda: kda.scaled_matmul(x.t(), ones, x, ones[:2].view(1, 2)), None)):
        a, b, native = both(call, monkeypatch)
        assert isinstance(a[0], type) and issubclass(a[0], Exception) and a == b
        assert native is None if refused_by is None else type(native) is refused_by


def test_captured():
    q, k, v, g, beta = qkv(140, 2, 2, True)
    cu = torch.tensor([0, 100, 140], dtype=torch.int32, device="cuda")
    call = lambda: kda.gated_delta_chunk_fwd(q, k, v, g, beta, cu)
    want = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = call()
    other.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
