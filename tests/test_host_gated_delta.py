"""Host-side refusals of the gated-delta, gated-norm and scaled-product entry points (no GPU: validation runs before any CUDA call),
the binding's checks of tensors, and pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from kda_chunked_prefill_gb300 import _lib
from oracle import delta as ref

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
OFF2, OFF8 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10008)
NAN = float("nan")
INVALID, UNSUPPORTED = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _lib.load_library(build_if_missing=True)


def _chunk(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, cu=FAKE, N=2, T=100, H=4, Hk=2, dk=128, dv=128, qs=256, ks=256, vs=512,
             s0=None, scale=0.1, o=FAKE, sT=None, status=None, ws=None, wsb=0)
    a.update(over)
    return lib.kda_gated_delta_chunk_fwd(*[a[k] for k in ("q", "k", "v", "g", "beta", "cu", "N", "T", "H", "Hk", "dk", "dv", "qs",
                                                          "ks", "vs", "s0", "scale", "o", "sT", "status", "ws", "wsb")], None)


def _decode(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, N=2, Tn=1, H=4, Hk=2, dk=128, dv=128, qs=256, ks=256, vs=512, s0=None,
             scale=0.1, o=FAKE, sT=None, status=None)
    a.update(over)
    return lib.kda_gated_delta_decode_fwd(*[a[k] for k in ("q", "k", "v", "g", "beta", "N", "Tn", "H", "Hk", "dk", "dv", "qs", "ks",
                                                           "vs", "s0", "scale", "o", "sT", "status")], None)


BAD = [({"dk": 64}, UNSUPPORTED), ({"dv": 256}, UNSUPPORTED), ({"H": 0}, INVALID), ({"Hk": 0}, INVALID),
       ({"Hk": 3, "qs": 384, "ks": 384}, INVALID), ({"N": -1}, INVALID), ({"qs": 248}, INVALID), ({"ks": 260}, INVALID),
       ({"vs": 504}, INVALID), ({"vs": 1 << 60}, UNSUPPORTED), ({"scale": NAN}, INVALID), ({"q": None}, INVALID),
       ({"g": None}, INVALID), ({"beta": None}, INVALID), ({"beta": OFF2}, INVALID), ({"o": None}, INVALID), ({"k": OFF8}, INVALID),
       ({"s0": OFF8}, INVALID), ({"sT": OFF8}, INVALID), ({"status": OFF2}, INVALID), ({"N": 2 ** 30, "H": 4}, INVALID)]


@pytest.mark.parametrize("over,code", BAD + [({"T": -1}, INVALID), ({"cu": None}, INVALID), ({"T": 2 ** 31}, UNSUPPORTED),
                                             ({"cu": OFF2}, INVALID)])
def test_chunk_refuses(lib, over, code):
    assert _chunk(lib, **over) == code


@pytest.mark.parametrize("over,code", BAD + [({"Tn": -1}, INVALID), ({"Tn": 65}, INVALID)])
def test_decode_refuses(lib, over, code):
    assert _decode(lib, **over) == code


def _norm(lib, **over):
    a = dict(x=FAKE, gate=FAKE, gs=512, w=FAKE, T=3, H=4, dv=128, eps=1e-5, fp32=0, silu=0, y=FAKE, ys=FAKE)
    a.update(over)
    return lib.kda_gated_rms_norm(*[a[k] for k in ("x", "gate", "gs", "w", "T", "H", "dv", "eps", "fp32", "silu", "y", "ys")], None)


@pytest.mark.parametrize("over,code", [
    ({"dv": 64}, UNSUPPORTED), ({"T": -1}, INVALID), ({"T": 2 ** 40}, UNSUPPORTED), ({"H": 0}, INVALID), ({"eps": 0.0}, INVALID),
    ({"eps": NAN}, INVALID), ({"eps": 1e-42}, INVALID), ({"fp32": 2}, INVALID), ({"silu": -1}, INVALID), ({"gs": 504}, INVALID), ({"gs": 516}, INVALID),
    ({"gs": 2 ** 40}, UNSUPPORTED), ({"x": None}, INVALID), ({"gate": OFF8}, INVALID), ({"w": OFF8}, INVALID), ({"y": OFF8}, INVALID),
    ({"ys": OFF2}, INVALID), ({"ys": None}, INVALID)])
def test_norm_refuses(lib, over, code):
    assert _norm(lib, **over) == code


def _product(lib, **over):
    a = dict(x=FAKE, xs=FAKE, per=1, w=FAKE, ws=FAKE, T=3, K=256, N=200, y=FAKE, status=None)
    a.update(over)
    return lib.kda_scaled_matmul(*[a[k] for k in ("x", "xs", "per", "w", "ws", "T", "K", "N", "y", "status")], None)


@pytest.mark.parametrize("over,code", [
    ({"T": -1}, INVALID), ({"T": 2 ** 31}, UNSUPPORTED), ({"K": 0}, INVALID), ({"K": 24}, UNSUPPORTED), ({"K": 2 ** 25}, UNSUPPORTED),
    ({"N": 0}, INVALID), ({"N": 2 ** 25}, UNSUPPORTED), ({"per": 2}, INVALID), ({"x": None}, INVALID), ({"xs": None}, INVALID),
    ({"w": OFF8}, INVALID), ({"x": OFF8}, INVALID), ({"y": OFF8}, INVALID), ({"ws": OFF2}, INVALID), ({"xs": OFF2}, INVALID),
    ({"status": OFF2}, INVALID)])
def test_product_refuses(lib, over, code):
    assert _product(lib, **over) == code


@pytest.mark.parametrize("withhold", [-2, -2 ** 31])
def test_debug_forms_refuse(lib, withhold):
    args = [FAKE] * 6 + [2, 100, 4, 2, 128, 128, 256, 256, 512, None, 0.1, FAKE, None, None, None, 0, None]
    assert lib.kda_gated_delta_chunk_fwd_debug(*args, withhold) == INVALID
    assert lib.kda_scaled_matmul_debug(FAKE, FAKE, 1, FAKE, FAKE, 3, 256, 200, FAKE, None, None, withhold) == INVALID


def test_calls_with_nothing_to_do(lib):
    assert _chunk(lib, N=0, T=0, q=None, k=None, v=None, g=None, beta=None, cu=None, o=None) == kda.KDA_OK
    assert _decode(lib, N=0, q=None, k=None, v=None, g=None, beta=None, o=None) == kda.KDA_OK
    assert _norm(lib, T=0, x=None, gate=None, w=None, y=None, ys=None) == kda.KDA_OK
    assert _product(lib, T=0, x=None, xs=None, w=None, ws=None, y=None) == kda.KDA_OK


def test_binding_refuses():
    t = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    g = torch.zeros(4, 2)
    with pytest.raises(ValueError):
        kda.gated_delta_chunk_fwd(t, t, t, g, g, torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError):
        kda.gated_delta_chunk_fwd(t, t, t, g[0], g, torch.tensor([0, 4], dtype=torch.int32))  # one decay per head
    with pytest.raises(ValueError):
        kda.gated_delta_decode_fwd(t, t, t, g, g, 4)
    with pytest.raises(ValueError):
        kda.gated_delta_decode_fwd(t, t, t, g, g, 4, in_place=True)
    with pytest.raises(ValueError):
        kda.gated_rms_norm(t, t, torch.ones(128))
    with pytest.raises(ValueError):
        kda.gated_rms_norm(t.flatten(1), t, torch.ones(128))
    x = torch.zeros(4, 256, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        kda.scaled_matmul(x, torch.ones(4), x, torch.ones(1, 2))


def test_native_calls_leave_what_is_not_plain(lib):
    """The native form of a plain call gives back what it does not take; the general one then says why."""
    if _lib._native is None:
        pytest.skip("the native calls are not built")
    t, g = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(4, 2)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    x = torch.zeros(4, 256, dtype=torch.float8_e4m3fn)
    n = _lib._native
    assert n.gated_delta_chunk(t, t, t, g, g, cu, None, None, True) is None
    assert n.gated_delta_chunk(None, t, t, g, g, 7, None, "x", True) is None
    assert n.gated_delta_decode(t, t, t, g, g, 4, None, None, False) is None
    assert n.gated_delta_decode(t, t, t, g, g, 2 ** 70, None, None, False) is None
    assert n.gated_rms_norm(t, t, torch.ones(128), 1e-5, 0) is None
    assert n.scaled_matmul(x, torch.ones(4), x, torch.ones(1, 2)) is None
    with pytest.raises(TypeError):
        n.scaled_matmul(x, x)


def test_oracle_recurrence_closed_forms():
    """With g = 0, beta = 1 and unit keys a token reads back what it wrote, repeated keys replace, orthogonal ones add up; beta =
    0 leaves the decayed state; the chunk's matrix form gives the same."""
    rng = np.random.default_rng(0)
    eye, v = np.eye(4), rng.standard_normal((3, 1, 5))
    k = eye[[0, 1, 0]][:, None]
    o, _, S, _ = ref.recurrence(k, k, v, np.zeros((3, 1)), np.ones((3, 1)), [3], None, 2.0)
    assert np.allclose(o, 2.0 * v) and np.allclose(S[0, 0, 0], v[2, 0]) and np.allclose(S[0, 0, 1], v[1, 0])
    s0 = rng.standard_normal((1, 1, 4, 5))
    _, _, S, _ = ref.recurrence(k, k, v, np.log(np.array([[.5], [.25], [1.]])), np.zeros((3, 1)), [3], s0, 1.0)
    assert np.allclose(S, s0 / 8)
    T, K, V = 7, 6, 5
    q, k, v = rng.standard_normal((T, 2, K)), rng.standard_normal((T, 2, K)), rng.standard_normal((T, 4, V))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    g, b, s0 = -rng.random((T, 4)), rng.random((T, 4)), rng.standard_normal((2, 4, K, V))
    o, off, S, E = ref.recurrence(q, k, v, g, b, [T - 2, 2], s0, 0.5, 4)
    assert (off > 0).all() and (E > 0).all()
    for h in range(4):
        G, kk, qq = np.cumsum(g[:T - 2, h]), k[:T - 2, h // 2], q[:T - 2, h // 2]
        pair = np.tril(np.exp(G[:, None] - G[None]))
        A = np.eye(T - 2) + np.tril(b[:T - 2, h, None] * (kk @ kk.T) * pair, -1)
        x = np.linalg.solve(A, b[:T - 2, h, None] * (v[:T - 2, h] - np.exp(G)[:, None] * (kk @ s0[0, h])))
        want = 0.5 * (np.exp(G)[:, None] * (qq @ s0[0, h]) + (qq @ kk.T * pair) @ x)
        assert np.allclose(o[:T - 2, h], want)
        assert np.allclose(S[0, h], np.exp(G[-1]) * s0[0, h] + (np.exp(G[-1] - G)[:, None] * kk).T @ x)


def test_oracle_norm_and_product():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    n = ref.gated_norm(x, np.zeros((1, 4)), [1, 2, 1, 1], 0.0, False)
    assert np.allclose(n, [[0.6, 1.6, 0, 0]])
    n = ref.gated_norm(x, np.full((1, 4), 2.0), [1, 2, 1, 1], 0.0, True)
    assert np.allclose(n, np.array([[1.2, 3.2, 0, 0]]) * 2 / (1 + np.exp(-2.0)))
    a, b = np.ones((2, 130)), np.ones((129, 130))
    ws = np.array([[1.0, 10.0], [100.0, 1000.0]])
    y, size = ref.scaled_matmul(a, np.array([1.0, -2.0]), b, ws)
    assert np.allclose(y[0, :128], 128 + 20) and np.allclose(y[1, 128], -2 * (12800 + 2000)) and np.allclose(size[1], -y[1])
    y, _ = ref.scaled_matmul(a, np.array([[1.0, 3.0], [5.0, 7.0]]), b, ws)
    assert np.allclose(y[1, 128], 5 * 12800 + 7 * 2000)
