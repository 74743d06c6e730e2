"""Host-side refusals of the linear-attention, state-cache and add-norm entry points (no GPU: validation runs before any CUDA
call), and the binding's checks of tensors."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from kda_chunked_prefill_gb300 import _lib
from oracle import linear as ref

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return _lib.load_library(build_if_missing=True)


def _chunk(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, cu=FAKE, N=2, T=100, H=4, Hk=2, dk=128, dv=128, qs=256, ks=256, vs=512, gt=1,
             s0=None, scale=0.1, o=FAKE, sT=None, status=None, ws=None, wsb=0)
    a.update(over)
    return lib.kda_linear_chunk_fwd(*[a[k] for k in ("q", "k", "v", "g", "cu", "N", "T", "H", "Hk", "dk", "dv", "qs", "ks", "vs",
                                                     "gt", "s0", "scale", "o", "sT", "status", "ws", "wsb")], None)


def _decode(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, N=2, Tn=1, H=4, Hk=2, dk=128, dv=128, qs=256, ks=256, vs=512, gt=1, s0=None,
             scale=0.1, o=FAKE, sT=None, status=None)
    a.update(over)
    return lib.kda_linear_decode_fwd(*[a[k] for k in ("q", "k", "v", "g", "N", "Tn", "H", "Hk", "dk", "dv", "qs", "ks", "vs",
                                                      "gt", "s0", "scale", "o", "sT", "status")], None)


BAD = [({"dk": 64}, kda.KDA_ERR_UNSUPPORTED), ({"dv": 256}, kda.KDA_ERR_UNSUPPORTED), ({"H": 0}, kda.KDA_ERR_INVALID_ARG),
       ({"Hk": 0}, kda.KDA_ERR_INVALID_ARG), ({"Hk": 3, "qs": 384, "ks": 384}, kda.KDA_ERR_INVALID_ARG),
       ({"N": -1}, kda.KDA_ERR_INVALID_ARG), ({"qs": 248}, kda.KDA_ERR_INVALID_ARG), ({"ks": 260}, kda.KDA_ERR_INVALID_ARG),
       ({"vs": 504}, kda.KDA_ERR_INVALID_ARG), ({"vs": 1 << 60}, kda.KDA_ERR_UNSUPPORTED), ({"gt": 2}, kda.KDA_ERR_INVALID_ARG),
       ({"scale": NAN}, kda.KDA_ERR_INVALID_ARG), ({"q": None}, kda.KDA_ERR_INVALID_ARG), ({"g": None}, kda.KDA_ERR_INVALID_ARG),
       ({"o": None}, kda.KDA_ERR_INVALID_ARG), ({"k": ctypes.c_void_p(0x10008)}, kda.KDA_ERR_INVALID_ARG),
       ({"s0": ctypes.c_void_p(0x10010)}, kda.KDA_ERR_INVALID_ARG), ({"sT": ctypes.c_void_p(0x10010)}, kda.KDA_ERR_INVALID_ARG),
       ({"status": ctypes.c_void_p(0x10002)}, kda.KDA_ERR_INVALID_ARG), ({"N": 2 ** 30, "H": 4}, kda.KDA_ERR_INVALID_ARG)]


@pytest.mark.parametrize("over,code", BAD + [({"T": -1}, kda.KDA_ERR_INVALID_ARG), ({"cu": None}, kda.KDA_ERR_INVALID_ARG),
                                             ({"T": 2 ** 31}, kda.KDA_ERR_UNSUPPORTED),
                                             ({"cu": ctypes.c_void_p(0x10002)}, kda.KDA_ERR_INVALID_ARG)])
def test_linear_chunk_refuses(lib, over, code):
    assert _chunk(lib, **over) == code


@pytest.mark.parametrize("withhold", [(-2, -1), (-1, -2), (0, -2 ** 31)])
def test_linear_chunk_debug_refuses(lib, withhold):
    args = [FAKE] * 5 + [2, 100, 4, 2, 128, 128, 256, 256, 512, 1, None, 0.1, FAKE, None, None, None, 0, None]
    assert lib.kda_linear_chunk_fwd_debug(*args, *withhold) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("over,code", BAD + [({"Tn": -1}, kda.KDA_ERR_INVALID_ARG), ({"Tn": 65}, kda.KDA_ERR_INVALID_ARG)])
def test_linear_decode_refuses(lib, over, code):
    assert _decode(lib, **over) == code


def test_calls_with_nothing_to_do(lib):
    assert _chunk(lib, N=0, T=0, q=None, k=None, v=None, g=None, cu=None, o=None) == kda.KDA_OK
    assert _decode(lib, N=0, q=None, k=None, v=None, g=None, o=None) == kda.KDA_OK
    assert _cache(lib, "store", M=0, state=None, slots=None) == kda.KDA_OK
    assert _norm(lib, rows=0, x=None, res=None, w=None, out=None, y=None, ys=None) == kda.KDA_OK


def _cache(lib, op, **over):
    a = dict(state=FAKE, slots=FAKE, M=3, H=2, dk=128, dv=128, S=5, codes=FAKE, scales=FAKE, status=None)
    a.update(over)
    if op == "store":
        return lib.kda_state_store(a["state"], a["slots"], a["M"], a["H"], a["dk"], a["dv"], a["S"], a["codes"], a["scales"],
                                   a["status"], None)
    return lib.kda_state_load(a["codes"], a["scales"], a["slots"], a["M"], a["H"], a["dk"], a["dv"], a["S"], a["state"],
                              a["status"], None)


@pytest.mark.parametrize("op", ["store", "load"])
@pytest.mark.parametrize("over,code", [
    ({"dk": 64}, kda.KDA_ERR_UNSUPPORTED), ({"dv": 64}, kda.KDA_ERR_UNSUPPORTED), ({"M": -1}, kda.KDA_ERR_INVALID_ARG),
    ({"H": 0}, kda.KDA_ERR_INVALID_ARG), ({"S": -1}, kda.KDA_ERR_INVALID_ARG), ({"state": None}, kda.KDA_ERR_INVALID_ARG),
    ({"slots": None}, kda.KDA_ERR_INVALID_ARG), ({"codes": None}, kda.KDA_ERR_INVALID_ARG),
    ({"scales": None}, kda.KDA_ERR_INVALID_ARG), ({"state": ctypes.c_void_p(0x10010)}, kda.KDA_ERR_INVALID_ARG),
    ({"codes": ctypes.c_void_p(0x10008)}, kda.KDA_ERR_INVALID_ARG), ({"scales": ctypes.c_void_p(0x10002)}, kda.KDA_ERR_INVALID_ARG),
    ({"M": 2 ** 30, "H": 4}, kda.KDA_ERR_INVALID_ARG)])
def test_state_cache_refuses(lib, op, over, code):
    assert _cache(lib, op, **over) == code


def _norm(lib, **over):
    a = dict(x=FAKE, res=FAKE, w=FAKE, rows=4, width=64, eps=1e-6, fp32=0, out=FAKE, y=FAKE, ys=FAKE)
    a.update(over)
    return lib.kda_add_rms_norm(a["x"], a["res"], a["w"], a["rows"], a["width"], a["eps"], a["fp32"], a["out"], a["y"], a["ys"],
                                None)


@pytest.mark.parametrize("over,code", [
    ({"rows": -1}, kda.KDA_ERR_INVALID_ARG), ({"rows": 2 ** 31}, kda.KDA_ERR_INVALID_ARG), ({"width": 0}, kda.KDA_ERR_INVALID_ARG),
    ({"width": 32769}, kda.KDA_ERR_UNSUPPORTED), ({"eps": 0.0}, kda.KDA_ERR_INVALID_ARG), ({"eps": NAN}, kda.KDA_ERR_INVALID_ARG),
    ({"eps": -1.0}, kda.KDA_ERR_INVALID_ARG), ({"fp32": 2}, kda.KDA_ERR_INVALID_ARG), ({"x": None}, kda.KDA_ERR_INVALID_ARG),
    ({"y": ctypes.c_void_p(0x10008)}, kda.KDA_ERR_INVALID_ARG), ({"ys": None}, kda.KDA_ERR_INVALID_ARG),
    ({"w": ctypes.c_void_p(0x10004)}, kda.KDA_ERR_INVALID_ARG), ({"out": ctypes.c_void_p(0x10004)}, kda.KDA_ERR_INVALID_ARG)])
def test_add_norm_refuses(lib, over, code):
    assert _norm(lib, **over) == code


def test_binding_refuses_cpu_tensors_and_bad_views():
    t = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kda.linear_chunk_fwd(t, t, t, torch.zeros(4, 2), torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError):
        kda.linear_decode_fwd(t, t, t, torch.zeros(4, 2), 4)
    with pytest.raises(ValueError):
        kda.state_load(torch.zeros(2, 1, 128, 128, dtype=torch.int8), torch.zeros(2, 1, 128), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        kda.add_rms_norm(t, t, torch.ones(128))
    cpu = t.get_device()
    assert _lib._heads_view(t, "q", 4, cpu) == 256
    assert _lib._heads_view(torch.zeros(4, 768, dtype=torch.bfloat16)[:, 256:512].view(4, 2, 128), "q", 4, cpu) == 768
    for bad in (t.transpose(0, 1).contiguous().transpose(0, 1), torch.zeros(4, 2, 256, dtype=torch.bfloat16)[:, :, ::2],
                torch.zeros(1, 2, 128, dtype=torch.bfloat16).expand(4, 2, 128),
                torch.zeros(4 * 260, dtype=torch.bfloat16).as_strided((4, 2, 128), (260, 128, 1))):
        with pytest.raises(ValueError):
            _lib._heads_view(bad, "q", 4, cpu)
    with pytest.raises(TypeError):
        _lib._heads_view(t.float(), "q", 4, cpu)


def test_the_package_imports_on_a_torch_without_cuda():
    """Inputs, constants and the host checks need no CUDA build of torch: there, its private CUDA bindings do not exist."""
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, name)\n"
            "import kda_chunked_prefill_gb300 as kda\n"
            "from kda_chunked_prefill_gb300 import inputs\n"
            "inputs.make_inputs([3], 1, seed=0)\n"
            "t = torch.zeros(4, 2, 128, dtype=torch.bfloat16)\n"
            "try: kda.add_rms_norm(t, t, torch.ones(128))\n"
            "except ValueError: print('refused')\n")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, 
                         cwd=os.path.dirname(os.path.dirname(kda.__file__)))
    assert run.returncode == 0 and run.stdout.strip() == "refused", run.stderr


def test_oracle_recurrence_closed_forms():
    """A constant decay and one repeated token give a geometric sum; shared heads read their group's query and key."""
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 1, 4)), rng.standard_normal((3, 1, 4)), rng.standard_normal((3, 2, 4))
    k[:], v[:] = k[0], v[0]
    g = np.log(np.array([0.5, 0.25]))
    o, size, S, A = ref.recurrence(q, k, v, g, [3], None, 2.0)
    for h, d in enumerate((0.5, 0.25)):
        want = (1 + d + d * d) * np.outer(k[0, 0], v[0, h])
        assert np.allclose(S[0, h], want) and np.allclose(A[0, h], np.abs(want))
        assert np.allclose(o[2, h], 2.0 * q[2, 0] @ want)
    assert (size >= np.abs(o) - 1e-12).all()
    o2, _, S2, _ = ref.recurrence(q, k, v, g, [0, 2, 0, 1], None, 2.0)
    assert np.allclose(S2[0], 0) and np.allclose(S2[1, 0], 1.5 * np.outer(k[0, 0], v[0, 0])) and np.allclose(o2[:2], o[:2])


def test_oracle_quantise_rows():
    x = np.zeros((1, 3, 4), dtype=np.float32)
    x[0, 0] = [127, 0.5, 1.5, -2.5]
    x[0, 1] = [-1, 0.25, 0, 1]
    codes, scales = ref.quantise_rows(x)
    assert codes[0, 0].tolist() == [127, 0, 2, -2] and scales[0, 0] == 1
    assert codes[0, 1].tolist() == [-127, 32, 0, 127] and codes[0, 2].tolist() == [0, 0, 0, 0] and scales[0, 2] == 0
