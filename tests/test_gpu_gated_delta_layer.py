"""A layer of the gated delta rule as its calls run: residual norm, projection, prompts and decoding, gated norm, output projection.

Each call is compared with 64 bits on the inputs that it was given, by the bounds of its own tests; and the whole, in 64 bits without any
rounding, with what comes out: e4m3 operands twice (2^-4 / sqrt(3) / sqrt(2) of a term on average, below 0.03 each, independent over the
sums), bf16 between the calls (below 0.002 each): below 0.1 in all (2-norm).
"""
import numpy as np
import pytest
import torch

import kda_chunked_prefill_gb300 as kda
from oracle import delta as ref
from oracle import linear as lref

pytestmark = pytest.mark.gpu
D, H, HK, WIDTH = 128, 4, 2, 384


def quantise(w):
    """Codes and a scale for each block of 128 x 128."""
    N, K = w.shape
    pad = torch.zeros(-(-N // 128) * 128, -(-K // 128) * 128, dtype=w.dtype)
    pad[:N, :K] = w
    s = pad.view(pad.shape[0] // 128, 128, -1, 128).abs().amax((1, 3)) / 448
    return (w / s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]).to(torch.float8_e4m3fn), s.float()


def layer(x, res, p, cu, states, steps):
    """The calls on the GPU; returns the output, the new residual, the states and what each call was given."""
    y, ys, res = kda.add_rms_norm(x, res, p["norm"], 1e-6)
    qkvz = kda.scaled_matmul(y, ys, p["w_in"], p["w_in_scale"], check=True)
    T = x.shape[0]
    at = np.cumsum([0, HK * D, HK * D, H * D, H * D, H, H])
    unit = lambda t: t / t.float().norm(dim=-1, keepdim=True).clamp_min(1e-6)
    q, k = (unit(qkvz[:, a:b].reshape(T, HK, D).float()).to(torch.bfloat16) for a, b in zip(at[:2], at[1:3]))
    v, z = qkvz[:, at[2]:at[3]].view(T, H, D), qkvz[:, at[3]:at[4]].view(T, H, D)  # slices of the projection
    beta = torch.sigmoid(qkvz[:, at[4]:at[5]].float())
    g = -torch.nn.functional.softplus(qkvz[:, at[5]:at[6]].float())
    if steps:
        o, states = kda.gated_delta_decode_fwd(q, k, v, g, beta, T // steps, states, in_place=True, check=True)
    else:
        o, states = kda.gated_delta_chunk_fwd(q, k, v, g, beta, cu, states, check=True)
    n, ns = kda.gated_rms_norm(o, z, p["onorm"], activation="silu")
    out = kda.scaled_matmul(n, ns, p["w_out"], p["w_out_scale"], check=True)
    return out, res, states, dict(y=y, ys=ys, qkvz=qkvz, q=q, k=k, v=v, z=z, beta=beta, g=g, o=o, n=n, ns=ns)


def layer64(x, res, p, lens, state):
    """All in 64 bits, from the weights that the codes stand for."""
    f = lambda t: t.double().cpu().numpy()
    h, y = lref.add_rms_norm(f(x), f(res), f(p["norm"]), 1e-6)
    deq = lambda c, s: f(c.float()) * np.repeat(np.repeat(f(s), 128, 0)[:c.shape[0]], 128, 1)[:, :c.shape[1]]
    qkvz = y @ deq(p["w_in"], p["w_in_scale"]).T
    T = len(y)
    at = np.cumsum([0, HK * D, HK * D, H * D, H * D, H, H])
    part = [qkvz[:, a:b] for a, b in zip(at[:-1], at[1:])]
    unit = lambda t: t / np.linalg.norm(t, axis=-1, keepdims=True)
    q, k = unit(part[0].reshape(T, HK, D)), unit(part[1].reshape(T, HK, D))
    o, _, S, _ = ref.recurrence(q, k, part[2].reshape(T, H, D), -np.log1p(np.exp(part[5])), 1 / (1 + np.exp(-part[4])), lens, state,
                                D ** -0.5)
    n = ref.gated_norm(o, part[3].reshape(T, H, D), f(p["onorm"]), 1e-5, True).reshape(T, -1)
    return n @ deq(p["w_out"], p["w_out_scale"]).T, h, S


def params(rng):
    w_in = torch.from_numpy(rng.standard_normal((2 * HK * D + 2 * H * D + 2 * H, WIDTH)) * WIDTH ** -0.5)
    w_out = torch.from_numpy(rng.standard_normal((WIDTH, H * D)) * (H * D) ** -0.5)
    p = {"norm": torch.from_numpy(1 + 0.1 * rng.standard_normal(WIDTH)).float(), "onorm": torch.from_numpy(1 + 0.1 * rng.standard_normal(D)).float()}
    p["w_in"], p["w_in_scale"] = quantise(w_in)
    p["w_out"], p["w_out_scale"] = quantise(w_out)
    return {n: t.cuda() for n, t in p.items()}


def rel(a, b):
    a = a.double().cpu().numpy()
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def check_calls(m, p, out):
    f = lambda t: t.double().cpu().numpy()
    for got, args in ((m["qkvz"], (m["y"], m["ys"], p["w_in"], p["w_in_scale"])), (out, (m["n"], m["ns"], p["w_out"], p["w_out_scale"]))):
        want, size = ref.scaled_matmul(*(f(t.float()) for t in args))
        assert (np.abs(f(got) - want) <= 2.0 ** -8 * 1.001 * np.abs(want) + 300 * ref.F * size + 1e-38).all()
    n = ref.gated_norm(f(m["o"]), f(m["z"]), f(p["onorm"]), 1e-5, True)
    assert (np.abs(f(m["ns"]) - np.abs(n).max(-1) / 448) <= 1e-5 * np.abs(n).max(-1) / 448).all()
    assert rel(m["n"].float().view(n.shape) * m["ns"][..., None], n) < 2.0 ** -4


def test_layer_prompts_then_steps():
    rng = np.random.default_rng(0)
    p = params(rng)
    lens = [150, 0, 1, 333]
    T = sum(lens)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda()
    x, res = bf(T, WIDTH), bf(T, WIDTH)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out, new, states, m = layer(x, res, p, cu, None, 0)
    check_calls(m, p, out)
    want, h, S = layer64(x, res, p, lens, None)
    assert rel(out, want) < 0.1 and rel(new, h) < 2.0 ** -8 and rel(states, S) < 0.1
    x, res = bf(12, WIDTH), bf(12, WIDTH)  # three drafted tokens of each sequence, on the states of the prompts
    before = states.double().cpu().numpy()
    out, _, states, m = layer(x, res, p, None, states, 3)
    check_calls(m, p, out)
    want, _, S = layer64(x, res, p, [3] * 4, before)
    assert rel(out, want) < 0.1 and rel(states, S) < 0.1


def test_layer_in_a_graph():
    """The calls captured together and replayed on new inputs give what they give one by one."""
    rng = np.random.default_rng(1)
    p = params(rng)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda()
    x, res = bf(140, WIDTH), bf(140, WIDTH)
    cu = torch.tensor([0, 100, 140], dtype=torch.int32, device="cuda")

    def calls():
        y, ys, r = kda.add_rms_norm(x, res, p["norm"], 1e-6)
        qkvz = kda.scaled_matmul(y, ys, p["w_in"], p["w_in_scale"])
        q, k = qkvz[:, :HK * D].view(140, HK, D) * 0.09, qkvz[:, HK * D:2 * HK * D].view(140, HK, D) * 0.09
        v, z = qkvz[:, 2 * HK * D:2 * HK * D + H * D].view(140, H, D), qkvz[:, 2 * HK * D + H * D:2 * HK * D + 2 * H * D].view(140, H, D)
        beta = torch.sigmoid(qkvz[:, -2 * H:-H].float())
        g = -torch.nn.functional.softplus(qkvz[:, -H:].float())
        o, s = kda.gated_delta_chunk_fwd(q, k, v, g, beta, cu)
        n, ns = kda.gated_rms_norm(o, z, p["onorm"])
        return kda.scaled_matmul(n, ns, p["w_out"], p["w_out_scale"]), s

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for _ in range(3):
        x.copy_(bf(140, WIDTH)), res.copy_(bf(140, WIDTH))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        now = calls()
        assert torch.equal(held[0], now[0]) and torch.equal(held[1], now[1])
