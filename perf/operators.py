"""The linear-attention, state-cache and norm operators as calls on given inputs: cases, their inputs, a plain form and a
64-bit form of each.

``own`` false: elementary torch operations in 32 bits (64 for sums of log decays). ``own`` true: the library's entry points.

  chunk   linear attention with a decay for each head over varlen-packed prompts, chunked form
  decode  the same recurrence for a few tokens per sequence on a carried state
  store   fp32 states -> slots of an int8 state cache with one fp32 scale per key row
  load    slots of that cache -> fp32 states
  norm    residual addition, RMS norm and e4m3 output with one fp32 scale per token
"""
import random

import torch

own = False

D = 128        # head dimension of keys and values
CHUNK = 128    # tokens per chunk of the plain form
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _chunk(seqs, tokens, heads, qk_heads, ragged, state, decay):
    return {"op": "chunk", "seqs": seqs, "tokens": tokens, "heads": heads, "qk_heads": qk_heads, "ragged": ragged,
            "state": state, "decay": decay}


def _decode(seqs, steps, heads, qk_heads, decay):
    return {"op": "decode", "seqs": seqs, "steps": steps, "heads": heads, "qk_heads": qk_heads, "decay": decay}


def _cache(op, rows, heads, slots, holes):
    return {"op": op, "rows": rows, "heads": heads, "slots": slots, "holes": holes}


def _norm(tokens, width):
    return {"op": "norm", "tokens": tokens, "width": width}


def listed():
    return [
        # the smallest prompt of the workloads: one short sequence, two heads; latency counts
        {"name": "chunk_256_H2", **_chunk(1, 256, 2, 2, False, False, "token")},
        # the headline batch: four prompts of 2048 tokens, 16 heads
        {"name": "chunk_4x2048_H16", **_chunk(4, 2048 * 4, 16, 16, False, False, "token")},
        # a serving batch on cached prefixes: odd lengths, an empty and a one-token prompt, query/key heads shared by two
        {"name": "chunk_ragged16_H16_state", **_chunk(16, 12189, 16, 8, True, True, "token")},
        # one long prompt with the few heads of a GPU under head-parallel sharding, a fixed decay for each head
        {"name": "chunk_1x65536_H4_state", **_chunk(1, 65536, 4, 4, False, True, "head")},
        # a large decode batch, one new token each
        {"name": "decode_256x1_H16", **_decode(256, 1, 16, 16, "token")},
        # a few sequences verifying four drafted tokens each
        {"name": "decode_3x4_H16", **_decode(3, 4, 16, 8, "head")},
        # a batch's final states into the prefix cache
        {"name": "store_256_H16", **_cache("store", 256, 16, 512, False)},
        # one sequence's state after its prompt
        {"name": "store_1_H16", **_cache("store", 1, 16, 64, False)},
        # the cached prefixes of a batch, some of whose sequences have none
        {"name": "load_256_H16", **_cache("load", 256, 16, 512, True)},
        # a few prefixes of a model with many heads
        {"name": "load_3_H96", **_cache("load", 3, 96, 16, False)},
        # the input of a layer for a prefill batch, width 16 heads x 128
        {"name": "norm_8192x2048", **_norm(8192, 2048)},
        # the same for a small decode batch, width 96 heads x 128
        {"name": "norm_7x12288", **_norm(7, 12288)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "decode", "decode", "store", "load", "norm", "norm"])
    heads = rng.choice([1, 2, 4, 5, 8, 16, 16, 32, 96])
    qk_heads = rng.choice([h for h in (heads, heads, heads // 2, heads // 4, 1) if h >= 1 and heads % h == 0])
    decay = rng.choice(["token", "token", "head"])
    if op == "chunk":
        tokens = _log_int(rng, 64, min(65536, 262144 // heads))
        seqs = _log_int(rng, 1, max(1, min(64, tokens // 16, 2048 // heads)))
        return _chunk(seqs, tokens, heads, qk_heads, seqs > 1, rng.random() < 0.5, decay)
    if op == "decode":
        seqs = _log_int(rng, 1, 4096 // heads)
        return _decode(seqs, rng.choice([1, 1, 1, 2, 3, 5, 8]), heads, qk_heads, decay)
    if op in ("store", "load"):
        rows = _log_int(rng, 1, 4096 // heads)
        return _cache(op, rows, heads, rows + _log_int(rng, 1, 1 + 4096 // heads), rng.random() < 0.5)
    width = rng.choice([128 * heads, _log_int(rng, 64, 16384), 8 * _log_int(rng, 8, 2048)])
    return _norm(_log_int(rng, 1, max(1, min(16384, (1 << 25) // width))), width)


def _lengths(case):
    """The sequence lengths of a chunk case: equal, or cut at random places, with an empty and a one-token sequence from four
    sequences on."""
    n, t = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [t // n + (1 if i < t % n else 0) for i in range(n)]
    rng = random.Random(1000003 * n + t)
    cuts = sorted(rng.randrange(t + 1) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [t])]
    if n >= 4:
        big = max(range(n), key=lambda i: lens[i])
        for place, want in ((n // 2, 0), (n - 1, 1)):
            if place != big and lens[big] + lens[place] > want:
                lens[big] += lens[place] - want
                lens[place] = want
    return lens


# ------------------------------------------------------------------ inputs
def _unit_rows(shape, gen):
    x = torch.randn(shape, device=DEV, generator=gen)
    return (x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-20)).to(torch.bfloat16)


def _decays(case, tokens, gen):
    """Log decays: a fixed one for each head, or -a_h * softplus(x) for each token and head."""
    h = case["heads"]
    if case["decay"] == "head":
        return -torch.exp2(-8.0 * (torch.rand(h, device=DEV, generator=gen) * 0.9 + 0.1))
    rate = torch.exp(torch.rand(h, device=DEV, generator=gen) * 4.0 - 5.0)
    return -rate * torch.log1p(torch.exp(torch.randn(tokens, h, device=DEV, generator=gen) + 1.0))


def _attention_inputs(case, tokens, gen):
    h, hk = case["heads"], case["qk_heads"]
    return {"q": _unit_rows((tokens, hk, D), gen), "k": _unit_rows((tokens, hk, D), gen),
            "v": torch.randn(tokens, h, D, device=DEV, generator=gen).to(torch.bfloat16),
            "g": _decays(case, tokens, gen), "scale": D ** -0.5}


def _states(rows, heads, gen):
    """States as they come out of a prompt: the key rows differ in size."""
    size = torch.exp(torch.randn(rows, heads, D, 1, device=DEV, generator=gen) * 0.7)
    return torch.randn(rows, heads, D, D, device=DEV, generator=gen).mul_(size * 0.2)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "chunk":
        lens = _lengths(case)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s.update(_attention_inputs(case, case["tokens"], gen))
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["lens"] = lens
        s["state"] = _states(len(lens), case["heads"], gen) if case["state"] else None
    elif op == "decode":
        s.update(_attention_inputs(case, case["seqs"] * case["steps"], gen))
        s["state"] = _states(case["seqs"], case["heads"], gen)
    elif op in ("store", "load"):
        rows, heads, slots = case["rows"], case["heads"], case["slots"]
        at = torch.randperm(slots, device=DEV, generator=gen)[:rows].to(torch.int32)
        if case["holes"]:
            at = torch.where(torch.rand(rows, device=DEV, generator=gen) < 0.25, torch.full_like(at, -1), at)
        s["slots"] = at
        s["codes"] = torch.randint(-127, 128, (slots, heads, D, D), device=DEV, generator=gen, dtype=torch.int8)
        s["scales"] = torch.rand(slots, heads, D, device=DEV, generator=gen) * 0.01
        if op == "store":
            s["state"] = _states(rows, heads, gen)
    else:
        t, d = case["tokens"], case["width"]
        s["x"] = torch.randn(t, d, device=DEV, generator=gen).to(torch.bfloat16)
        s["residual"] = (torch.randn(t, d, device=DEV, generator=gen) * 3.0).to(torch.bfloat16)
        s["weight"] = 1.0 + 0.2 * torch.randn(d, device=DEV, generator=gen)
        s["eps"] = 1e-6
    return s


# ------------------------------------------------------------------ plain forms
def _per_token(g, tokens):
    return g.expand(tokens, -1) if g.dim() == 1 else g


def _plain_chunk(s):
    q, k, v, lens, state = s["q"], s["k"], s["v"], s["lens"], s["state"]
    t, h = v.shape[0], v.shape[1]
    lens_t = torch.tensor(lens)
    per = (lens_t + CHUNK - 1) // CHUNK                                   # chunks of each sequence
    seq = torch.repeat_interleave(torch.arange(len(lens)), per)           # sequence of each chunk
    first = torch.cumsum(per, 0) - per                                    # first chunk of each sequence
    local = torch.arange(int(per.sum())) - first[seq]
    start = (torch.cumsum(lens_t, 0) - lens_t)[seq] + local * CHUNK
    left = lens_t[seq] - local * CHUNK
    seq, first, start, left = seq.to(DEV), first.to(DEV), start.to(DEV), left.to(DEV)
    lane = torch.arange(CHUNK, device=DEV)
    valid = lane[None] < left[:, None]                                    # [NC, C]
    idx = torch.where(valid, start[:, None] + lane[None], 0)

    def rows(x):                                                          # [NC, H, C, D], zeros behind a sequence
        x = x.float()[idx] * valid[..., None, None]
        x = x.repeat_interleave(h // x.shape[2], 2) if x.shape[2] != h else x
        return x.permute(0, 2, 1, 3)

    qc, kc, vc = rows(q), rows(k), rows(v)
    g = _per_token(s["g"], t).double()[idx] * valid[..., None]
    cum = g.permute(0, 2, 1).cumsum(-1)                                   # [NC, H, C]
    total = cum[..., -1]                                                  # [NC, H]
    low = torch.tril(torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV))
    pair = torch.where(low, cum[..., :, None] - cum[..., None, :], -torch.inf).exp().float()
    out = (qc @ kc.transpose(-1, -2) * pair) @ vc
    add = (kc * (total[..., None] - cum).exp().float()[..., None]).transpose(-1, -2) @ vc  # each chunk's own state
    nc = add.shape[0]
    upto = total.cumsum(0)                                                # [NC, H] log decay up to a chunk's end
    before = upto - total
    same = seq[:, None] == seq[None, :]
    earlier = torch.arange(nc, device=DEV)[:, None] > torch.arange(nc, device=DEV)[None, :]
    carry = torch.where((same & earlier)[None], before.t()[:, :, None] - upto.t()[:, None, :], -torch.inf).exp().float()
    flat = add.permute(1, 0, 2, 3).reshape(h, nc, D * D)
    entry = (carry @ flat).reshape(h, nc, D, D).permute(1, 0, 2, 3)       # state before each chunk
    if state is not None:
        entry = entry + (before - before[first[seq]]).exp().float()[..., None, None] * state[seq]
    out = out + cum.exp().float()[..., None] * (qc @ entry)
    o = torch.zeros(t, h, D, device=DEV)
    o[idx[valid]] = out.permute(0, 2, 1, 3)[valid] * s["scale"]
    mine = torch.arange(len(lens), device=DEV)[:, None] == seq[None, :]   # [N, NC]
    last = torch.cumsum(per, 0).to(DEV) - 1
    some = (lens_t > 0).to(DEV)
    end = upto[last.clamp_min(0)]                                         # [N, H]
    keep = torch.where(mine[None], end.t()[:, :, None] - upto.t()[:, None, :], -torch.inf).exp().float()
    final = (keep @ flat).reshape(h, len(lens), D, D).permute(1, 0, 2, 3)
    if state is not None:
        whole = torch.where(some[:, None], end - before[first.clamp_max(nc - 1)], 0.0).exp().float()
        final = final + whole[..., None, None] * state
    return {"o": o.to(torch.bfloat16), "state": final.contiguous()}


def _plain_decode(s):
    case, v = s["case"], s["v"]
    n, tn, h = case["seqs"], case["steps"], case["heads"]
    rep = h // case["qk_heads"]
    # the few tokens of a sequence at once: o_t = sum_{u<=t} e^{G_t-G_u} (q_t.k_u) v_u + e^{G_t} S^T q_t
    q = s["q"].float().repeat_interleave(rep, 1).reshape(n, tn, h, D).transpose(1, 2)
    k = s["k"].float().repeat_interleave(rep, 1).reshape(n, tn, h, D).transpose(1, 2)
    v = v.float().reshape(n, tn, h, D).transpose(1, 2)
    cum = _per_token(s["g"], n * tn).double().reshape(n, tn, h).transpose(1, 2).cumsum(-1)
    low = torch.tril(torch.ones(tn, tn, dtype=torch.bool, device=DEV))
    pair = torch.where(low, cum[..., :, None] - cum[..., None, :], -torch.inf).exp().float()
    o = (q @ k.transpose(-1, -2) * pair) @ v + cum.exp().float()[..., None] * (q @ s["state"])
    end = cum[..., -1:]
    final = (k * (end - cum).exp().float()[..., None]).transpose(-1, -2) @ v + end.exp().float()[..., None] * s["state"]
    o = (o * s["scale"]).transpose(1, 2).reshape(n * tn, h, D)
    return {"o": o.to(torch.bfloat16), "state": final}


def _plain_store(s):
    x = s["state"]
    amax = x.abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, 127.0)                                    # tensors on both sides: one IEEE division each
    scale = amax / top
    inverse = torch.where(amax > 0, top / amax, 0.0)
    codes = (x * inverse).round().clamp(-127, 127).to(torch.int8)
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    s["codes"][at] = codes[keep]
    s["scales"][at] = scale[keep][..., 0]
    return {"codes": s["codes"], "scales": s["scales"]}


def _plain_load(s):
    at = s["slots"].long()
    x = s["codes"][at.clamp_min(0)].float() * s["scales"][at.clamp_min(0)][..., None]
    return torch.where((at >= 0)[:, None, None, None], x, 0.0)


def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    amax = y.abs().amax(-1, keepdim=True)
    inverse = torch.where(amax > 0, 448.0 / amax, 0.0)
    q = (y * inverse).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return {"residual": h.to(torch.bfloat16), "y": q, "scale": (amax / 448.0)[:, 0]}


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"chunk": _plain_chunk, "decode": _plain_decode, "store": _plain_store, "load": _plain_load,
                "norm": _plain_norm}[op](s)
    import kda_chunked_prefill_gb300 as kda
    if op == "chunk":
        o, state = kda.linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["cu_seqlens"], s["state"], scale=s["scale"])
        return {"o": o, "state": state}
    if op == "decode":
        o, state = kda.linear_decode_fwd(s["q"], s["k"], s["v"], s["g"], s["case"]["seqs"], s["state"], scale=s["scale"])
        return {"o": o, "state": state}
    if op == "store":
        kda.state_store(s["state"], s["slots"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "load":
        return kda.state_load(s["codes"], s["scales"], s["slots"])
    y, scale, residual = kda.add_rms_norm(s["x"], s["residual"], s["weight"], s["eps"])
    return {"residual": residual, "y": y, "scale": scale}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    h = case.get("heads", 0)
    if op in ("chunk", "decode"):
        t = case["tokens"] if op == "chunk" else case["seqs"] * case["steps"]
        reads = op == "decode" or case["state"]
        g = 4 * (t * h if case["decay"] == "token" else h)
        states = 4 * D * D * case["seqs"] * h * (2 if reads else 1)
        return {"bytes": 2 * D * t * (2 * case["qk_heads"] + 2 * h) + g + states, "flops": 4 * D * D * t * h}
    if op in ("store", "load"):
        live = case["rows"] * (0.75 if case["holes"] else 1.0)  # rows with a slot; the others' states are still written as zeros
        states = case["rows"] if op == "load" else live
        return {"bytes": h * (4 * D * D * states + (D * D + 4 * D) * live) + 4 * case["rows"], "flops": 2 * live * h * D * D}
    t, d = case["tokens"], case["width"]
    return {"bytes": t * d * (2 + 2 + 2 + 1) + 4 * t + 4 * d, "flops": 6 * t * d}


# ------------------------------------------------------------------ 64 bits
def _recurrence(q, k, v, g, lens, state, scale):
    """S = e^g S + k v^T, o = scale S^T q, token by token for all sequences and heads at once, in 64 bits."""
    h = v.shape[1]
    n, longest = len(lens), max(lens)
    lens_t = torch.tensor(lens, device=DEV)
    starts = torch.cumsum(lens_t, 0) - lens_t
    q = q.repeat_interleave(h // q.shape[1], 1)
    k = k.repeat_interleave(h // k.shape[1], 1)
    g = _per_token(g, v.shape[0])
    S = torch.zeros(n * h, D, D, dtype=torch.float64, device=DEV)
    if state is not None:
        S += state.double().reshape(n * h, D, D)
    o = torch.zeros(v.shape[0] + 1, h, D, dtype=torch.float64, device=DEV)  # the last row takes what has no token
    for t0 in range(0, longest, 256):
        steps = min(256, longest - t0)
        at = starts[:, None] + t0 + torch.arange(steps, device=DEV)[None]
        live = (t0 + torch.arange(steps, device=DEV)[None]) < lens_t[:, None]
        at = torch.where(live, at, 0)
        on = live[..., None]
        qs = (q[at].double() * on[..., None]).permute(1, 0, 2, 3).reshape(steps, n * h, D, 1)
        ks = (k[at].double() * on[..., None]).permute(1, 0, 2, 3).reshape(steps, n * h, D, 1)
        vs = (v[at].double() * on[..., None]).permute(1, 0, 2, 3).reshape(steps, n * h, 1, D)
        ds = (g[at].double() * on).exp().permute(1, 0, 2).reshape(steps, n * h, 1, 1)
        outs = []
        for u in range(steps):
            S.mul_(ds[u]).addcmul_(ks[u], vs[u])
            outs.append((S * qs[u]).sum(1))
        rows = torch.stack(outs).reshape(steps, n, h, D).permute(1, 0, 2, 3)
        o[torch.where(live, at, v.shape[0])] = rows * scale
    return {"o": o[:-1], "state": S.reshape(n, h, D, D)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "chunk":
        return _recurrence(s["q"], s["k"], s["v"], s["g"], s["lens"], s["state"], s["scale"])
    if op == "decode":
        return _recurrence(s["q"], s["k"], s["v"], s["g"], [case["steps"]] * case["seqs"], s["state"], s["scale"])
    if op == "store":
        scales = s["scales"].double()
        for row, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                scales[slot] = s["state"][row].double().abs().max(-1).values / 127.0
        return {"codes": None, "scales": scales}
    if op == "load":
        out = torch.zeros(case["rows"], case["heads"], D, D, dtype=torch.float64, device=DEV)
        for row, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                out[row] = s["codes"][slot].double() * s["scales"][slot].double()[..., None]
        return out
    x = s["x"].double() + s["residual"].double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[1] + s["eps"]).sqrt() * s["weight"].double()
    scale = y.abs().max(-1).values / 448.0
    return {"residual": x, "y": y / scale[:, None], "scale": scale}
