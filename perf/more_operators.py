"""The gated-delta-rule layer's operators as calls on given inputs: cases, their inputs, a plain form and a 64-bit form of each.

``own`` false: elementary torch operations in 32 bits (64 for sums of log decays). ``own`` true: the library's entry points.

  delta    the delta rule with one decay for each head over varlen-packed prompts, chunked form
  step     the same recurrence for a few tokens per sequence on a carried state
  gate     RMS norm of each head's output row, its gate, and e4m3 output with one fp32 scale per token and head
  product  e4m3 activations (a scale per row, or per row and 128 channels) times an e4m3 weight with a scale per 128 x 128 block
"""
import random

import torch

own = False

D = 128        # head dimension of keys and values
CHUNK = 64     # tokens per chunk of the plain form
BLOCK = 128    # channels and outputs that share a scale of the weight
DEV = "cuda"


# ------------------------------------------------------------------ cases
def _delta(seqs, tokens, heads, qk_heads, ragged, state):
    return {"op": "delta", "seqs": seqs, "tokens": tokens, "heads": heads, "qk_heads": qk_heads, "ragged": ragged, "state": state}


def _step(seqs, steps, heads, qk_heads):
    return {"op": "step", "seqs": seqs, "steps": steps, "heads": heads, "qk_heads": qk_heads}


def _gate(tokens, heads, silu, wide):
    return {"op": "gate", "tokens": tokens, "heads": heads, "silu": silu, "wide": wide}


def _product(rows, outs, width, blocks):
    return {"op": "product", "rows": rows, "outs": outs, "width": width, "blocks": blocks}


def listed():
    return [
        # the smallest prompt of the workloads: one short sequence, two heads; latency counts
        {"name": "delta_256_H2", **_delta(1, 256, 2, 2, False, False)},
        # the headline batch: four prompts of 2048 tokens, 16 heads
        {"name": "delta_4x2048_H16", **_delta(4, 2048 * 4, 16, 16, False, False)},
        # a serving batch on cached prefixes: odd lengths, an empty and a one-token prompt, query/key heads shared by two
        {"name": "delta_ragged16_H16_state", **_delta(16, 12189, 16, 8, True, True)},
        # one long prompt with the few heads of a GPU under head-parallel sharding
        {"name": "delta_1x65536_H4_state", **_delta(1, 65536, 4, 4, False, True)},
        # a large decode batch, one new token each
        {"name": "step_256x1_H16", **_step(256, 1, 16, 16)},
        # a few sequences verifying four drafted tokens each
        {"name": "step_3x4_H16", **_step(3, 4, 16, 8)},
        # the headline batch's outputs on their way to the output projection
        {"name": "gate_8192_H16", **_gate(8192, 16, True, False)},
        # a small decode batch of a model with many heads, from KDA's fp32 outputs
        {"name": "gate_7_H96", **_gate(7, 96, False, True)},
        # the headline batch's projection to q, k, v: 3 x 16 heads of 128 from width 2048, rows scaled as the norm leaves them
        {"name": "product_8192_2048_to_6144", **_product(8192, 6144, 2048, False)},
        # the output projection of the headline batch, one scale per token and head
        {"name": "product_8192_2048_to_2048", **_product(8192, 2048, 2048, True)},
        # a decode batch's projection to q, k, v and the gates of decay and delta rule (2 x 16 more outputs)
        {"name": "product_256_2048_to_6176", **_product(256, 6176, 2048, False)},
        # a small decode batch through the output projection of a model with 96 heads
        {"name": "product_7_12288_to_12288", **_product(7, 12288, 12288, True)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "step", "step", "gate", "gate", "product", "product", "product"])
    heads = rng.choice([1, 2, 4, 5, 8, 16, 16, 32, 96])
    qk_heads = rng.choice([h for h in (heads, heads, heads // 2, heads // 4, 1) if h >= 1 and heads % h == 0])
    if op == "delta":
        tokens = _log_int(rng, 64, min(65536, 262144 // heads))
        seqs = _log_int(rng, 1, max(1, min(64, tokens // 16, 2048 // heads)))
        return _delta(seqs, tokens, heads, qk_heads, seqs > 1, rng.random() < 0.5)
    if op == "step":
        seqs = _log_int(rng, 1, 4096 // heads)
        return _step(seqs, rng.choice([1, 1, 1, 2, 3, 5, 8]), heads, qk_heads)
    if op == "gate":
        return _gate(_log_int(rng, 1, max(1, 262144 // heads)), heads, rng.random() < 0.5, rng.random() < 0.3)
    width = rng.choice([128 * heads, 128 * heads, 16 * _log_int(rng, 1, 768)])
    outs = rng.choice([128 * heads, _log_int(rng, 1, 12288), 8 * _log_int(rng, 1, 1536)])
    return _product(_log_int(rng, 1, max(1, min(16384, (1 << 36) // (width * outs)))), outs, width, rng.random() < 0.5)


def _lengths(case):
    """The sequence lengths of a delta case: equal, or cut at random places, with an empty and a one-token sequence from four
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
    """What a projection, its SiLU and the normalisation leave: unit rows with a common part."""
    x = torch.randn(shape, device=DEV, generator=gen)
    x = x / (1.0 + torch.exp(-x))
    return (x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-20)).to(torch.bfloat16)


def _attention_inputs(case, tokens, gen):
    h, hk = case["heads"], case["qk_heads"]
    rate = torch.exp(torch.rand(h, device=DEV, generator=gen) * 4.0 - 5.0)
    return {"q": _unit_rows((tokens, hk, D), gen), "k": _unit_rows((tokens, hk, D), gen),
            "v": torch.randn(tokens, h, D, device=DEV, generator=gen).to(torch.bfloat16),
            "g": -rate * torch.log1p(torch.exp(torch.randn(tokens, h, device=DEV, generator=gen) + 1.0)),
            "beta": 1.0 / (1.0 + torch.exp(-torch.randn(tokens, h, device=DEV, generator=gen))), "scale": D ** -0.5}


def _states(rows, heads, gen):
    """States as they come out of a prompt: the key rows differ in size."""
    size = torch.exp(torch.randn(rows, heads, D, 1, device=DEV, generator=gen) * 0.7)
    return torch.randn(rows, heads, D, D, device=DEV, generator=gen).mul_(size * 0.2)


def _per_block(scale, width):
    """A scale per 128 channels (or one for all) -> one for each channel."""
    return scale.repeat_interleave(BLOCK, -1)[..., :width]


def _to_e4m3(x, block_rows, block_cols):
    """Codes of x and their scales, one for each block: its largest magnitude / 448."""
    r, c = x.shape
    rb, cb = -(-r // block_rows), -(-c // block_cols)
    pad = torch.zeros(rb * block_rows, cb * block_cols, device=DEV)
    pad[:r, :c] = x.abs()
    scale = (pad.view(rb, block_rows, cb, block_cols).amax((1, 3)) / 448.0).clamp_min(1e-20)
    each = scale.repeat_interleave(block_rows, 0)[:r].repeat_interleave(block_cols, 1)[:, :c]
    return (x / each).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "delta":
        lens = _lengths(case)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s.update(_attention_inputs(case, case["tokens"], gen))
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["lens"] = lens
        s["state"] = _states(len(lens), case["heads"], gen) if case["state"] else None
    elif op == "step":
        s.update(_attention_inputs(case, case["seqs"] * case["steps"], gen))
        s["state"] = _states(case["seqs"], case["heads"], gen)
    elif op == "gate":
        t, h = case["tokens"], case["heads"]
        size = torch.exp(torch.randn(t, h, 1, device=DEV, generator=gen))
        x = torch.randn(t, h, D, device=DEV, generator=gen) * size * 0.1
        s["x"] = x if case["wide"] else x.to(torch.bfloat16)
        s["gate"] = (torch.randn(t, h, D, device=DEV, generator=gen) * 1.5).to(torch.bfloat16)
        s["weight"] = 1.0 + 0.2 * torch.randn(D, device=DEV, generator=gen)
        s["eps"] = 1e-5
    else:
        rows, outs, width = case["rows"], case["outs"], case["width"]
        x = torch.randn(rows, width, device=DEV, generator=gen) * torch.exp(torch.randn(rows, 1, device=DEV, generator=gen))
        s["x"], scale = _to_e4m3(x, 1, BLOCK if case["blocks"] else width)
        s["x_scale"] = scale if case["blocks"] else scale[:, 0].contiguous()
        w = torch.randn(outs, width, device=DEV, generator=gen) * width ** -0.5
        s["weight"], s["weight_scale"] = _to_e4m3(w, BLOCK, BLOCK)
    return s


# ------------------------------------------------------------------ plain forms
def _inverse(a):
    """(I + a)^-1 for strictly lower triangular a [..., C, C], C a power of two: blocks of twice the size in each round,
    [[P, 0], [a21, Q]] with P and Q inverted already has -Q a21 P below its diagonal."""
    c = a.shape[-1]
    t = torch.eye(c, device=a.device).expand_as(a).contiguous()
    size = 1
    while size < c:
        n = c // (2 * size)
        at = torch.arange(n, device=a.device)
        tb = t.view(*t.shape[:-2], n, 2 * size, n, 2 * size)
        ab = a.view(*a.shape[:-2], n, 2 * size, n, 2 * size)
        low = ab[..., at, size:, at, :size]
        # (the two index tensors put the blocks' dimension first)
        tb[..., at, size:, at, :size] = -(tb[..., at, size:, at, size:] @ low @ tb[..., at, :size, at, :size])
        size *= 2
    return t


def _plain_delta(s):
    q, k, v, lens, state = s["q"], s["k"], s["v"], s["lens"], s["state"]
    t, h = v.shape[0], v.shape[1]
    lens_t = torch.tensor(lens)
    per = (lens_t + CHUNK - 1) // CHUNK                                   # chunks of each sequence
    seq = torch.repeat_interleave(torch.arange(len(lens)), per)           # sequence of each chunk
    first = torch.cumsum(per, 0) - per                                    # first chunk of each sequence
    local = torch.arange(int(per.sum())) - first[seq]
    start = (torch.cumsum(lens_t, 0) - lens_t)[seq] + local * CHUNK
    left = lens_t[seq] - local * CHUNK
    seq, local, start, left = seq.to(DEV), local.to(DEV), start.to(DEV), left.to(DEV)
    lane = torch.arange(CHUNK, device=DEV)
    valid = lane[None] < left[:, None]                                    # [NC, C]
    idx = torch.where(valid, start[:, None] + lane[None], 0)

    def rows(x):                                                          # [NC, H, C, ...], zeros behind a sequence
        x = x[idx] * valid.view(*valid.shape, *[1] * (x.dim() - 1))
        x = x.repeat_interleave(h // x.shape[2], 2) if x.shape[2] != h else x
        return x.transpose(1, 2)

    qc, kc, vc, beta = rows(q.float()), rows(k.float()), rows(v.float()), rows(s["beta"])
    cum = rows(s["g"].double()).cumsum(-1)                                # [NC, H, C]
    total = cum[..., -1:]
    low = torch.tril(torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV))
    pair = torch.where(low, cum[..., :, None] - cum[..., None, :], -torch.inf).exp().float()
    kk = kc @ kc.transpose(-1, -2)
    inv = _inverse(torch.tril(kk * pair * beta[..., None], -1)) * beta[..., None, :]
    u = inv @ vc                                                          # v_new = u - w S
    w = inv @ (kc * cum.exp().float()[..., None])
    ke = (kc * (total - cum).exp().float()[..., None]).transpose(-1, -2)
    # each chunk's map of the state, S -> keep S + add; then of all chunks of its sequence up to it, by doubling
    keep = total.exp().float()[..., None] * torch.eye(D, device=DEV) - ke @ w
    add = ke @ u
    span, longest = 1, int(per.max()) if len(lens) else 0
    while span < longest:
        has = torch.nonzero(local >= span)[:, 0]                          # the chunk `span` before is of the same sequence
        add_has = keep[has] @ add[has - span] + add[has]
        keep_has = keep[has] @ keep[has - span]
        add[has], keep[has] = add_has, keep_has
        span *= 2
    zero = torch.zeros(len(lens), h, D, D, device=DEV) if state is None else state
    after = keep @ zero[seq] + add
    entry = torch.where((local > 0)[:, None, None, None], after.roll(1, 0), zero[seq])
    new = u - w @ entry
    out = (qc * cum.exp().float()[..., None]) @ entry + ((qc @ kc.transpose(-1, -2)) * pair) @ new
    o = torch.zeros(t, h, D, device=DEV)
    o[idx[valid]] = out.transpose(1, 2)[valid] * s["scale"]
    final = zero.clone()
    some = torch.nonzero(per > 0)[:, 0]
    final[some.to(DEV)] = after[(first + per - 1)[some].to(DEV)]
    return {"o": o.to(torch.bfloat16), "state": final}


def _plain_step(s):
    case, v, beta = s["case"], s["v"], s["beta"]
    n, tn, h = case["seqs"], case["steps"], case["heads"]
    rep = h // case["qk_heads"]

    def rows(x):                                                          # [N, H, Tn, D]
        return x.float().repeat_interleave(h // x.shape[1], 1).reshape(n, tn, h, D).transpose(1, 2)

    q, k, v = rows(s["q"]), rows(s["k"]), rows(v)
    beta = beta.reshape(n, tn, h).transpose(1, 2)
    cum = s["g"].double().reshape(n, tn, h).transpose(1, 2).cumsum(-1)
    low = torch.tril(torch.ones(tn, tn, dtype=torch.bool, device=DEV))
    pair = torch.where(low, cum[..., :, None] - cum[..., None, :], -torch.inf).exp().float()
    size = 1 << (tn - 1).bit_length()
    a = torch.zeros(n, h, size, size, device=DEV)
    a[..., :tn, :tn] = torch.tril(k @ k.transpose(-1, -2) * pair * beta[..., None], -1)
    decay = cum.exp().float()[..., None]
    new = _inverse(a)[..., :tn, :tn] @ (beta[..., None] * (v - decay * (k @ s["state"])))
    o = decay * (q @ s["state"]) + (q @ k.transpose(-1, -2) * pair) @ new
    end = cum[..., -1:]
    final = end.exp().float()[..., None] * s["state"] + (k * (end - cum).exp().float()[..., None]).transpose(-1, -2) @ new
    return {"o": (o * s["scale"]).transpose(1, 2).reshape(n * tn, h, D).to(torch.bfloat16), "state": final}


def _plain_gate(s):
    x, g = s["x"].float(), s["gate"].float()
    act = 1.0 / (1.0 + torch.exp(-g))
    if s["case"]["silu"]:
        act = act * g
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"] * act
    amax = y.abs().amax(-1, keepdim=True)
    inverse = torch.where(amax > 0, 448.0 / amax, 0.0)
    q = (y * inverse).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return {"y": q.flatten(1), "scale": (amax / 448.0)[..., 0]}


def _plain_product(s):
    x, w = s["x"].float(), s["weight"].float()
    x_scale = s["x_scale"] if s["case"]["blocks"] else s["x_scale"][:, None]
    x = x * (_per_block(x_scale, x.shape[1]) if s["case"]["blocks"] else x_scale)
    w = w * _per_block(s["weight_scale"].repeat_interleave(BLOCK, 0)[:w.shape[0]], w.shape[1])
    return (x @ w.t()).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"delta": _plain_delta, "step": _plain_step, "gate": _plain_gate, "product": _plain_product}[op](s)
    import kda_chunked_prefill_gb300 as kda
    if op == "delta":
        o, state = kda.gated_delta_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu_seqlens"], s["state"],
                                             scale=s["scale"])
        return {"o": o, "state": state}
    if op == "step":
        o, state = kda.gated_delta_decode_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["case"]["seqs"], s["state"],
                                              scale=s["scale"])
        return {"o": o, "state": state}
    if op == "gate":
        y, scale = kda.gated_rms_norm(s["x"], s["gate"], s["weight"], s["eps"],
                                      activation="silu" if s["case"]["silu"] else "sigmoid")
        return {"y": y, "scale": scale}
    return kda.scaled_matmul(s["x"], s["x_scale"], s["weight"], s["weight_scale"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("delta", "step"):
        h = case["heads"]
        t = case["tokens"] if op == "delta" else case["seqs"] * case["steps"]
        reads = op == "step" or case["state"]
        states = 4 * D * D * case["seqs"] * h * (2 if reads else 1)
        return {"bytes": 2 * D * t * (2 * case["qk_heads"] + 2 * h) + 8 * t * h + states, "flops": 6 * D * D * t * h}
    if op == "gate":
        t, h = case["tokens"], case["heads"]
        return {"bytes": t * h * (D * ((4 if case["wide"] else 2) + 2 + 1) + 4) + 4 * D, "flops": 12 * t * h * D}
    rows, outs, width = case["rows"], case["outs"], case["width"]
    blocks = -(-width // BLOCK)
    scales = rows * (blocks if case["blocks"] else 1) + blocks * -(-outs // BLOCK)
    return {"bytes": rows * width + outs * width + 2 * rows * outs + 4 * scales, "flops": 2 * rows * outs * width}


# ------------------------------------------------------------------ 64 bits
def _recurrence(q, k, v, g, beta, lens, state, scale):
    """S <- e^g S;  S <- S + beta k (v - k^T S)^T;  o = scale S^T q, token by token for all sequences and heads at once."""
    h = v.shape[1]
    n, longest = len(lens), max(lens)
    lens_t = torch.tensor(lens, device=DEV)
    starts = torch.cumsum(lens_t, 0) - lens_t
    q = q.repeat_interleave(h // q.shape[1], 1)
    k = k.repeat_interleave(h // k.shape[1], 1)
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
        qs = (q[at].double() * on[..., None]).permute(1, 0, 2, 3).reshape(steps, n * h, 1, D)
        ks = (k[at].double() * on[..., None]).permute(1, 0, 2, 3).reshape(steps, n * h, D, 1)
        vs = v[at].double().permute(1, 0, 2, 3).reshape(steps, n * h, 1, D)
        ds = (g[at].double() * on).exp().permute(1, 0, 2).reshape(steps, n * h, 1, 1)
        bs = (beta[at].double() * on).permute(1, 0, 2).reshape(steps, n * h, 1, 1)
        outs = []
        for u in range(steps):
            S.mul_(ds[u])
            S.addcmul_(ks[u], bs[u] * (vs[u] - torch.bmm(ks[u].transpose(1, 2), S)))
            outs.append(torch.bmm(qs[u], S))
        rows = torch.stack(outs).reshape(steps, n, h, D).permute(1, 0, 2, 3)
        o[torch.where(live, at, v.shape[0])] = rows * scale
    return {"o": o[:-1], "state": S.reshape(n, h, D, D)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "delta":
        return _recurrence(s["q"], s["k"], s["v"], s["g"], s["beta"], s["lens"], s["state"], s["scale"])
    if op == "step":
        return _recurrence(s["q"], s["k"], s["v"], s["g"], s["beta"], [case["steps"]] * case["seqs"], s["state"], s["scale"])
    if op == "gate":
        x, g = s["x"].double(), s["gate"].double()
        y = x / (x.pow(2).sum(-1, keepdim=True) / D + s["eps"]).sqrt() * s["weight"].double() / (1 + (-g).exp())
        y = y * g if case["silu"] else y
        scale = y.abs().max(-1).values / 448.0
        return {"y": (y / scale[..., None]).flatten(1), "scale": scale}
    x, w = s["x"], s["weight"]
    rows, outs, width = case["rows"], case["outs"], case["width"]
    y = torch.zeros(rows, outs, dtype=torch.float64, device=DEV)
    per_out = torch.arange(outs, device=DEV) // BLOCK
    for b in range(-(-width // BLOCK)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK].double() @ w[:, b * BLOCK:(b + 1) * BLOCK].double().t()
        part *= (s["x_scale"][:, b] if case["blocks"] else s["x_scale"]).double()[:, None]
        y += part * s["weight_scale"][per_out, b].double()[None]
    return y
