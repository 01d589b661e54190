"""What a transformer block holds between its linears, as cases to measure:
the gated residual with the norms around it, rotary positions of several axes,
and attention, each with its gradients.

Formulas:

  residual_norm       hn = h, or norm(h) gp with a norm after the block,
                      s = alpha x + gate hn (rounded to the rows' type),
                      y = norm(s) g + b; gate, gp, g, b belong to the row's
                      group; norm(v) = (v - mean) rstd, or v rstd (rms), with
                      rstd = 1 / sqrt(mean of the squares + eps)
  residual_norm_grad  with t = ds + the norm's gradient of dy g at s:
                      dx = alpha t, dgate = sum t hn, dgp = sum t gate hhat,
                      dh = t gate, or the norm's gradient of t gate gp at h,
                      dg = sum dy shat, db = sum dy (sums over a group's rows)
  rope                a pair (u, v) of a head's elements turns by the angle
                      position[axis of the pair] freq[pair]; the gradient
                      turns back
  attention           o = softmax(scale q k^T) v over the keys that the mask
                      keeps (causal: key j <= query i + keys - queries), lse
                      the logarithm of the softmax's denominator; a row
                      without keys is 0 and -inf
  attention_grad      p = exp(scale q k^T - lse), dv = p^T do,
                      ds = p (do v^T - sum_d do o), dq = scale ds k,
                      dk = scale ds^T q; shared heads add up
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one conditioning token: nothing but latency
        {"name": "residual_norm 1x1536", "op": "residual_norm", "rows": 1, "channels": 1536, "groups": 1, "dtype": "bf16",
         "params": "bf16", "kind": "rms", "post": True, "one_plus": False},
        # between a block's attention and its MLP: two images of 4096 tokens, modulated per sample
        {"name": "residual_norm 8192x4096 modulated", "op": "residual_norm", "rows": 8192, "channels": 4096, "groups": 2,
         "dtype": "bf16", "params": "bf16", "kind": "layer", "post": False, "one_plus": True},
        # the same in training
        {"name": "residual_norm_grad 8192x4096 modulated", "op": "residual_norm_grad", "rows": 8192, "channels": 4096,
         "groups": 2, "dtype": "bf16", "params": "bf16", "kind": "layer", "post": False, "one_plus": True},
        # a text stream with norms on both sides of its blocks, a width that no vector divides
        {"name": "residual_norm_grad 5003x1283 rms post fp16", "op": "residual_norm_grad", "rows": 5003, "channels": 1283,
         "groups": 1, "dtype": "fp16", "params": "fp32", "kind": "rms", "post": True, "one_plus": True},
        # queries and keys of 512 text tokens and a 64 x 64 image: time, height and width
        {"name": "rope 4608 tokens 24 heads", "op": "rope", "samples": 1, "tokens": 4608, "heads": 24, "kv_heads": 24, "dim": 128,
         "pairs": "8,28,28", "interleaved": True, "inverse": False, "dtype": "bf16", "positions": "int32"},
        # gradients of a video's ragged clip in 32 bits, halves of the head turned, fractional frame times
        {"name": "rope_grad 2x1003 tokens fp32", "op": "rope", "samples": 2, "tokens": 1003, "heads": 12, "kv_heads": 4, "dim": 80,
         "pairs": "8,12,12", "interleaved": False, "inverse": True, "dtype": "fp32", "positions": "fp32"},
        # joint attention of text and image, part of the text padding
        {"name": "attention 4608 tokens 24 heads", "op": "attention", "samples": 1, "queries": 4608, "keys": 4608, "heads": 24,
         "kv_heads": 24, "dim": 128, "causal": False, "mask": True, "dtype": "bf16"},
        # one token of a text stream over a long cache with shared heads
        {"name": "attention 1 query 65536 keys", "op": "attention", "samples": 1, "queries": 1, "keys": 65536, "heads": 32,
         "kv_heads": 8, "dim": 128, "causal": True, "mask": False, "dtype": "bf16"},
        # a text encoder's causal attention, every size ragged
        {"name": "attention causal 2x1531 fp16", "op": "attention", "samples": 2, "queries": 1531, "keys": 1601, "heads": 12,
         "kv_heads": 4, "dim": 72, "causal": True, "mask": False, "dtype": "fp16"},
        # training the joint attention
        {"name": "attention_grad 4608 tokens 24 heads", "op": "attention_grad", "samples": 1, "queries": 4608, "keys": 4608,
         "heads": 24, "kv_heads": 24, "dim": 128, "causal": False, "mask": True, "dtype": "bf16"},
        # cross attention of image tokens to a short padded prompt
        {"name": "attention_grad 2x4096 queries 77 keys", "op": "attention_grad", "samples": 2, "queries": 4096, "keys": 77,
         "heads": 20, "kv_heads": 20, "dim": 64, "causal": False, "mask": True, "dtype": "bf16"},
        # training the causal text encoder with shared heads
        {"name": "attention_grad causal 2x1531 fp16", "op": "attention_grad", "samples": 2, "queries": 1531, "keys": 1601,
         "heads": 12, "kv_heads": 4, "dim": 72, "causal": True, "mask": False, "dtype": "fp16"},
    ]


def _spread(rng, lo, hi, step=1):
    """A size of [lo, hi], spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["residual_norm", "residual_norm_grad", "rope", "attention", "attention", "attention_grad",
                     "attention_grad"])
    if op in ("residual_norm", "residual_norm_grad"):
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        channels = _spread(rng, 33, 8192)
        rows = _spread(rng, 1, min(16384, 8192 * 4096 // channels // (2 if dtype == "fp32" else 1)))
        return {"op": op, "rows": rows, "channels": channels, "groups": rng.randint(1, min(rows, 4)), "dtype": dtype,
                "params": rng.choice([dtype, "fp32"]), "kind": rng.choice(["layer", "rms"]), "post": rng.random() < 0.5,
                "one_plus": rng.random() < 0.5}
    kv_heads = _spread(rng, 1, 16)
    heads = kv_heads * _spread(rng, 1, max(1, 32 // kv_heads))
    samples, dtype = rng.randint(1, 4), rng.choice(["bf16", "bf16", "fp16"])
    if op == "rope":
        interleaved = rng.random() < 0.5
        pairs = [rng.randint(1, 20) if interleaved else 8 * rng.randint(1, 2) for _ in range(rng.randint(1, 4))]
        dim = (2 * sum(pairs) + 7) // 8 * 8 + rng.choice([0, 8, 16])
        tokens = _spread(rng, 1, 4608 * 48 * 128 // (samples * (heads + kv_heads) * dim) // 2)
        return {"op": op, "samples": samples, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "pairs": ",".join(map(str, pairs)), "interleaved": interleaved, "inverse": rng.random() < 0.5,
                "dtype": rng.choice([dtype, "fp32"]), "positions": rng.choice(["int32", "fp32"])}
    dim = _spread(rng, 16, 128, 8)
    queries = _spread(rng, 1, 8192 // samples)
    most = min(4608 * 4608 * 24 // (samples * queries * heads), (1 << 26) // (samples * kv_heads * dim), 65536)
    return {"op": op, "samples": samples, "queries": queries, "keys": _spread(rng, 1, max(1, most)), "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "causal": rng.random() < 0.5, "mask": rng.random() < 0.5, "dtype": dtype}


def _rows_per_group(rows, groups):
    return -(-rows // groups)


def _pairs(case):
    return [int(p) for p in case["pairs"].split(",")]


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _stream_of_activations(gen, rows, channels, dtype):
    """A residual stream: unit normal, one channel in a hundred much larger,
    with an offset of its own per channel."""
    big = torch.rand(channels, device="cuda", generator=gen) < 0.01
    return ((_randn(gen, rows, channels) + 0.25 * _randn(gen, channels)) * torch.where(big, 20.0, 1.0)).to(dtype)


def _parameters(gen, case):
    """Gate, shift, scale and post-norm weight of each group: slices of what a
    modulation layer gives, or a norm's own parameters."""
    g, c, dtype = case["groups"], case["channels"], TYPES[case["params"]]
    if g > 1:
        m = (0.3 * _randn(gen, g, 4 * c)).to(dtype)
        gate, bias, weight, post = (m[:, i * c:(i + 1) * c] for i in range(4))
        if not case["one_plus"]:
            weight, post = weight + 1, post + 1
    else:
        gate, bias, weight, post = ((0.3 * _randn(gen, c)).to(dtype) for _ in range(4))
        if not case["one_plus"]:
            weight, post = weight + 1, post + 1
    return {"gate": gate, "bias": bias, "weight": weight, "post": post if case["post"] else None}


def _stats(v, kind):
    """(mean, rstd) of the rows in 64 bits, as float32; the mean of rms is None."""
    v = v.double()
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    rstd = ((v - mean).square().mean(1) + EPS).rsqrt().float()
    return [mean[:, 0].float(), rstd] if kind == "layer" else [rstd]


def _prepare_residual_norm(case, gen):
    rows, c, dtype = case["rows"], case["channels"], TYPES[case["dtype"]]
    state = {"case": dict(case), "x": _stream_of_activations(gen, rows, c, dtype), "h": _randn(gen, rows, c).to(dtype)}
    state.update(_parameters(gen, case))
    if case["op"] == "residual_norm_grad":
        # x is here the stream that the forward left, with the statistics of its rows
        state["s"] = state.pop("x")
        stats = _stats(state["s"], case["kind"]) + (_stats(state["h"], case["kind"]) if case["post"] else [])
        state["stats"] = torch.stack(stats)
        state["dy"] = (_randn(gen, rows, c) * torch.exp(_randn(gen, c)) / 16).to(dtype)
        state["ds"] = (_randn(gen, rows, c) / 4).to(dtype)
    return state


def _prepare_rope(case, gen):
    b, n, d, dtype = case["samples"], case["tokens"], case["dim"], TYPES[case["dtype"]]
    pairs = _pairs(case)
    heads = case["heads"] + case["kv_heads"]
    qk = _randn(gen, b, n, heads, d).to(dtype)   # as a projection leaves them, side by side
    # a text part at the origin, then the places of a grid, or frame times
    side = max(1, int(math.sqrt(n)))
    at = torch.arange(n, device="cuda")
    pos = [at // (side * side), at % (side * side) // side, at % side, at][:len(pairs)]
    pos = torch.stack(pos, 1) + torch.randint(0, 1000, (len(pairs),), device="cuda", generator=gen)
    pos[: n // 9] = 0
    pos = pos.to(torch.int32) if case["positions"] == "int32" else pos.float() * 0.5 + 0.125
    freqs = torch.cat([THETA ** (-torch.arange(p, dtype=torch.float64) / p) for p in pairs]).cuda()
    return {"case": dict(case), "q": qk[:, :, :case["heads"]], "k": qk[:, :, case["heads"]:], "positions": pos, "freqs": freqs}


def _prepare_attention(case, gen):
    b, lq, lk, h, hk, d = (case[n] for n in ("samples", "queries", "keys", "heads", "kv_heads", "dim"))
    dtype = TYPES[case["dtype"]]
    state = {"case": dict(case), "mask": None}
    if lq == lk:   # one projection's output, side by side
        qkv = _randn(gen, b, lq, h + 2 * hk, d)
        qkv[:, :, :h] *= 1.5
        state["q"], state["k"], state["v"] = qkv.to(dtype).split([h, hk, hk], 2)
    else:
        state["q"] = (1.5 * _randn(gen, b, lq, h, d)).to(dtype)
        state["k"], state["v"] = _randn(gen, b, lk, 2 * hk, d).to(dtype).split([hk, hk], 2)
    if case["mask"]:   # a prompt's padding: keys from a random place of the first part on
        text = max(1, lk // 9) if lk > 200 else lk
        length = torch.randint(0, text + 1, (b, 1), device="cuda", generator=gen)
        at = torch.arange(lk, device="cuda")[None]
        state["mask"] = (at < length) | (at >= text)
    if case["op"] == "attention_grad":
        state["o"], state["lse"] = _plain_attention(state)
        state["do"] = (_randn(gen, b, lq, h, d) * torch.exp(0.5 * _randn(gen, b, lq, h, 1)) / 8).to(dtype)
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("residual_norm", "residual_norm_grad"):
        return _prepare_residual_norm(case, gen)
    return _prepare_rope(case, gen) if case["op"] == "rope" else _prepare_attention(case, gen)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _of_rows(p, case):
    """A parameter's value for each row, in 32 bits."""
    if p.dim() == 1:
        return p.float()[None]
    of_row = torch.arange(case["rows"], device=p.device) // _rows_per_group(case["rows"], case["groups"])
    return p.float()[of_row]


def _plain_norm(v, kind):
    stats = []
    if kind == "layer":
        mean = v.mean(1)
        v = v - mean[:, None]
        stats.append(mean)
    rstd = (v.square().mean(1) + EPS).rsqrt()
    return v * rstd[:, None], stats + [rstd]


def _plain_residual_norm(state):
    case, dtype = state["case"], state["x"].dtype
    one = 1.0 if case["one_plus"] else 0.0
    hn, post_stats = state["h"].float(), []
    if case["post"]:
        hn, post_stats = _plain_norm(hn, case["kind"])
        hn = hn * (_of_rows(state["post"], case) + one)
    s = (state["x"].float() + _of_rows(state["gate"], case) * hn).to(dtype)
    shat, stats = _plain_norm(s.float(), case["kind"])
    y = shat * (_of_rows(state["weight"], case) + one) + _of_rows(state["bias"], case)
    return s, y.to(dtype), torch.stack(stats + post_stats)


def _plain_norm_grad(d, vhat, rstd, kind):
    d = d - vhat * (d * vhat).mean(1, keepdim=True) - (d.mean(1, keepdim=True) if kind == "layer" else 0.0)
    return d * rstd[:, None]


def _group_sums(v, like, case):
    if like.dim() == 1:
        return v.sum(0).to(like.dtype)
    g, run_of = case["groups"], _rows_per_group(case["rows"], case["groups"])
    v = torch.cat([v, v.new_zeros(g * run_of - v.shape[0], v.shape[1])])
    return v.view(g, run_of, -1).sum(1).to(like.dtype)


def _plain_residual_norm_grad(state):
    case, dtype, kind = state["case"], state["s"].dtype, state["case"]["kind"]
    one = 1.0 if case["one_plus"] else 0.0
    n = 2 if kind == "layer" else 1
    stats, post_stats = state["stats"][:n], state["stats"][n:]

    def centred(v, st):
        v = v.float() - st[0][:, None] if kind == "layer" else v.float()
        return v * st[-1][:, None]

    dy = state["dy"].float()
    shat = centred(state["s"], stats)
    t = state["ds"].float() + _plain_norm_grad(dy * (_of_rows(state["weight"], case) + one), shat, stats[-1], kind)
    gate = _of_rows(state["gate"], case)
    hn, dh, dpost = state["h"].float(), t * gate, None
    if case["post"]:
        hhat, gain = centred(state["h"], post_stats), _of_rows(state["post"], case) + one
        hn = hhat * gain
        dpost = _group_sums(dh * hhat, state["post"], case)
        dh = _plain_norm_grad(dh * gain, hhat, post_stats[-1], kind)
    out = [t.to(dtype), dh.to(dtype), _group_sums(t * hn, state["gate"], case), _group_sums(dy * shat, state["weight"], case),
           _group_sums(dy, state["bias"], case)]
    return out + [dpost] if case["post"] else out


def _plain_rope(state):
    case, pos = state["case"], state["positions"].double()
    pairs = _pairs(case)
    axis = torch.repeat_interleave(torch.arange(len(pairs)), torch.tensor(pairs)).to(pos.device)
    angle = pos[:, axis] * state["freqs"]
    if case["inverse"]:
        angle = -angle
    cos, sin = angle.cos().float()[None, :, None], angle.sin().float()[None, :, None]
    n = sum(pairs)
    out = []
    for x in (state["q"], state["k"]):
        y = x.float().clone()
        if case["interleaved"]:
            u, v = y[..., 0:2 * n:2].clone(), y[..., 1:2 * n:2].clone()
            y[..., 0:2 * n:2], y[..., 1:2 * n:2] = u * cos - v * sin, u * sin + v * cos
        else:
            u, v = y[..., :n].clone(), y[..., n:2 * n].clone()
            y[..., :n], y[..., n:2 * n] = u * cos - v * sin, u * sin + v * cos
        out.append(y.to(x.dtype))
    return tuple(out)


def _visible(case, mask, sample, device):
    """[queries][keys] of a sample: which keys each query sees; None for all."""
    lq, lk = case["queries"], case["keys"]
    see = None
    if case["causal"]:
        see = torch.arange(lk, device=device)[None] <= torch.arange(lq, device=device)[:, None] + (lk - lq)
    if mask is not None:
        see = mask[sample][None] if see is None else see & mask[sample][None]
    return see


def _heads(state, name, sample, kv):
    """A key head's part of a tensor: [1][length][dim], or its group of query
    heads [group][length][dim], in 32 bits."""
    t, group = state[name][sample], state["case"]["heads"] // state["case"]["kv_heads"]
    t = t[:, kv:kv + 1] if name in ("k", "v") else t[:, kv * group:(kv + 1) * group]
    return t.transpose(0, 1).float().contiguous()


def _plain_attention(state):
    case, q = state["case"], state["q"]
    b, lq, h, d = q.shape
    o = torch.empty(b, lq, h, d, dtype=q.dtype, device=q.device)
    lse = torch.empty(b, h, lq, device=q.device)
    group = h // case["kv_heads"]
    for i in range(b):
        see = _visible(case, state["mask"], i, q.device)
        for kv in range(case["kv_heads"]):
            k, v = _heads(state, "k", i, kv)[0], _heads(state, "v", i, kv)[0]
            s = torch.matmul(_heads(state, "q", i, kv), k.t()) / math.sqrt(d)
            if see is not None:
                s = s.masked_fill(~see, -math.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m.clamp(min=-3e38))
            total = p.sum(-1, keepdim=True)
            heads = slice(kv * group, (kv + 1) * group)
            o[i, :, heads] = (torch.matmul(p, v) / total.clamp(min=1e-30)).transpose(0, 1).to(q.dtype)
            lse[i, heads] = (m + torch.log(total))[..., 0]
    return o, lse


def _plain_attention_grad(state):
    case = state["case"]
    q, k = state["q"], state["k"]
    scale, group = 1 / math.sqrt(case["dim"]), case["heads"] // case["kv_heads"]
    dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, k))
    for i in range(case["samples"]):
        see = _visible(case, state["mask"], i, q.device)
        for kv in range(case["kv_heads"]):
            heads = slice(kv * group, (kv + 1) * group)
            q1, do, o = (_heads(state, n, i, kv) for n in ("q", "do", "o"))
            k1, v1 = _heads(state, "k", i, kv)[0], _heads(state, "v", i, kv)[0]
            p = torch.exp(torch.matmul(q1, k1.t()) * scale - state["lse"][i, heads, :, None])
            if see is not None:
                p = p.masked_fill(~see, 0.0)
            dv[i, :, kv] = torch.matmul(p.flatten(0, 1).t(), do.flatten(0, 1)).to(q.dtype)
            ds = p * (torch.matmul(do, v1.t()) - (do * o).sum(-1, keepdim=True)) * scale
            if see is not None:
                ds = ds.masked_fill(~see, 0.0)
            dq[i, :, heads] = torch.matmul(ds, k1).transpose(0, 1).to(q.dtype)
            dk[i, :, kv] = torch.matmul(ds.flatten(0, 1).t(), q1.flatten(0, 1)).to(q.dtype)
    return dq, dk, dv


def _own(state):
    import bit_svdquant_diffusion_amd as S

    case, op = state["case"], state["case"]["op"]
    if op == "residual_norm":
        return S.residual_norm_forward(state["x"], state["h"], state["gate"], state["weight"], state["bias"],
                                       post_weight=state["post"], kind=case["kind"], eps=EPS, one_plus=case["one_plus"],
                                       rows_per_group=_rows_per_group(case["rows"], case["groups"]))
    if op == "residual_norm_grad":
        out = S.residual_norm_backward(state["dy"], state["s"], state["h"], state["stats"], state["gate"], state["weight"],
                                       post_weight=state["post"], ds=state["ds"], kind=case["kind"], one_plus=case["one_plus"],
                                       rows_per_group=_rows_per_group(case["rows"], case["groups"]))
        return out if case["post"] else out[:5]
    if op == "rope":
        return S.rope(state["q"], state["k"], state["positions"], state["freqs"], _pairs(case),
                      interleaved=case["interleaved"], inverse=case["inverse"])
    if op == "attention":
        return S.attention_forward(state["q"], state["k"], state["v"], key_mask=state["mask"], causal=case["causal"])
    return S.attention_backward(state["do"], state["q"], state["k"], state["v"], state["o"], state["lse"],
                                key_mask=state["mask"], causal=case["causal"])


def run(state):
    if own:
        return _own(state)
    return {"residual_norm": _plain_residual_norm, "residual_norm_grad": _plain_residual_norm_grad, "rope": _plain_rope,
            "attention": _plain_attention, "attention_grad": _plain_attention_grad}[state["case"]["op"]](state)


def work(case):
    op, e = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op in ("residual_norm", "residual_norm_grad"):
        rows, c, g, p = case["rows"], case["channels"], case["groups"], 4 if case["params"] == "fp32" else 2
        post = 1 if case["post"] else 0
        stats = 4 * rows * (1 + post) * (2 if case["kind"] == "layer" else 1)
        if op == "residual_norm":
            return {"bytes": 4 * rows * c * e + (3 + post) * g * c * p + stats, "flops": (12 + 8 * post) * rows * c}
        return {"bytes": 6 * rows * c * e + (5 + 2 * post) * g * c * p + stats, "flops": (20 + 12 * post) * rows * c}
    b, h, hk, d = case["samples"], case["heads"], case["kv_heads"], case["dim"]
    if op == "rope":
        n = case["tokens"]
        pairs = _pairs(case)
        return {"bytes": 2 * b * n * (h + hk) * d * e + 4 * n * len(pairs) + 8 * sum(pairs),
                "flops": 6 * b * n * (h + hk) * sum(pairs)}
    lq, lk = case["queries"], case["keys"]
    pairs = lq * lk
    if case["causal"]:   # the pairs that a query sees
        first = lk - lq + 1
        seen = max(0, min(lq, lq + first - 1))   # queries that see a key
        pairs = seen * (max(first, 1) + lk) // 2
    q, kv, lse = b * lq * h * d * e, b * lk * hk * d * e, 4 * b * h * lq
    mask = b * lk if case["mask"] else 0
    if op == "attention":
        return {"bytes": 2 * q + 2 * kv + lse + mask, "flops": 4 * b * h * d * pairs}
    return {"bytes": 4 * q + 4 * kv + lse + mask, "flops": 10 * b * h * d * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(state):
    """(rows of a group, its parameters in 64 bits) of each group."""
    case = state["case"]
    one = 1.0 if case["one_plus"] else 0.0
    run_of = _rows_per_group(case["rows"], case["groups"])
    for g in range(case["groups"]):
        def of(name, add=0.0):
            p = state[name]
            return None if p is None else (p if p.dim() == 1 else p[g]).double() + add
        yield slice(g * run_of, min((g + 1) * run_of, case["rows"])), of("gate"), of("weight", one), of("bias"), of("post", one)


def _exact_norm(v, kind):
    """(norm(v), mean, rstd) of float64 rows."""
    n = v.shape[1]
    mean = v.sum(1) / n if kind == "layer" else torch.zeros_like(v[:, 0])
    off = v - mean[:, None]
    rstd = 1 / torch.sqrt((off * off).sum(1) / n + EPS)
    return off * rstd[:, None], mean, rstd


def _exact_residual_norm(state):
    kind, x = state["case"]["kind"], state["x"]
    s = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    y = torch.zeros_like(s)
    stats = torch.zeros(4, x.shape[0], dtype=torch.float64, device=x.device)
    for rows, gate, weight, bias, post in _exact_rows(state):
        hn = state["h"][rows].double()
        if not hn.shape[0]:
            continue
        if post is not None:
            hn, stats[2, rows], stats[3, rows] = _exact_norm(hn, kind)
            hn = hn * post
        s[rows] = x[rows].double() + gate * hn
        shat, stats[0, rows], stats[1, rows] = _exact_norm(s[rows].to(x.dtype).double(), kind)
        y[rows] = shat * weight + bias
    keep = [0, 1] if kind == "layer" else [1]
    if state["post"] is not None:
        keep += [2, 3] if kind == "layer" else [3]
    return s, y, stats[keep]


def _exact_residual_norm_grad(state):
    case, kind, s = state["case"], state["case"]["kind"], state["s"]
    stats = state["stats"].double()
    zero = torch.zeros(s.shape[0], dtype=torch.float64, device=s.device)
    n = 2 if kind == "layer" else 1
    mean, rstd = (stats[0], stats[1]) if kind == "layer" else (zero, stats[0])
    if case["post"]:
        hmean, hrstd = (stats[n], stats[n + 1]) if kind == "layer" else (zero, stats[n])
    dx = torch.zeros(s.shape, dtype=torch.float64, device=s.device)
    dh = torch.zeros_like(dx)
    sums = [torch.zeros(case["groups"], s.shape[1], dtype=torch.float64, device=s.device) for _ in range(4)]

    def through(d, hat, r):
        c = d.shape[1]
        inner = c * d - hat * (d * hat).sum(1, keepdim=True)
        if kind == "layer":
            inner = inner - d.sum(1, keepdim=True)
        return r[:, None] / c * inner

    for g, (rows, gate, weight, _, post) in enumerate(_exact_rows(state)):
        dy, h = state["dy"][rows].double(), state["h"][rows].double()
        if not h.shape[0]:
            continue
        shat = (s[rows].double() - mean[rows, None]) * rstd[rows, None]
        t = state["ds"][rows].double() + through(dy * weight, shat, rstd[rows])
        dx[rows], back = t, t * gate
        sums[1][g], sums[2][g] = (dy * shat).sum(0), dy.sum(0)
        if post is None:
            dh[rows], sums[0][g] = back, (t * h).sum(0)
        else:
            hhat = (h - hmean[rows, None]) * hrstd[rows, None]
            sums[0][g], sums[3][g] = (t * hhat * post).sum(0), (back * hhat).sum(0)
            dh[rows] = through(back * post, hhat, hrstd[rows])
    flat = state["gate"].dim() == 1
    sums = [v[0] if flat else v for v in sums]
    return [dx, dh] + (sums if case["post"] else sums[:3])


def _exact_rope(state):
    case, pos = state["case"], state["positions"].double()
    pairs, turn = _pairs(case), -1.0 if case["inverse"] else 1.0
    n = sum(pairs)
    out = []
    for x in (state["q"], state["k"]):
        y = x.double().clone()
        pair = 0
        for axis, count in enumerate(pairs):
            for _ in range(count):
                u, v = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + n)
                z = torch.polar(torch.ones_like(pos[:, axis]), turn * pos[:, axis] * state["freqs"][pair])
                z = z[None, :, None] * torch.complex(x[..., u].double(), x[..., v].double())
                y[..., u], y[..., v] = z.real, z.imag
                pair += 1
        out.append(y)
    return tuple(out)


def _exact_attention(case, state):
    """One query head at a time, in 64 bits; the gradients with the o and the
    lse that the forward left."""
    q, k, v = state["q"], state["k"], state["v"]
    b, lq, h, d = q.shape
    grad, group = case["op"] == "attention_grad", h // case["kv_heads"]
    o = torch.zeros(b, lq, h, d, dtype=torch.float64, device=q.device)
    lse = torch.zeros(b, h, lq, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(o), *(torch.zeros(k.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    for i in range(b):
        seen = torch.ones(lq, case["keys"], dtype=torch.bool, device=q.device)
        if case["causal"]:
            seen = seen.tril(case["keys"] - lq)
        if state["mask"] is not None:
            seen = seen & state["mask"][i]
        for head in range(h):
            q1, k1, v1 = q[i, :, head].double(), k[i, :, head // group].double(), v[i, :, head // group].double()
            s = torch.where(seen, torch.mm(q1, k1.t().contiguous()) * d ** -0.5, -math.inf)
            if not grad:
                lse[i, head] = torch.logsumexp(s, 1)
                p = torch.where(seen, torch.exp(s - lse[i, head][:, None]), 0.0)
                o[i, :, head] = torch.mm(p, v1)
                continue
            do = state["do"][i, :, head].double()
            p = torch.where(seen, torch.exp(s - state["lse"][i, head].double()[:, None]), 0.0)
            delta = (do * state["o"][i, :, head].double()).sum(1)
            ds = p * (torch.mm(do, v1.t().contiguous()) - delta[:, None]) * d ** -0.5
            dq[i, :, head] = torch.mm(ds, k1)
            dk[i, :, head // group] += torch.mm(ds.t().contiguous(), q1)
            dv[i, :, head // group] += torch.mm(p.t().contiguous(), do)
    return (dq, dk, dv) if grad else (o, lse)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "residual_norm":
        return _exact_residual_norm(state)
    if case["op"] == "residual_norm_grad":
        return _exact_residual_norm_grad(state)
    return _exact_rope(state) if case["op"] == "rope" else _exact_attention(case, state)
