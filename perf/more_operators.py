"""The operators that take in a prompt: cases, plain forms and definitions.

A step of many requests, whole prompts and single tokens mixed, runs through a
decoder's layers.  Into a projection goes the normed residual stream, in 16 bits
or as the 8-bit codes and scales that the fused linear layer takes
(``add_rms_norm`` and its gradient, for training).  Beside the projection stands
a low-rank adapter for each request (``lora``).  The new tokens, whose keys and
values have been appended to a paged cache, attend to it: to all of it, or to a
sliding window and the first few places (``ChunkAttention``).

``run`` computes a case in elementary torch operations in 32 bits, or with
``own`` set through the package's entry points.  ``exact`` is each operator's
definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one decode step of seven sequences, the input of an FP8 projection: latency
        dict(name="norm_step", op="norm", dtype="bf16", tokens=7, width=4096, quant="token", residual=True, keep=False),
        # a long prompt into a projection with block scales, the odd token count of packed requests
        dict(name="norm_prompt", op="norm", dtype="bf16", tokens=8191, width=5120, quant="block", residual=True, keep=False),
        # backward pass of a training micro-batch: gradient of the residual stream and of the weight
        dict(name="norm_backward", op="norm_backward", dtype="bf16", tokens=16384, width=4096, quant="none", residual=True, keep=True),
        # a short follow-up question in a running chat: latency
        dict(name="chunk_few", op="attention", dtype="bf16", batch=1, chunk_low=33, chunk_high=33, ctx_low=200, ctx_high=200, q_heads=32, kv_heads=8, dim=128, page=16, heads_first=False, window=0, sinks=0),
        # a decode step of 64 sequences in a layer with a window
        dict(name="window_step", op="attention", dtype="bf16", batch=64, chunk_low=1, chunk_high=1, ctx_low=900, ctx_high=32768, q_heads=32, kv_heads=8, dim=128, page=16, heads_first=False, window=4096, sinks=4),
        # prompts of uneven lengths in a layer with a window, many query heads for each cached one
        dict(name="window_prompt", op="attention", dtype="f16", batch=5, chunk_low=700, chunk_high=4001, ctx_low=0, ctx_high=2500, q_heads=64, kv_heads=8, dim=128, page=64, heads_first=True, window=1024, sinks=16),
        # pieces of long documents: few rows, a long cache that has to be split
        dict(name="chunk_long", op="attention", dtype="bf16", batch=2, chunk_low=512, chunk_high=512, ctx_low=65536, ctx_high=98304, q_heads=32, kv_heads=8, dim=128, page=64, heads_first=False, window=0, sinks=0),
        # one whole prompt from its first token on: the products bound it
        dict(name="chunk_prompt", op="attention", dtype="bf16", batch=1, chunk_low=8192, chunk_high=8192, ctx_low=0, ctx_high=0, q_heads=32, kv_heads=8, dim=128, page=128, heads_first=False, window=0, sinks=0),
        # one token each of five requests with small adapters: latency
        dict(name="lora_step", op="lora", dtype="bf16", sequences=5, prompts=0, tokens=5, inputs=4096, outputs=4096, rank=16, adapters=8, base=True),
        # a decode step of 64 requests, nearly each with an adapter of its own: their weights bound it
        dict(name="lora_many", op="lora", dtype="bf16", sequences=64, prompts=0, tokens=64, inputs=4096, outputs=12288, rank=64, adapters=64, base=True),
        # a few prompts: the activations bound it
        dict(name="lora_prompt", op="lora", dtype="bf16", sequences=5, prompts=5, tokens=8191, inputs=5120, outputs=5120, rank=64, adapters=8, base=True),
        # two prompts among single tokens, a wide input, large adapters
        dict(name="lora_mixed", op="lora", dtype="f16", sequences=33, prompts=2, tokens=6031, inputs=12288, outputs=4096, rank=128, adapters=16, base=False),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "attention", "attention", "attention", "lora", "lora"])
    if op in ("norm", "norm_backward"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        width = _spread(rng, 64, 16384)
        quant = "none" if op == "norm_backward" else rng.choice(["none", "token", "token", "block"])
        width = width // 128 * 128 + 128 if quant == "block" else max(64, width // rng.choice([1, 2, 8, 8]) * rng.choice([1, 2, 8, 8]))
        most = (8191 * 5120 if op == "norm" else 16384 * 4096) * 2 // BYTES[dtype] // width
        return dict(op=op, dtype=dtype, tokens=_spread(rng, 1, min(most, 32768)), width=min(width, 16384), quant=quant,
                    residual=rng.random() < 0.75, keep=quant == "none" or rng.random() < 0.3)
    if op == "attention":
        kv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 4, 5, 7, 8])
        dim = rng.choice([64, 80, 96, 128, 128])
        window = rng.choice([0, 0, _spread(rng, 16, 8192)])
        sinks = rng.choice([0, 1, 4, 64]) if window else 0
        chunk = 1 if rng.random() < 0.3 else _spread(rng, 2, 8192)
        batch = _spread(rng, 1, 64)
        # no more cached values than the long case, no more products than half the whole prompt squared
        chunk = max(1, min(chunk, 8192 * 32 * 128 // (batch * kv * group * dim)))
        seen = 8192 * 4096 * 32 * 128 // (batch * chunk * kv * group * dim)
        most = min((65536 + 98304) * 8 * 128 // (batch * kv * dim), 131072, max(0, seen - chunk // 2) if not window else 131072)
        high = _spread(rng, 1, most + 1) - 1
        return dict(op=op, dtype=rng.choice(["bf16", "f16"]), batch=batch, chunk_low=max(1, chunk // rng.choice([1, 3])), chunk_high=chunk,
                    ctx_low=rng.choice([0, high // 2, high]), ctx_high=high, q_heads=kv * group, kv_heads=kv, dim=dim,
                    page=rng.choice([8, 16, 24, 32, 48, 64, 128, 256]), heads_first=rng.random() < 0.5, window=window, sinks=sinks)
    rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
    inputs, outputs = (_spread(rng, 16, 1536) * 8 for _ in range(2))
    adapters = _spread(rng, 1, 32)
    sequences = _spread(rng, 1, 64)
    prompts = rng.choice([0, sequences, rng.randint(0, sequences)])
    base = rng.random() < 0.7
    most = 6031 * (12288 + 4096) // (inputs + outputs * (1 + base))
    tokens = sequences if prompts == 0 else max(sequences, _spread(rng, sequences, max(sequences, min(most, 8192))))
    return dict(op=op, dtype=rng.choice(["bf16", "f16"]), sequences=sequences, prompts=prompts, tokens=tokens, inputs=inputs, outputs=outputs,
                rank=rank, adapters=adapters, base=base)


def _lengths(case):
    """Cached lengths and new tokens of each sequence, by the case alone; each seed gets them in another order."""
    r = np.random.RandomState(case["batch"] * 7919 + case["chunk_high"])
    ctx = r.randint(case["ctx_low"], case["ctx_high"] + 1, case["batch"])
    ctx[0], ctx[-1] = case["ctx_low"], case["ctx_high"]
    n = r.randint(case["chunk_low"], case["chunk_high"] + 1, case["batch"])
    n[-1] = case["chunk_high"]
    return ctx, n


def _requests(case):
    """Tokens and adapter of each sequence, by the case alone: prompts share what single tokens leave; one in eight has no adapter."""
    r = np.random.RandomState(case["sequences"] * 7919 + case["tokens"])
    n = np.ones(case["sequences"], np.int64)
    if case["prompts"]:
        share = r.dirichlet(np.full(case["prompts"], 3.0))
        extra = np.floor(share * (case["tokens"] - case["sequences"])).astype(np.int64)
        extra[0] += case["tokens"] - case["sequences"] - extra.sum()
        n[:case["prompts"]] += extra
    adapter = r.permutation(max(case["adapters"], case["sequences"]))[:case["sequences"]] % case["adapters"]
    adapter[r.random_sample(case["sequences"]) < 0.125] = -1
    adapter[0] = max(adapter[0], 0)
    return n, adapter


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("norm", "norm_backward"):
        values = case["tokens"] * case["width"]
        if op == "norm_backward":
            return {"bytes": 4 * values * e + case["width"] * (e + 4), "flops": 12 * values}
        codes = {"none": 0, "token": values + 4 * case["tokens"], "block": values + values // 32}[case["quant"]]
        return {"bytes": values * e * (1 + 2 * case["residual"] + case["keep"]) + codes + case["width"] * e, "flops": 8 * values}
    if op == "attention":
        ctx, n = _lengths(case)
        pairs = keys = 0
        for c, m in zip(ctx.tolist(), n.tolist()):
            place = np.arange(c, c + m, dtype=np.int64)
            if case["window"]:
                low = np.maximum(place - case["window"] + 1, 0)
                pairs += int((place + 1 - low + np.minimum(low, case["sinks"])).sum())
                keys += int(c + m - low[0] + min(low[0], case["sinks"]))
            else:
                pairs += int((place + 1).sum())
                keys += c + m
        bytes_ = 2 * keys * case["kv_heads"] * case["dim"] * e + 2 * int(n.sum()) * case["q_heads"] * case["dim"] * e
        return {"bytes": bytes_ + 4 * -(-keys // case["page"]), "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    n, adapter = _requests(case)
    held = len(set(adapter[adapter >= 0].tolist())) * case["rank"] * (case["inputs"] + case["outputs"])
    with_one = int(n[adapter >= 0].sum())
    moved = with_one * case["inputs"] + case["tokens"] * case["outputs"] * (1 + case["base"])
    return {"bytes": (moved + held) * e, "flops": 2 * with_one * case["rank"] * (case["inputs"] + case["outputs"])}


# ----------------------------------------------------------------- inputs ---

def _prepare_norm(case, gen, s):
    dt, t, k = DTYPES[case["dtype"]], case["tokens"], case["width"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    # a residual stream has a few columns that are far larger than the rest
    column = 1 + 12 * (torch.rand(k, generator=gen, device="cuda") < 0.003).float()
    s["weight"] = (1 + 0.2 * normal(k)).to(dt)
    if case["op"] == "norm_backward":
        s["sum"] = (normal(t, k) * 2 * column).to(dt)
        s["d_out"] = (normal(t, k) * 0.1).to(dt)
        s["d_sum"] = (normal(t, k) * 0.1).to(dt) if case["residual"] else None
        return
    s["x"] = normal(t, k).to(dt)
    s["residual"] = (normal(t, k) * 2 * column).to(dt) if case["residual"] else None


def _prepare_attention(case, gen, s):
    dt, d, hq, hk, page = DTYPES[case["dtype"]], case["dim"], case["q_heads"], case["kv_heads"], case["page"]
    rng = np.random.RandomState(s["seed"] % (1 << 31))
    ctx, n = _lengths(case)
    order = rng.permutation(len(ctx))
    ctx, n = ctx[order], n[order]
    total, lens = int(n.sum()), ctx + n
    need = -(-lens // page)
    pages = int(need.sum()) + 2
    free = rng.permutation(pages)
    table = np.full((len(ctx), int(need.max()) + 1), -1, np.int32)  # entries past a sequence's length hold nothing
    at = 0
    for b in range(len(ctx)):
        table[b, :need[b]] = free[at:at + need[b]]
        at += need[b]
    s["max_len"], s["max_chunk"], s["window"], s["sinks"] = int(lens.max()), case["chunk_high"], case["window"], case["sinks"]
    s["q"] = torch.randn((total, hq, d), generator=gen, device="cuda").to(dt)
    shape = (pages, hk, page, d) if case["heads_first"] else (pages, page, hk, d)
    s["block_table"] = torch.from_numpy(table).cuda()
    s["context_lens"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
    s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    # slots that hold no token have whatever was there before: not a number stands for it
    used = np.zeros((pages, page), bool)
    for b in range(len(ctx)):
        used.reshape(-1)[(table[b, :need[b], None].astype(np.int64) * page + np.arange(page)).reshape(-1)[:lens[b]]] = True
    used = torch.from_numpy(used).cuda()
    used = used[:, None, :, None] if case["heads_first"] else used[:, :, None, None]
    for name in ("k_cache", "v_cache"):
        c = torch.randn(shape, generator=gen, device="cuda", dtype=dt).masked_fill_(~used, math.nan)
        s[name] = c.permute(0, 2, 1, 3) if case["heads_first"] else c
    s["scale"] = d ** -0.5
    if own:
        import epilogue_tcgen05_tmem_gb300 as eg
        s["plan"] = eg.ChunkAttention(hq, hk, d, case["dtype"], page, max_batch=case["batch"], max_chunk=case["chunk_high"])


def _prepare_lora(case, gen, s):
    dt, r = DTYPES[case["dtype"]], case["rank"]
    rng = np.random.RandomState(s["seed"] % (1 << 31))
    n, adapter = _requests(case)
    order = rng.permutation(len(n))
    n, adapter = n[order], adapter[order]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dt)

    s["x"] = normal(case["tokens"], case["inputs"])
    s["a"] = normal(case["adapters"], r, case["inputs"], scale=case["inputs"] ** -0.5)
    s["b"] = normal(case["adapters"], case["outputs"], r, scale=r ** -0.5)
    s["scales"] = (0.5 + torch.rand(case["adapters"], generator=gen, device="cuda")).float()
    s["seq_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    s["adapter"] = torch.from_numpy(adapter.astype(np.int32)).cuda()
    s["base"] = normal(case["tokens"], case["outputs"]) if case["base"] else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"op": case["op"], "seed": seed, "quant": case.get("quant"), "keep": case.get("keep")}
    if case["op"] in ("norm", "norm_backward"):
        _prepare_norm(case, gen, s)
    elif case["op"] == "attention":
        _prepare_attention(case, gen, s)
    else:
        _prepare_lora(case, gen, s)
    return s


# ------------------------------------------------------------ plain forms ---

def _plain_norm(s):
    x = s["x"]
    total = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    z = total.float()
    h = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out = {}
    if s["residual"] is not None:
        out["sum"] = total
    if s["keep"]:
        out["out"] = h.to(x.dtype)
    if s["quant"] != "none":
        part = h.unflatten(-1, (-1, 128)) if s["quant"] == "block" else h
        most = part.abs().amax(-1, keepdim=True)
        scale = torch.where(most > 0, most / E4M3_MAX, 1.0)
        out["codes"] = (part / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(h.shape)
        out["scales"] = scale.squeeze(-1)
    return out


def _plain_norm_backward(s):
    z, d, w = s["sum"].float(), s["d_out"].float(), s["weight"].float()
    r = torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS)
    h = z * r
    g = d * w
    dx = r * (g - h * (g * h).mean(-1, keepdim=True))
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].float()
    return {"dx": dx.to(s["sum"].dtype), "d_weight": (d * h).sum(0)}


def _plain_attention(s):
    """Queries in blocks of the window's length (one block without a window): each against the places that any of its
    tokens can see."""
    q, start, ctx = s["q"], s["q_start"].long(), s["context_lens"].long()
    page, hk, d = s["k_cache"].shape[1:]
    total, hq = q.shape[:2]
    window, sinks, chunk = s["window"], s["sinks"], s["max_chunk"]
    batch, group, dev = ctx.shape[0], hq // hk, q.device
    n = start[1:] - start[:-1]
    each = min(chunk, max(window, 128)) if window else chunk
    blocks = -(-chunk // each)
    step = torch.arange(blocks * each, device=dev).view(blocks, each)
    place = ctx[:, None, None] + step                                     # [batch, block, token]
    if window:
        low = (place[:, :, :1] - window + 1).clamp(min=sinks)
        at = torch.cat([torch.arange(sinks, device=dev).expand(batch, blocks, -1), low + torch.arange(min(window + each, s["max_len"]), device=dev)], -1)
    else:
        at = torch.arange(s["max_len"], device=dev).expand(batch, blocks, -1)
    held = at < (ctx + n)[:, None, None]                                  # [batch, block, key]
    entry = (at // page).clamp(max=s["block_table"].shape[1] - 1)
    pages = torch.gather(s["block_table"].long(), 1, entry.flatten(1)).view(at.shape).clamp(min=0)
    k = torch.where(held[..., None, None], s["k_cache"][pages, at % page].float(), 0.0)
    v = torch.where(held[..., None, None], s["v_cache"][pages, at % page].float(), 0.0)
    token = (start[:-1, None, None] + step).clamp(max=total - 1)
    rows = q[token].float().view(batch, blocks, each, hk, group, d).permute(0, 1, 3, 4, 2, 5).reshape(batch, blocks, hk, -1, d)
    score = torch.matmul(rows, k.permute(0, 1, 3, 4, 2)).view(batch, blocks, hk, group, each, -1) * s["scale"]
    far = place[..., None] - at[:, :, None, :]                            # [batch, block, token, key]
    sees = (far >= 0) & held[:, :, None, :]
    if window:
        sees &= (far < window) | (at[:, :, None, :] < sinks)
    score.masked_fill_(~sees[:, :, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    weight = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(weight == 0, 1.0, weight))
    o = torch.matmul(p.view(batch, blocks, hk, group * each, -1), v.permute(0, 1, 3, 2, 4)).view(batch, blocks, hk, group, each, d)
    seq = torch.searchsorted(start, torch.arange(total, device=dev), right=True) - 1
    t = torch.arange(total, device=dev) - start[seq]
    return o[seq, t // each, :, :, t % each].reshape(total, hq, d).to(q.dtype)


def _plain_lora(s):
    x, a, b = s["x"], s["a"], s["b"]
    tokens, (adapters, rank, inputs) = x.shape[0], a.shape
    seq = torch.searchsorted(s["seq_start"].long(), torch.arange(tokens, device=x.device), right=True) - 1
    whose = s["adapter"].long()[seq]
    # every adapter's products, of which a token keeps its own
    mine = torch.where(whose[:, None] == torch.arange(adapters, device=x.device), s["scales"], 0.0)
    h = (x.float() @ a.float().view(-1, inputs).T).view(tokens, adapters, rank) * mine[..., None]
    y = h.view(tokens, -1) @ b.float().permute(0, 2, 1).reshape(adapters * rank, -1)
    return (y if s["base"] is None else s["base"].float() + y).to(x.dtype)


PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "attention": _plain_attention, "lora": _plain_lora}


# ------------------------------------------------------------ entry points --

def _own(s):
    import epilogue_tcgen05_tmem_gb300 as eg
    op = s["op"]
    if op == "norm":
        quant = {"none": None, "token": "e4m3", "block": "e4m3_block"}[s["quant"]]
        r = eg.add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant=quant, keep_out=s["keep"])
        out = {}
        if s["residual"] is not None:
            out["sum"] = r.sum
        if s["keep"]:
            out["out"] = r.out
        if quant:
            out["codes"] = r.codes.view(torch.float8_e4m3fn)
            out["scales"] = r.scales if s["quant"] == "block" else r.scales.view(-1)
        return out
    if op == "norm_backward":
        dx, dw = eg.add_rms_norm_backward(s["d_out"], s["sum"], s["weight"], eps=EPS, d_sum=s["d_sum"])
        return {"dx": dx, "d_weight": dw}
    if op == "attention":
        return s["plan"].run(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["context_lens"], s["q_start"], window=s["window"], sinks=s["sinks"],
                             scale=s["scale"])
    return eg.lora(s["x"], s["a"], s["b"], s["seq_start"], s["adapter"], scales=s["scales"], base=s["base"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------ definitions ---

def _exact_norm(s):
    x = s["x"]
    total = x.double() if s["residual"] is None else x.double() + s["residual"].double()
    stored = total.to(x.dtype).double()
    norm = (stored.pow(2).sum(-1, keepdim=True) / stored.shape[-1] + EPS).sqrt()
    h = s["weight"].double() * stored / norm
    out = {}
    if s["residual"] is not None:
        out["sum"] = total
    if s["keep"]:
        out["out"] = h
    if s["quant"] != "none":
        parts = h.view(h.shape[0], -1, 128 if s["quant"] == "block" else h.shape[1])
        scale = parts.abs().max(-1).values / E4M3_MAX
        scale[scale == 0] = 1.0
        out["codes"] = (parts / scale[..., None]).view(h.shape)
        out["scales"] = scale if s["quant"] == "block" else scale[:, 0]
    return out


def _exact_norm_backward(s):
    z, d = s["sum"].double(), s["d_out"].double()
    k = z.shape[1]
    mean = z.pow(2).sum(-1, keepdim=True) / k + EPS
    g = d * s["weight"].double()
    # the derivative of z / sqrt(mean) by z, applied to g
    dx = g / mean.sqrt() - z * (g * z).sum(-1, keepdim=True) / (k * mean.pow(1.5))
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].double()
    return {"dx": dx, "d_weight": torch.einsum("tk,tk->k", d, z / mean.sqrt())}


def _exact_attention(s):
    q, page = s["q"], s["k_cache"].shape[1]
    total, hq, d = q.shape
    hk = s["k_cache"].shape[2]
    start, ctx, table = s["q_start"].tolist(), s["context_lens"].tolist(), s["block_table"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for b in range(len(ctx)):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        length = ctx[b] + n
        ids = torch.tensor([table[b][j] for j in range(-(-length // page))], device=q.device)
        place = torch.arange(ctx[b], length, device=q.device)[:, None]
        j = torch.arange(length, device=q.device)
        hidden = j > place
        if s["window"]:
            hidden |= (j <= place - s["window"]) & (j >= s["sinks"])
        for h in range(hk):
            keys = s["k_cache"][ids, :, h].reshape(-1, d)[:length].double()
            values = s["v_cache"][ids, :, h].reshape(-1, d)[:length].double()
            for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                score = (q[start[b]:start[b + 1], g].double() @ keys.T * s["scale"]).masked_fill_(hidden, -math.inf)
                out[start[b]:start[b + 1], g] = torch.softmax(score, 1) @ values
    return out


def _exact_lora(s):
    start, adapter = s["seq_start"].tolist(), s["adapter"].tolist()
    out = torch.zeros((s["x"].shape[0], s["b"].shape[1]), dtype=torch.float64, device=s["x"].device)
    if s["base"] is not None:
        out += s["base"].double()
    for b, of in enumerate(adapter):
        if of >= 0:
            rows = slice(start[b], start[b + 1])
            inner = torch.einsum("tk,rk->tr", s["x"][rows].double(), s["a"][of].double())
            out[rows] += s["scales"][of].double() * torch.einsum("tr,nr->tn", inner, s["b"][of].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "attention": _exact_attention, "lora": _exact_lora}[case["op"]](s)
