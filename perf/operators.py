"""The attention-side operators of a decoder layer: cases, plain forms and definitions.

Four operators stand around the fused linear layer.  The projection of a layer
gives queries, keys and values; they are normed per head and rotated by their
positions (``qk_norm_rope`` and its gradient, for training); while serving the
same step appends keys and values to a paged cache (``kv_append``); the tokens
of a drafted tree, or one token, attend to that cache (``TreeAttention``); and
the head's logits are scored: log probabilities of given tokens, entropy and
the top alternatives, with their gradient (``token_logprobs``).

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


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # a handful of prompt tokens of a small model: latency; neighbouring pairs rotated, part of the head only
        dict(name="rope_few", op="rope_forward", dtype="f16", tokens=37, q_heads=12, kv_heads=4, dim=96, rot=48, pairs=True, norm=True),
        # forward pass of a training micro-batch, packed documents (a ragged token count)
        dict(name="rope_forward", op="rope_forward", dtype="bf16", tokens=8191, q_heads=32, kv_heads=8, dim=128, rot=128, pairs=False, norm=True),
        # its backward pass at twice the tokens: gradients of queries, keys and both norm weights
        dict(name="rope_backward", op="rope_backward", dtype="bf16", tokens=16384, q_heads=32, kv_heads=8, dim=128, rot=128, pairs=False, norm=True),
        # one decode step of seven sequences: latency
        dict(name="append_step", op="append", dtype="bf16", tokens=7, q_heads=32, kv_heads=8, dim=128, rot=128, pairs=False, norm=True, page=16, heads_first=False),
        # a long prompt written into the cache, heads-first pages that are no power of two, no norm
        dict(name="append_prompt", op="append", dtype="f16", tokens=24593, q_heads=32, kv_heads=8, dim=128, rot=64, pairs=True, norm=False, page=48, heads_first=True),
        # one token of one sequence over a short cache: latency
        dict(name="attend_token", op="attention", dtype="bf16", batch=1, tree=1, ctx_low=517, ctx_high=517, q_heads=32, kv_heads=8, dim=128, page=16, heads_first=False, chain=True),
        # one token each of two sequences over long caches: the cache has to be split over the whole GPU
        dict(name="attend_long", op="attention", dtype="bf16", batch=2, tree=1, ctx_low=98304, ctx_high=131072, q_heads=32, kv_heads=8, dim=128, page=64, heads_first=True, chain=True),
        # drafted trees of up to 13 tokens, ragged caches, one of them empty
        dict(name="attend_tree", op="attention", dtype="bf16", batch=24, tree=13, ctx_low=0, ctx_high=9001, q_heads=32, kv_heads=8, dim=128, page=16, heads_first=False, chain=False),
        # wide trees with many query heads for each cached head: the products bound it
        dict(name="attend_wide", op="attention", dtype="f16", batch=16, tree=64, ctx_low=3800, ctx_high=8200, q_heads=64, kv_heads=8, dim=128, page=128, heads_first=False, chain=False),
        # the last positions of a few drafts, an odd vocabulary, five alternatives each: latency
        dict(name="score_few", op="score", dtype="f32", rows=5, vocab=50021, top=5),
        # scoring a batch of prompts: all positions, the usual count of alternatives
        dict(name="score_prompts", op="score", dtype="bf16", rows=4096, vocab=131072, top=20),
        # policy-gradient step: gradient of log probability and entropy to the logits
        dict(name="score_backward", op="score_backward", dtype="f32", rows=2048, vocab=100003, top=0),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["rope_forward", "rope_backward", "append", "attention", "attention", "attention", "score", "score_backward"])
    if op in ("rope_forward", "rope_backward", "append"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        kv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2])
        # no more values than the largest listed case of its kind has
        most = {"rope_forward": 8191 * 40 * 128, "rope_backward": 16384 * 40 * 128, "append": 24593 * 48 * 128}[op]
        most = most * 2 // BYTES[dtype] // ((kv * group + 2 * kv) * dim)
        case = dict(op=op, dtype=dtype, tokens=_spread(rng, 1, min(most, 32768)), q_heads=kv * group, kv_heads=kv, dim=dim, rot=rot,
                    pairs=rng.random() < 0.4, norm=rng.random() < 0.7 or op == "rope_backward")
        if op == "append":
            case.update(page=rng.choice([1, 8, 16, 24, 32, 64, 128]), heads_first=rng.random() < 0.5)
        return case
    if op == "attention":
        kv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 4, 5, 7, 8])
        dim = rng.choice([64, 80, 96, 128, 128])
        tree = 1 if rng.random() < 0.4 else _spread(rng, 2, 64)
        batch = _spread(rng, 1, 48)
        # no more cached values than the long case, no more products than the wide one
        most = min(2 * 131072 * 8 * 128 // (batch * kv * dim), 16 * 64 * 64 * 8200 * 128 // (batch * tree * kv * group * dim), 131072)
        high = _spread(rng, 1, max(1, most))
        low = rng.choice([0, high // 2, high])
        return dict(op=op, dtype=rng.choice(["bf16", "f16"]), batch=batch, tree=tree, ctx_low=low, ctx_high=high, q_heads=kv * group, kv_heads=kv,
                    dim=dim, page=rng.choice([8, 16, 24, 32, 48, 64, 128, 256]), heads_first=rng.random() < 0.5, chain=tree == 1 or rng.random() < 0.3)
    dtype = rng.choice(["bf16", "f16", "f32"])
    vocab = _spread(rng, 1000, 160000)
    most = (4096 * 131072 if op == "score" else 2048 * 100003) * 2 // BYTES[dtype] // vocab
    return dict(op=op, dtype=dtype, rows=_spread(rng, 1, min(most, 8192)), vocab=vocab, top=rng.choice([0, 1, 5, 20]) if op == "score" else 0)


def _lengths(case):
    """Cached lengths and drafted tokens of each sequence, by the case alone; each seed gets them in another order."""
    r = np.random.RandomState(case["batch"] * 7919 + case["tree"])
    ctx = r.randint(case["ctx_low"], case["ctx_high"] + 1, case["batch"])
    ctx[0], ctx[-1] = case["ctx_low"], case["ctx_high"]
    n = r.randint((case["tree"] + 1) // 2, case["tree"] + 1, case["batch"])
    n[-1] = case["tree"]
    return ctx, n


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("rope_forward", "rope_backward", "append"):
        values = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        side = case["tokens"] * (8 + 4 * case["rot"])  # position and its row of the table
        weights = 2 * case["dim"] * e if case["norm"] else 0
        if op == "rope_forward":
            return {"bytes": 2 * values * e + side + weights, "flops": 8 * values}
        if op == "rope_backward":
            return {"bytes": 3 * values * e + side + weights + 8 * case["dim"], "flops": 16 * values}
        appended = case["tokens"] * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * (values + appended) * e + side + weights + 8 * case["tokens"], "flops": 8 * values}
    if op == "attention":
        ctx, n = _lengths(case)
        keys, tokens = int((ctx + n).sum()), int(n.sum())
        pairs = int((ctx * n + n).sum())
        bytes_ = 2 * keys * case["kv_heads"] * case["dim"] * e + 2 * tokens * case["q_heads"] * case["dim"] * e
        return {"bytes": bytes_ + 4 * int((-(-(ctx + n) // case["page"])).sum()), "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    logits = case["rows"] * case["vocab"]
    if op == "score":
        return {"bytes": logits * e + case["rows"] * (8 + 12 + 12 * case["top"]), "flops": 5 * logits}
    return {"bytes": 2 * logits * e + case["rows"] * 24, "flops": 6 * logits}


# ----------------------------------------------------------------- inputs ---

def _positions(gen, tokens):
    """Positions of packed documents: they count up and start again."""
    start = torch.rand(tokens, generator=gen, device="cuda") < 1 / 700
    at = torch.arange(tokens, device="cuda")
    return at - torch.cummax(torch.where(start, at, torch.zeros_like(at)), 0).values


def _table(count, rot):
    """Cosines, then sines, of each position."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(count, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _prepare_rope(case, gen, s):
    dt, d, hq, hk, t = DTYPES[case["dtype"]], case["dim"], case["q_heads"], case["kv_heads"], case["tokens"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    # queries, keys and values are parts of one projection's output
    qkv = (normal(t, hq + 2 * hk, d) * 1.5).to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    s["q_weight"] = (1 + 0.2 * normal(d)).to(dt) if case["norm"] else None
    s["k_weight"] = (1 + 0.2 * normal(d)).to(dt) if case["norm"] else None
    s["positions"] = _positions(gen, t)
    s["table"] = _table(max(4096, t), case["rot"])
    if case["op"] == "rope_backward":
        s["dq_out"], s["dk_out"] = (normal(t, hq, d) * 0.1).to(dt), (normal(t, hk, d) * 0.1).to(dt)
    if case["op"] == "append":
        page = case["page"]
        pages = -(-t // page) + 3
        shape = (pages, hk, page, d) if case["heads_first"] else (pages, page, hk, d)
        for name in ("k_cache", "v_cache"):
            c = normal(*shape).to(dt)
            s[name] = c.permute(0, 2, 1, 3) if case["heads_first"] else c
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda")
        s["slots"] = order[at // page] * page + at % page
        if t > 4:
            s["slots"][t // 2] = -1  # a padded token: nothing is appended


def _ancestors(rng, n):
    """Which tokens of a random drafted tree each token sees: its ancestors and itself."""
    sees = np.zeros((n, n), bool)
    for i in range(n):
        if i and rng.random_sample() < 0.9:
            sees[i] = sees[rng.randint(max(0, i - 8), i)]
        sees[i, i] = True
    return sees


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
    mask = np.zeros((total, -(-case["tree"] // 32)), np.uint32)
    at = row = 0
    for b in range(len(ctx)):
        table[b, :need[b]] = free[at:at + need[b]]
        at += need[b]
        sees = np.zeros((n[b], mask.shape[1] * 32), bool)
        sees[:, :n[b]] = _ancestors(rng, n[b])
        mask[row:row + n[b]] = np.packbits(sees, axis=1, bitorder="little").view(np.uint32)
        row += n[b]
    s["max_len"], s["max_tree"] = int(lens.max()), case["tree"]
    s["q"] = torch.randn((total, hq, d), generator=gen, device="cuda").to(dt)
    shape = (pages, hk, page, d) if case["heads_first"] else (pages, page, hk, d)
    s["block_table"] = torch.from_numpy(table).cuda()
    s["context_lens"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
    s["q_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
    s["mask"] = None if case["chain"] else torch.from_numpy(mask.view(np.int32)).cuda()
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
        s["plan"] = eg.TreeAttention(hq, hk, d, case["dtype"], page, max_batch=case["batch"], max_tree=case["tree"])


def _prepare_score(case, gen, s):
    rows, vocab = case["rows"], case["vocab"]
    x = torch.randn((rows, vocab), generator=gen, device="cuda", dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32).mul_(2.5)
    x[:, vocab - vocab // 100:] = -math.inf  # a vocabulary padded up, its last entries masked
    s["logits"] = x.to(DTYPES[case["dtype"]])
    s["tokens"] = torch.randint(0, vocab - vocab // 100, (rows,), generator=gen, device="cuda")
    if rows > 4:
        s["tokens"][rows // 3] = -1  # a position without a given token
    s["top"] = case["top"]
    if case["op"] == "score_backward":
        lse, entropy = [], []
        for part in s["logits"].split(256):
            y = part.double()
            z = torch.logsumexp(y, 1)
            lse.append(z)
            y = (y - z[:, None]).clamp_(min=-1e4)
            entropy.append(-(y.exp() * y).sum(1))
        s["lse"], s["entropy"] = torch.cat(lse).float(), torch.cat(entropy).float()
        s["d_logprob"] = torch.randn((rows,), generator=gen, device="cuda")
        s["d_entropy"] = torch.randn((rows,), generator=gen, device="cuda") * 0.05


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"op": case["op"], "seed": seed, "rot": case.get("rot"), "pairs": case.get("pairs")}
    if case["op"] in ("rope_forward", "rope_backward", "append"):
        _prepare_rope(case, gen, s)
    elif case["op"] == "attention":
        _prepare_attention(case, gen, s)
    else:
        _prepare_score(case, gen, s)
    return s


# ------------------------------------------------------------ plain forms ---

def _split(x, rot, pairs):
    """The two halves of the rotated part, and the rest."""
    if pairs:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _join(a, b, rest, pairs):
    if pairs:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _rotation(s):
    row = s["table"][s["positions"]][:, None, :]
    return row[..., :s["rot"] // 2], row[..., s["rot"] // 2:]


def _norm_rope(x, weight, cos, sin, s):
    z = x.float()
    if weight is not None:
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS) * weight.float()
    a, b, rest = _split(z, s["rot"], s["pairs"])
    return _join(a * cos - b * sin, b * cos + a * sin, rest, s["pairs"]).to(x.dtype)


def _norm_rope_backward(dy, x, weight, cos, sin, s):
    a, b, rest = _split(dy.float(), s["rot"], s["pairs"])
    dz = _join(a * cos + b * sin, b * cos - a * sin, rest, s["pairs"])
    z = x.float()
    r = torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS)
    h = z * r
    g = dz * weight.float()
    dx = r * (g - h * (g * h).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dz * h).sum((0, 1))


def _plain_rope(s):
    cos, sin = _rotation(s)
    return {"q": _norm_rope(s["q"], s["q_weight"], cos, sin, s), "k": _norm_rope(s["k"], s["k_weight"], cos, sin, s)}


def _plain_rope_backward(s):
    cos, sin = _rotation(s)
    dq, dwq = _norm_rope_backward(s["dq_out"], s["q"], s["q_weight"], cos, sin, s)
    dk, dwk = _norm_rope_backward(s["dk_out"], s["k"], s["k_weight"], cos, sin, s)
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def _plain_append(s):
    cos, sin = _rotation(s)
    q = _norm_rope(s["q"], s["q_weight"], cos, sin, s)
    k = _norm_rope(s["k"], s["k_weight"], cos, sin, s)
    page = s["k_cache"].shape[1]
    put = s["slots"] >= 0
    # a token without a slot writes what the first slot gets, so nothing of it stays
    slot = torch.where(put, s["slots"], s["slots"][0])
    keep = put[:, None, None]
    s["k_cache"][slot // page, slot % page] = torch.where(keep, k, k[:1])
    s["v_cache"][slot // page, slot % page] = torch.where(keep, s["v"], s["v"][:1])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    q, start, ctx = s["q"], s["q_start"].long(), s["context_lens"].long()
    page, hk, d = s["k_cache"].shape[1:]
    total, hq = q.shape[:2]
    batch, tree = ctx.shape[0], s["max_tree"]
    n = start[1:] - start[:-1]
    at = torch.arange(s["max_len"], device="cuda")
    filled = (at < (ctx + n)[:, None])[:, :, None, None]
    pages = s["block_table"][:, at // page].long().clamp(min=0)
    k = torch.where(filled, s["k_cache"][pages, at % page].float(), 0.0)
    v = torch.where(filled, s["v_cache"][pages, at % page].float(), 0.0)
    step = torch.arange(tree, device="cuda")
    token = (start[:-1, None] + step).clamp(max=total - 1)
    rows = q[token].float().view(batch, tree, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(batch, hk, -1, d)
    score = torch.matmul(rows, k.permute(0, 2, 3, 1)).view(batch, hk, hq // hk, tree, -1) * s["scale"]
    drafted = (at - ctx[:, None])[:, None, :]  # [batch, 1, key]: the key's place in its tree
    if s["mask"] is None:
        sees = drafted <= step[:, None]
    else:
        bit = drafted.clamp(min=0, max=s["mask"].shape[1] * 32 - 1).expand(-1, tree, -1)
        sees = (drafted < 0) | ((torch.gather(s["mask"][token], 2, bit // 32) >> (bit % 32)) & 1).bool()
    sees = (sees & (drafted < n[:, None, None]))[:, None, None]
    score = torch.where(sees, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total_p = p.sum(-1, keepdim=True)
    p = p / torch.where(total_p == 0, 1.0, total_p)
    o = torch.matmul(p.view(batch, hk, -1, s["max_len"]), v.permute(0, 2, 1, 3)).view(batch, hk, hq // hk, tree, d)
    seq = torch.searchsorted(start, torch.arange(total, device="cuda"), right=True) - 1
    return o[seq, :, :, torch.arange(total, device="cuda") - start[seq]].reshape(total, hq, d).to(q.dtype)


def _ordered(x):
    """Whole numbers that are ordered as the values of x are."""
    i = (x + 0.0).view(torch.int32)
    return torch.where(i < 0, i ^ 0x7FFFFFFF, i)


def _plain_score(s):
    x = s["logits"].float()
    lse = torch.logsumexp(x, 1)
    logp = x - lse[:, None]
    given = torch.gather(logp, 1, s["tokens"].clamp(min=0)[:, None])[:, 0]
    out = {"logprob": torch.where(s["tokens"] >= 0, given, 0.0), "lse": lse}
    out["entropy"] = -torch.where(logp == -math.inf, 0.0, torch.exp(logp) * logp).sum(1)
    if s["top"]:
        # one whole number for value and place, so that of equal values the lowest place comes first
        place = x.shape[1] - 1 - torch.arange(x.shape[1], device="cuda")
        key = torch.topk((_ordered(x).long() << 32) + place, s["top"], dim=1).values
        out["top_ids"] = x.shape[1] - 1 - (key & 0xFFFFFFFF)
        out["top_logprobs"] = torch.gather(logp, 1, out["top_ids"])
    return out


def _plain_score_backward(s):
    x = s["logits"].float()
    logp = x - s["lse"][:, None]
    p = torch.exp(logp)
    inner = torch.where(p > 0, logp + s["entropy"][:, None], 0.0)
    put = s["tokens"] >= 0
    d = -p * (torch.where(put, s["d_logprob"], 0.0)[:, None] + s["d_entropy"][:, None] * inner)
    d.scatter_add_(1, s["tokens"].clamp(min=0)[:, None], torch.where(put, s["d_logprob"], 0.0)[:, None])
    return d.to(s["logits"].dtype)


PLAIN = {"rope_forward": _plain_rope, "rope_backward": _plain_rope_backward, "append": _plain_append,
         "attention": _plain_attention, "score": _plain_score, "score_backward": _plain_score_backward}


# ------------------------------------------------------------ entry points --

def _own(s):
    import epilogue_tcgen05_tmem_gb300 as eg
    op = s["op"]
    if op == "rope_forward":
        q, k = eg.qk_norm_rope(s["q"], s["k"], s["table"], positions=s["positions"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                               eps=EPS, pairs=s["pairs"])
        return {"q": q, "k": k}
    if op == "rope_backward":
        dq, dk, dwq, dwk = eg.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["table"], positions=s["positions"],
                                                    q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, pairs=s["pairs"])
        return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}
    if op == "append":
        q = eg.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], q=s["q"], cos_sin=s["table"], positions=s["positions"],
                         q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, pairs=s["pairs"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "attention":
        return s["plan"].run(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["context_lens"], s["q_start"], mask=s["mask"], scale=s["scale"])
    if op == "score":
        r = eg.token_logprobs(s["logits"], s["tokens"], top=s["top"])
        out = {"logprob": r.logprob, "lse": r.lse, "entropy": r.entropy}
        if s["top"]:
            out.update(top_ids=r.top_ids, top_logprobs=r.top_logprobs)
        return out
    return eg.token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], s["d_logprob"], s["d_entropy"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------ definitions ---

def _exact_rotate(z, s, turn):
    """Each rotated pair of coordinates as a complex number, turned by its angle (turn 1) or back (turn -1)."""
    half = s["rot"] // 2
    row = s["table"].double()[s["positions"]]
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if s["pairs"] else (i, i + half)
    y = torch.complex(z[..., first], z[..., second]) * torch.complex(row[:, :half], turn * row[:, half:])[:, None]
    out = z.clone()
    out[..., first], out[..., second] = y.real, y.imag
    return out


def _exact_rope(x, weight, s):
    z = x.double()
    if weight is not None:
        z = weight.double() * z / (z.pow(2).sum(-1, keepdim=True) / z.shape[-1] + EPS).sqrt()
    return _exact_rotate(z, s, 1)


def _exact_rope_backward(dy, x, weight, s):
    dz, z = _exact_rotate(dy.double(), s, -1), x.double()
    mean = z.pow(2).sum(-1, keepdim=True) / z.shape[-1] + EPS
    g = dz * weight.double()
    # the derivative of z / sqrt(mean) by z, applied to g
    return g / mean.sqrt() - z * (g * z).sum(-1, keepdim=True) / (z.shape[-1] * mean.pow(1.5)), (dz * z / mean.sqrt()).sum((0, 1))


def _exact_attention(s):
    q, page = s["q"].double(), s["k_cache"].shape[1]
    total, hq, d = q.shape
    hk = s["k_cache"].shape[2]
    start, ctx, table = s["q_start"].tolist(), s["context_lens"].tolist(), s["block_table"].tolist()
    out = torch.zeros_like(q)
    for b in range(len(ctx)):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        ids = torch.tensor([table[b][j] for j in range(-(-(ctx[b] + n) // page))], device="cuda")
        sees = torch.ones((n, ctx[b] + n), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            sees[:, ctx[b]:] = torch.ones((n, n), device="cuda").tril() > 0
        else:
            words = s["mask"][start[b]:start[b + 1]].cpu().numpy()
            bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little")[:, :n]
            sees[:, ctx[b]:] = torch.from_numpy(bits > 0).cuda()
        for h in range(hk):
            keys = s["k_cache"][ids, :, h].reshape(-1, d)[:ctx[b] + n].double()
            values = s["v_cache"][ids, :, h].reshape(-1, d)[:ctx[b] + n].double()
            for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                score = (q[start[b]:start[b + 1], g] @ keys.T * s["scale"]).masked_fill(~sees, -math.inf)
                out[start[b]:start[b + 1], g] = torch.softmax(score, 1) @ values
    return out


def _exact_score(s):
    parts = []
    for x, token in zip(s["logits"].split(256), s["tokens"].split(256)):
        y = x.double()
        top = y.max(1, keepdim=True).values
        w = (y - top).exp()
        lse = top[:, 0] + w.sum(1).log()
        logp = y - lse[:, None]
        given = logp[torch.arange(len(token), device="cuda"), token.clamp(min=0)]
        finite = logp.masked_fill(y == -math.inf, 0.0)
        parts.append([given.masked_fill(token < 0, 0.0), lse, -(finite * logp.exp()).sum(1), torch.sort(logp, 1, descending=True).values[:, :s["top"]]])
    given, lse, entropy, top = (torch.cat(p) for p in zip(*parts))
    out = {"logprob": given, "lse": lse, "entropy": entropy}
    if s["top"]:
        out.update(top_ids=None, top_logprobs=top)
    return out


def _exact_score_backward(s):
    parts = []
    for r in range(0, len(s["tokens"]), 256):
        e = slice(r, r + 256)
        y, token = s["logits"][e].double(), s["tokens"][e]
        logp = y - s["lse"][e].double()[:, None]
        one = torch.zeros_like(y)
        has = (token >= 0).nonzero()[:, 0]
        one[has, token[has]] = 1.0
        p = logp.exp()
        by_logprob = s["d_logprob"][e].double()[:, None] * (token >= 0)[:, None] * (one - p)
        by_entropy = s["d_entropy"][e].double()[:, None] * p * (logp.clamp(min=-1e4) + s["entropy"][e].double()[:, None])
        parts.append((by_logprob - by_entropy))
    return torch.cat(parts)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope_forward":
        return {"q": _exact_rope(s["q"], s["q_weight"], s), "k": _exact_rope(s["k"], s["k_weight"], s)}
    if case["op"] == "rope_backward":
        dq, dwq = _exact_rope_backward(s["dq_out"], s["q"], s["q_weight"], s)
        dk, dwk = _exact_rope_backward(s["dk_out"], s["k"], s["k_weight"], s)
        return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}
    if case["op"] == "append":
        k = _exact_rope(s["k"], s["k_weight"], s)
        page = s["k_cache"].shape[1]
        at = (s["slots"] >= 0).nonzero()[:, 0]
        slot = s["slots"][at]
        out = {"q": _exact_rope(s["q"], s["q_weight"], s), "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        out["k_cache"][slot // page, slot % page] = k[at]
        out["v_cache"][slot // page, slot % page] = s["v"][at].double()
        return out
    return {"attention": _exact_attention, "score": _exact_score, "score_backward": _exact_score_backward}[case["op"]](s)
