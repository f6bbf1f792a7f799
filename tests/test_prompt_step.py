"""The example of a decoder layer that takes in prompts and single tokens: its
packing on the CPU, and the whole step on the GPU against 64-bit arithmetic."""
import pytest
import torch

import epilogue_tcgen05_tmem_gb300 as eg
from epilogue_tcgen05_tmem_gb300 import prompt_step as P


def test_pack_requests():
    r = P.pack_requests([3, 1], [5, 0], [[7, 2, 3], [4, 9, 1]], [1, -1], page_size=4, max_chunk=4, device="cpu")
    assert r.q_start.tolist() == [0, 3, 4] and r.context_lens.tolist() == [5, 0] and r.adapter.tolist() == [1, -1]
    assert r.positions.tolist() == [5, 6, 7, 0]
    assert r.slots.tolist() == [2 * 4 + 1, 2 * 4 + 2, 2 * 4 + 3, 4 * 4]


def test_requests_that_do_not_fit_are_refused():
    with pytest.raises(ValueError, match="max_chunk"):
        P.pack_requests([3], [0], [[0]], [0], page_size=4, max_chunk=2, device="cpu")
    with pytest.raises(ValueError, match="pages"):
        P.pack_requests([3], [2], [[0]], [0], page_size=4, max_chunk=4, device="cpu")
    with pytest.raises(ValueError, match="adapters"):
        P.pack_requests([3], [0], [[0]], [0, 1], page_size=4, max_chunk=4, device="cpu")
    with pytest.raises(ValueError):
        P.pack_requests([3, 1], [0], [[0], [1]], [0, 1], page_size=4, max_chunk=4, device="cpu")


def _step_in_64_bits(layer, x, residual, lengths, ctx, table, adapters, page, cache):
    """This layer's output from the definitions, rounded where the layer's steps are."""
    d = torch.float64
    bf = lambda t: t.to(torch.bfloat16).to(d)  # noqa: E731
    hq, hk, dim = layer.q_heads, layer.kv_heads, layer.head_dim
    s = bf(x.to(d) + residual.to(d))
    h = s * (s.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * layer.norm.to(d)
    scale = h.abs().amax(-1, keepdim=True) / 448
    codes = (h / scale).float().to(torch.float8_e4m3fn).to(d)
    weight = layer.w_qkv.view(torch.float8_e4m3fn).to(d) * layer.s_qkv.to(d)[:, None]
    added = torch.zeros(len(x), weight.shape[0], dtype=d, device="cuda")
    at = 0
    for n, a in zip(lengths, adapters):
        if a >= 0:
            added[at:at + n] = layer.lora_scales[a].to(d) * (bf(h[at:at + n]) @ layer.lora_a[a].to(d).T @ layer.lora_b[a].to(d).T)
        at += n
    heads = bf(codes * scale @ weight.T + bf(added)).view(len(x), hq + 2 * hk, dim)

    def turn(t, w, position):
        t = t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.to(d)
        c, sn = layer.cos_sin[position].to(d)[:, None].split(dim // 2, -1)
        a, b = t.split(dim // 2, -1)
        return bf(torch.cat([a * c - b * sn, b * c + a * sn], -1))

    out, at = [], 0
    for b, n in enumerate(lengths):
        position = torch.arange(ctx[b], ctx[b] + n, device="cuda")
        q = turn(heads[at:at + n, :hq], layer.q_norm, position)
        place = [table[b][i // page] * page + i % page for i in range(ctx[b])]
        past_k, past_v = (c.to(d).flatten(0, 1)[place] for c in cache)
        k = torch.cat([past_k, turn(heads[at:at + n, hq:hq + hk], layer.k_norm, position)]).repeat_interleave(hq // hk, 1)
        v = torch.cat([past_v, heads[at:at + n, hq + hk:]]).repeat_interleave(hq // hk, 1)
        far = position[:, None] - torch.arange(ctx[b] + n, device="cuda")
        sees = (far >= 0) & ((layer.window == 0) | (far < layer.window) | (torch.arange(ctx[b] + n, device="cuda") < layer.sinks))
        p = torch.softmax(torch.einsum("ihd,jhd->hij", q, k).mul(dim ** -0.5).masked_fill(~sees, -torch.inf), -1)
        out.append(bf(torch.einsum("hij,jhd->ihd", p, v)).flatten(1))
        at += n
    return s, torch.cat(out) @ layer.w_output.to(d).T


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 2)])
def test_step(window, sinks):
    lengths, ctx, adapters, page = [90, 1, 140, 1], [0, 200, 33, 7], [1, 0, -1, 2], 16
    pages = 16
    table = torch.randperm(4 * pages, generator=torch.Generator().manual_seed(1)).view(4, pages).tolist()
    requests = P.pack_requests(lengths, ctx, table, adapters, page, 140)
    tokens = sum(lengths)
    layer = P.PromptLayer(tokens, 256, 8, 2, 64, page, 4, 140, 16, 3, window, sinks, max_positions=400, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = [torch.randn(4 * pages, page, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2)]
    before = [c.clone() for c in cache]
    x, residual = (torch.randn(tokens, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    first = residual.clone()
    got = layer.run(x, residual, requests, *cache)
    s, ref = _step_in_64_bits(layer, x, first, lengths, ctx, table, adapters, page, before)
    assert torch.equal(residual.double(), s)
    # Both sides round every stage, and a value near the middle of two codes or
    # of two 16-bit values may go the other way: an E4M3 code by an eighth of a
    # value of at most 4, times a weight of 1 / 16; the projections, below 8, by
    # 2^-5.  Attention averages values, and the output's 512 weights of size
    # 2^-4.5 add up what is left with either sign: 2^-4 is two such steps.
    assert ((got.double() - ref).abs() <= 2.0 ** -4).all()
    changed = (cache[0] != before[0]).flatten(0, 1).any(-1).any(-1).nonzero()[:, 0]
    assert torch.equal(changed, requests.slots.sort().values)
    assert eg.lora_device_status() == eg.EG_OK and layer.attention.device_status() == eg.EG_OK


@pytest.mark.gpu
def test_a_captured_step_replays_with_new_inputs():
    page, table = 16, [[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11]]
    layer = P.PromptLayer(42, 256, 8, 2, 64, page, 3, 41, 16, 2, max_positions=64, seed=3)
    g = torch.Generator(device="cuda").manual_seed(6)
    cache = [torch.randn(12, page, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2)]
    requests = P.pack_requests([40, 1, 1], [0, 20, 7], table, [0, 1, -1], page, 41)
    x, residual = (torch.randn(42, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    layer.run(x, residual, requests, *cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = layer.run(x, residual, requests, *cache)
    later = P.pack_requests([1, 12, 29], [63, 5, 30], table, [1, -1, 0], page, 41)
    for mine, new in zip(vars(requests).values(), vars(later).values()):
        mine.copy_(new)
    x.copy_(torch.randn(42, 256, generator=g, device="cuda"))
    kept, held = residual.clone(), [c.clone() for c in cache]
    graph.replay()
    torch.cuda.synchronize()
    got, sums = replayed.clone(), residual.clone()
    residual.copy_(kept)
    for c, old in zip(cache, held):
        c.copy_(old)
    assert torch.equal(layer.run(x, residual, later, *cache), got) and torch.equal(residual, sums)


@pytest.mark.gpu
def test_inputs_that_are_not_the_plans_are_refused():
    layer = P.PromptLayer(6, 256, 8, 2, 64, 16, 2, 5, max_positions=64)
    cache = [torch.zeros(2, 16, 2, 64, device="cuda").bfloat16() for _ in range(2)]
    requests = P.pack_requests([5, 1], [5, 7], [[0], [1]], [0, 0], 16, 5)
    x = torch.zeros(6, 256, device="cuda").bfloat16()
    for bad in (x[:5], x[:, :128], x.float(), x.cpu(), torch.zeros(256, 6, device="cuda").bfloat16().t(), x.flatten()):
        with pytest.raises(ValueError, match="x must be"):
            layer.run(bad, x, requests, *cache)
        with pytest.raises(ValueError, match="residual must be"):
            layer.run(x, bad, requests, *cache)
    with pytest.raises(ValueError, match="6 tokens"):
        layer.run(x, x, P.pack_requests([5], [5], [[0]], [0], 16, 5), *cache)
    torch.cuda.synchronize()
    assert all((c == 0).all() for c in cache)
