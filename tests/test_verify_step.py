"""The example of a decoder layer that verifies drafted trees: its packing on
the CPU, and the whole step on the GPU against 64-bit arithmetic."""
import pytest
import torch

from epilogue_tcgen05_tmem_gb300 import verify_step as V


def test_pack_trees():
    t = V.pack_trees([[-1, 0, 0, 1], [-1]], [5, 0], [[7, 2, 3], [4, 9, 1]], page_size=4, max_tree=4, device="cpu")
    assert t.q_start.tolist() == [0, 4, 5]
    assert t.mask.tolist() == [[0b1], [0b11], [0b101], [0b1011], [0b1]]
    assert t.positions.tolist() == [5, 6, 6, 7, 0]
    assert t.slots.tolist() == [2 * 4 + 1, 2 * 4 + 2, 2 * 4 + 3, 3 * 4, 4 * 4]


def test_pack_trees_of_more_than_a_word():
    t = V.pack_trees([list(range(-1, 39))], [0], [[0]], page_size=64, max_tree=40, device="cpu")
    assert t.mask.shape == (40, 2)
    assert t.mask[31].tolist() == [-1, 0] and t.mask[39].tolist() == [-1, 0xFF]


def test_a_draft_before_its_parent_is_refused():
    with pytest.raises(ValueError, match="parent"):
        V.pack_trees([[1, -1]], [0], [[0]], page_size=4, max_tree=2, device="cpu")


def test_a_tree_of_more_drafts_than_the_plan_takes_is_refused():
    """Its last rows would not be attended (and their mask bits would be lost)."""
    V.pack_trees([[-1, 0]], [0], [[0]], page_size=4, max_tree=2, device="cpu")
    for drafts, most in ((3, 2), (40, 33), (33, 32)):
        with pytest.raises(ValueError, match="max_tree"):
            V.pack_trees([[-1], list(range(-1, drafts - 1))], [0, 0], [[0], [1]], page_size=64, max_tree=most, device="cpu")


def _step_in_64_bits(layer, hidden, parents, ctx, table, page, cache):
    """Log probabilities from the definitions; the projections' outputs are rounded to 16 bits, as the layer's are."""
    d = torch.float64
    bf = lambda x: x.to(torch.bfloat16).to(d)  # noqa: E731
    hq, hk, dim = layer.q_heads, layer.kv_heads, layer.head_dim
    heads = bf(hidden.to(d) @ layer.w_qkv.to(d).T).view(len(hidden), hq + 2 * hk, dim)

    def turn(x, weight, position):
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight.to(d)
        c, s = layer.cos_sin[position].to(d).split(dim // 2)
        a, b = x.split(dim // 2, -1)
        return bf(torch.cat([a * c - b * s, b * c + a * s], -1))

    rows, at = [], 0
    for b, tree in enumerate(parents):
        place = [table[b][i // page] * page + i % page for i in range(ctx[b])]
        past_k, past_v = (c.to(d).flatten(0, 1)[place] for c in cache)
        depth, path, ks, vs = [], [], [], []
        for i, parent in enumerate(tree):
            depth.append(depth[parent] + 1 if parent >= 0 else 0)
            path.append((path[parent] if parent >= 0 else []) + [i])
            ks.append(turn(heads[at + i, hq:hq + hk], layer.k_norm, ctx[b] + depth[i]))
            vs.append(heads[at + i, hq + hk:])
        for i in range(len(tree)):
            q = turn(heads[at + i, :hq], layer.q_norm, ctx[b] + depth[i]).view(hk, hq // hk, dim)
            k = torch.cat([past_k] + [ks[j][None] for j in path[i]])
            v = torch.cat([past_v] + [vs[j][None] for j in path[i]])
            p = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * dim ** -0.5, -1)
            rows.append(torch.einsum("hgt,thd->hgd", p, v).reshape(-1))
        at += len(tree)
    states = bf(bf(torch.stack(rows)) @ layer.w_output.to(d).T + hidden.to(d))
    logp = torch.log_softmax(bf(states @ layer.w_head.to(d).T), -1)
    return logp


@pytest.mark.gpu
@pytest.mark.parametrize("branching", [False, True])
def test_step(branching):
    ctx, page, sizes = [37, 0, 300], 16, [9, 4, 11]
    parents = [[(i - 1) // 2 if branching and i else i - 1 for i in range(n)] for n in sizes]
    pages = 20
    table = torch.randperm(3 * pages, generator=torch.Generator().manual_seed(1)).view(3, pages).tolist()
    trees = V.pack_trees(parents, ctx, table, page, 11)
    layer = V.VerifyLayer(sum(sizes), 256, 8, 2, 64, 1000, page, 3, 11, max_positions=400, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    cache = [torch.randn(3 * pages, page, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2)]
    before = [c.clone() for c in cache]
    hidden = torch.randn(sum(sizes), 256, generator=g, device="cuda").bfloat16()
    following = torch.randint(-1, 1000, (sum(sizes),), generator=g, device="cuda")
    got = layer.run(hidden, trees, *cache, next_tokens=following, top=4)
    logp = _step_in_64_bits(layer, hidden, parents, ctx, table, page, before)
    # Every stage is rounded to 16 bits on both sides, and a value near the
    # middle of two may go the other way.  States are below 4 in size, where a
    # step is 2^-6, and the head's sums (256 weights of size 1/16) keep that
    # size; the logits are below 4 too, and lse moves by no more than they do:
    # 3 x 2^-6 in all.
    tol = 2.0 ** -4
    given = torch.where(following < 0, 0.0, logp.gather(1, following.clamp(min=0)[:, None])[:, 0])
    assert ((got.logprob.double() - given).abs() <= tol).all()
    assert ((got.top_logprobs.double() - logp.topk(4).values).abs() <= tol).all()
    assert torch.equal(got.top_ids, layer.logits.float().sort(dim=1, descending=True, stable=True).indices[:, :4])
    # the appended places changed, and no other
    changed = (cache[0] != before[0]).flatten(0, 1).any(-1).any(-1).nonzero()[:, 0]
    assert torch.equal(changed, trees.slots.sort().values)


@pytest.mark.gpu
def test_states_that_are_not_the_plans_are_refused():
    """Before any launch: fewer rows, another type or another layout would be read out of range."""
    layer = V.VerifyLayer(6, 256, 8, 2, 64, 1000, 16, 2, 3, max_positions=64)
    cache = [torch.zeros(2, 16, 2, 64, device="cuda").bfloat16() for _ in range(2)]
    parents = [[-1, 0, 1], [-1, 0, 0]]
    trees = V.pack_trees(parents, [5, 7], [[0], [1]], 16, 3)
    hidden = torch.zeros(6, 256, device="cuda").bfloat16()
    for bad in (hidden[:5], hidden[:, :128], hidden.float(), hidden.cpu(), torch.zeros(256, 6, device="cuda").bfloat16().t(), hidden.flatten()):
        with pytest.raises(ValueError, match="hidden must be"):
            layer.run(bad, trees, *cache)
    with pytest.raises(ValueError, match="6 drafts"):
        layer.run(hidden, V.pack_trees(parents[:1], [5], [[0]], 16, 3), *cache)
    torch.cuda.synchronize()
    assert all((c == 0).all() for c in cache)


@pytest.mark.gpu
def test_a_captured_step_replays_with_new_inputs():
    parents, page = [[-1, 0, 1], [-1, 0, 0]], 16
    table = [[0, 1, 2, 3], [4, 5, 6, 7]]
    layer = V.VerifyLayer(6, 256, 8, 2, 64, 1000, page, 2, 3, max_positions=64, seed=3)
    g = torch.Generator(device="cuda").manual_seed(6)
    cache = [torch.randn(8, page, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2)]
    trees = V.pack_trees(parents, [20, 7], table, page, 3)
    hidden = torch.randn(6, 256, generator=g, device="cuda").bfloat16()
    layer.run(hidden, trees, *cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = layer.run(hidden, trees, *cache)
    later = V.pack_trees(parents, [33, 60], table, page, 3)
    for mine, new in zip(vars(trees).values(), vars(later).values()):
        mine.copy_(new)
    hidden.copy_(torch.randn(6, 256, generator=g, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in replayed]
    called = layer.run(hidden, later, *cache)
    assert all(torch.equal(a, b) for a, b in zip(got, called))
