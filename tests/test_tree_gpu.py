"""Attention of drafted trees over a paged cache on the GPU against the 64-bit
definition."""
import ctypes
import math

import numpy as np
import pytest
import torch

import epilogue_tcgen05_tmem_gb300 as eg
from epilogue_tcgen05_tmem_gb300 import decoder
from tests import _decoder_helpers as H

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from epilogue_tcgen05_tmem_gb300 import _build
    _build.build()
    eg.lib()


def _pack(sees, words):
    """Truth values [n, n] as int32 words [n, words], bit u of token t."""
    bits = np.zeros((sees.shape[0], words * 32), bool)
    bits[:, :sees.shape[1]] = sees
    return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32))


def _tree(rng, n):
    sees = np.zeros((n, n), bool)
    for i in range(n):
        if i and rng.random_sample() < 0.9:
            sees[i] = sees[rng.randint(0, i)]
        sees[i, i] = True
    return sees


class Case:
    """Sequences with contexts ctx and drafted counts n; slots without a token hold NaN, table entries past the pages -1."""

    def __init__(self, dtype, hq, hk, dim, page, ctx, n, chain=False, heads_first=False, seed=0, scale=1.0, max_tree=None):
        rng = np.random.RandomState(seed)
        g = torch.Generator().manual_seed(seed)
        self.hq, self.hk, self.dim, self.page, self.dtype = hq, hk, dim, page, dtype
        self.ctx, self.n = np.array(ctx), np.array(n)
        self.max_tree = max_tree or max(1, int(max(n)))
        total, lens = int(self.n.sum()), self.ctx + self.n
        need = -(-lens // page)
        pages = int(need.sum()) + 2
        free = rng.permutation(pages)
        table = np.full((len(ctx), max(1, int(need.max()))), -1, np.int32)
        used, at = np.zeros((pages, page), bool), 0
        for b in range(len(ctx)):
            table[b, :need[b]] = free[at:at + need[b]]
            at += need[b]
            for j in range(lens[b]):
                used[table[b, j // page], j % page] = True
        self.table = table
        self.q = H.rand(g, total, hq, dim, dtype=dtype, scale=scale)
        self.sees = [np.tril(np.ones((k, k), bool)) if chain else _tree(rng, k) for k in n]
        words = -(-self.max_tree // 32)
        self.mask = None if chain else torch.cat([_pack(s, words) for s in self.sees]) if total else torch.zeros(0, words, dtype=torch.int32)
        hole = torch.from_numpy(~used)[:, :, None, None]
        self.kv = [H.rand(g, pages, page, hk, dim, dtype=dtype).masked_fill(hole, math.nan) for _ in range(2)]
        self.heads_first = heads_first
        self.scale = dim ** -0.5

    def device(self):
        kv = [c.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) if self.heads_first else c.cuda() for c in self.kv]
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
        return dict(q=self.q.cuda(), k_cache=kv[0], v_cache=kv[1], block_table=i32(self.table), context_lens=i32(self.ctx),
                    q_start=i32(np.concatenate([[0], np.cumsum(self.n)])), mask=None if self.mask is None else self.mask.cuda())

    def plan(self):
        return eg.TreeAttention(self.hq, self.hk, self.dim, self.dtype, self.page, max_batch=len(self.ctx), max_tree=self.max_tree)

    def reference(self):
        """(o, lse, sum of p |v|, largest sum of |q k| scale) in 64 bits."""
        total = self.q.shape[0]
        o, mass = (torch.zeros(total, self.hq, self.dim, dtype=torch.float64) for _ in range(2))
        lse, size = torch.full((total, self.hq), -INF, dtype=torch.float64), torch.zeros(total, self.hq, dtype=torch.float64)
        row = 0
        for b in range(len(self.ctx)):
            length = int(self.ctx[b] + self.n[b])
            at = torch.arange(length)
            pages = torch.from_numpy(self.table[b].astype(np.int64))[at // self.page]
            k, v = (c[pages, at % self.page].double() for c in self.kv)
            for t in range(int(self.n[b])):
                keep = torch.cat([torch.ones(int(self.ctx[b]), dtype=torch.bool), torch.from_numpy(self.sees[b][t])])
                kk, vv = k[keep].repeat_interleave(self.hq // self.hk, 1), v[keep].repeat_interleave(self.hq // self.hk, 1)
                if kk.shape[0]:
                    q = self.q[row].double()
                    s = torch.einsum("hd,jhd->jh", q, kk) * self.scale
                    p = torch.softmax(s, 0)
                    o[row] = torch.einsum("jh,jhd->hd", p, vv)
                    mass[row] = torch.einsum("jh,jhd->hd", p, vv.abs())
                    lse[row] = torch.logsumexp(s, 0)
                    size[row] = (torch.einsum("hd,jhd->jh", q.abs(), kk.abs()) * self.scale).amax(0)
                row += 1
        return o, lse, mass, size


def _check(case, o, lse=None):
    ref, ref_lse, mass, size = case.reference()
    u = H.UNIT[case.dtype]
    # scores: products are exact, their sum in float32 is off by a few units
    # of the sum of magnitudes; that moves a weight by as much, relatively.
    # Weights are rounded to the type for the product with the values.
    ds = 2.0 ** -21 * size[..., None] + 2.0 ** -20
    bound = u * ref.abs() + (u + 2 * ds) * mass + H.TINY[case.dtype]
    over = (o.cpu().double() - ref).abs() - bound
    assert not torch.isnan(over).any() and (over.numel() == 0 or over.max().item() <= 0), over.max()
    if lse is not None:
        a = lse.cpu().double()
        assert ((a == ref_lse) | ((a - ref_lse).abs() <= ds[..., 0] + 2.0 ** -21 * ref_lse.abs())).all()


def _run(case, **kw):
    d = case.device()
    plan = case.plan()
    lse = torch.full((case.q.shape[0], case.hq), 7.0, device="cuda")
    o = plan.run(**d, lse=lse, **kw)
    torch.cuda.synchronize()
    assert plan.device_status() == eg.EG_OK
    plan.close()
    return o, lse


CASES = [
    # dtype, q heads, kv heads, head_dim, page, contexts, drafted, chain, heads first
    ("bf16", 8, 2, 128, 16, [1], [1], True, False),
    ("bf16", 8, 8, 128, 16, [0], [1], True, False),                      # nothing cached but the token itself
    ("bf16", 32, 8, 128, 16, [517], [1], True, False),
    ("f16", 32, 8, 128, 64, [127, 128, 129, 255, 256, 257], [1] * 6, True, True),
    ("bf16", 4, 1, 64, 8, [5000], [3], False, False),
    ("bf16", 10, 2, 80, 24, [700, 0, 33], [7, 2, 1], False, True),
    ("f16", 7, 1, 96, 48, [300, 1000], [13, 9], False, False),
    ("bf16", 16, 2, 128, 128, [900, 40, 0], [64, 0, 33], False, False),  # a sequence without drafted tokens
    ("f16", 8, 1, 8, 16, [100], [5], False, True),
    ("bf16", 5, 1, 40, 32, [61, 62, 63, 64], [1, 2, 3, 4], True, False),
    ("bf16", 12, 3, 128, 256, [2000, 1], [40, 17], False, True),
    ("f16", 8, 8, 128, 16, [250], [200], False, False),                  # more rows than a tile, one head each
    ("bf16", 16, 1, 64, 16, [130], [70], False, False),                  # many rows for one cached head
    ("bf16", 32, 4, 128, 32, [3000], [256], True, False),
    ("f16", 2, 1, 72, 40, list(range(0, 400, 7)), [1 + i % 4 for i in range(58)], False, False),
    ("bf16", 64, 8, 128, 16, [17000], [1], True, False),
    # items of two row tiles and of one side by side, each over several CTAs
    ("bf16", 32, 2, 128, 16, [6000, 0, 2500, 77], [17, 24, 9, 8], False, False),
    ("f16", 40, 1, 64, 32, [9000, 4000], [30, 3], False, False),
    # more sequences than a CTA has threads
    ("bf16", 4, 2, 64, 8, [37 * i % 300 for i in range(900)], [i % 3 for i in range(900)], False, False),
]


@pytest.mark.parametrize("dtype,hq,hk,dim,page,ctx,n,chain,heads_first", CASES)
def test_against_definition(dtype, hq, hk, dim, page, ctx, n, chain, heads_first):
    c = Case(dtype, hq, hk, dim, page, ctx, n, chain, heads_first)
    _check(c, *_run(c))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 64, 65])
def test_rows_of_a_tile(n):
    c = Case("bf16", 8, 2, 64, 16, [200, 77], [n, max(1, n - 1)], False, seed=n)
    _check(c, *_run(c))


@pytest.mark.parametrize("length", [1, 7, 63, 64, 65, 127, 128, 129, 383, 384, 385, 1023])
def test_lengths_around_tiles(length):
    c = Case("f16", 4, 2, 128, 8, [length, length + 1], [2, 1], False, seed=length)
    _check(c, *_run(c))


def test_large_scores():
    """Rows whose maximum keeps rising along the keys, and weights that underflow."""
    c = Case("bf16", 8, 2, 128, 16, [4000], [4], False, scale=6.0, seed=5)
    k = c.kv[0]
    for j in range(4000):
        k[c.table[0, j // 16], j % 16] *= 0.2 + j / 2000
    _check(c, *_run(c))


def test_rows_that_attend_to_nothing():
    c = Case("bf16", 8, 2, 64, 16, [0, 0, 50], [4, 1, 3], False, seed=6)
    c.sees[0][1] = False
    c.sees[0][3] = False
    c.sees[1][0] = False
    c.sees[2][2] = False
    c.mask = torch.cat([_pack(s, 1) for s in c.sees])
    o, lse = _run(c)
    _check(c, o, lse)
    assert (o[[1, 3, 4]] == 0).all() and (lse[[1, 3, 4]] == -INF).all() and torch.isfinite(lse[[0, 2, 5, 6, 7]]).all()


@pytest.mark.parametrize("bad", [math.nan, INF])
@pytest.mark.parametrize("ctx", [0, 120, 5000])
def test_masked_places_may_hold_anything(bad, ctx):
    """Keys and values of drafted tokens that a row does not attend to are not finite: its result is as without them."""
    c = Case("bf16", 8, 2, 128, 16, [ctx], [9], False, seed=7)
    c.sees[0][:, 4] = False
    c.sees[0][4] = np.eye(9, dtype=bool)[4]  # only token 4 attends to itself
    c.mask = _pack(c.sees[0], 1)
    j = ctx + 4
    for cache in c.kv:
        cache[c.table[0, j // 16], j % 16] = bad
    o, lse = _run(c)
    keep = [t for t in range(9) if t != 4]
    assert torch.isnan(o[4]).all() or torch.isinf(o[4]).any()
    assert torch.isfinite(o[keep]).all() and torch.isfinite(lse[keep]).all()
    for cache in c.kv:
        cache[c.table[0, j // 16], j % 16] = 0.0
    ref, ref_lse, mass, size = c.reference()
    over = (o.cpu().double() - ref).abs() - (H.UNIT["bf16"] * (ref.abs() + mass) + 2 * (2.0 ** -21 * size[..., None] + 2.0 ** -20) * mass)
    assert over[keep].max() <= 0


def test_infinite_values_of_seen_places_reach_the_result():
    c = Case("f16", 4, 2, 64, 16, [10], [3], True, seed=8)
    c.kv[1][c.table[0, 0], 3, 0, 5] = INF
    c.kv[1][c.table[0, 0], 11, 1, 6] = -INF  # drafted token 1: seen by tokens 1 and 2
    o, _ = _run(c)
    o = o.cpu()
    assert (o[:, :2, 5] == INF).all() and (o[1:, 2:, 6] == -INF).all() and torch.isfinite(o[0, 2:]).all()


def test_infinite_drafted_values_reach_the_rows_of_both_tiles():
    """More rows than one tile: the tiles share the drafted keys, one comes to them after the other, and the rows of each that attend to
    the value get it."""
    many, ctx = 200, 900
    c = Case("bf16", 8, 1, 128, 16, [ctx] * many, [32] * many, True, seed=9)
    for b in range(many):
        c.kv[1][c.table[b, (ctx + 2) // 16], (ctx + 2) % 16, 0, 7] = INF  # drafted token 2
    o, _ = _run(c)
    o = o.cpu().view(many, 32, 8, 128)
    assert (o[:, 2:, :, 7] == INF).all() and torch.isfinite(o[:, :2]).all() and torch.isfinite(o[..., :7]).all()


def test_same_every_time_and_on_another_stream():
    c = Case("bf16", 32, 8, 128, 16, [3000, 20, 0, 911], [5, 1, 3, 8], False, seed=9)
    d, plan = c.device(), c.plan()
    first = plan.run(**d)
    for _ in range(3):
        assert torch.equal(plan.run(**d), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = plan.run(**d, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(o, first)
    plan.close()


def test_a_new_plan_is_ready_for_any_stream():
    """A plan made while the default stream is busy, with its first run on a stream that does not wait for that one: its counters are clear
    by then (the items are split over CTAs, and a count left over would leave them unjoined)."""
    c = Case("bf16", 8, 2, 128, 16, [5000, 900], [1, 1], True, seed=14)
    d = c.device()
    out, lse = torch.zeros_like(d["q"]), torch.zeros(2, 8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s of the default stream
    plan = c.plan()
    assert torch.cuda.default_stream().query()
    plan.run(**d, out=out, lse=lse, stream=s.cuda_stream)
    s.synchronize()
    _check(c, out, lse)
    plan.close()


def test_a_reported_plan_is_ready_for_any_stream():
    """The same for the clear that follows a report."""
    c = Case("bf16", 8, 2, 128, 16, [5000, 900], [1, 1], True, seed=15)
    d, plan = c.device(), c.plan()
    out, s = torch.zeros_like(d["q"]), torch.cuda.Stream()
    plan.set_test_stall(5_000_000, 1)
    plan.run(**d, out=out)
    assert plan.device_status() == eg.EG_ERR_DEVICE_TIMEOUT
    plan.set_test_stall(0, 0)
    plan.run(**d, out=out, stream=s.cuda_stream)
    s.synchronize()
    _check(c, out)
    assert plan.device_status() == eg.EG_OK
    plan.close()


def test_graph_replays_with_new_lengths():
    """Lengths, tables and queries are read on the device: one captured graph serves later steps."""
    a = Case("bf16", 16, 4, 128, 16, [600, 31], [2, 2], True, seed=10)
    b = Case("bf16", 16, 4, 128, 16, [1900, 7], [2, 2], True, seed=11)
    da, db = a.device(), b.device()
    pages = max(da["k_cache"].shape[0], db["k_cache"].shape[0])
    width = max(da["block_table"].shape[1], db["block_table"].shape[1])

    def wide(d):
        kv = [torch.cat([d[n], torch.zeros(pages - d[n].shape[0], *d[n].shape[1:], dtype=d[n].dtype, device="cuda")]) for n in ("k_cache", "v_cache")]
        t = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
        t[:, :d["block_table"].shape[1]] = d["block_table"]
        return dict(d, k_cache=kv[0], v_cache=kv[1], block_table=t)

    da, db = wide(da), wide(db)
    plan = eg.TreeAttention(16, 4, 128, "bf16", 16, max_batch=2, max_tree=2)
    out = torch.empty_like(da["q"])
    plan.run(**da, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(**da, out=out)
    graph.replay()
    _check(a, out)
    for n in ("q", "k_cache", "v_cache", "block_table", "context_lens", "q_start"):
        da[n].copy_(db[n])
    graph.replay()
    _check(b, out)
    plan.close()


def test_lengths_beyond_the_limits_are_cut():
    """Lengths that the table or the plan does not hold read nothing outside of them."""
    c = Case("bf16", 4, 2, 64, 16, [30, 30], [2, 2], True, seed=12)
    d, plan = c.device(), c.plan()
    before = plan.run(**d)
    d["context_lens"][1] = 1 << 30
    o = plan.run(**d)
    torch.cuda.synchronize()
    assert plan.device_status() == eg.EG_OK and torch.equal(o[:2], before[:2])
    d["context_lens"][1] = -5
    d["q_start"][2] = 1 << 20
    o = plan.run(**d)
    torch.cuda.synchronize()
    assert plan.device_status() == eg.EG_OK and torch.equal(o[:2], before[:2])
    plan.close()


@pytest.mark.parametrize("ctx", [3, 6000])
def test_rows_of_no_sequence_are_left_as_they_were(ctx):
    """Before the first sequence, after the last, and past max_tree; the others are as without them."""
    c = Case("bf16", 8, 2, 64, 16, [ctx, 40, 0], [4, 7, 3], True, seed=16, max_tree=5)
    d, plan = c.device(), c.plan()
    d["q_start"][0] = 2                  # its rows 0 and 1 are no sequence's: the other two are tokens 0 and 1
    d["q_start"][3] = 13                 # row 13 neither
    out, lse = torch.full_like(d["q"], 7.0), torch.full((14, 8), 7.0, device="cuda")
    plan.run(**d, out=out, lse=lse)
    torch.cuda.synchronize()
    assert plan.device_status() == eg.EG_OK
    left = [0, 1, 9, 10, 13]             # 9 and 10: past max_tree of the second sequence
    assert (out[left] == 7).all() and (lse[left] == 7).all()
    own = [2, 3, 4, 5, 6, 7, 8, 11, 12]
    alone = Case("bf16", 8, 2, 64, 16, [ctx, 40, 0], [2, 5, 2], True, seed=16, max_tree=5)
    alone.q, alone.kv, alone.table = c.q[own], c.kv, c.table
    _check(alone, out[own], lse[own])
    plan.close()


def test_a_wait_that_runs_out_is_reported():
    c = Case("bf16", 8, 2, 128, 16, [900, 0], [5, 2], False, seed=13)
    d, plan = c.device(), c.plan()
    plan.set_test_stall(5_000_000, 1)
    plan.run(**d)
    torch.cuda.synchronize()
    assert plan.device_status() == eg.EG_ERR_DEVICE_TIMEOUT
    assert plan.device_status() == eg.EG_OK  # reported once
    plan.set_test_stall(0, 0)
    _check(c, plan.run(**d))
    assert plan.device_status() == eg.EG_OK
    plan.close()


def test_a_plan_of_another_device_is_refused():
    """Found on the host: the plan's record of its device (after its problem) is set to another one, and nothing is launched."""
    c = Case("bf16", 4, 2, 64, 16, [30], [2], True)
    d, plan = c.device(), c.plan()
    problem = decoder.eg_tree_problem.from_address(plan.handle)
    assert (problem.q_heads, problem.page_size, problem.max_tree) == (4, 16, 2)
    its = ctypes.c_int.from_address(plan.handle + ctypes.sizeof(problem))
    assert its.value == torch.cuda.current_device()
    its.value += 1
    try:
        with pytest.raises(eg.EgError, match="device") as e:
            plan.run(**d)
        assert e.value.status == eg.EG_ERR_INVALID_ARG
        assert plan.device_status() == eg.EG_ERR_INVALID_ARG
    finally:
        its.value -= 1
    _check(c, plan.run(**d))
    assert plan.device_status() == eg.EG_OK
    plan.close()


def test_nothing_to_do():
    c = Case("bf16", 4, 2, 64, 16, [30], [2], True)
    d, plan = c.device(), c.plan()
    e = plan.run(d["q"][:0], d["k_cache"], d["v_cache"], d["block_table"][:0], d["context_lens"][:0], d["q_start"][:1])
    assert e.shape == (0, 4, 64)
    plan.close()


def test_heads_that_do_not_fit_a_tile_are_refused():
    for group in (17, 19, 136):
        with pytest.raises(eg.EgError, match="do not fit a tile") as e:
            eg.TreeAttention(group, 1, 64)
        assert e.value.status == eg.EG_ERR_UNSUPPORTED
    for group in (16, 18, 40, 128):
        eg.TreeAttention(group, 1, 64).close()


def test_refusals():
    c = Case("bf16", 4, 2, 64, 16, [30], [2], False)
    d, plan = c.device(), c.plan()
    bad = [dict(q=d["q"].half()), dict(q=d["q"][:, :2]), dict(q=d["q"].transpose(1, 2)), dict(k_cache=d["k_cache"][:, :8]),
           dict(v_cache=d["v_cache"].float()), dict(block_table=d["block_table"].long()), dict(context_lens=d["context_lens"].long()),
           dict(q_start=d["q_start"][:1]), dict(mask=d["mask"][:1]), dict(q=d["q"].cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            plan.run(**dict(d, **kw))
    for kw in (dict(mask=d["mask"][:, :0].contiguous()), dict(scale=math.nan), dict(scale=-1.0), dict(scale=0.0)):
        with pytest.raises(eg.EgError) as e:
            plan.run(**dict(d, **kw))
        assert e.value.status == eg.EG_ERR_INVALID_ARG
    odd = torch.zeros(3, 16, 2, 68, dtype=torch.bfloat16, device="cuda")[..., :64]  # rows off 16-byte boundaries
    with pytest.raises(eg.EgError) as e:
        plan.run(**dict(d, k_cache=odd, v_cache=odd))
    assert e.value.status == eg.EG_ERR_INVALID_ARG
    plan.close()
    for kw, status in ((dict(q_heads=3, kv_heads=2), eg.EG_ERR_INVALID_ARG), (dict(head_dim=136), eg.EG_ERR_UNSUPPORTED),
                       (dict(head_dim=60), eg.EG_ERR_UNSUPPORTED), (dict(page_size=12), eg.EG_ERR_UNSUPPORTED),
                       (dict(max_tree=257), eg.EG_ERR_UNSUPPORTED), (dict(max_batch=0), eg.EG_ERR_UNSUPPORTED), (dict(dtype="f32"), eg.EG_ERR_UNSUPPORTED)):
        with pytest.raises(eg.EgError) as e:
            eg.TreeAttention(**dict(dict(q_heads=4, kv_heads=2, head_dim=64), **kw))
        assert e.value.status == status
