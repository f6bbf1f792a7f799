"""Attention of chunks of new tokens over a paged cache on the GPU against the
64-bit definition."""
import ctypes
import math

import numpy as np
import pytest
import torch

import epilogue_tcgen05_tmem_gb300 as eg
from epilogue_tcgen05_tmem_gb300 import prompt
from tests import _decoder_helpers as H

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from epilogue_tcgen05_tmem_gb300 import _build
    _build.build()
    eg.lib()


class Case:
    """Sequences with contexts ctx and n new tokens; slots without a token hold
    NaN, table entries past the pages -1."""

    def __init__(self, dtype, hq, hk, dim, page, ctx, n, window=0, sinks=0, heads_first=False, seed=0, scale=1.0, max_chunk=None):
        rng = np.random.RandomState(seed)
        g = torch.Generator().manual_seed(seed)
        self.hq, self.hk, self.dim, self.page, self.dtype = hq, hk, dim, page, dtype
        self.ctx, self.n, self.window, self.sinks = np.array(ctx), np.array(n), window, sinks
        self.max_chunk = max_chunk or max(1, int(max(n)))
        total, lens = int(self.n.sum()), self.ctx + self.n
        need = -(-lens // page)
        pages = int(need.sum()) + 2
        free = rng.permutation(pages)
        table = np.full((len(ctx), max(1, int(need.max()))), -1, np.int32)
        used, at = np.zeros((pages, page), bool), 0
        for b in range(len(ctx)):
            table[b, :need[b]] = free[at:at + need[b]]
            at += need[b]
            j = np.arange(lens[b])
            used[table[b, j // page], j % page] = True
        self.table = table
        self.q = H.rand(g, total, hq, dim, dtype=dtype, scale=scale)
        hole = torch.from_numpy(~used)[:, :, None, None]
        self.kv = [H.rand(g, pages, page, hk, dim, dtype=dtype).masked_fill(hole, math.nan) for _ in range(2)]
        self.heads_first = heads_first
        self.scale = dim ** -0.5

    def device(self):
        kv = [c.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) if self.heads_first else c.cuda() for c in self.kv]
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
        return dict(q=self.q.cuda(), k_cache=kv[0], v_cache=kv[1], block_table=i32(self.table), context_lens=i32(self.ctx),
                    q_start=i32(np.concatenate([[0], np.cumsum(self.n)])), window=self.window, sinks=self.sinks)

    def plan(self):
        return eg.ChunkAttention(self.hq, self.hk, self.dim, self.dtype, self.page, max_batch=len(self.ctx), max_chunk=self.max_chunk)

    def places(self, b):
        """Slots of sequence b's places: (page, place in the page)."""
        at = np.arange(int(self.ctx[b] + self.n[b]))
        return torch.from_numpy(self.table[b][at // self.page].astype(np.int64)), torch.from_numpy(at % self.page)

    def sees(self, b):
        i = np.arange(self.ctx[b], self.ctx[b] + self.n[b])[:, None]
        j = np.arange(self.ctx[b] + self.n[b])
        return torch.from_numpy((j <= i) & ((self.window == 0) | (i - j < self.window) | (j < self.sinks)))

    def reference(self):
        """(o, lse, sum of p |v|, largest sum of |q k| scale) in 64 bits, on the GPU (matrix products of the definition)."""
        total, group = self.q.shape[0], self.hq // self.hk
        o, mass = (torch.zeros(total, self.hq, self.dim, dtype=torch.float64) for _ in range(2))
        lse, size = torch.full((total, self.hq), -INF, dtype=torch.float64), torch.zeros(total, self.hq, dtype=torch.float64)
        row = 0
        for b in range(len(self.ctx)):
            n = int(self.n[b])
            rows = slice(row, row + n)
            row += n
            if n == 0:
                continue
            k, v = (c[self.places(b)].cuda().double() for c in self.kv)
            hidden = ~self.sees(b).cuda()
            for h in range(self.hq):
                q = self.q[rows, h].cuda().double()
                kk = k[:, h // group]
                s = (q @ kk.T * self.scale).masked_fill(hidden, -INF)
                p = torch.softmax(s, 1)
                o[rows, h], mass[rows, h] = (p @ v[:, h // group]).cpu(), (p @ v[:, h // group].abs()).cpu()
                lse[rows, h] = torch.logsumexp(s, 1).cpu()
                size[rows, h] = (q.abs() @ kk.abs().T * self.scale).masked_fill(hidden, 0.0).amax(1).cpu()
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
    # dtype, q heads, kv heads, head_dim, page, contexts, new tokens, window, sinks, heads first
    ("bf16", 8, 2, 128, 16, [1], [1], 0, 0, False),
    ("bf16", 8, 8, 128, 16, [0], [1], 0, 0, False),
    ("bf16", 32, 8, 128, 16, [200], [33], 0, 0, False),
    ("bf16", 32, 8, 128, 16, [0], [700], 0, 0, False),
    ("f16", 8, 1, 128, 64, [0, 77, 128], [300, 129, 1], 0, 0, True),
    ("bf16", 4, 4, 64, 8, [900], [515], 0, 0, False),                          # one head each: 256 tokens an item
    ("bf16", 10, 2, 80, 24, [700, 0, 33], [70, 2, 301], 0, 0, True),           # groups of 5
    ("f16", 7, 1, 96, 48, [300, 1000], [130, 90], 0, 0, False),                # of 7
    ("bf16", 6, 2, 72, 40, [11, 0], [350, 86], 0, 0, False),                   # of 3
    ("bf16", 16, 1, 64, 16, [130], [270], 0, 0, False),
    ("bf16", 128, 1, 64, 16, [50, 0], [9, 2], 0, 0, False),                    # a token fills a tile
    ("bf16", 32, 8, 128, 16, [9000], [300], 0, 0, False),                      # a few items over many CTAs
    ("f16", 64, 8, 128, 128, [20000], [1], 0, 0, False),
    ("bf16", 32, 8, 128, 16, [0, 5, 1000], [600, 1000, 150], 128, 0, False),
    ("bf16", 32, 8, 128, 16, [0, 5, 1000], [600, 1000, 150], 100, 4, False),
    ("f16", 8, 2, 64, 8, [3, 2000, 40], [2, 333, 64], 1, 1, True),             # a window of the token itself
    ("bf16", 8, 2, 64, 8, [3, 2000, 40], [2, 333, 64], 37, 300, True),         # more first places than a tile
    ("bf16", 5, 1, 40, 24, [100, 4000], [200, 1], 129, 7, False),
    ("bf16", 8, 1, 8, 16, [100], [50], 63, 130, True),
    ("f16", 32, 4, 128, 32, [5000, 300, 0], [1, 1, 1], 256, 4, False),         # decoding with a window
    ("bf16", 32, 8, 128, 16, [70 * i for i in range(64)], [1] * 64, 1024, 5, False),
    ("bf16", 8, 2, 128, 16, [100, 3000], [40, 600], 100000, 3, False),         # a window that reaches everything
    ("bf16", 8, 2, 128, 16, [100, 3000], [40, 600], 2 ** 31 - 1, 2 ** 31 - 1, False),
    ("f16", 2, 1, 72, 40, list(range(0, 400, 7)), [1 + 5 * (i % 4) for i in range(58)], 90, 10, False),
    # caches above what the L2 keeps: row groups go through them as teams of eight, four, two, and not
    ("bf16", 32, 8, 128, 64, [9000, 8500], [512, 512], 0, 0, False),
    ("f16", 32, 8, 128, 64, [17000], [251], 0, 0, True),
    ("bf16", 32, 8, 128, 64, [9000, 8001], [100, 120], 0, 0, False),
    ("bf16", 32, 8, 128, 64, [9000, 8500, 40], [512, 130, 1], 0, 0, False),
    ("bf16", 32, 8, 128, 64, [12000, 11000], [512, 500], 9000, 5, False),
    # more sequences than a CTA has threads, some without tokens
    ("bf16", 4, 2, 64, 8, [37 * i % 300 for i in range(900)], [i % 3 for i in range(900)], 0, 0, False),
    ("bf16", 4, 2, 64, 8, [37 * i % 300 for i in range(900)], [5 * (i % 3) for i in range(900)], 50, 9, False),
]


@pytest.mark.parametrize("dtype,hq,hk,dim,page,ctx,n,window,sinks,heads_first", CASES)
def test_against_definition(dtype, hq, hk, dim, page, ctx, n, window, sinks, heads_first):
    c = Case(dtype, hq, hk, dim, page, ctx, n, window, sinks, heads_first)
    _check(c, *_run(c))


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191])
@pytest.mark.parametrize("window", [0, 64])
def test_rows_around_tiles(n, window):
    c = Case("bf16", 8, 2, 64, 16, [200, 77], [n, max(1, n - 1)], window, 2 if window else 0, seed=n)
    _check(c, *_run(c))


@pytest.mark.parametrize("length", [1, 7, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1023])
@pytest.mark.parametrize("window,sinks", [(0, 0), (127, 0), (128, 1), (129, 128), (200, 129)])
def test_lengths_and_windows_around_tiles(length, window, sinks):
    c = Case("f16", 4, 2, 128, 8, [length, length + 1], [2, 1], window, sinks, seed=length)
    _check(c, *_run(c))


def test_one_plan_serves_layers_with_and_without_a_window():
    c = Case("bf16", 16, 4, 128, 16, [300, 0, 2000], [260, 90, 1], seed=4)
    plan = c.plan()
    for c.window, c.sinks in ((0, 0), (70, 4), (0, 0), (500, 0)):
        _check(c, plan.run(**c.device()))
    plan.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_scores(dtype):
    """Rows whose maximum keeps rising along the keys, and weights that underflow."""
    c = Case(dtype, 8, 2, 128, 16, [3000], [300], scale=6.0, seed=5)
    k = c.kv[0]
    for j in range(3300):
        k[c.table[0, j // 16], j % 16] *= 0.2 + j / 2000
    _check(c, *_run(c))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_place_far_above_the_rest(dtype):
    """A score that is far above those of the tiles before it, in the first and in the second half of a tile, and as far above those after."""
    for at in (700, 760, 5):
        c = Case(dtype, 8, 2, 128, 16, [900], [140], scale=2.0, seed=at)
        page, place = c.table[0, at // 16], at % 16
        c.kv[0][page, place] = (c.q[:, ::4].float().mean(0) * 60).to(c.q.dtype)[:c.hk]
        c.kv[0][page, place, 0] = (c.q[70, 1].float() * 4).to(c.q.dtype)
        _check(c, *_run(c))


@pytest.mark.parametrize("bad", [math.nan, INF, -INF])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (40, 3)])
@pytest.mark.parametrize("ctx,n", [(0, 150), (500, 150), (400, 1)])
def test_places_that_a_token_does_not_attend_to_may_hold_anything(bad, window, sinks, ctx, n):
    """Keys and values of one place are not finite: rows that do not attend to it are as without them."""
    for j in (ctx + n // 2, max(ctx - 20, 0), 100 if ctx + n > 100 else 0, 5):
        c = Case("bf16", 8, 2, 128, 16, [ctx], [n], window, sinks, seed=7)
        page, place = c.table[0, j // 16], j % 16
        for cache in c.kv:
            cache[page, place] = bad
        seen = c.sees(0)[:, j]
        o, lse = _run(c)
        assert not torch.isfinite(o.cpu()[seen]).all(2).any()
        assert torch.isfinite(o.cpu()[~seen]).all() and torch.isfinite(lse.cpu()[~seen]).all()
        for cache in c.kv:
            cache[page, place] = 0.0
        ref, ref_lse, mass, size = c.reference()
        over = (o.cpu().double() - ref).abs() - (H.UNIT["bf16"] * (ref.abs() + mass) + 2 * (2.0 ** -21 * size[..., None] + 2.0 ** -20) * mass)
        assert (~seen).sum() == 0 or over[~seen].max() <= 0


def test_infinite_values_of_seen_places_reach_the_result():
    for window, sinks in ((0, 0), (60, 4)):
        c = Case("f16", 8, 2, 64, 16, [10], [300], window, sinks, seed=8)
        for place, value in ((3, INF), (11, -INF), (200, INF)):
            c.kv[1][c.table[0, place // 16], place % 16, 0, place % 8] = value
        o = _run(c)[0].cpu()
        sees = c.sees(0)
        for place, value in ((3, INF), (11, -INF), (200, INF)):
            if place == 11:
                continue  # column 3 has place 3 too: where both are seen the sum is not a number
            others = sees[:, 11] if place == 3 else torch.zeros(300, dtype=torch.bool)
            rows = sees[:, place] & ~others
            assert (o[rows][:, :4, place % 8] == value).all()
        none = ~(sees[:, 3] | sees[:, 11] | sees[:, 200])
        assert torch.isfinite(o[none]).all() and torch.isfinite(o[:, 4:]).all()


def test_pages_outside_the_window_need_not_exist():
    """Table entries of pages that no token attends to are invalid, or another sequence's."""
    for sinks in (0, 5):
        c = Case("bf16", 8, 2, 128, 16, [2000, 1500], [3, 40], 100, sinks, seed=9)
        d = c.device()
        for b, (ctx, lost) in enumerate(((2000, -1), (1500, 1 << 30))):
            first = (ctx - 100 + 1) // 16
            d["block_table"][b, (sinks + 15) // 16:first] = lost
        plan = c.plan()
        o = plan.run(**d)
        torch.cuda.synchronize()
        assert plan.device_status() == eg.EG_OK
        _check(c, o)
        plan.close()


def test_queries_and_results_by_strides():
    """Queries inside a projection's output, results inside a wider tensor."""
    c = Case("bf16", 8, 2, 64, 16, [40, 300], [150, 20], 64, 2, seed=10)
    d, plan = c.device(), c.plan()
    wide = torch.full((170, 12, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = d["q"]
    out = torch.full((170, 16, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    plan.run(**dict(d, q=wide[:, :8]), out=out[:, 4:12, 64:])
    _check(c, out[:, 4:12, 64:])
    out[:, 4:12, 64:] = 5.0
    assert (out == 5).all()
    plan.close()


@pytest.mark.parametrize("page", [8, 16, 40, 256])
@pytest.mark.parametrize("layout", ["keys and values in turn", "wide heads", "heads first, keys and values in turn"])
def test_caches_by_strides(page, layout):
    """Caches that are parts of other tensors, small pages (boxes of both halves of the columns, where the strides allow them) and large."""
    c = Case("bf16", 8, 2, 128, page, [700, 90], [150, 1], 200, 3, seed=page)
    d, plan = c.device(), c.plan()
    pages = d["k_cache"].shape[0]
    if layout == "keys and values in turn":
        both = torch.full((pages, 2, page, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
        k, v = both[:, 0], both[:, 1]
    elif layout == "wide heads":
        k, v = torch.full((2, pages, page, 2, 192), math.nan, dtype=torch.bfloat16, device="cuda")[..., 64:]
    else:
        both = torch.full((pages, 2, 2, page, 128), math.nan, dtype=torch.bfloat16, device="cuda")
        k, v = both[:, 0].permute(0, 2, 1, 3), both[:, 1].permute(0, 2, 1, 3)
    k.copy_(d["k_cache"]), v.copy_(d["v_cache"])
    _check(c, plan.run(**dict(d, k_cache=k, v_cache=v)))
    d["block_table"][1, 1:] = torch.where(d["block_table"][1, 1:] < 0, 1 << 30, d["block_table"][1, 1:])  # past the pages: any number
    _check(c, plan.run(**dict(d, k_cache=k, v_cache=v)))
    assert plan.device_status() == eg.EG_OK
    plan.close()


def test_offsets_past_32_bits():
    """Pages behind 2^31 elements of the cache, also where values that are not finite are read again."""
    c = Case("bf16", 8, 2, 128, 256, [700, 60], [150, 10], seed=43)
    d, plan = c.device(), c.plan()
    pages, used = 33000, d["k_cache"].shape[0]
    assert (pages - used) * 256 * 2 * 128 > 1 << 31
    d["block_table"] = torch.where(d["block_table"] < 0, -1, d["block_table"] + (pages - used))
    for name in ("k_cache", "v_cache"):
        cache = torch.full((pages, 256, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
        cache[-used:] = d[name]
        d[name] = cache
    o = plan.run(**d)
    _check(c, o)
    d["v_cache"][int(d["block_table"][1, 0]), 0, 1, 5] = INF  # the second sequence's first place, cached head 1
    again = plan.run(**d)
    assert (again[150:, 4:, 5] == INF).all()
    again[150:, 4:, 5] = o[150:, 4:, 5]
    assert torch.equal(again, o)
    assert plan.device_status() == eg.EG_OK
    plan.close()


@pytest.mark.parametrize("dtype,dim,hq,hk,window", [("f16", 80, 12, 3, 0), ("bf16", 128, 12, 3, 0), ("bf16", 64, 8, 2, 0), ("f16", 128, 8, 1, 200)])
def test_many_sequences_whose_last_rows_are_few(dtype, dim, hq, hk, window):
    """A CTA goes from pairs of row tiles to single ones and back; every run gives the same bits."""
    rng = np.random.RandomState(dim)
    n = rng.randint(247, 744, 47)
    c = Case(dtype, hq, hk, dim, 64, np.zeros_like(n), n, window, 4 if window else 0, heads_first=True, seed=dim)
    d, plan = c.device(), c.plan()
    outs = [plan.run(**d) for _ in range(40)]
    _check(c, outs[0])
    assert all(torch.equal(o, outs[0]) for o in outs)
    assert plan.device_status() == eg.EG_OK
    plan.close()


def test_same_every_time_and_on_another_stream():
    c = Case("bf16", 32, 8, 128, 16, [3000, 20, 0, 911], [50, 1, 300, 8], 700, 3, seed=9)
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


def test_new_and_reported_plans_are_ready_for_any_stream():
    c = Case("bf16", 8, 2, 128, 16, [5000, 900], [1, 1], seed=14)
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
    plan.set_test_stall(5_000_000, 1)
    plan.run(**d, out=out)
    assert plan.device_status() == eg.EG_ERR_DEVICE_TIMEOUT
    assert plan.device_status() == eg.EG_OK  # reported once
    plan.set_test_stall(0, 0)
    plan.run(**d, out=out, stream=s.cuda_stream)
    s.synchronize()
    _check(c, out)
    assert plan.device_status() == eg.EG_OK
    plan.close()


def test_a_wait_that_runs_out_is_reported():
    c = Case("bf16", 8, 2, 128, 16, [900, 0], [500, 2], 300, 3, seed=13)
    d, plan = c.device(), c.plan()
    plan.set_test_stall(5_000_000, 1)
    plan.run(**d)
    torch.cuda.synchronize()
    assert plan.device_status() == eg.EG_ERR_DEVICE_TIMEOUT
    plan.set_test_stall(0, 0)
    _check(c, plan.run(**d))
    plan.close()


def test_graph_replays_with_new_lengths():
    """Lengths, tables and queries are read on the device: one captured graph serves later steps."""
    n = [70, 3]
    a = Case("bf16", 16, 4, 128, 16, [600, 31], n, 200, 4, seed=10)
    b = Case("bf16", 16, 4, 128, 16, [1900, 7], n, 200, 4, seed=11)
    da, db = a.device(), b.device()
    pages = max(da["k_cache"].shape[0], db["k_cache"].shape[0])
    width = max(da["block_table"].shape[1], db["block_table"].shape[1])

    def wide(d):
        kv = [torch.cat([d[x], torch.zeros(pages - d[x].shape[0], *d[x].shape[1:], dtype=d[x].dtype, device="cuda")]) for x in ("k_cache", "v_cache")]
        t = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
        t[:, :d["block_table"].shape[1]] = d["block_table"]
        return dict(d, k_cache=kv[0], v_cache=kv[1], block_table=t)

    da, db = wide(da), wide(db)
    plan = a.plan()
    out = torch.empty_like(da["q"])
    plan.run(**da, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(**da, out=out)
    graph.replay()
    _check(a, out)
    for x in ("q", "k_cache", "v_cache", "block_table", "context_lens", "q_start"):
        da[x].copy_(db[x])
    graph.replay()
    _check(b, out)
    plan.close()


@pytest.mark.parametrize("window", [0, 5])
def test_lengths_beyond_the_limits_are_cut(window):
    """Lengths that the table or the plan does not hold read nothing outside of them."""
    c = Case("bf16", 4, 2, 64, 16, [30, 30], [40, 20], window, seed=12)
    d, plan = c.device(), c.plan()
    before = plan.run(**d)
    for ctx, end in ((1 << 30, 60), (2 ** 31 - 1, 60), (-5, 60), (-2 ** 31, 1 << 20), (30, 2 ** 31 - 1)):
        d["context_lens"][1], d["q_start"][2] = ctx, end
        lse = torch.full((60, 4), 7.0, device="cuda")
        o = plan.run(**d, lse=lse)
        torch.cuda.synchronize()
        assert plan.device_status() == eg.EG_OK and torch.equal(o[:40], before[:40])
        if ctx >= 1 << 30 and window:  # from its fifth token on the window lies past the table: nothing is attended to
            assert (o[44:] == 0).all() and (lse[44:] == -INF).all()
    plan.close()


@pytest.mark.parametrize("ctx", [3, 6000])
def test_rows_of_no_sequence_are_left_as_they_were(ctx):
    """Before the first sequence, after the last, and past max_chunk; the others are as without them."""
    c = Case("bf16", 8, 2, 64, 16, [ctx, 40, 0], [4, 77, 3], seed=16, max_chunk=70)
    d, plan = c.device(), c.plan()
    d["q_start"][0] = 2                  # its rows 0 and 1 are no sequence's: the other two are tokens 0 and 1
    d["q_start"][3] = 83                 # row 83 neither
    out, lse = torch.full_like(d["q"], 7.0), torch.full((84, 8), 7.0, device="cuda")
    plan.run(**d, out=out, lse=lse)
    torch.cuda.synchronize()
    assert plan.device_status() == eg.EG_OK
    left = [0, 1, *range(74, 81), 83]    # 74 to 80: past max_chunk of the second sequence
    assert (out[left] == 7).all() and (lse[left] == 7).all()
    own = [i for i in range(84) if i not in left]
    alone = Case("bf16", 8, 2, 64, 16, [ctx, 40, 0], [2, 70, 2], seed=16, max_chunk=70)
    alone.q, alone.kv, alone.table = c.q[own], c.kv, c.table
    _check(alone, out[own], lse[own])
    plan.close()


def test_a_plan_of_another_device_is_refused():
    """Found on the host: the plan's record of its device (after its problem) is set to another one, and nothing is launched."""
    c = Case("bf16", 4, 2, 64, 16, [30], [2])
    d, plan = c.device(), c.plan()
    problem = prompt.eg_chunk_problem.from_address(plan.handle)
    assert (problem.q_heads, problem.page_size, problem.max_chunk) == (4, 16, 2)
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
    plan.close()


def test_nothing_to_do():
    c = Case("bf16", 4, 2, 64, 16, [30, 4], [2, 1])
    d, plan = c.device(), c.plan()
    e = plan.run(d["q"][:0], d["k_cache"], d["v_cache"], d["block_table"][:0], d["context_lens"][:0], d["q_start"][:1])
    assert e.shape == (0, 4, 64)
    out = torch.full_like(d["q"], 7.0)
    plan.run(**dict(d, q_start=torch.zeros_like(d["q_start"])), out=out)  # sequences without new tokens
    assert (out == 7).all() and plan.device_status() == eg.EG_OK
    plan.close()


def test_agrees_with_tree_attention_on_a_chain():
    """The same rows through both operators: each within its own error."""
    c = Case("bf16", 16, 4, 128, 16, [900, 5], [40, 64], seed=18)
    d = c.device()
    d.pop("window"), d.pop("sinks")
    tree = eg.TreeAttention(16, 4, 128, "bf16", 16, max_batch=2, max_tree=64)
    _check(c, tree.run(**d))
    _check(c, *_run(c))
    tree.close()


def test_refusals():
    c = Case("bf16", 4, 2, 64, 16, [30], [2])
    d, plan = c.device(), c.plan()
    bad = [dict(q=d["q"].half()), dict(q=d["q"][:, :2]), dict(q=d["q"].transpose(1, 2)), dict(k_cache=d["k_cache"][:, :8]),
           dict(v_cache=d["v_cache"].float()), dict(block_table=d["block_table"].long()), dict(context_lens=d["context_lens"].long()),
           dict(q_start=d["q_start"][:1]), dict(q=d["q"].cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            plan.run(**dict(d, **kw))
    for kw in (dict(scale=math.nan), dict(scale=-1.0), dict(scale=0.0), dict(window=-1), dict(window=8, sinks=-1), dict(sinks=4)):
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
                       (dict(max_chunk=2 ** 20 + 1), eg.EG_ERR_UNSUPPORTED), (dict(max_batch=0), eg.EG_ERR_UNSUPPORTED), (dict(dtype="f32"), eg.EG_ERR_UNSUPPORTED)):
        with pytest.raises(eg.EgError) as e:
            eg.ChunkAttention(**dict(dict(q_heads=4, kv_heads=2, head_dim=64), **kw))
        assert e.value.status == status
    for group in (17, 19, 136):
        with pytest.raises(eg.EgError, match="do not fit a tile"):
            eg.ChunkAttention(group, 1, 64)
