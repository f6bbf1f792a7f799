"""lora on the GPU against 64-bit arithmetic."""
import math

import pytest
import torch

import epilogue_tcgen05_tmem_gb300 as eg
from tests import _decoder_helpers as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from epilogue_tcgen05_tmem_gb300 import _build
    _build.build()
    eg.lib()


class Case:
    """Sequences of n rows with adapters `of` (-1: none)."""

    def __init__(self, dtype, n, of, inputs, outputs, rank, adapters, base=True, scales=True, seed=0, size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.n, self.of = dtype, n, of
        rows = sum(n)
        self.x = H.rand(g, rows, inputs, dtype=dtype, scale=size)
        self.a = H.rand(g, adapters, rank, inputs, dtype=dtype, scale=inputs ** -0.5)
        self.b = H.rand(g, adapters, outputs, rank, dtype=dtype, scale=rank ** -0.5)
        self.scales = torch.rand(adapters, generator=g) + 0.5 if scales else None
        self.base = H.rand(g, rows, outputs, dtype=dtype) if base else None

    def device(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        start = [0]
        for k in self.n:
            start.append(start[-1] + k)
        on = lambda t: None if t is None else t.cuda()  # noqa: E731
        return dict(x=on(self.x), a=on(self.a), b=on(self.b), seq_start=torch.tensor(start, **i32), adapter=torch.tensor(self.of, **i32),
                    scales=on(self.scales), base=on(self.base))

    def reference(self):
        """(out, bound) in 64 bits.  The first product's sums are float32: off by
        a few units of the sum of magnitudes (the products of 16-bit values are
        exact; the tensor cores' sums keep 2^-21 of their largest terms); h goes
        on as two parts, 2^-16 (bf16: two of 2^-8 - a half step each, and 2^-24
        of the row's largest for fp16's small ones) off."""
        out, bound = [], []
        row = 0
        for k, which in zip(self.n, self.of):
            rows = slice(row, row + k)
            row += k
            y = torch.zeros(k, self.b.shape[1], dtype=torch.float64) if self.base is None else self.base[rows].double()
            e = torch.zeros_like(y)
            if 0 <= which < self.a.shape[0] and k:
                x, a, b = self.x[rows].double(), self.a[which].double(), self.b[which].double()
                s = 1.0 if self.scales is None else self.scales[which].double()
                h, size = x @ a.T, x.abs() @ a.abs().T
                y = y + s * (h @ b.T)
                e = s * ((2.0 ** -20 * size + 2.0 ** -15 * h.abs() + 2.0 ** -22 * h.abs().amax(1, keepdim=True)) @ b.abs().T) + 2.0 ** -20 * s * (h.abs() @ b.abs().T)
            out.append(y)
            bound.append(e)
        out, bound = torch.cat(out), torch.cat(bound)
        return out, bound + H.UNIT[self.dtype] * (out.abs() + bound) + H.TINY[self.dtype]


def _check(case, out):
    ref, bound = case.reference()
    over = (out.cpu().double() - ref).abs() - bound
    assert not torch.isnan(over).any() and (over.numel() == 0 or over.max().item() <= 0), over.max()


def _run(case, **kw):
    out = eg.lora(**case.device(), **kw)
    assert eg.lora_device_status() == eg.EG_OK
    return out


CASES = [
    # dtype, rows of the sequences, adapters, inputs, outputs, rank, bank, base
    ("bf16", [1], [0], 64, 64, 16, 1, True),
    ("bf16", [1], [0], 8, 8, 8, 1, False),
    ("f16", [1, 1, 1, 1, 1], [3, 0, -1, 1, 3], 4096, 4096, 16, 4, True),
    ("bf16", [17], [1], 200, 136, 24, 2, True),
    ("bf16", [16, 17, 15, 1], [0, 1, 2, 0], 512, 1000, 32, 3, True),
    ("f16", [128, 129, 127], [2, 0, 1], 1024, 512, 64, 3, True),
    ("bf16", [300, 1, 0, 40, 5], [1, 0, 2, -1, 7], 1288, 2056, 64, 3, True),    # one without rows, one without an adapter, one outside the bank
    ("bf16", [700], [0], 5120, 640, 128, 1, False),
    ("f16", [3, 260], [1, 0], 2000, 264, 72, 2, True),
    ("bf16", [5, 200], [1, 0], 640, 1544, 104, 2, True),
    ("bf16", [1] * 64, [i % 60 - 1 for i in range(64)], 1024, 3200, 64, 59, True),
    ("f16", [1] * 31 + [900, 50], [(5 * i) % 16 for i in range(33)], 4104, 1032, 128, 16, False),
    ("bf16", [i % 4 for i in range(700)], [i % 9 - 1 for i in range(700)], 72, 88, 8, 8, True),  # more sequences than a CTA has threads
    ("bf16", [2000], [0], 64, 40, 40, 1, True),
    ("bf16", [9, 400], [0, 1], 12288, 128, 16, 2, True),
]


@pytest.mark.parametrize("dtype,n,of,inputs,outputs,rank,adapters,base", CASES)
def test_against_definition(dtype, n, of, inputs, outputs, rank, adapters, base):
    c = Case(dtype, n, of, inputs, outputs, rank, adapters, base, seed=len(n))
    _check(c, _run(c))


@pytest.mark.parametrize("rank", range(8, 129, 8))
@pytest.mark.parametrize("n", [[2, 33], [130]])
def test_ranks(rank, n):
    c = Case("bf16", n, [1, 0][:len(n)], 520, 264, rank, 2, scales=False, seed=rank)
    _check(c, _run(c))


@pytest.mark.parametrize("size", [1e-4, 2000.0])
def test_fp16_keeps_its_range(size):
    """h beyond fp16's largest value, and in its subnormal numbers, with results that fit."""
    c = Case("f16", [1, 40], [0, 1], 4096, 256, 32, 2, base=False, size=size)
    c.a, c.b = c.a * (16 if size > 1 else 1), c.b * (2.0 ** -8 if size > 1 else 64)
    c.a, c.b = c.a.half(), c.b.half()
    _check(c, _run(c))


def test_in_place_by_strides_and_rows_of_no_sequence():
    g = torch.Generator().manual_seed(2)
    for n in ([3, 7], [150, 60]):
        c = Case("bf16", n, [1, 0], 256, 384, 16, 2, seed=3)
        d, rows = c.device(), sum(n)
        wide_x = H.rand(g, rows + 9, 800).cuda()
        wide_x[4:4 + rows, 8:264] = d["x"]
        wide = H.rand(g, rows + 9, 1024).cuda()
        wide[4:4 + rows, 128:512] = d["base"]
        kept = wide.clone()
        view = wide[:, 128:512]
        d.update(x=wide_x[:, 8:264], seq_start=d["seq_start"] + 4, base=view)
        assert eg.lora(**d, out=view) is view
        assert eg.lora_device_status() == eg.EG_OK
        _check(c, view[4:4 + rows])
        wide[4:4 + rows, 128:512] = kept[4:4 + rows, 128:512]
        assert torch.equal(wide, kept)


def test_rows_without_an_adapter_are_the_base():
    c = Case("bf16", [5, 130], [-1, 9], 64, 200, 16, 2)
    d = c.device()
    assert torch.equal(eg.lora(**d), d["base"])
    d.update(base=None)
    out = torch.full((135, 200), math.nan, dtype=torch.bfloat16, device="cuda")
    assert (eg.lora(**d, out=out) == 0).all()
    # an empty bank
    e = dict(d, a=d["a"][:0], b=d["b"][:0], scales=d["scales"][:0])
    assert (eg.lora(**e) == 0).all()


@pytest.mark.parametrize("n", [[1, 1], [40, 100]])
def test_rows_that_are_not_finite_stay_alone(n):
    c = Case("bf16", n, [0, 1], 512, 256, 16, 2, seed=6)
    good, row = c.reference()[0], n[0]
    for bad in (math.nan, math.inf):
        c.x[row, 77] = bad
        out = _run(c).cpu().double()
        assert not torch.isfinite(out[row]).any()
        rest = torch.arange(sum(n)) != row
        assert ((out - good).abs()[rest] <= 2.0 ** -6 * (1 + good.abs()[rest])).all()
    # weights of an adapter that another sequence has
    c = Case("bf16", n, [0, 1], 512, 256, 16, 3, seed=7)
    c.a[0], c.b[0], c.a[2], c.b[2] = math.nan, math.inf, math.nan, math.nan
    out = _run(c)
    assert torch.isnan(out[:n[0]]).all()
    c.a[0], c.b[0] = 0, 0
    ref, bound = c.reference()
    assert ((out.cpu().double() - ref).abs() <= bound)[n[0]:].all()


def test_same_every_time_on_another_stream_and_with_two_calls_at_once():
    c = Case("bf16", [1, 300, 20, 1], [0, 1, 2, 1], 1024, 1024, 64, 3, seed=8)
    d = c.device()
    first = eg.lora(**d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(8):
        for s in streams:
            got.append(eg.lora(**d, stream=s.cuda_stream))
    torch.cuda.synchronize()
    assert eg.lora_device_status() == eg.EG_OK
    assert all(torch.equal(o, first) for o in got)


def test_graph_replays_with_new_sequences():
    a = Case("bf16", [1, 200, 3], [0, 1, 2], 512, 512, 32, 4, seed=9)
    b = Case("bf16", [100, 4, 100], [3, -1, 0], 512, 512, 32, 4, seed=10)
    da, db = a.device(), b.device()
    out = torch.empty_like(da["base"])
    eg.lora(**da, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.lora(**da, out=out)
    graph.replay()
    _check(a, out)
    for name, t in da.items():
        t.copy_(db[name])
    graph.replay()
    _check(b, out)


def test_sequences_past_the_rows_are_cut():
    c = Case("bf16", [4, 6], [0, 1], 64, 64, 8, 2, seed=11)
    d = c.device()
    d["seq_start"][2] = 1 << 30
    _check(c, eg.lora(**d))
    d["seq_start"][0] = -(1 << 31)
    _check(c, eg.lora(**d))
    assert eg.lora_device_status() == eg.EG_OK


def test_a_wait_that_runs_out_is_reported():
    for n in ([1], [200, 3]):
        c = Case("bf16", n, list(range(len(n))), 4096, 512, 16, 2, seed=12)
        d = c.device()
        eg.prompt.lora_set_test_stall(5_000_000, 1)
        try:
            eg.lora(**d)
            assert eg.lora_device_status() == eg.EG_ERR_DEVICE_TIMEOUT
            assert eg.lora_device_status() == eg.EG_OK  # reported once
        finally:
            eg.prompt.lora_set_test_stall(0, 0)
        _check(c, _run(c))


@pytest.mark.parametrize("act", ["none", "silu"])
def test_beside_a_linear_plan(act):
    """The adapters' part goes into the plan as the residual before its activation; or is added to the plan's output."""
    c = Case("bf16", [1, 60, 3], [0, -1, 1], 256, 512, 16, 2, base=False, seed=13)
    d = c.device()
    g = torch.Generator().manual_seed(14)
    w = H.rand(g, 512, 256, scale=1 / 16)
    plan = eg.Plan(64, 512, 256, act=act, residual=True, residual_pre_act=True)
    y = torch.empty(64, 512, dtype=torch.bfloat16, device="cuda")
    part = eg.lora(**d)
    plan.run(d["x"], w.cuda(), y, residual=part)
    torch.cuda.synchronize()
    assert plan.device_status() == eg.EG_OK
    v = c.x.double() @ w.double().T + part.cpu().double()
    ref = v * torch.sigmoid(v) if act == "silu" else v
    assert ((y.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4).all()
    if act == "none":
        plain = eg.Plan(64, 512, 256)
        plain.run(d["x"], w.cuda(), y)
        c.base = y.cpu()
        _check(c, eg.lora(**dict(d, base=y), out=y))


def test_offsets_past_32_bits():
    c = Case("bf16", [5, 130], [1, 0], 64, 8200, 16, 2, seed=41)
    rows, last = 262150, sum(c.n)
    assert (rows - last) * 8200 > 1 << 31
    d = c.device()
    wide = torch.full((rows, 8200), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide.clone()
    x = wide[:, 8:72]
    x[-last:], out[-last:] = d["x"], d["base"]
    eg.lora(**dict(d, x=x, seq_start=d["seq_start"] + (rows - last), base=out, out=out))
    assert eg.lora_device_status() == eg.EG_OK
    _check(c, out[-last:])
    assert (out[:-last] == 7).all()


def test_nothing_to_do():
    c = Case("bf16", [4], [0], 64, 64, 8, 2)
    d = c.device()
    out = torch.full((4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    eg.lora(**dict(d, seq_start=d["seq_start"][:1], adapter=d["adapter"][:0]), out=out)
    assert (out == 7).all()
    assert eg.lora(**dict(d, x=d["x"][:0], base=d["base"][:0])).shape == (0, 64)


def test_refusals():
    c = Case("bf16", [4], [0], 64, 64, 8, 2)
    d = c.device()
    bad = [dict(x=d["x"].half()), dict(x=d["x"].cpu()), dict(x=d["x"][0]), dict(a=d["a"][:1]), dict(a=d["a"][:, :, :32]), dict(b=d["b"].transpose(1, 2)),
           dict(seq_start=d["seq_start"].long()), dict(adapter=d["adapter"].long()), dict(seq_start=d["seq_start"][:1]), dict(scales=d["scales"].double()),
           dict(base=d["base"][:2]), dict(out=d["base"].half())]
    for kw in bad:
        with pytest.raises(ValueError):
            eg.lora(**dict(d, **kw))
    f = {k: t.float() if t.is_floating_point() else t for k, t in d.items()}
    odd = torch.zeros(4, 65, dtype=torch.bfloat16, device="cuda")
    for kw, status in ((f, eg.EG_ERR_UNSUPPORTED), (dict(d, x=odd[:, 1:]), eg.EG_ERR_INVALID_ARG), (dict(d, base=odd[:, 1:]), eg.EG_ERR_INVALID_ARG),
                       (dict(d, out=odd[:, :64]), eg.EG_ERR_INVALID_ARG), (dict(d, out=d["base"][:1].expand(4, 64)), eg.EG_ERR_INVALID_ARG)):
        with pytest.raises(eg.EgError) as e:
            eg.lora(**kw)
        assert e.value.status == status
    for inputs, outputs, rank in ((60, 64, 8), (64, 60, 8), (64, 64, 12), (64, 64, 136)):
        c = Case("bf16", [4], [0], inputs, outputs, rank, 2)
        with pytest.raises(eg.EgError) as e:
            eg.lora(**c.device())
        assert e.value.status == eg.EG_ERR_UNSUPPORTED
