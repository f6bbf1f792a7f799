"""add_rms_norm and its gradient on the GPU against 64-bit arithmetic."""
import math

import pytest
import torch

import epilogue_tcgen05_tmem_gb300 as eg
from tests._decoder_helpers import DT, F32, TINY, UNIT, directional, rand

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from epilogue_tcgen05_tmem_gb300 import _build
    _build.build()
    eg.lib()


def _steps(width):
    """Longest chain of float32 operations behind a normed value: the squares
    one thread adds (32, or a 256th of the row), halved by the root, two trees
    of 5 halved too, rsqrtf (2 units), two products, the scale."""
    return max(32, width // 256) / 2 + 16


def _reference(x, weight, residual, eps):
    z = x.double() if residual is None else (x.double() + residual.double()).to(x.dtype).double()
    return z, z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * weight.double()


def _check_out(out, h, dtype, width):
    bound = UNIT[dtype] * h.abs() * (1 + 1e-3) + _steps(width) * F32 * h.abs() + TINY[dtype]
    assert ((out.cpu().double() - h).abs() <= bound).all()


def _check_codes(r, h, quant, width):
    block = 128 if quant == "e4m3_block" else width
    parts = h.view(h.shape[0], -1, block)
    scale = parts.abs().amax(-1) / (127 if quant == "int8" else 448)
    scale[scale.float() == 0] = 1.0
    got = r.scales.cpu().double().view(scale.shape)
    rel = (_steps(width) + 2) * F32
    assert ((got - scale).abs() <= rel * scale + 2.0 ** -149).all()
    codes = r.codes.cpu()
    value = (codes.double() if quant == "int8" else codes.view(torch.float8_e4m3fn).double()).view(parts.shape)
    exact = parts / got[..., None]
    # half a step of the code, and what float32 may be off before the rounding
    half = 0.5 if quant == "int8" else torch.maximum(exact.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10))
    assert ((value - exact).abs() <= half * (1 + 1e-5) + 2 * rel * exact.abs()).all()
    assert value.abs().max() <= (127 if quant == "int8" else 448)


SHAPES = [(1, 1), (3, 7), (5, 8), (4, 64), (9, 100), (1, 128), (17, 256), (6, 1000), (5, 1024), (3, 1032), (7, 4096), (2, 5120), (2, 8200), (3, 16384), (1, 40000), (1, 65536),
          (21, 9), (10, 333), (9, 1001), (17, 4099), (6, 8202), (9, 12001), (5, 16383), (2, 20001)]  # rows at every place of a vector


@pytest.mark.parametrize("rows,width", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(rows, width, dtype, residual):
    g = torch.Generator().manual_seed(rows * 1000 + width)
    x, w = rand(g, rows, width, dtype=dtype, scale=2.0), (1 + 0.3 * torch.randn(width, generator=g)).to(DT[dtype])
    res = rand(g, rows, width, dtype=dtype, scale=5.0) if residual else None
    z, h = _reference(x, w, res, EPS)
    xc, wc, rc = x.cuda(), w.cuda(), res.cuda() if residual else None
    for quant in (None, "e4m3", "int8") + (("e4m3_block",) if width % 128 == 0 else ()):
        r = eg.add_rms_norm(xc, wc, rc, EPS, quant=quant, keep_out=True)
        assert torch.equal(r.sum.cpu().double(), z)
        assert (r.sum is xc) != residual
        _check_out(r.out, h, dtype, width)
        if quant:
            _check_codes(r, h, quant, width)
        assert torch.equal(xc.cpu(), x)
    assert eg.add_rms_norm(xc, wc, rc, quant="int8").out is None


@pytest.mark.parametrize("shift", [0, 1])
def test_norm_of_strided_rows_in_place(shift):
    """Rows inside a wider tensor, at an aligned and an odd place; sum over the
    residual and out over x."""
    g = torch.Generator().manual_seed(3)
    rows, width = 11, 384
    for quant in (None, "e4m3_block", "e4m3"):
        wide = rand(g, rows, 3 * width + 8, scale=1.5).cuda()
        x, res = wide[:, shift:shift + width], wide[:, 8 + width + shift:8 + 2 * width + shift]
        w = rand(g, width).cuda()
        z, h = _reference(x.cpu(), w.cpu(), res.cpu(), 1e-5)
        kept = wide.clone()
        r = eg.add_rms_norm(x, w, res, 1e-5, quant=quant, out=x, sum_out=res)
        assert r.sum is res and r.out is x
        assert torch.equal(res.cpu().double(), z)
        _check_out(x, h, "bf16", width)
        if quant:
            _check_codes(r, h, quant, width)
        inside = torch.zeros(wide.shape[1], dtype=torch.bool)
        inside[shift:shift + width] = inside[8 + width + shift:8 + 2 * width + shift] = True
        assert torch.equal(wide[:, ~inside], kept[:, ~inside])
        # the norm over its own input, without a residual
        y = kept[:, :width] if shift == 0 else kept[:, 1:1 + width]
        _, h = _reference(y.cpu(), w.cpu(), None, 1e-5)
        r = eg.add_rms_norm(y, w, None, 1e-5, quant=quant, out=y)
        _check_out(y, h, "bf16", width)
        if quant:
            _check_codes(r, h, quant, width)


@pytest.mark.parametrize("width", [100, 2500, 5000, 9000, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tensors_at_different_places_of_a_vector(width, dtype):
    """x at an odd place, the others not: element by element, the gradient too."""
    g = torch.Generator().manual_seed(width)
    rows = 7
    wide = rand(g, rows, width + 3, dtype=dtype).cuda()
    x, res, w = wide[:, 1:1 + width], rand(g, rows, width, dtype=dtype).cuda(), rand(g, width, dtype=dtype).cuda()
    z, h = _reference(x.cpu(), w.cpu(), res.cpu(), EPS)
    for quant in (None, "e4m3", "int8"):
        r = eg.add_rms_norm(x, w, res, EPS, quant=quant, keep_out=True)
        assert torch.equal(r.sum.cpu().double(), z)
        _check_out(r.out, h, dtype, width)
        if quant:
            _check_codes(r, h, quant, width)
    dx, dw = eg.add_rms_norm_backward(x, res, w, EPS, d_sum=r.sum)
    ref, size, ref_w, size_w = _gradient(x.cpu(), res.cpu(), w.cpu(), r.sum.cpu(), EPS)
    assert ((dx.cpu().double() - ref).abs() <= UNIT[dtype] * ref.abs() + (3 * _steps(width) + 8) * F32 * size + TINY[dtype]).all()
    assert ((dw.cpu().double() - ref_w).abs() <= (_steps(width) + 57) * F32 * size_w + 1e-37).all()


def test_rows_beside_others_are_left_as_they_were():
    """Odd rows with others between them, in place: the vectors at their ends hold elements of those."""
    g = torch.Generator().manual_seed(31)
    wide = rand(g, 40, 2 * 333 + 7).cuda()
    res, w, d = rand(g, 40, 2 * 333 + 7).cuda(), rand(g, 333).cuda(), rand(g, 40, 2 * 333 + 7).cuda()
    kept = [t.clone() for t in (wide, res, d)]
    x, r, dd = (t[:, 328:328 + 333] for t in (wide, res, d))
    z, h = _reference(x.cpu(), w.cpu(), r.cpu(), EPS)
    eg.add_rms_norm(x, w, r, EPS, out=x, sum_out=r)
    assert torch.equal(r.cpu().double(), z)
    _check_out(x, h, "bf16", 333)
    ref, size, ref_w, size_w = _gradient(dd.cpu(), r.cpu(), w.cpu(), None, EPS)
    dx, dw = eg.add_rms_norm_backward(dd, r, w, EPS, dx=dd)
    # not bit for bit what another alignment gives: a thread's elements, so the order of a row's sum, go by it
    assert ((dx.cpu().double() - ref).abs() <= UNIT["bf16"] * ref.abs() + (3 * _steps(333) + 8) * F32 * size + TINY["bf16"]).all()
    assert ((dw.cpu().double() - ref_w).abs() <= (_steps(333) + 57) * F32 * size_w + 1e-37).all()
    for t, old in zip((wide, res, d), kept):
        t[:, 328:328 + 333] = old[:, 328:328 + 333]
        assert torch.equal(t, old)


def test_a_residual_broadcast_over_rows():
    g = torch.Generator().manual_seed(5)
    x, w, res = rand(g, 6, 512), rand(g, 512), rand(g, 1, 512)
    z, h = _reference(x, w, res, EPS)
    r = eg.add_rms_norm(x.cuda(), w.cuda(), res.cuda().expand(6, 512))
    assert torch.equal(r.sum.cpu().double(), z)
    _check_out(r.out, h, "bf16", 512)


@pytest.mark.parametrize("width", [200, 256])
def test_rows_of_zeros_infinities_and_nan(width):
    x = torch.randn(6, width, generator=torch.Generator().manual_seed(1))
    x[1] = 0
    x[2, 5] = math.inf
    x[3, width - 1] = math.nan
    x[4] *= 1e-30                       # the mean of squares is far below eps
    w = torch.ones(width)
    for quant in ("e4m3", "int8") + (("e4m3_block",) if width % 128 == 0 else ()):
        r = eg.add_rms_norm(x.cuda(), w.cuda(), quant=quant, keep_out=True)
        out, scales, codes = r.out.cpu(), r.scales.cpu().view(6, -1), r.codes.cpu().view(torch.int8)
        assert (out[1] == 0).all() and (scales[1] == 1).all() and (codes[1] == 0).all()
        assert math.isnan(out[2, 5]) and torch.isnan(out[3]).all()
        assert torch.isnan(scales[2, 5 // 128 if quant == "e4m3_block" else 0]) and torch.isnan(scales[3]).all()
        fine = torch.tensor([0, 4, 5])
        assert torch.isfinite(out[fine]).all() and torch.isfinite(scales[fine]).all()
        _, h = _reference(x[fine], w, None, EPS)
        _check_out(out[fine], h, "f32", width)


def test_scales_near_the_smallest_number():
    """h = 15.998 w for the one value that is not zero (eps takes 0.002), in
    units of 2^-149: w = 1e-43 is 71 of them, h 1136; a / 448 = 2.54 is 3 units
    and the code 1136 / 3 = 378.7, 384 as E4M3; a / 127 = 8.9 is 9 units and the
    code 126.  w of one unit gives h of 16, whose scale is below half a unit:
    the scale is 1 and the code 0."""
    x = torch.zeros(2, 256)
    x[0, 3] = 1.0
    unit = 2.0 ** -149
    for weight, by in ((1e-43, {"e4m3": (3, 384), "e4m3_block": (3, 384), "int8": (9, 126)}), (unit, None)):
        w = torch.full((256,), weight)
        for quant in ("e4m3", "int8", "e4m3_block"):
            r = eg.add_rms_norm(x.cuda(), w.cuda(), quant=quant)
            scales = r.scales.cpu().double().view(2, -1)
            codes = r.codes.cpu().double() if quant == "int8" else r.codes.cpu().view(torch.float8_e4m3fn).double()
            if by:
                assert scales[0, 0] == by[quant][0] * unit and codes[0, 3] == by[quant][1]
                scales[0, 0], codes[0, 3] = 1, 0
            assert (codes == 0).all() and (scales == 1).all()


def test_no_rows():
    x, w = torch.empty(0, 256, device="cuda", dtype=torch.bfloat16), torch.ones(256, device="cuda", dtype=torch.bfloat16)
    r = eg.add_rms_norm(x, w, x, quant="e4m3_block")
    assert r.codes.shape == (0, 256) and r.scales.shape == (0, 2) and r.sum.shape == (0, 256)
    dx, dw = eg.add_rms_norm_backward(x, x, w)
    assert dx.shape == (0, 256) and torch.equal(dw, torch.zeros_like(dw))


def test_equal_inputs_give_equal_bits_on_any_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(8)
    x, res, w = rand(g, 300, 2048).cuda(), rand(g, 300, 2048).cuda(), rand(g, 2048).cuda()
    d = rand(g, 300, 2048).cuda()

    def call(**kw):
        r = eg.add_rms_norm(x, w, res, quant="e4m3", keep_out=True, **kw)
        return [r.out, r.sum, r.codes, r.scales, *eg.add_rms_norm_backward(d, r.sum, w, d_sum=d, **kw)]

    first = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = call(stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    new = rand(g, 300, 2048).cuda()
    x.copy_(new)
    graph.replay()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(call(), held))
    assert not torch.equal(held[0], first[0])


@pytest.mark.parametrize("quant,scale", [("e4m3", "token_channel"), ("int8", "token_channel"), ("e4m3_block", "block")])
def test_codes_go_into_a_linear_plan(quant, scale):
    g = torch.Generator().manual_seed(9)
    rows, width, outputs = 33, 512, 256
    x, res, w = rand(g, rows, width).cuda(), rand(g, rows, width, scale=3.0).cuda(), rand(g, width).cuda()
    r = eg.add_rms_norm(x, w, res, quant=quant)
    weight = torch.randn(outputs, width, generator=g)
    if quant == "int8":
        codes_w = (weight * 40).round().clamp(-127, 127).to(torch.int8)
        values = codes_w.double()
    else:
        codes_w = weight.to(torch.float8_e4m3fn)
        values, codes_w = codes_w.double(), codes_w.view(torch.uint8)
    s_w = torch.rand((outputs // 128, width // 128) if scale == "block" else outputs, generator=g) + 0.5
    y = torch.empty(rows, outputs, dtype=torch.bfloat16, device="cuda")
    plan = eg.Plan(rows, outputs, width, "int8" if quant == "int8" else "e4m3", scale)
    plan.run(r.codes, codes_w.cuda(), y, s_a=r.scales, s_w=s_w.cuda())
    torch.cuda.synchronize()
    assert plan.device_status() == eg.EG_OK
    a = r.codes.cpu().double() if quant == "int8" else r.codes.cpu().view(torch.float8_e4m3fn).double()
    s_a = r.scales.cpu().double()
    if scale == "block":
        a = a * s_a.repeat_interleave(128, 1)
        ref = a @ (values * s_w.double().repeat_interleave(128, 0).repeat_interleave(128, 1)).T
        size = a.abs() @ (values * s_w.double().repeat_interleave(128, 0).repeat_interleave(128, 1)).abs().T
    else:
        ref = (a * s_a[:, None]) @ (values * s_w.double()[:, None]).T
        size = (a * s_a[:, None]).abs() @ (values * s_w.double()[:, None]).abs().T
    # one rounding to bf16; the products' sums in float32 (E4M3 sums keep 14 bits at least)
    assert ((y.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * size).all()


def test_a_plan_may_start_while_the_norm_runs():
    """A linear plan as the norm's programmatic dependent: its inputs are the codes and scales of this call, not of the last one."""
    g = torch.Generator().manual_seed(11)
    rows, width, outputs = 64, 2048, 512
    w, weight = rand(g, width).cuda(), torch.randn(outputs, width, generator=g).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    s_w = (torch.rand(outputs, generator=g) + 0.5).cuda()
    plans = [eg.Plan(rows, outputs, width, "e4m3", "token_channel", pdl=pdl) for pdl in (True, False)]
    inputs = [(rand(g, rows, width).cuda(), rand(g, rows, width, scale=3.0).cuda()) for _ in range(12)]
    got = []
    for plan in plans:
        outs = [torch.empty(rows, outputs, dtype=torch.bfloat16, device="cuda") for _ in inputs]
        for (x, res), y in zip(inputs, outs):
            r = eg.add_rms_norm(x, w, res, quant="e4m3")
            plan.run(r.codes, weight, y, s_a=r.scales, s_w=s_w)
        torch.cuda.synchronize()
        assert plan.device_status() == eg.EG_OK
        got.append(outs)
    assert all(torch.equal(a, b) for a, b in zip(*got))


# --------------------------------------------------------------- gradient --

def _gradient(d_out, z, weight, d_sum, eps):
    d, z, w = d_out.double(), z.double(), weight.double()
    m = (z * z).mean(-1, keepdim=True) + eps
    g = d * w
    dx = g / m.sqrt() - z * (g * z).mean(-1, keepdim=True) / m ** 1.5
    # what float32 may be off: of each part of dx, and of the row's sum before it cancels
    size = (g / m.sqrt()).abs() + z.abs() * (g * z).abs().mean(-1, keepdim=True) / m ** 1.5
    if d_sum is not None:
        dx, size = dx + d_sum.double(), size + d_sum.double().abs()
    terms = d * z / m.sqrt()
    return dx, size, terms.sum(0), terms.abs().sum(0)


@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (2, 8), (40, 100), (7, 256), (700, 264), (1300, 64), (5, 1000), (9, 4096), (2, 8200), (3, 16384), (1, 40000),
                                        (21, 9), (400, 333), (1300, 1001), (700, 77), (310, 4099), (6, 8202), (9, 12001), (5, 16383), (2, 20001)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("with_sum", [True, False])
def test_gradient(rows, width, dtype, with_sum):
    g = torch.Generator().manual_seed(rows * 77 + width)
    z, d, w = rand(g, rows, width, dtype=dtype, scale=3.0), rand(g, rows, width, dtype=dtype), rand(g, width, dtype=dtype)
    ds = rand(g, rows, width, dtype=dtype) if with_sum else None
    dx, dw = eg.add_rms_norm_backward(d.cuda(), z.cuda(), w.cuda(), EPS, d_sum=ds.cuda() if with_sum else None)
    ref, size, ref_w, size_w = _gradient(d, z, w, ds, EPS)
    bound = UNIT[dtype] * ref.abs() + (3 * _steps(width) + 8) * F32 * size + TINY[dtype]
    assert ((dx.cpu().double() - ref).abs() <= bound).all()
    # rows one CTA adds in turn (there are 608), then trees of 32 and of 19
    steps = _steps(width) + rows / 600 + 56
    assert ((dw.cpu().double() - ref_w).abs() <= steps * F32 * size_w + 1e-37).all()


@pytest.mark.parametrize("width", [96, 100])
def test_gradient_against_differences(width):
    g = torch.Generator().manual_seed(21)
    z, w = torch.randn(5, width, generator=g), torch.randn(width, generator=g)
    d, ds = torch.randn(5, width, generator=g), torch.randn(5, width, generator=g)
    dx, dw = eg.add_rms_norm_backward(d.cuda(), z.cuda(), w.cuda(), 1e-3, d_sum=ds.cuda())

    def f(zz, ww):
        return ((zz / torch.sqrt((zz * zz).mean(-1, keepdim=True) + 1e-3) * ww) * d.double() + zz * ds.double()).sum().item()

    for _ in range(3):
        u, v = torch.randn(5, width, generator=g).double(), torch.randn(width, generator=g).double()
        by_z = directional(lambda t: f(t, w.double()), z.double(), u, 1e-5)
        by_w = directional(lambda t: f(z.double(), t), w.double(), v, 1e-5)
        # the difference's own error is some 1e-9; the gradient's float32 errors add up over 5 * width values of size 1
        assert abs((dx.cpu().double() * u).sum().item() - by_z) <= 64 * F32 * 5 * width + 1e-6
        assert abs((dw.cpu().double() * v).sum().item() - by_w) <= 64 * F32 * 5 * width + 1e-6


def test_gradient_in_place_and_strided():
    g = torch.Generator().manual_seed(23)
    rows, width = 30, 512
    z, d, ds, w = (rand(g, rows, width) for _ in range(3)), None, None, rand(g, width).cuda()
    z, d, ds = z
    ref = eg.add_rms_norm_backward(d.cuda(), z.cuda(), w, d_sum=ds.cuda())
    wide = torch.zeros(rows, 2 * width + 16, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + width] = z.cuda()
    for over in ("d", "ds"):
        dc, dsc = d.cuda(), ds.cuda()
        dx, dw = eg.add_rms_norm_backward(dc, wide[:, 8:8 + width], w, d_sum=dsc, dx=dc if over == "d" else dsc)
        assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])
    # a gradient broadcast over the rows (as a mean's is)
    one = rand(g, 1, width)
    a = eg.add_rms_norm_backward(one.cuda().expand(rows, width), z.cuda(), w)
    b = eg.add_rms_norm_backward(one.cuda().repeat(rows, 1), z.cuda(), w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("width", [1001, 512])
def test_gradient_in_place_of_many_rows(width):
    """Rows that share a vector with the next one's start, over the gradient they come from; and two calls at once."""
    g = torch.Generator().manual_seed(width)
    rows = 2003
    z, d, ds = (rand(g, rows, width).cuda() for _ in range(3))
    w = rand(g, width).cuda()
    ref = eg.add_rms_norm_backward(d, z, w, d_sum=ds)
    for over in range(2):
        both = [d.clone(), ds.clone()]
        dx, dw = eg.add_rms_norm_backward(both[0], z, w, d_sum=both[1], dx=both[over])
        assert dx is both[over] and torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [eg.add_rms_norm_backward(d, z, w, d_sum=ds, stream=s.cuda_stream) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref[0]) and torch.equal(y, ref[1]) for x, y in got)


def test_offsets_past_32_bits():
    g = torch.Generator().manual_seed(31)
    rows, width, last = 524297, 4104, 5
    assert rows * width > 1 << 31
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    x[-last:] = rand(g, last, width, scale=2.0).cuda()
    res, w = rand(g, 1, width).cuda(), rand(g, width).cuda()
    big = eg.add_rms_norm(x, w, res.expand(rows, width), quant="e4m3", keep_out=True)
    small = eg.add_rms_norm(x[-last:], w, res.expand(last, width), quant="e4m3", keep_out=True)
    for a, b in zip(big, small):
        assert torch.equal(a[-last:], b)
    total = big.sum
    del big
    d = x
    d.zero_()
    d[-1] = rand(g, width).cuda()  # one row: the weight's gradient is its product, whatever the order of sums
    dx, dw = eg.add_rms_norm_backward(d, total, w)
    one = eg.add_rms_norm_backward(d[-last:], total[-last:], w)
    assert torch.equal(dx[-last:], one[0]) and torch.equal(dw, one[1]) and dx[:last].abs().max() == 0


def test_refusals_of_the_binding():
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for bad in (lambda: eg.add_rms_norm(x.cpu(), w), lambda: eg.add_rms_norm(x[0], w), lambda: eg.add_rms_norm(x, w[:32]),
                lambda: eg.add_rms_norm(x, w.half()), lambda: eg.add_rms_norm(x.double(), w.double()), lambda: eg.add_rms_norm(x, w, x[:2]),
                lambda: eg.add_rms_norm(x.T, w), lambda: eg.add_rms_norm(x, w, quant="e5m2"), lambda: eg.add_rms_norm(x, w, sum_out=x),
                lambda: eg.add_rms_norm(x, w, x, out=x.half()), lambda: eg.add_rms_norm_backward(x[:2], x, w),
                lambda: eg.add_rms_norm_backward(x, x, w, d_sum=x.half())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(eg.EgError, match="128"):
        eg.add_rms_norm(x, w, quant="e4m3_block")
    with pytest.raises(eg.EgError, match="apart"):
        eg.add_rms_norm(x, w, out=x[:1].expand(4, 64))
