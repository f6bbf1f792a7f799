"""Log probabilities, entropy, top alternatives and their gradient on the GPU
against the 64-bit definitions."""
import math

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


def _reference(x, tokens, top):
    """(logprob, lse, entropy, ids, top logprobs) in 64 bits; rows of -inf alone have a value of their own."""
    y = x.double()
    m = y.max(1, keepdim=True).values
    nothing = m[:, 0] == -INF
    e = torch.where(nothing[:, None], 0.0, torch.exp(y - torch.where(m == -INF, 0.0, m)))
    s = e.sum(1)
    lse = torch.where(nothing, -INF, m[:, 0] + s.log())
    logp = torch.where(nothing[:, None], -INF, y - lse[:, None])
    p = torch.exp(logp)
    ent = -torch.where(p > 0, p * logp, 0.0).sum(1)
    given = (tokens >= 0) & (tokens < x.shape[1])
    lp = torch.where(given, logp.gather(1, torch.where(given, tokens, 0)[:, None])[:, 0], 0.0)
    order = torch.sort(y, dim=1, descending=True, stable=True).indices[:, :top]
    return lp, lse, ent, order, logp.gather(1, order)


def _check(got, x, tokens, top):
    lp, lse, ent, ids, best = _reference(x, tokens, top)
    # y = (x - m) log2 e is a fused product of relative error 2^-24 (and the
    # rounded constant's 2^-25), 2^y has 2 ulp; sums over up to 2^18 values are
    # joined pairwise over threads after runs of at most 2^12: the mean error of
    # such a run of positive values is far below 2^-19
    tol = lambda ref: 2.0 ** -19 * (1 + ref.abs())  # noqa: E731
    # entropy cancels lse against the mean of x
    spread = torch.where(torch.isfinite(x.double()), x.double(), 0.0).abs().amax(1)
    for name, a, b, t in (("lse", got.lse, lse, tol(lse)), ("logprob", got.logprob, lp, tol(lp) + 2.0 ** -22 * spread),
                          ("entropy", got.entropy, ent, tol(ent) + 2.0 ** -21 * spread)):
        a = a.cpu().double()
        same = a == b
        assert (same | ((a - b).abs() <= t)).all(), (name, (a - b).abs().max())
    if top:
        assert torch.equal(got.top_ids.cpu(), ids)
        b = got.top_logprobs.cpu().double()
        assert ((b == best) | ((b - best).abs() <= tol(best) + 2.0 ** -22 * spread[:, None])).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 7, 7), (1, 50021, 5), (2, 131072, 20), (5, 4097, 32), (200, 1000, 1),
                                            (400, 8191, 0), (1, 200003, 32), (33, 32000, 20)])
def test_forward(dtype, rows, vocab, top):
    g = torch.Generator().manual_seed(rows + vocab)
    x = H.rand(g, rows, vocab, dtype=dtype, scale=2.5)
    if vocab > 100:
        x[:, vocab - vocab // 100:] = -INF
    tokens = torch.randint(-1, vocab + 1, (rows,), generator=g)
    _check(eg.token_logprobs(x.cuda(), tokens.cuda(), top=top), x, tokens, top)


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 4000, 130000), ("f32", 2500, 20011), ("f16", 9000, 1003)])
def test_many_rows_are_the_same_every_time(dtype, rows, vocab):
    """More rows than CTAs: each takes several, and the next one's loads overlap the end of the one before."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 2.5).to(H.DT[dtype])
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    first = eg.token_logprobs(x, tokens, top=20)
    ref = torch.cat([torch.logsumexp(part.double(), 1) for part in x.split(500)])
    assert ((first.lse.double() - ref).abs() <= 2.0 ** -19 * (1 + ref)).all()
    for _ in range(30):
        assert all(torch.equal(a, b) for a, b in zip(eg.token_logprobs(x, tokens, top=20), first))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab,top", [(1, 1), (37, 32), (1003, 20), (1003, 0), (14001, 32)])
def test_many_short_rows(dtype, vocab, top):
    """As many rows as fill the machine several times, ordinary ones and such as make every value a candidate or none."""
    rows = 1500
    g = torch.Generator().manual_seed(vocab)
    x = H.rand(g, rows, vocab, dtype=dtype, scale=2.5)
    at = torch.arange(vocab, dtype=torch.float32).to(x.dtype)
    x[7::50] = at / 64
    x[8::50] = -at / 64
    x[9::50] = 3.0
    x[10::50] = torch.finfo(x.dtype).min
    x[11::50] = -INF
    x[12::50, : vocab // 2] = -INF
    tokens = torch.randint(-1, vocab + 1, (rows,), generator=g)
    _check(eg.token_logprobs(x.cuda(), tokens.cuda(), top=top), x, tokens, top)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("order", ["rising", "falling", "equal", "two values", "few"])
def test_top_of_ordered_and_equal_logits(dtype, order):
    """Values that would all be candidates: the selection runs often, and ties go to the lowest id."""
    vocab = 70001
    at = torch.arange(vocab, dtype=torch.float32)
    x = {"rising": at / 1000, "falling": -at / 1000, "equal": torch.full_like(at, 3.0), "two values": (at % 977 == 500).float(),
         "few": torch.where(at % 30011 == 7, 1.0, -INF)}[order].to(H.DT[dtype])[None].repeat(2, 1)
    tokens = torch.tensor([7, 69999])
    _check(eg.token_logprobs(x.cuda(), tokens.cuda(), top=32), x, tokens, 32)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_of_the_lowest_values(dtype):
    lowest = torch.finfo(H.DT[dtype]).min
    x = torch.full((6, 5000), lowest, dtype=H.DT[dtype])
    x[1] = -INF
    x[2, 17] = -INF                      # the lowest value and less
    x[3] = -INF
    x[3, 4999] = lowest
    x[4, 33] = 1.0                       # one real logit among masked ones
    x[5] = torch.finfo(H.DT[dtype]).max
    tokens = torch.tensor([3, 3, 3, 4999, 33, 0])
    _check(eg.token_logprobs(x.cuda(), tokens.cuda(), top=3), x, tokens, 3)


def test_infinite_and_undefined_logits():
    x = torch.zeros(3, 3000)
    x[0, 5], x[1, 7], x[2, 2999] = INF, math.nan, math.nan
    r = eg.token_logprobs(x.cuda(), torch.tensor([0, 0, 2999]).cuda(), top=2)
    assert r.lse[0].item() == INF and math.isnan(r.logprob[0].item()) and math.isnan(r.entropy[0].item())
    assert r.top_ids[0].tolist() == [5, 0]
    for row in (1, 2):
        assert all(torch.isnan(t[row]).all() for t in (r.lse, r.logprob, r.entropy, r.top_logprobs)) and (r.top_ids[row] == -1).all()


@pytest.mark.parametrize("rows,vocab,top", [(5, 50021, 5), (700, 9000, 3), (2, 200, 0), (1500, 1000, 20)])
def test_a_wait_that_runs_out_is_reported(rows, vocab, top):
    """By a cluster for a row, CTAs of either size and short rows; not to be taken for a NaN among the logits."""
    g = torch.Generator().manual_seed(rows)
    x = H.rand(g, rows, vocab, dtype="f32", scale=2.5)
    tokens = torch.randint(0, vocab, (rows,), generator=g)
    xd, td = x.cuda(), tokens.cuda()
    decoder.token_logprobs_set_test_stall(5_000_000, 1)
    try:
        r = eg.token_logprobs(xd, td, top=top)
        torch.cuda.synchronize()
        assert eg.token_logprobs_device_status() == eg.EG_ERR_DEVICE_TIMEOUT
        assert eg.token_logprobs_device_status() == eg.EG_OK  # reported once
    finally:
        decoder.token_logprobs_set_test_stall(0, 0)
    assert all(torch.isnan(t).all() for t in (r.lse, r.logprob, r.entropy))
    if top:
        assert torch.isnan(r.top_logprobs).all() and (r.top_ids == -1).all()
    x[0, 7] = math.nan
    _check(eg.token_logprobs(xd, td, top=top), xd.cpu(), tokens, top)
    assert torch.isnan(eg.token_logprobs(x.cuda(), td, top=top).lse[0]) and eg.token_logprobs_device_status() == eg.EG_OK


@pytest.mark.parametrize("hook", [False, True])
def test_the_limit_of_a_wait(hook, monkeypatch):
    """From the hook or from EG_WAIT_CAP_MS, as the other kernels have it."""
    x, tokens = torch.zeros(2, 5000, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    monkeypatch.setenv("EG_WAIT_CAP_MS", "40" if not hook else "4000")
    decoder.token_logprobs_set_test_stall(40_000_000 if hook else 0, 1)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    try:
        begin.record()
        eg.token_logprobs(x, tokens)
        end.record()
        assert eg.token_logprobs_device_status() == eg.EG_ERR_DEVICE_TIMEOUT
    finally:
        decoder.token_logprobs_set_test_stall(0, 0)
    assert 30 < begin.elapsed_time(end) < 1000


def test_rows_of_a_wider_tensor():
    """A row stride that leaves rows off 16-byte boundaries, and no tokens."""
    g = torch.Generator().manual_seed(3)
    wide = H.rand(g, 9, 5003, scale=2.0)
    x = wide[:, 1:4096]
    r = eg.token_logprobs(wide.cuda()[:, 1:4096], top=4)
    _check(r, x, torch.full((9,), -1), 4)
    d = eg.token_logprobs_backward(wide.cuda()[:, 1:4096], torch.full((9,), 11).cuda(), r.lse, r.entropy, torch.ones(9, device="cuda"))
    _check_grad(d, x, torch.full((9,), 11), r.lse, r.entropy, torch.ones(9), torch.zeros(9))


def _check_grad(d, x, tokens, lse, entropy, gl, ge):
    y = x.double()
    lse, entropy, gl, ge = (t.cpu().double()[:, None] for t in (lse, entropy, gl, ge))
    logp = y - lse
    p = torch.exp(logp)
    given = ((tokens >= 0) & (tokens < x.shape[1]))[:, None]
    one = torch.zeros_like(y)
    one.scatter_(1, torch.where(given, tokens[:, None], 0), given.double())
    inner = torch.where(p > 0, logp + entropy, 0.0)
    ref = gl * given * (one - p) - ge * p * inner
    n = H.name_of(d)
    # p: 2 ulp of 2^y, and y's rounding (2^-24 |y|, twice); the bracket's
    # two products
    mass = p * ((gl * given).abs() + ge.abs() * (logp.clamp(min=-200).abs() + entropy.abs())) + one * gl.abs()
    tol = H.UNIT[n] * ref.abs() + mass * H.F32 * (16 + 4 * logp.clamp(min=-200).abs()) + H.TINY[n] + 2.0 ** -125
    assert ((d.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 7), (2, 100003), (300, 1001), (17, 8192)])
def test_backward(dtype, rows, vocab):
    g = torch.Generator().manual_seed(rows * vocab)
    x = H.rand(g, rows, vocab, dtype=dtype, scale=2.5)
    if vocab > 100:
        x[:, -vocab // 100:] = -INF
    tokens = torch.randint(-1, vocab + 1, (rows,), generator=g)
    r = eg.token_logprobs(x.cuda(), tokens.cuda())
    gl, ge = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    xd = x.cuda()
    d = eg.token_logprobs_backward(xd, tokens.cuda(), r.lse, r.entropy, gl.cuda(), ge.cuda())
    _check_grad(d, x, tokens, r.lse, r.entropy, gl, ge)
    only = eg.token_logprobs_backward(xd, tokens.cuda(), r.lse, None, gl.cuda())
    _check_grad(only, x, tokens, r.lse, r.entropy, gl, torch.zeros(rows))
    assert eg.token_logprobs_backward(xd, tokens.cuda(), r.lse, r.entropy, gl.cuda(), ge.cuda(), out=xd) is xd
    assert torch.equal(xd, d)


def test_backward_is_the_difference_quotient():
    g = torch.Generator().manual_seed(9)
    x = (torch.randn(4, 501, generator=g) * 2).cuda()
    tokens = torch.randint(0, 501, (4,), generator=g).cuda()
    gl, ge = torch.randn(4, generator=g).cuda(), torch.randn(4, generator=g).cuda()

    def loss(x):
        r = eg.token_logprobs(x, tokens)
        return (r.logprob.double() * gl + r.entropy.double() * ge).sum().item()

    r = eg.token_logprobs(x, tokens)
    d = eg.token_logprobs_backward(x, tokens, r.lse, r.entropy, gl, ge)
    step = torch.randn(4, 501, generator=g).cuda()
    want = H.directional(loss, x, step, 1e-2)
    # the quotient's error: h^2 / 6 of a third derivative of order one, and
    # float32 results of order 10 over h
    assert abs((d.double() * step).sum().item() - want) <= 2e-3 * (d.double().norm() * step.double().norm()).item()


def test_backward_of_a_row_of_nothing_is_zero():
    x = torch.full((2, 600), -INF)
    x[1] = 0.0
    r = eg.token_logprobs(x.cuda(), torch.tensor([3, 3]).cuda())
    one = torch.ones(2, device="cuda")
    d = eg.token_logprobs_backward(x.cuda(), torch.tensor([3, 3]).cuda(), r.lse, r.entropy, one, one)
    assert (d[0] == 0).all() and torch.isfinite(d[1]).all()


def test_no_rows_and_refusals():
    e = torch.empty(0, 100, device="cuda")
    assert eg.token_logprobs(e, torch.empty(0, dtype=torch.int64, device="cuda"), top=3).top_ids.shape == (0, 3)
    x = torch.zeros(2, 100, device="cuda")
    t = torch.zeros(2, dtype=torch.int64, device="cuda")
    z = torch.zeros(2, device="cuda")
    for call in (lambda: eg.token_logprobs(x.double(), t), lambda: eg.token_logprobs(x, t.int()), lambda: eg.token_logprobs(x, t[:1]),
                 lambda: eg.token_logprobs(x.t(), t), lambda: eg.token_logprobs(x.cpu(), t.cpu()),
                 lambda: eg.token_logprobs_backward(x, t, z, z, z, z, out=x[:, :50]),
                 lambda: eg.token_logprobs_backward(x, t, z.double(), z)):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: eg.token_logprobs(x, t, top=33), eg.EG_ERR_UNSUPPORTED),
                         (lambda: eg.token_logprobs(x[:, :3], t, top=4), eg.EG_ERR_INVALID_ARG),
                         (lambda: eg.token_logprobs(x[:, :0], t), eg.EG_ERR_INVALID_ARG),
                         (lambda: eg.token_logprobs_backward(x, t, z, None, z, z), eg.EG_ERR_INVALID_ARG)):
        with pytest.raises(eg.EgError) as e:
            call()
        assert e.value.status == status
