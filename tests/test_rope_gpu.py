"""Head norm with rotation, its gradient, and the paged append, on the GPU
against the 64-bit definitions."""
import pytest
import torch

import epilogue_tcgen05_tmem_gb300 as eg
from tests import _decoder_helpers as H

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from epilogue_tcgen05_tmem_gb300 import _build
    _build.build()
    eg.lib()


def _inputs(dtype, t, hq, hk, dim, rot, norm, seed=0, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    qkv = H.rand(g, t, hq + 2 * hk, dim, dtype=dtype, scale=scale)
    d = {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "v": qkv[:, hq + hk:]}
    d["qw"] = (1 + 0.3 * torch.randn(dim, generator=g)).to(H.DT[dtype]) if norm else None
    d["kw"] = (1 + 0.3 * torch.randn(dim, generator=g)).to(H.DT[dtype]) if norm else None
    d["pos"] = torch.randint(0, 700, (t,), generator=g)
    d["table"] = H.table(700, rot) if rot else None
    d["gen"] = g
    qkv_dev = qkv.cuda()  # views of one tensor, as a projection leaves them
    d["dev"] = {"q": qkv_dev[:, :hq], "k": qkv_dev[:, hq:hq + hk], "v": qkv_dev[:, hq + hk:]}
    for n in ("qw", "kw", "pos", "table"):
        d["dev"][n] = None if d[n] is None else d[n].cuda()
    return d


SHAPES = [
    # dtype, tokens, q heads, kv heads, head_dim, rot_dim, pairs, norm
    ("bf16", 1, 32, 8, 128, 128, False, True),
    ("bf16", 37, 32, 8, 128, 128, False, True),
    ("f16", 300, 12, 4, 96, 48, True, True),
    ("bf16", 5, 5, 1, 64, 64, False, False),
    ("f32", 19, 7, 7, 128, 64, False, True),
    ("f32", 3, 2, 1, 256, 256, True, True),
    ("bf16", 11, 3, 2, 256, 128, False, True),
    ("f16", 8, 8, 2, 192, 192, True, False),
    ("bf16", 9, 10, 2, 80, 40, False, True),    # pairs of four-element chunks
    ("f16", 13, 4, 4, 72, 36, True, True),      # a chunk rotated in part
    ("bf16", 6, 3, 1, 50, 22, False, True),     # no chunk fits
    ("f32", 4, 2, 2, 6, 2, True, True),
    ("bf16", 4, 2, 2, 2, 2, False, True),
    ("bf16", 7, 4, 2, 128, 0, False, True),     # norm alone
    ("bf16", 4097, 4, 1, 64, 64, False, True),
    ("f16", 2500, 33, 3, 128, 128, False, True),
]


@pytest.mark.parametrize("dtype,t,hq,hk,dim,rot,pairs,norm", SHAPES)
def test_forward(dtype, t, hq, hk, dim, rot, pairs, norm):
    d = _inputs(dtype, t, hq, hk, dim, rot, norm)
    v = d["dev"]
    q, k = eg.qk_norm_rope(v["q"], v["k"], v["table"], positions=v["pos"], q_weight=v["qw"], k_weight=v["kw"], eps=EPS, pairs=pairs)
    H.assert_rounded(q, H.norm_rope(d["q"], d["qw"], d["table"], d["pos"], pairs, EPS), "q")
    H.assert_rounded(k, H.norm_rope(d["k"], d["kw"], d["table"], d["pos"], pairs, EPS), "k")


@pytest.mark.parametrize("dtype,t,hq,hk,dim,rot,pairs,norm", SHAPES)
def test_backward(dtype, t, hq, hk, dim, rot, pairs, norm):
    d = _inputs(dtype, t, hq, hk, dim, rot, norm, seed=1)
    v = d["dev"]
    dq_out, dk_out = (H.rand(d["gen"], t, h, dim, dtype=dtype) for h in (hq, hk))
    got = eg.qk_norm_rope_backward(dq_out.cuda(), dk_out.cuda(), v["q"], v["k"], v["table"], positions=v["pos"],
                                   q_weight=v["qw"], k_weight=v["kw"], eps=EPS, pairs=pairs)
    for dx, dw, dy, x, w in ((got[0], got[2], dq_out, d["q"], d["qw"]), (got[1], got[3], dk_out, d["k"], d["kw"])):
        ref, dw_ref, mass = H.norm_rope_backward(dy, x, w, d["table"], d["pos"], pairs, EPS)
        # g and h * mean cancel: the error is a few units of either
        H.assert_rounded(dx, ref, "dx", steps=64 + dim // 4)
        if w is None:
            assert dw is None
            continue
        # each term has a few roundings, and the longest chain of additions
        # is a warp's rows, then the joins over lanes, warps and CTAs
        chain = 32 + t * x.shape[1] // 32 + 64
        assert ((dw.cpu().double() - dw_ref).abs() <= chain * H.F32 * mass + 1e-30).all()


def test_backward_is_the_difference_quotient():
    d = _inputs("f32", 9, 4, 2, 128, 128, True, seed=2)
    v = d["dev"]
    g = d["gen"]
    cq, ck = torch.randn(9, 4, 128, generator=g).cuda(), torch.randn(9, 2, 128, generator=g).cuda()

    def loss(q, k, qw, kw):
        yq, yk = eg.qk_norm_rope(q, k, v["table"], positions=v["pos"], q_weight=qw, k_weight=kw, eps=EPS)
        return ((yq.double() * cq).sum() + (yk.double() * ck).sum()).item()

    at = [v["q"].contiguous(), v["k"].contiguous(), v["qw"], v["kw"]]
    grads = eg.qk_norm_rope_backward(cq, ck, at[0], at[1], v["table"], positions=v["pos"], q_weight=at[2], k_weight=at[3], eps=EPS)
    for i in range(4):
        step = torch.randn(at[i].shape, generator=g).cuda()
        want = H.directional(lambda x: loss(*at[:i], x, *at[i + 1:]), at[i], step, 1e-2)
        have = (grads[i].double() * step).sum().item()
        # the quotient's own error: h^2 / 6 of the third derivative, and the
        # float32 outputs' rounding over h
        assert abs(have - want) <= 2e-3 * (grads[i].double().norm() * step.double().norm()).item()


def test_backward_is_the_same_every_time():
    d = _inputs("bf16", 3001, 8, 2, 128, 128, True, seed=3)
    v = d["dev"]
    dy = [H.rand(d["gen"], 3001, h, 128).cuda() for h in (8, 2)]
    runs = [eg.qk_norm_rope_backward(*dy, v["q"], v["k"], v["table"], positions=v["pos"], q_weight=v["qw"], k_weight=v["kw"]) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_forward_in_place_and_default_positions():
    d = _inputs("bf16", 50, 6, 2, 128, 128, True, seed=4)
    q, k = d["dev"]["q"].contiguous(), d["dev"]["k"].contiguous()
    out = eg.qk_norm_rope(q, k, d["dev"]["table"], q_weight=d["dev"]["qw"], k_weight=d["dev"]["kw"], eps=EPS, q_out=q, k_out=k)
    assert out[0] is q and out[1] is k
    pos = torch.arange(50)
    H.assert_rounded(q, H.norm_rope(d["q"], d["qw"], d["table"], pos, False, EPS))
    H.assert_rounded(k, H.norm_rope(d["k"], d["kw"], d["table"], pos, False, EPS))


def test_strided_and_misaligned_views():
    """Heads-first storage, and rows that start off a 16-byte boundary."""
    g = torch.Generator().manual_seed(5)
    t, hq, hk, dim = 21, 4, 2, 64
    base_q = H.rand(g, hq, t, dim)
    base_k = H.rand(g, t, hk, dim + 3)
    tab, pos = H.table(64, 64), torch.arange(t)
    q, k = base_q.permute(1, 0, 2), base_k[..., 3:]
    qd, kd = base_q.cuda().permute(1, 0, 2), base_k.cuda()[..., 3:]
    yq, yk = eg.qk_norm_rope(qd, kd, tab.cuda())
    H.assert_rounded(yq, H.norm_rope(q, None, tab, pos, False, EPS))
    H.assert_rounded(yk, H.norm_rope(k, None, tab, pos, False, EPS))


def test_position_outside_the_table_is_not_a_number():
    tab = H.table(16, 64).cuda()
    x = torch.ones(3, 1, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (-1, 16, 1 << 40):
        pos = torch.tensor([3, bad, 15], device="cuda")
        q, _ = eg.qk_norm_rope(x, x, tab, positions=pos)
        assert torch.isnan(q[1, 0, :64]).all() and not torch.isnan(q[1, 0, 64:]).any()
        assert not torch.isnan(q[0]).any() and not torch.isnan(q[2]).any()


def test_values_past_the_rotation_keep_infinities():
    tab = H.table(16, 64).cuda()
    x = torch.ones(2, 1, 128, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 100] = float("inf")
    q, _ = eg.qk_norm_rope(x, x, tab)
    assert torch.isinf(q[0, 0, 100]) and torch.isfinite(q[0, 0, :100]).all() and torch.isfinite(q[0, 0, 101:]).all()


def test_no_tokens():
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    tab = H.table(16, 64).cuda()
    q, k = eg.qk_norm_rope(e, e, tab, q_weight=w, k_weight=w)
    assert q.shape == e.shape and k.shape == e.shape
    _, _, dqw, dkw = eg.qk_norm_rope_backward(e, e, e, e, tab, q_weight=w, k_weight=w)
    assert (dqw == 0).all() and (dkw == 0).all()


# ------------------------------------------------------------------ append --

@pytest.mark.parametrize("dtype,t,hq,hk,dim,rot,pairs,norm", SHAPES)
@pytest.mark.parametrize("page,heads_first", [(16, False), (5, True)])
def test_append(dtype, t, hq, hk, dim, rot, pairs, norm, page, heads_first):
    d = _inputs(dtype, t, hq, hk, dim, rot, norm, seed=6)
    v = d["dev"]
    pages = t // page + 2
    shape = (pages, hk, page, dim) if heads_first else (pages, page, hk, dim)
    before = [H.rand(d["gen"], *shape, dtype=dtype) for _ in range(2)]
    dev = [c.cuda() for c in before]
    view = (lambda c: c.permute(0, 2, 1, 3)) if heads_first else (lambda c: c)
    slots = torch.randperm(pages * page, generator=d["gen"])[:t]
    if t > 2:
        slots[1], slots[2] = -1, pages * page + 3  # neither is in the cache
    q = eg.kv_append(v["k"], v["v"], view(dev[0]), view(dev[1]), slots.cuda(), q=v["q"], cos_sin=v["table"], positions=v["pos"],
                     q_weight=v["qw"], k_weight=v["kw"], eps=EPS, pairs=pairs)
    H.assert_rounded(q, H.norm_rope(d["q"], d["qw"], d["table"], d["pos"], pairs, EPS), "q")
    put = [i for i in range(t) if 0 <= slots[i] < pages * page]
    ref_k = H.norm_rope(d["k"], d["kw"], d["table"], d["pos"], pairs, EPS)
    at = slots[put]
    have_k, have_v = (view(c).cpu() for c in dev)
    H.assert_rounded(have_k[at // page, at % page], ref_k[put], "k")
    assert torch.equal(have_v[at // page, at % page], d["v"][put])
    # nothing else of the cache is written
    for c, b in zip((have_k, have_v), before):
        b = view(b).clone()
        b[at // page, at % page] = c[at // page, at % page]
        assert torch.equal(c, b)


def test_append_without_queries_or_rotation():
    g = torch.Generator().manual_seed(7)
    k, v = H.rand(g, 4, 2, 64), H.rand(g, 4, 2, 64)
    kc, vc = (torch.zeros(3, 8, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([0, 23, 9, 4], device="cuda")
    assert eg.kv_append(k.cuda(), v.cuda(), kc, vc, slots) is None
    assert torch.equal(kc.view(24, 2, 64)[slots.cpu()].cpu(), k) and torch.equal(vc.view(24, 2, 64)[slots.cpu()].cpu(), v)


def test_append_on_another_stream():
    g = torch.Generator().manual_seed(8)
    k, v, q = H.rand(g, 64, 2, 128), H.rand(g, 64, 2, 128), H.rand(g, 64, 8, 128)
    kc, vc = (torch.zeros(8, 8, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tab = H.table(64, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = [x.cuda() for x in (k, v, q, tab)]
    s.wait_stream(torch.cuda.current_stream())
    y = eg.kv_append(a[0], a[1], kc, vc, torch.arange(64, device="cuda"), q=a[2], cos_sin=a[3], stream=s.cuda_stream)
    s.synchronize()
    H.assert_rounded(y, H.norm_rope(q, None, tab, torch.arange(64), False, EPS))
    assert torch.equal(vc.view(64, 2, 128).cpu(), v)


def test_append_on_a_stream_that_waits_for_its_inputs():
    """Every input, the slots too, is made before the stream waits for it, and is kept until the stream is done."""
    g = torch.Generator().manual_seed(9)
    k, v, q = H.rand(g, 64, 2, 128), H.rand(g, 64, 2, 128), H.rand(g, 64, 8, 128)
    slots, tab = torch.randperm(64, generator=g), H.table(64, 128)
    kc, vc = (torch.zeros(8, 8, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    a = [x.cuda() for x in (k, v, q, tab, slots)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = eg.kv_append(a[0], a[1], kc, vc, a[4], q=a[2], cos_sin=a[3], stream=s.cuda_stream)
    s.synchronize()
    H.assert_rounded(y, H.norm_rope(q, None, tab, torch.arange(64), False, EPS))
    H.assert_rounded(kc.view(64, 2, 128)[a[4]], H.norm_rope(k, None, tab, torch.arange(64), False, EPS))
    assert torch.equal(vc.view(64, 2, 128).cpu()[slots], v)


def test_refusals():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    tab = H.table(16, 64).cuda()
    for call in (lambda: eg.qk_norm_rope(x.double(), x.double(), tab),
                 lambda: eg.qk_norm_rope(x, x[:3], tab),
                 lambda: eg.qk_norm_rope(x, x, tab.half()),
                 lambda: eg.qk_norm_rope(x, x, tab, positions=torch.zeros(4, dtype=torch.int32, device="cuda")),
                 lambda: eg.qk_norm_rope(x, x, tab, q_weight=torch.ones(64, device="cuda")),
                 lambda: eg.qk_norm_rope(x.cpu(), x.cpu(), tab),
                 lambda: eg.qk_norm_rope(x.transpose(1, 2), x.transpose(1, 2), tab),
                 lambda: eg.qk_norm_rope(x, x, tab, q_out=x[:, :1]),
                 lambda: eg.kv_append(x, x, x.view(1, 4, 2, 64), x.view(1, 4, 2, 64), None),
                 lambda: eg.kv_append(x, x, x.view(1, 4, 2, 64), x.view(2, 2, 2, 64), torch.arange(4, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: eg.qk_norm_rope(x, x, H.table(16, 66).cuda()),
                 lambda: eg.qk_norm_rope(x, x, tab[:, :63].contiguous()),
                 lambda: eg.qk_norm_rope(x, x, tab[:0]),
                 lambda: eg.qk_norm_rope(x, x, tab, q_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"), eps=-1.0)):
        with pytest.raises(eg.EgError) as e:
            call()
        assert e.value.status == eg.EG_ERR_INVALID_ARG
    wide = torch.zeros(4, 2, 320, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(eg.EgError) as e:
        eg.qk_norm_rope(wide, wide, None)
    assert e.value.status == eg.EG_ERR_UNSUPPORTED
