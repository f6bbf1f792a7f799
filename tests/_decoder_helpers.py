"""Definitions in 64 bits of the operators between a decoder's linear layers
(numpy-like torch code on the CPU, written from the formulas), and the error
bounds that their tests share."""
import math

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# largest relative error of one rounding to the type (2^-p for a significand of
# p bits: 8, 11 and 24), and half its smallest step
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
F32 = 2.0 ** -24


def name_of(t):
    return {v: k for k, v in DT.items()}[t.dtype]


def table(count, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(count, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def pair_places(rot, pairs):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)


def turn(z, cos_sin, positions, pairs, sign):
    """Rotate the pairs of z [T, H, D] by sign times their angle."""
    rot = cos_sin.shape[1] if cos_sin is not None else 0
    out = z.clone()
    if rot:
        a, b = pair_places(rot, pairs)
        row = cos_sin.double()[positions][:, None]
        c, s = row[..., :rot // 2], sign * row[..., rot // 2:]
        out[..., a] = z[..., a] * c - z[..., b] * s
        out[..., b] = z[..., b] * c + z[..., a] * s
    return out


def norm_rope(x, weight, cos_sin, positions, pairs, eps):
    z = x.double()
    if weight is not None:
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * weight.double()
    return turn(z, cos_sin, positions, pairs, 1.0)


def norm_rope_backward(dy, x, weight, cos_sin, positions, pairs, eps):
    """(dx, dw, sum of the magnitudes that dw adds up)."""
    dz = turn(dy.double(), cos_sin, positions, pairs, -1.0)
    if weight is None:
        return dz, None, None
    z = x.double()
    m = (z * z).mean(-1, keepdim=True) + eps
    g = dz * weight.double()
    dx = g / m.sqrt() - z * (g * z).mean(-1, keepdim=True) / m ** 1.5
    terms = dz * z / m.sqrt()
    return dx, terms.sum((0, 1)), terms.abs().sum((0, 1))


def assert_rounded(y, ref, what="", steps=24):
    """y is ref rounded once to its type, after float32 arithmetic whose error
    is a few units of the largest value of the row (`steps`: the longest chain
    of float32 operations a value goes through, each at most half an ulp)."""
    n = name_of(y)
    y = y.detach().cpu().double()
    assert y.shape == ref.shape, what
    amp = ref.abs().amax(-1, keepdim=True)
    bound = UNIT[n] * ref.abs() + steps * F32 * amp + TINY[n]
    over = (y - ref).abs() - bound
    assert not torch.isnan(over).any() and over.max().item() <= 0 if over.numel() else True, \
        f"{what}: {over.max().item():.3g} over the bound"


def directional(f, x, d, h):
    """Central difference of the scalar f at x along d."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def rand(gen, *shape, dtype="bf16", scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(DT[dtype])


def log2_ceil(n):
    return int(math.ceil(math.log2(max(n, 2))))
