"""Plain 64-bit forms of the operators on weights in 4 bits, and the tolerances
of their tests.

u = 2^-24 is float32's rounding unit. A sum of terms taken in float32 with at
most k roundings on any term's way is within k u of the sum of the terms'
absolute values. Products are exact (a value is a bfloat16 number, a float32
activation three of them), so:

* Product over K: at most one rounding for each term added (K, three times that
  for float32 activations, whose later parts are 2^-8 and 2^-16 of the first:
  K (1 + 2^-7) in all), one for each group's scale (K / 32), at most 64 for the
  parts that are joined: SUM(K) = 1.05 K + 64.
* Layer: g and u are such products; a = g u is one rounding more; y's sum over
  d_ff neurons takes a scale, a product (2) and at most d_ff + 64 additions.
* A value that is stored in bfloat16 is off by half a unit, 2^-8 of it.

Quantisation and its inverse are compared bit for bit.
"""
import torch

U32, UBF = 2.0 ** -24, 2.0 ** -8
AMAX_MIN, AMAX_MAX = 2.0 ** -64, 2.0 ** 127
VALUES = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                      dtype=torch.float64)
# ties between neighbours, and whether a tie goes to the upper one (even code)
TIES = ((.25, False), (.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
        (5., False))


def terms(K):
    return 1.05 * K + 64


def six_bits(v):
    """float64 to the nearest number of six significant bits, ties to even."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.round(m * 64) / 64, e)


def quant(w, group):
    """(q, scale) as the layout defines them, bit for bit."""
    w = w.detach().cpu().double()
    R, C = w.shape
    cp = -(-C // 128) * 128
    p = torch.zeros(R, cp, dtype=torch.float64)
    p[:, :C] = w
    p = p.view(R, cp // group, group)
    amax = p.abs().amax(2)
    bad = ~torch.isfinite(p).all(2)
    s = six_bits(amax.nan_to_num(1.0, 1.0).clamp(AMAX_MIN, AMAX_MAX) / 6)
    code = torch.zeros_like(p)
    for tie, up in TIES:
        border = tie * s[:, :, None]
        code += (p.abs() >= border) if up else (p.abs() > border)
    # what is negative keeps its sign, rounded to zero or not
    code = (code + 8 * torch.signbit(p)).to(torch.uint8)
    code[bad] = 0
    code = code.view(R, cp)
    s[bad] = float("nan")
    return code[:, ::2] + 16 * code[:, 1::2], s.t().contiguous().to(torch.bfloat16)


def values(q, scale, cols, group):
    """The float64 matrix that (q, scale) stands for."""
    q, s = q.cpu(), scale.cpu().double()
    c = torch.stack((q & 15, q >> 4), 2).flatten(1)
    return (VALUES[c.int()] * s.t().repeat_interleave(group, 1))[:, :cols]


def matmul(x, w):
    """x w^T and the sums of its terms' absolute values, float64."""
    x = x.detach().cpu().double()
    return x @ w.t(), x.abs() @ w.t().abs()


def bound(mag, ref, K, dtype):
    """How far a product over K may be from ref."""
    b = terms(K) * U32 * mag
    return b + (UBF * (ref.abs() + b) if dtype == torch.bfloat16 else 0)


def layer(x, wg, wu, wd):
    """y and how far a float32 layer may be from it."""
    x, d, f = x.detach().cpu().double(), x.shape[1], wg.shape[0]
    (g, mg), (u, mu) = matmul(x, wg), matmul(x, wu)
    eg, eu = terms(d) * U32 * mg, terms(d) * U32 * mu
    h = g.clamp(min=0)
    a = h * u
    ea = torch.where(g > -eg, eg * u.abs() + (h + eg) * eu + 2 * U32 * a.abs(), 0 * g)
    y = a @ wd
    return y, ea @ wd.abs() + terms(f) * U32 * ((a.abs() + ea) @ wd.abs())
