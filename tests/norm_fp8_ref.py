"""Plain 64-bit forms of the residual norm, the block quantisation and the
8-bit product, and the tolerances of their tests.

u = 2^-24 is float32's rounding unit, 2^-8 bfloat16's. A sum of terms taken
in float32 with at most k roundings on any term's way is within k u of the sum
of the terms' absolute values; the constants below count those roundings.

* Norm (d <= 16384). The sum of squares: at most 64 in a lane, 6 over a wave,
  2 over the waves, the square of a rounded h (2): 74, halved by the root; the
  mean, the root, the quotient and two products: 6. NORM = 64 covers
  74 / 2 + 6 on n, relative to |n|.
* Norm's gradient: each of its three terms carries r (43), its own products
  (4), and the second a mean over d (74) with r again: at most 128 u of the
  sum of the terms' absolute values. dgain: a term carries 48, and its sum over
  T <= 8192 rows at most 8192 / 512 = 16 in a workgroup's lane, 4 over its
  waves, 32 + 16 over the partial rows: 128 u covers 48 + 68.
* Product: 128 products in one matrix instruction, at most one rounding for
  each addition (128), a scale (2), one addition for each block of 128 k and,
  where k is split, one for each of at most 64 parts.
* Product with fast sums: each of eight products is kept to 13 bits below the
  largest, so an eight is off by at most 8 * 2^-13 of its terms' sum: FAST.
* A value that is stored is off by half a unit of its type once more.
"""
import torch

U32, UBF = 2.0 ** -24, 2.0 ** -8
NORM, GRAD = 64 * U32, 128 * U32
FAST = 8 * 2.0 ** -13
AMAX_MIN, E4M3_MAX = 2.0 ** -64, 448.0


def ustore(dtype):
    return UBF + 2 * U32 if dtype == torch.bfloat16 else U32


def rmsnorm(x, gain, eps, residual=None):
    """(n, h) in float64."""
    h = x.double() if residual is None else x.double() + residual.double()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h * r * gain.double(), h


def rmsnorm_bwd(dn, h, gain, eps, dres=None):
    """(dh, dgain) and the sums of their terms' absolute values, in float64."""
    dn, h, gain = dn.double(), h.double(), gain.double()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    xh, dg = h * r, dn * gain
    dh = r * (dg - xh * (dg * xh).mean(1, keepdim=True))
    mag = r * (dg.abs() + xh.abs() * (dg * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        dh, mag = dh + dres.double(), mag + dres.double().abs()
    return dh, (dn * xh).sum(0), mag, (dn * xh).abs().sum(0)


def to_e4m3(y):
    """float64 to the nearest e4m3 value, ties to even (|y| <= 448)."""
    step = 2 * half_step(y)
    return (torch.round(y / step) * step).float().to(torch.float8_e4m3fn)


def quant(x, block_rows):
    """(q, scale) as the layout defines them, bit for bit: the scale is the
    32-bit quotient amax / 448, q the e4m3 value nearest to x / scale (in 64
    bits no quotient of two floats is rounded onto or across a tie)."""
    x = x.float()
    R, C = x.shape
    rb, cb = -(-R // block_rows), -(-C // 128)
    p = torch.zeros((rb * block_rows, cb * 128), dtype=torch.float32)
    p[:R, :C] = x
    b = p.view(rb, block_rows, cb, 128)
    s = b.abs().amax(dim=(1, 3)).clamp(min=AMAX_MIN) / E4M3_MAX
    q = to_e4m3(b.double() / s.double()[:, None, :, None]).view(rb * block_rows, cb * 128)[:R]
    return q, s.t().contiguous()


def dequant(q, scale, block_rows):
    s = scale.double().t().repeat_interleave(block_rows, 0)[:q.shape[0]]
    return q.double() * s.repeat_interleave(128, 1)


def half_step(y):
    """Half the distance between e4m3 values around y (float64)."""
    _, e = torch.frexp(y)
    return torch.ldexp(torch.ones_like(y), e.clamp(min=-5) - 5)


def assert_within(got, ref, tol, what):
    got, ref, tol = got.detach().cpu().double(), ref.detach().cpu(), tol.detach().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, (got - ref).abs() / (tol + 1e-300), 0.0)))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: "
                             f"{got.flatten()[i]!r} against {ref.flatten()[i]!r} "
                             f"+- {tol.flatten()[i]!r}")
