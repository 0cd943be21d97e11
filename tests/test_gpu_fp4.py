"""The operators on weights in 4 bits against their 64-bit forms (fp4_ref)."""
import pytest
import torch

import fp4_ref as ref
from activation_sparse_ffn_gemm_amd import _lib as tw

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF = torch.float32, torch.bfloat16
GROUPS = (32, 64, 128)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weights(R, C, seed, dtype=F32, scale=0.05):
    g = gen(seed)
    w = torch.randn(R, C, generator=g) * scale * torch.exp(torch.randn(R, 1, generator=g))
    return torch.where(torch.rand(R, C, generator=g) < 0.01, 8 * w, w).to(dtype)


def quantised(R, C, group, seed, scale=0.05):
    """(Fp4 on the GPU, its float64 values)."""
    q, s = ref.quant(weights(R, C, seed, scale=scale), group)
    return tw.Fp4(q.to(DEV), s.to(DEV), C, group), ref.values(q, s, C, group)


def within(got, want, tol):
    d = (got.detach().cpu().double() - want).abs()
    assert bool((d <= tol).all()), f"off by {float((d - tol).max()):.3e} past the tolerance"


def same(got, q, s):
    assert torch.equal(got.scale.cpu().view(torch.int16)[~s.isnan()],
                       s.view(torch.int16)[~s.isnan()])
    assert torch.equal(got.scale.cpu().isnan(), s.isnan())
    assert torch.equal(got.q.cpu(), q)


# ---------------------------------------------------------------- quantisation
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("R,C", [(1, 1), (1, 128), (3, 31), (33, 130), (70, 999), (5, 512),
                                 (257, 640)])
@pytest.mark.parametrize("dtype", (F32, BF))
def test_quant(R, C, group, dtype):
    w = weights(R, C, R * 1000 + C, dtype)
    same(tw.fp4_quant(w.to(DEV), group=group), *ref.quant(w, group))


@pytest.mark.parametrize("group", GROUPS)
def test_quant_ties_and_ends(group):
    """Every tie of the grid and its neighbours, and amaxes over the whole range."""
    rows = []
    for e in (-126, -80, -64, -10, 0, 60, 120, 124):
        for m in (32, 33, 47, 63):
            s = m / 32 * 2.0 ** e
            v = torch.tensor([t * s for t, _ in ref.TIES] + [6 * s], dtype=torch.float64).float()
            up = torch.nextafter(v, torch.full_like(v, float("inf")))
            dn = torch.nextafter(v, torch.zeros_like(v))
            r = torch.cat((v, up[:-1], dn, -v, torch.zeros(1)))
            rows.append(torch.nn.functional.pad(r, (0, 128 - r.numel())))
    big = torch.zeros(4, 128)
    big[0, 3], big[1, :5], big[2, 100] = 3.4028234e38, 3.0e38, -2.0 ** 127
    big[3] = 1e-40
    w = torch.cat((torch.stack(rows), big))
    same(tw.fp4_quant(w.to(DEV), group=group), *ref.quant(w, group))


@pytest.mark.parametrize("dtype", (F32, BF))
def test_quant_not_finite(dtype):
    w = weights(40, 300, 3, dtype)
    w[1, 5], w[2, 299], w[3, 128], w[4, 40] = (float(v) for v in ("nan", "inf", "-inf", "nan"))
    w[4, 41] = float("inf")
    for group in GROUPS:
        same(tw.fp4_quant(w.to(DEV), group=group), *ref.quant(w, group))
        v = tw.fp4_dequant(tw.fp4_quant(w.to(DEV), group=group)).cpu()
        j = 40 // group * group
        assert v[4, j:min(j + group, 300)].isnan().all() and v[0].isfinite().all()


def test_quant_strided_and_given():
    big = weights(37, 700, 9).to(DEV)
    for view in (big[:, 3:403], big[::2, 1:130], big[5:6, :77], big[:0]):
        out = tw.empty_fp4(view.shape[0], view.shape[1], 64, DEV)
        assert tw.fp4_quant(view, group=64, out=out) is out
        same(out, *ref.quant(view.cpu(), 64))


# ---------------------------------------------------------------- its inverse
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("R,C", [(1, 1), (5, 130), (33, 999), (7, 2056), (64, 256)])
def test_dequant(R, C, group):
    w4, v = quantised(R, C, group, 7 * R + C)
    for dtype in (F32, BF):
        got = tw.fp4_dequant(w4, out_dtype=dtype)
        assert got.dtype == dtype and torch.equal(got.cpu().double(), v)
    wide = torch.full((R, C + 9), 7.0, dtype=BF, device=DEV)
    tw.fp4_dequant(w4, out=wide[:, 3:3 + C])
    assert torch.equal(wide[:, 3:3 + C].cpu().double(), v)
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 3 + C:] == 7).all())
    assert torch.equal(w4.float().cpu().double(), v)


def test_dequant_every_code():
    """All 256 bytes, on scales that are powers of two, of six bits, and of eight
    (whose products with three are rounded)."""
    q = torch.arange(256, dtype=torch.uint8).view(4, 64).repeat(3, 1)
    s = torch.tensor([1.0] * 4 + [63 / 32] * 4 + [255 / 128] * 4).to(BF).view(1, 12)
    w4 = tw.Fp4(q.to(DEV), s.to(DEV), 128, 128)
    v = ref.values(q, s, 128, 128)
    assert torch.equal(tw.fp4_dequant(w4, out_dtype=F32).cpu().double(), v)
    assert torch.equal(tw.fp4_dequant(w4).cpu(), v.float().to(BF))


# ---------------------------------------------------------------- products
SIZES = [(1, 1, 1), (1, 16, 128), (2, 17, 130), (3, 100, 256), (4, 33, 640), (5, 31, 1090),
         (7, 260, 384), (16, 300, 2304), (17, 129, 512), (21, 64, 999), (22, 45, 256),
         (50, 515, 896), (64, 100, 1280), (65, 130, 200), (130, 257, 320), (333, 300, 1090)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("group", GROUPS)
def test_matmul(T, N, K, group):
    w4, w = quantised(N, K, group, N + K)
    for xdt, odt in ((BF, BF), (F32, F32), (BF, F32), (F32, BF)):
        x = torch.randn(T, K, generator=gen(T)).to(xdt)
        want, mag = ref.matmul(x, w)
        got = tw.fp4_matmul(x.to(DEV), w4, out_dtype=odt)
        assert got.dtype == odt and got.shape == (T, N)
        within(got, want, ref.bound(mag, want, K, odt))


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("group", GROUPS)
def test_matmul_dx(T, N, K, group):
    w4, w = quantised(N, K, group, N + K)
    for xdt, odt in ((BF, BF), (F32, F32), (BF, F32), (F32, BF)):
        dy = torch.randn(T, N, generator=gen(T)).to(xdt)
        want, mag = ref.matmul(dy, w.t())
        got = tw.fp4_matmul_dx(dy.to(DEV), w4, out_dtype=odt)
        assert got.dtype == odt and got.shape == (T, K)
        within(got, want, ref.bound(mag, want, N, odt))


@pytest.mark.parametrize("T,N,K", [(1, 33, 700), (3, 200, 300), (13, 77, 1000), (40, 90, 500),
                                   (200, 300, 260), (600, 520, 384)])
@pytest.mark.parametrize("dtype", (F32, BF))
def test_products_exact_on_integers(T, N, K, dtype):
    """Whole numbers whose sums stay below 2^24: every order of addition gives
    the same result, and a wrong index another."""
    g = gen(T + N)
    code = torch.randint(0, 16, (N, -(-K // 128) * 128), generator=g).to(torch.uint8)
    code[:, K:] = 0
    for group in GROUPS:
        s = torch.randint(1, 4, (code.shape[1] // group, N), generator=g).to(BF) * 2
        w4 = tw.Fp4((code[:, ::2] + 16 * code[:, 1::2]).to(DEV), s.to(DEV), K, group)
        w = ref.values(w4.q, w4.scale, K, group)
        x = torch.randint(-3, 4, (T, K), generator=g).to(dtype)
        dy = torch.randint(-3, 4, (T, N), generator=g).to(dtype)
        assert torch.equal(tw.fp4_matmul(x.to(DEV), w4, out_dtype=F32).cpu().double(),
                           x.double() @ w.t())
        assert torch.equal(tw.fp4_matmul_dx(dy.to(DEV), w4, out_dtype=F32).cpu().double(),
                           dy.double() @ w)


# ---------------------------------------------------------------- the layer
@pytest.mark.parametrize("T,d,f", [(1, 64, 128), (1, 2304, 1024), (2, 128, 256), (5, 256, 1024),
                                   (6, 192, 384), (16, 1024, 640), (17, 576, 256), (33, 448, 512),
                                   (64, 320, 1280), (3, 4096, 384)])
@pytest.mark.parametrize("group", GROUPS)
def test_layer(T, d, f, group):
    for dtype, off in ((BF, -2.0), (F32, -2.0), (BF, 0.0)):
        x = torch.randn(T, d, generator=gen(T))
        x[:, 0] = 1
        w = []
        for i in range(3):
            m = torch.randn(f, d, generator=gen(10 + i)) / (f if i == 2 else d) ** 0.5
            if i == 0:
                m[:, 0] = off
            q, s = ref.quant(m, group)
            w.append((tw.Fp4(q.to(DEV), s.to(DEV), d, group), ref.values(q, s, d, group)))
        x = x.to(dtype)
        want, tol = ref.layer(x, *(v for _, v in w))
        got = tw.fp4_decode_fwd(x.to(DEV), *(m for m, _ in w))
        assert got.dtype == F32
        within(got, want, tol)
