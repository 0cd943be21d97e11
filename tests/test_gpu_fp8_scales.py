"""8-bit products whose scales are very small or very large: the product of
two scales may be denormal or infinite where the result is not. Tolerances as
derived in norm_fp8_ref, and half of the smallest denormal for each of the
roundings of a sum that lies among the denormals."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
import norm_fp8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, E4 = torch.float32, torch.float8_e4m3fn
# sizes that between them take every kernel, whole and split contractions
SIZES = [(1, 300, 700), (1, 4100, 300), (4100, 16, 300), (4100, 20, 1000),
         (4100, 100, 700), (2049, 1000, 700), (2000, 4100, 700), (2000, 6000, 700),
         (1, 16, 70000), (520, 20, 40000), (130, 6000, 8192)]
KERNELS = {"fp8_mm_rows_1x1", "fp8_mm_rows_1x2", "fp8_mm_rows_2x2", "fp8_mm_rows_2x2_8",
           "fp8_mm_tile64", "fp8_mm_tile128", "fp8_mm_tile192", "fp8_mm_tile256", "fp8_mm_join"}


def _codes(rows, cols, g):
    q = (torch.randn((rows, -(-cols // 128) * 128), generator=g) * 60).abs().clamp(max=448)
    q[:, cols:] = 0
    return q.to(E4).to(DEV)


def _matrix(rows, cols, block_rows, exponent, seed):
    """Positive codes (sums without cancellation), scales of random
    significands around 2^exponent."""
    g = torch.Generator().manual_seed(seed)
    s = (1 + torch.rand((-(-cols // 128), -(-rows // block_rows)), generator=g)) * 2.0 ** exponent
    return tw.Fp8(_codes(rows, cols, g), s.to(DEV), cols, block_rows)


def _value(m):
    return ref.dequant(m.q, m.scale, m.block_rows)


def _within(got, want, tol, what):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(off[bad].max()), float(want[bad][0]))


@pytest.mark.parametrize("ea,eb", [(-73, -73), (-70, -60), (-72, 100), (102, -73), (60, 20)])
def test_scales_of_every_size(ea, eb):
    names, timer = set(), tw.KernelTimer()
    for M, N, K in SIZES:
        for rb in (128, 1):
            a, b = _matrix(M, K, 1, ea - 1, 1), _matrix(N, K, rb, eb, 2)
            da, db = _value(a), _value(b)
            want = da @ db.t()
            nkb = a.scale.shape[0]
            for fast in (False, True):
                print("[case] scales", ea, eb, M, N, K, rb, fast, flush=True)
                got = tw.fp8_matmul(a, b, out_dtype=F32, fast_sums=fast, timing=timer)
                torch.cuda.synchronize()
                names |= {n for n, _ in timer.collect()}
                rel = (128 + 2 + nkb + 64) * ref.U32 + ref.U32 + (ref.FAST if fast else 0)
                _within(got, want, rel * want + (nkb + 66) * 2.0 ** -150,
                                  f"{M} {N} {K} {rb} {fast}")
    assert names == KERNELS, names


@pytest.mark.parametrize("ea,eb", [(70, 70), (100, 90)])
def test_zero_sums_of_large_scales(ea, eb):
    """Rows of a that meet zeros of b only: the result is 0 though the scales'
    product is past float32; where terms meet it is infinite."""
    for M, N, K in SIZES:
        for rb in (128, 1):
            a, b = _matrix(M, K, 1, ea, 1), _matrix(N, K, rb, eb, 2)
            a.q.view(torch.uint8)[0::2, 0::2] = 0  # even rows: odd k alone
            b.q.view(torch.uint8)[:, 1::2] = 0     # b: even k alone
            for fast in (False, True):
                print("[case] zero sums", ea, eb, M, N, K, rb, fast, flush=True)
                got = tw.fp8_matmul(a, b, out_dtype=F32, fast_sums=fast)
                torch.cuda.synchronize()
                assert (got[0::2] == 0).all(), (M, N, K, rb, fast)
                assert (got[1::2] == float("inf")).all()


@pytest.mark.parametrize("M,N,K", [(2000, 4100, 256), (130, 300, 256)])
def test_scales_that_are_not_numbers(M, N, K):
    """Scales of zero, below zero, infinite and NaN on either side."""
    for rb in (128, 1):
        a, b = _matrix(M, K, 1, 0, 1), _matrix(N, K, rb, 0, 2)
        a.scale[0, :4] = torch.tensor([0.0, -2.5, float("inf"), float("nan")], device=DEV)
        b.scale[1, 0], b.scale[1, 1] = 0.0, -3.5
        last = b.scale.shape[1] - 1
        b.scale[0, last] = float("inf")
        for fast in (False, True):
            print("[case] odd scales", M, N, K, rb, fast, flush=True)
            got = tw.fp8_matmul(a, b, out_dtype=F32, fast_sums=fast)
            torch.cuda.synchronize()
            n0 = last * rb
            fin = [i for i in range(M) if i not in (2, 3)]
            want = _value(a)[fin] @ _value(b)[:n0].t()
            mag = _value(a)[fin].abs() @ _value(b)[:n0].abs().t()
            rel = (128 + 4 + 64) * ref.U32 + (ref.FAST if fast else 0)
            _within(got[fin][:, :n0], want, rel * mag, f"{M} {N} {K} {rb} {fast}")
            assert (got[2, :n0] == float("inf")).all() and got[3].isnan().all()
            assert not got[:, n0:].isfinite().any()


@pytest.mark.parametrize("M,N,K", [(4173, 4226, 300), (2500, 6151, 641), (24577, 513, 384),
                                   (1029, 2811, 640), (50, 2304, 1000)])
@pytest.mark.parametrize("sign", [False, True], ids=["positive", "signed"])
def test_scales_of_all_sizes_at_once(M, N, K, sign):
    """Every block and every row its own size, from the smallest scale to 2^40:
    tokens whose factor is a normal float beside tokens where it is not, in
    workgroups that go on to further tiles, whole and cut."""
    for rb in (128, 1):
        a, b = _matrix(M, K, 1, 0, 1), _matrix(N, K, rb, 0, 2)
        g = torch.Generator(DEV).manual_seed(M)
        for m in (a, b):
            m.scale *= 2.0 ** torch.randint(-73, 41, m.scale.shape, generator=g, device=DEV)
            if sign:
                m.scale *= torch.randint(0, 2, m.scale.shape, generator=g, device=DEV) * 2.0 - 1
        da, db = _value(a), _value(b)
        want, mag = da @ db.t(), da.abs() @ db.abs().t()
        nkb = a.scale.shape[0]
        for fast in (False, True):
            print("[case] mixed scales", M, N, K, rb, fast, flush=True)
            got = tw.fp8_matmul(a, b, out_dtype=F32, fast_sums=fast)
            torch.cuda.synchronize()
            rel = (128 + 2 + nkb + 64) * ref.U32 + ref.U32 + (ref.FAST if fast else 0)
            _within(got, want, rel * mag + (nkb + 66) * 2.0 ** -150, f"{M} {N} {K} {rb} {fast}")
