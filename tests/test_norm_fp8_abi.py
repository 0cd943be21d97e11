"""Refusals of the norm, the quantisation and the 8-bit product, through the
C-ABI and through the Python calls, and the 64-bit forms that their GPU tests
compare with (CPU only: every call here ends before anything is launched)."""
import ctypes

import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
import norm_fp8_ref as ref

FAKE = 0x100000  # 16-byte aligned, never dereferenced
F32, BF, E4 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
NULL, SHAPE, DTYPE, ALIGN, WS = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def L():
    return tw.load()


def mat(rows=4, cols=256, ld=None, dt=tw.TWELL_BF16, p=FAKE):
    return tw.MatC(rows, cols, cols if ld is None else ld, dt, p)


def fp8(rows=4, cols=256, br=1, q=FAKE, s=FAKE):
    return tw.Fp8C(rows, cols, br, q, s)


def _r(x):
    return None if x is None else ctypes.byref(x)


def test_rmsnorm_fwd_refusals(L):
    def f(x=mat(), res=mat(), gain=FAKE, gdt=tw.TWELL_F32, eps=1e-6, h=mat(), n=mat(), n8=None):
        return L.twell_rmsnorm_fwd(_r(x), _r(res), gain, gdt, eps, _r(h), _r(n), _r(n8), None,
                                   None)
    assert f(x=None) == f(gain=0) == f(h=None) == f(n=None) == NULL
    assert f(n=mat(p=0)) == f(res=mat(p=0)) == NULL
    assert f(n=None, n8=fp8(q=0)) == f(n=None, n8=fp8(s=0)) == NULL
    assert f(gdt=2) == f(x=mat(dt=5)) == f(n=mat(dt=-1)) == DTYPE
    assert f(h=mat(dt=tw.TWELL_F32)) == DTYPE                      # h not of residual's type
    assert f(x=mat(cols=0)) == f(x=mat(rows=-1)) == f(x=mat(cols=tw.NORM_COLS + 1)) == SHAPE
    assert f(res=mat(rows=5)) == f(n=mat(cols=255)) == f(x=mat(ld=255)) == SHAPE
    assert f(x=mat(ld=-1)) == f(x=mat(ld=(1 << 31) + 1)) == SHAPE
    assert f(n8=fp8()) == SHAPE                                      # both outputs
    assert f(res=None) == SHAPE                                      # h without a residual
    assert f(n=None, n8=fp8(br=128)) == f(n=None, n8=fp8(cols=255)) == SHAPE
    for eps in (float("nan"), float("inf"), -1e-6):
        assert f(eps=eps) == SHAPE
    assert f(x=mat(p=FAKE + 1)) == f(gain=FAKE + 2) == f(n=None, n8=fp8(q=FAKE + 4)) == ALIGN
    assert f(n=None, n8=fp8(s=FAKE + 2)) == ALIGN
    z = mat(rows=0, p=0)
    assert f(x=z, res=z, h=z, n=z) == 0                              # no rows: nothing to do


def test_rmsnorm_bwd_refusals(L):
    need = L.twell_rmsnorm_bwd_workspace_bytes(4, 256)
    assert need >= 256 * 4
    assert L.twell_rmsnorm_bwd_workspace_bytes(0, 256) == 0
    for r, c in ((-1, 256), (4, 0), (4, tw.NORM_COLS + 1), ((1 << 28) + 1, 64)):
        assert L.twell_rmsnorm_bwd_workspace_bytes(r, c) == 0

    def f(dn=mat(), h=mat(), gain=FAKE, gdt=tw.TWELL_F32, eps=1e-6, dres=mat(), dh=mat(),
          dg=FAKE, ws=FAKE, nb=need):
        return L.twell_rmsnorm_bwd(_r(dn), _r(h), gain, gdt, eps, _r(dres), _r(dh), dg, ws, nb,
                                   None, None)
    assert f(dn=None) == f(h=None) == f(gain=0) == f(dh=None) == f(dg=0) == NULL
    assert f(h=mat(p=0)) == NULL
    assert f(gdt=7) == f(dres=mat(dt=3)) == DTYPE
    assert f(dn=mat(rows=3)) == f(dh=mat(cols=128)) == f(eps=-1.0) == SHAPE
    assert f(dg=FAKE + 2) == f(ws=FAKE + 8) == f(dh=mat(p=FAKE + 1)) == ALIGN
    assert f(nb=need - 1) == f(ws=0) == WS


def test_fp8_quant_refusals(L):
    def f(x=mat(), o=fp8(), t=fp8(256, 4)):
        return L.twell_fp8_quant(_r(x), _r(o), _r(t), None, None)
    assert f(x=None) == f(o=None, t=None) == f(x=mat(p=0)) == f(o=fp8(q=0)) == NULL
    assert f(x=mat(dt=9)) == DTYPE
    assert f(o=fp8(5)) == f(t=fp8(4, 256)) == f(o=fp8(br=64), t=None) == SHAPE
    assert f(o=fp8(br=128)) == SHAPE                                 # block_rows differ
    assert f(x=mat(rows=-1)) == SHAPE
    big = 1 << 28
    assert f(x=mat(big, big, big), o=fp8(big, big), t=None) == SHAPE  # 2^42 tiles
    assert f(x=mat(p=FAKE + 1)) == f(t=fp8(256, 4, q=FAKE + 8)) == ALIGN
    assert f(x=mat(rows=0, p=0), o=fp8(0, q=0, s=0), t=fp8(256, 0, q=0, s=0)) == 0


def test_fp8_matmul_refusals(L):
    def f(a=fp8(), b=fp8(8, 256, 128), o=mat(4, 8), sums=0, ws=FAKE, nb=1 << 40):
        return L.twell_fp8_matmul(_r(a), _r(b), _r(o), sums, ws, nb, None, None)
    assert f(a=None) == f(b=None) == f(o=None) == f(a=fp8(q=0)) == f(o=mat(4, 8, p=0)) == NULL
    assert f(o=mat(4, 8, dt=4)) == DTYPE
    assert f(b=fp8(8, 255)) == f(o=mat(4, 9)) == f(o=mat(5, 8)) == f(o=mat(4, 8, ld=7)) == SHAPE
    assert f(a=fp8(br=2)) == f(a=fp8(rows=-1)) == f(sums=2) == f(sums=-1) == SHAPE
    big = 1 << 28
    assert f(a=fp8(big), b=fp8(big), o=mat(big, big)) == SHAPE
    assert f(a=fp8(q=FAKE + 8)) == f(b=fp8(8, s=FAKE + 1)) == f(ws=FAKE + 4) == ALIGN
    assert f(a=fp8(0, q=0, s=0), o=mat(0, 8, p=0)) == 0
    for args in ((-1, 4, 4), (4, -1, 4), (4, 4, -1), (big, big, 4)):
        assert L.twell_fp8_matmul_workspace_bytes(*args) == 0
    for M, N, K in ((1, 2304, 6144), (300, 256, 8192), (1, 1, 1 << 20)):
        need = L.twell_fp8_matmul_workspace_bytes(M, N, K)
        if need:
            assert f(fp8(M, K), fp8(N, K), mat(M, N), nb=need - 1) == WS
            assert f(fp8(M, K), fp8(N, K), mat(M, N), ws=0, nb=0) == WS


def _raises(match, fn, *a, **k):
    with pytest.raises(tw.TwellError, match=match):
        fn(*a, **k)


def test_python_refusals():
    x, g = torch.zeros(4, 200), torch.zeros(200)
    _raises("x: expected", tw.rmsnorm_fwd, g, g)
    _raises("gain: shape", tw.rmsnorm_fwd, x, torch.zeros(199))
    _raises("unsupported dtype", tw.rmsnorm_fwd, x.half(), g)
    _raises("unsupported dtype", tw.rmsnorm_fwd, x, g.half())
    _raises("residual: shape", tw.rmsnorm_fwd, x, g, residual=x[:3])
    _raises("h: dtype", tw.rmsnorm_fwd, x, g, residual=x, h=x.to(BF))
    _raises("h: written only", tw.rmsnorm_fwd, x, g, h=x)
    _raises("out: dtype", tw.rmsnorm_fwd, x, g, out=x)
    _raises("out: expected an Fp8", tw.rmsnorm_fwd, x, g, out=x, out_dtype=E4)
    _raises("out.scale: shape", tw.rmsnorm_fwd, x, g, out_dtype=E4,
            out=tw.Fp8(torch.zeros(4, 256).to(E4), torch.zeros(4, 2), 200))
    _raises("consecutive", tw.rmsnorm_fwd, x.t().contiguous().t(), g)
    _raises("rows must not overlap", tw.rmsnorm_fwd, x[:1].expand(4, 200), g)
    _raises("GPU only", tw.rmsnorm_fwd, x, g)
    _raises("h: shape", tw.rmsnorm_bwd, x, x[:, :100], g)
    _raises("dgain: dtype", tw.rmsnorm_bwd, x, x, g, dgain=g.to(BF))
    _raises("workspace", tw.rmsnorm_bwd, x, x, g, workspace=torch.zeros(4))
    _raises("GPU only", tw.rmsnorm_bwd, x, x, g)
    _raises("layout", tw.fp8_quant, x, layout="both ways")
    _raises("block_rows", tw.fp8_quant, x, block_rows=64)
    _raises("out_t: not written", tw.fp8_quant, x, out_t=tw.empty_fp8(200, 4, 1, "cpu"))
    _raises("out: block_rows", tw.fp8_quant, x, out=tw.empty_fp8(4, 200, 128, "cpu"))
    _raises("out: 100 columns", tw.fp8_quant, x, out=tw.empty_fp8(4, 100, 1, "cpu"))
    _raises("GPU only", tw.fp8_quant, x)
    a, b = tw.empty_fp8(4, 200, 1, "cpu"), tw.empty_fp8(6, 200, 128, "cpu")
    _raises("b: 256 columns", tw.fp8_matmul, a, tw.empty_fp8(6, 256, 128, "cpu"))
    _raises("a: expected an Fp8", tw.fp8_matmul, x, b)
    _raises("a.q: shape", tw.fp8_matmul, tw.Fp8(a.q[:, :200], a.scale, 200), b)
    _raises("a.q: dtype", tw.fp8_matmul, tw.Fp8(a.q.float(), a.scale, 200), b)
    _raises("out: shape", tw.fp8_matmul, a, b, out=torch.zeros(4, 5, dtype=BF))
    _raises("unsupported dtype", tw.fp8_matmul, a, b, out_dtype=torch.float16)
    _raises("GPU only", tw.fp8_matmul, a, b)


def test_fp8_values():
    m = tw.Fp8(torch.arange(6, dtype=F32).repeat(256, 1).t().contiguous().to(E4),
               torch.tensor([[1.0], [0.5]]), 200, 128)
    assert m.rows == 6 and m.float().shape == (6, 200)
    assert m.float()[5, 127] == 5 and m.float()[5, 128] == 2.5


def test_reference_gradient_by_differences():
    g = torch.Generator().manual_seed(0)
    d = torch.float64
    x, res = torch.randn(3, 11, generator=g, dtype=d), torch.randn(3, 11, generator=g, dtype=d)
    gain, w, v = (torch.randn(s, generator=g, dtype=d) for s in (11, (3, 11), (3, 11)))

    def loss(x_, gain_):
        n, h = ref.rmsnorm(x_, gain_, 1e-2, res)
        return float((w * n).sum() + (v * h).sum())

    dh, dg, mag, gmag = ref.rmsnorm_bwd(w, x + res, gain, 1e-2, v)
    assert (dh.abs() <= mag + 1e-12).all() and (dg.abs() <= gmag + 1e-12).all()
    e = 1e-6
    for t in range(3):
        for j in range(11):
            p, m = x.clone(), x.clone()
            p[t, j] += e
            m[t, j] -= e
            assert abs((loss(p, gain) - loss(m, gain)) / (2 * e) - float(dh[t, j])) < 1e-7
    for j in range(11):
        p, m = gain.clone(), gain.clone()
        p[j] += e
        m[j] -= e
        assert abs((loss(x, p) - loss(x, m)) / (2 * e) - float(dg[j])) < 1e-7


def test_reference_quantisation():
    """A block whose values are the e4m3 grid itself comes back exactly; one
    planted wrong scale or value is seen by the bound of the norm's test."""
    grid = torch.arange(0x7F, dtype=torch.uint8).view(E4).float()
    x = torch.cat([grid, torch.zeros(1)])[None] * 0.125
    q, s = ref.quant(x, 1)
    assert torch.equal(ref.dequant(q, s, 1).float(), x)
    y = torch.linspace(-448, 448, 4001, dtype=torch.float64)
    near = y.float().to(E4).double()
    assert ((near - y).abs() <= ref.half_step(y) + y.abs() * 2 * ref.U32).all()
    assert not ((near * 1.13 - y).abs() <= ref.half_step(y)).all()
    with pytest.raises(AssertionError):
        ref.assert_within(near * 1.13, y, ref.half_step(y), "planted")
