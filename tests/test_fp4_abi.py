"""Refusals of the calls on weights in 4 bits, through the C-ABI and through the
Python calls, and the 64-bit forms that their GPU tests compare with (CPU only:
every call here ends before anything is launched)."""
import ctypes

import pytest
import torch

import fp4_ref as ref
from activation_sparse_ffn_gemm_amd import _lib as tw

FAKE = 0x100000  # 16-byte aligned, never dereferenced
F32, BF = torch.float32, torch.bfloat16
NULL, SHAPE, DTYPE, ALIGN, WS = -1, -2, -3, -4, -5
BIG = 1 << 28


@pytest.fixture(scope="module")
def L():
    return tw.load()


def mat(rows=4, cols=256, ld=None, dt=tw.TWELL_BF16, p=FAKE):
    return bytes(tw.MatC(rows, cols, cols if ld is None else ld, dt, p))


def fp4(rows=8, cols=256, group=64, q=FAKE, s=FAKE):
    return bytes(tw.Fp4C(rows, cols, group, q, s))


def test_quant_refusals(L):
    def f(x=mat(8), o=fp4()):
        return L.twell_fp4_quant(x, o, None, None)
    assert f(x=None) == f(o=None) == f(x=mat(8, p=0)) == f(o=fp4(q=0)) == f(o=fp4(s=0)) == NULL
    assert f(x=mat(8, dt=4)) == DTYPE
    assert f(x=mat(7)) == f(x=mat(8, 255)) == f(x=mat(8, ld=255)) == f(o=fp4(group=16)) == SHAPE
    assert f(o=fp4(rows=-1)) == f(o=fp4(BIG + 1), x=mat(BIG + 1)) == f(x=mat(8, ld=-1)) == SHAPE
    assert f(o=fp4(q=FAKE + 8)) == f(o=fp4(s=FAKE + 1)) == f(x=mat(8, p=FAKE + 1)) == ALIGN
    assert f(x=mat(0, p=0), o=fp4(0, q=0, s=0)) == f(x=mat(8, 0, p=0), o=fp4(8, 0, q=0, s=0)) == 0


def test_dequant_refusals(L):
    def f(w=fp4(), o=mat(8)):
        return L.twell_fp4_dequant(w, o, None, None)
    assert f(w=None) == f(o=None) == f(w=fp4(q=0)) == f(o=mat(8, p=0)) == NULL
    assert f(o=mat(8, dt=-1)) == DTYPE
    assert f(o=mat(9)) == f(o=mat(8, 128)) == f(w=fp4(group=0)) == f(o=mat(8, ld=1)) == SHAPE
    assert f(w=fp4(q=FAKE + 1)) == f(o=mat(8, p=FAKE + 1)) == ALIGN
    assert f(w=fp4(0, q=0, s=0), o=mat(0, p=0)) == 0


@pytest.mark.parametrize("dx", (False, True))
def test_product_refusals(L, dx):
    call = L.twell_fp4_matmul_dx if dx else L.twell_fp4_matmul
    size = L.twell_fp4_matmul_dx_workspace_bytes if dx else L.twell_fp4_matmul_workspace_bytes
    a, b = (8, 256) if dx else (256, 8)  # columns of x and of the result

    def f(x=mat(4, a), w=fp4(), o=mat(4, b), ws=FAKE, nb=1 << 40):
        return call(x, w, o, ws, nb, None, None)
    assert f(x=None) == f(w=None) == f(o=None) == f(x=mat(4, a, p=0)) == f(w=fp4(q=0)) == NULL
    assert f(o=mat(4, b, p=0)) == NULL
    assert f(x=mat(4, a, dt=2)) == f(o=mat(4, b, dt=7)) == DTYPE
    assert f(x=mat(4, a + 1)) == f(o=mat(4, b + 1)) == f(o=mat(5, b)) == SHAPE
    assert f(x=mat(4, a, ld=a - 1)) == f(o=mat(4, b, ld=b - 1)) == f(w=fp4(group=48)) == SHAPE
    assert f(x=mat(-1, a), o=mat(-1, b)) == SHAPE
    long = (1 << 21) + 1
    if dx:
        assert f(x=mat(4, long), w=fp4(long)) == SHAPE
    else:
        assert f(x=mat(4, long), w=fp4(8, long)) == SHAPE
    many = (1 << 27) + 1  # tokens, of pieces of 16 x 128
    assert f(x=mat(many, a), o=mat(many, b), w=fp4(8, 256)) == SHAPE
    assert f(w=fp4(q=FAKE + 8)) == f(w=fp4(s=FAKE + 1)) == f(ws=FAKE + 4) == ALIGN
    assert f(x=mat(4, a, p=FAKE + 1)) == f(o=mat(4, b, p=FAKE + 1)) == ALIGN
    assert f(x=mat(0, a, p=0), o=mat(0, b, p=0)) == 0
    for args in ((tw.TWELL_BF16, -1, 8, 8), (tw.TWELL_BF16, 4, -1, 8), (tw.TWELL_F32, 4, 8, -1),
                 (9, 4, 8, 8), (tw.TWELL_BF16, BIG, BIG, 8), (tw.TWELL_BF16, 0, 8, 256)):
        assert size(*args) == 0
    # float32 is laid out anew: that much workspace at least, and no less is taken
    for T in (1, 5, 6, 70, 300):
        need = size(tw.TWELL_F32, T, 256, 512)
        assert need >= T * (256 if dx else 512) * 6
        x, o = ((256, 512) if dx else (512, 256))
        args = mat(T, x, dt=tw.TWELL_F32), fp4(256, 512), mat(T, o)
        assert call(*args, FAKE, T * x * 6 - 1, None, None) == WS
        assert call(*args, None, need, None, None) == WS


def test_layer_refusals(L):
    def f(x=mat(4, 256), g=fp4(128), u=fp4(128), d=fp4(128), y=FAKE, ws=FAKE, nb=1 << 40):
        return L.twell_fp4_decode_fwd(x, g, u, d, y, ws, nb, None, None)
    assert f(x=None) == f(g=None) == f(u=None) == f(d=None) == f(y=0) == NULL
    assert f(x=mat(4, 256, p=0)) == f(u=fp4(128, q=0)) == f(d=fp4(128, s=0)) == NULL
    assert f(x=mat(4, 256, dt=3)) == DTYPE
    assert f(x=mat(65, 256)) == f(x=mat(-1, 256)) == f(x=mat(4, 200)) == f(x=mat(4, 4160)) == SHAPE
    assert f(g=fp4(100)) == f(u=fp4(256)) == f(d=fp4(128, 192)) == f(u=fp4(128, group=32)) == SHAPE
    assert f(g=fp4(32896), u=fp4(32896), d=fp4(32896)) == f(x=mat(4, 256, ld=255)) == SHAPE
    assert f(y=FAKE + 4) == f(ws=FAKE + 8) == f(d=fp4(128, q=FAKE + 4)) == ALIGN
    assert f(x=mat(0, 256, p=0), y=0) == 0
    for dt, T in ((tw.TWELL_BF16, 1), (tw.TWELL_BF16, 64), (tw.TWELL_F32, 5), (tw.TWELL_F32, 40)):
        need = L.twell_fp4_decode_workspace_bytes(dt, T, 256, 128)
        assert need >= T * 128 * 4
        assert f(x=mat(T, 256, dt=dt), ws=0, nb=need) == WS
        assert f(x=mat(T, 256, dt=dt), nb=T * 128 * 4 - 1) == WS
    for args in ((7, 1, 256, 128), (1, 65, 256, 128), (1, -1, 256, 128), (1, 1, 100, 128),
                 (1, 1, 256, 100)):
        assert L.twell_fp4_decode_workspace_bytes(*args) == 0


def _raises(match, fn, *a, **k):
    with pytest.raises(tw.TwellError, match=match):
        fn(*a, **k)


def test_python_refusals():
    x = torch.zeros(4, 200)
    w = tw.empty_fp4(6, 200, 64, "cpu")
    assert w.q.shape == (6, 128) and w.scale.shape == (4, 6) and w.rows == 6
    _raises("w: expected", tw.fp4_quant, x[0])
    _raises("group: 16", tw.fp4_quant, x, group=16)
    _raises("unsupported dtype", tw.fp4_quant, x.half())
    _raises("consecutive", tw.fp4_quant, x.t().contiguous().t())
    _raises("out: group 64", tw.fp4_quant, x, out=tw.empty_fp4(4, 200, 64, "cpu"))
    _raises("out: 100 columns", tw.fp4_quant, x, out=tw.empty_fp4(4, 100, 128, "cpu"))
    _raises("out.q: shape", tw.fp4_quant, x, out=tw.empty_fp4(5, 200, 128, "cpu"))
    _raises("GPU only", tw.fp4_quant, x)
    _raises("w: expected an Fp4", tw.fp4_dequant, x)
    _raises("out: shape", tw.fp4_dequant, w, out=torch.zeros(6, 199, dtype=BF))
    _raises("unsupported dtype", tw.fp4_dequant, w, out_dtype=torch.float16)
    _raises("GPU only", tw.fp4_dequant, w)
    _raises("w.q: dtype", tw.fp4_matmul, x, tw.Fp4(w.q.float(), w.scale, 200, 64))
    _raises("w.scale: dtype", tw.fp4_matmul, x, tw.Fp4(w.q, w.scale.float(), 200, 64))
    _raises("w.scale: shape", tw.fp4_matmul, x, tw.Fp4(w.q, w.scale, 200, 32))
    _raises("w.group", tw.fp4_matmul, x, tw.Fp4(w.q, w.scale, 200, 256))
    _raises("contiguous", tw.fp4_matmul, x, tw.Fp4(w.q.t().contiguous().t(), w.scale, 200, 64))
    _raises("x: 199 columns, w has 200 columns", tw.fp4_matmul, x[:, 1:], w)
    _raises("dy: 200 columns, w has 6 rows", tw.fp4_matmul_dx, x, w)
    _raises("out: shape", tw.fp4_matmul, x, w, out=torch.zeros(4, 7, dtype=BF))
    _raises("out: dtype", tw.fp4_matmul, x, w, out=torch.zeros(4, 6))
    _raises("workspace", tw.fp4_matmul, x, w, workspace=torch.zeros(4))
    _raises("GPU only", tw.fp4_matmul, x, w)
    _raises("GPU only", tw.fp4_matmul_dx, x[:, :6], w)
    x = torch.zeros(4, 128)
    m = [tw.empty_fp4(128, 128, 64, "cpu") for _ in range(3)]
    _raises("at most 64", tw.fp4_decode_fwd, torch.zeros(65, 128), *m)
    _raises("wg_t: expected an Fp4", tw.fp4_decode_fwd, x, m[0].q, m[1], m[2])
    _raises("wu_t: group", tw.fp4_decode_fwd, x, m[0], tw.empty_fp4(128, 128, 32, "cpu"), m[2])
    _raises("wd: 256 columns", tw.fp4_decode_fwd, x, m[0], m[1], tw.empty_fp4(128, 256, 64, "cpu"))
    _raises("wg_t: 256 columns", tw.fp4_decode_fwd, x, tw.empty_fp4(128, 256, 64, "cpu"), m[1], m[2])
    _raises("y: dtype", tw.fp4_decode_fwd, x, *m, y=x.to(BF))
    _raises("GPU only", tw.fp4_decode_fwd, x, *m)


# ---------------------------------------------------------------- the 64-bit forms
def test_ref_rounds_to_the_nearest_value():
    """Against a search over all values; ties to the even code."""
    g = torch.Generator().manual_seed(0)
    w = torch.randn(50, 128, generator=g)
    w[0, :8] = torch.tensor([6., .25, .75, 1.25, 1.75, 2.5, 3.5, 5.])  # scale 1: ties
    w[0, 8:] = 0
    q, s = ref.quant(w, 128)
    v = ref.values(q, s, 128, 128)
    code = torch.stack((q & 15, q >> 4), 2).flatten(1).int()
    sc = s.double()[0][:, None, None]
    far = (w.double()[:, :, None] - ref.VALUES * sc).abs()
    least = far.min(2).values
    assert torch.equal((w.double() - v).abs(), least)
    tie = (far == least[:, :, None]) & (ref.VALUES.abs() != v.abs()[:, :, None] / sc)
    assert not (tie.any(2) & (code % 2 == 1)).any()
    assert code[0, :8].tolist() == [7, 0, 2, 2, 4, 4, 6, 6]


def test_ref_scale_has_six_bits_and_exact_products():
    amax = torch.exp(torch.linspace(-40, 80, 4001, dtype=torch.float64))
    w = torch.zeros(4001, 32)
    w[:, 7] = amax.float()
    _, s = ref.quant(w, 32)
    s = s[0].double()  # (of the padding's groups: those of zeros)
    m, _ = torch.frexp(s)
    assert torch.equal(m * 64, torch.round(m * 64))
    assert ((s * 6 / amax.float().double()).log2().abs() < 2.0 ** -5).all()
    for v in ref.VALUES:
        assert torch.equal((s * v).float().to(BF).double(), s * v)


def test_fp4_float_is_the_format():
    q, s = ref.quant(torch.randn(9, 300, generator=torch.Generator().manual_seed(1)), 64)
    assert torch.equal(tw.Fp4(q, s, 300, 64).float().double(), ref.values(q, s, 300, 64))
    assert ctypes.sizeof(tw.Fp4C) == len(tw._pack_fp8(1, 2, 32, 3, 4))
