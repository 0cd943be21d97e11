"""The norm's 8-bit output is the e4m3 value nearest to n / scale, as the layout
defines it, and not to a float32 of it. The kernel's quotient is off by a few
roundings of 64 bits and two Newton steps of 2^-40 each, so by less than 2^-37;
only a quotient that near to a tie may go either way."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
import norm_fp8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF, E4 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
EPS, NEAR = 1e-6, 2.0 ** -37


def _blocks(t):
    """[T][d] as [T][blocks][128], zeros past d."""
    T, d = t.shape
    p = torch.zeros((T, -(-d // 128) * 128), dtype=t.dtype, device=t.device)
    p[:, :d] = t
    return p.view(T, -1, 128)


def _not_nearest(q, y):
    """How many of q are not the nearest value to y."""
    return int(((q.double() - y).abs() > ref.half_step(y) + NEAR * y.abs()).sum())


CASES = [(1, 7, F32, None), (1, 128, BF, BF), (1, 2304, F32, BF), (1, 2311, BF, F32),
         (1, 16384, F32, BF), (2, 8192, F32, F32), (1029, 999, BF, F32), (8192, 2048, F32, BF),
         (8192, 2048, BF, None), (1024, 16000, F32, BF), (65536, 256, F32, F32)]


@pytest.mark.parametrize("T,d,xt,rt", CASES, ids=lambda v: str(v).replace("torch.", ""))
def test_nearest(T, d, xt, rt):
    print("[case] rmsnorm_fwd nearest", T, d, xt, rt, flush=True)
    g = torch.Generator(DEV).manual_seed(T + d)
    x = torch.randn((T, d), generator=g, device=DEV).to(xt)
    res = None if rt is None else torch.randn((T, d), generator=g, device=DEV).to(rt)
    gain = 1 + 0.3 * torch.randn(d, generator=g, device=DEV)
    n, _ = tw.rmsnorm_fwd(x, gain, residual=res, eps=EPS, out_dtype=E4)
    torch.cuda.synchronize()
    want, h = ref.rmsnorm(x, gain, EPS, res)
    want = _blocks(want)
    amax = want.abs().amax(2).clamp(min=ref.AMAX_MIN)
    s = n.scale.t().double()
    assert ((s * 448 - amax).abs() <= amax * (ref.U32 + NEAR)).all()
    y = want / s[:, :, None]
    assert _not_nearest(n.q.view(T, -1, 128), y) == 0
    if (T, d, xt) == (8192, 2048, F32):  # the check sees 32-bit arithmetic
        h, s, gain = h.cpu().float(), n.scale.t().cpu(), gain.cpu()
        r = 1 / torch.sqrt((h ** 2).mean(1, keepdim=True) + EPS)
        f = _blocks(h * r * gain) / s[:, :, None]
        assert _not_nearest(f.to(E4), y.cpu()) > 0
