"""The residual norm of more rows than one launch takes (a grid has fewer than
2^32 threads), up to the most that a call takes."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
import norm_fp8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF, E4 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-6


def _chunks(T, n=1 << 24):
    return [slice(t, min(T, t + n)) for t in range(0, T, n)]


# 16 lanes a row: 2^32 threads from 2^28 rows on, the most a call takes
@pytest.mark.parametrize("T,d", [(1 << 28, 1), ((1 << 28) - 5, 3)])
@pytest.mark.parametrize("out", [BF, E4], ids=["bf16", "e4m3"])
def test_forward_of_many_rows(T, d, out):
    print("[case] rmsnorm_fwd of many rows", T, d, out, flush=True)
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.randn((T, d), generator=g, device=DEV, dtype=BF)
    res = torch.randn((T, d), generator=g, device=DEV, dtype=BF)
    gain = 1 + 0.3 * torch.randn(d, generator=g, device=DEV)
    n, h = tw.rmsnorm_fwd(x, gain, residual=res, eps=EPS, out_dtype=out)
    torch.cuda.synchronize()
    for s in _chunks(T):
        want, wh = ref.rmsnorm(x[s], gain, EPS, res[s])
        assert ((h[s].double() - wh).abs() <= wh.abs() * (ref.ustore(BF) + ref.U32)).all(), s
        if out == BF:
            got, tol = n[s], want.abs() * (ref.NORM + ref.ustore(BF)) + 1e-37
        else:
            q = n.q[s]
            assert not q[:, d:].view(torch.uint8).any(), s
            sc = n.scale[0, s].double()[:, None]
            y = want / sc
            got = q[:, :d].double() * sc
            tol = sc * (ref.half_step(y) + y.abs() * (ref.NORM + 2 * ref.U32))
        assert ((got.double() - want).abs() <= tol).all(), s
