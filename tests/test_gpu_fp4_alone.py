"""Few tokens and weights in 4 bits: a token's results are the same bits alone and
beside others, as long as the few-token kernels take them."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
from test_gpu_fp4 import BF, DEV, F32
from test_gpu_fp4_calls import coded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,group", [(1000, 2304, 64), (6144, 2304, 128), (16400, 4096, 32),
                                       (20001, 2200, 128), (32768, 1100, 64)])
def test_product(N, K, group):
    w4, _ = coded(N, K, group, N)
    for dtype, counts in ((BF, (1, 2, 5, 9, 16, 20, 32)), (F32, (1, 2, 3, 5, 9, 10))):
        g = torch.Generator(DEV).manual_seed(K)
        x = torch.randn(counts[-1], K, generator=g, device=DEV).to(dtype)
        alone = torch.cat([tw.fp4_matmul(x[t:t + 1], w4, out_dtype=F32) for t in range(len(x))])
        for T in counts:
            timer = tw.KernelTimer()
            y = tw.fp4_matmul(x[:T], w4, out_dtype=F32, timing=timer)
            assert torch.equal(y, alone[:T]), (T, dtype)
            assert timer.collect()[-1][0] == "fp4_rows"


@pytest.mark.parametrize("d,f", [(1024, 2816), (2304, 16512)])
def test_layer(d, f):
    ms = [coded(f, d, 64, i)[0] for i in range(3)]
    for dtype, counts in ((BF, (1, 4, 9, 16)), (F32, (1, 2, 3, 5))):
        x = torch.randn(16, d, generator=torch.Generator(DEV).manual_seed(d), device=DEV).to(dtype)
        alone = torch.cat([tw.fp4_decode_fwd(x[t:t + 1], *ms) for t in range(16)])
        for T in counts:
            timer = tw.KernelTimer()
            y = tw.fp4_decode_fwd(x[:T], *ms, timing=timer)
            assert torch.equal(y, alone[:T]), (T, dtype)
            assert "fp4_gate_up" in [name for name, _ in timer.collect()]
