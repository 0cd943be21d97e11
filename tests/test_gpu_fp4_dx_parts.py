"""The gradient of few tokens through weights in 4 bits, its contraction in several
parts of one or more steps: whole numbers, compared exactly with 64 bits."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
from test_gpu_fp4 import BF, DEV, F32

pytestmark = pytest.mark.gpu

# rows of W (the contraction), columns: parts of one to four steps, a last one of
# few rows, one part only
SIZES = [(5632, 4096), (6144, 2304), (6144, 4096), (9216, 2304), (11008, 2048), (14336, 4096),
         (2816, 5632), (5001, 4000), (513, 384), (1300, 20000), (700, 33000)]


def whole(N, K, group, seed):
    """(Fp4 of any codes on scales 2, 4 and 6, its float64 values), on the GPU."""
    g = torch.Generator(DEV).manual_seed(seed)
    code = torch.randint(0, 16, (N, -(-K // 128) * 128), generator=g, device=DEV,
                         dtype=torch.uint8)
    code[:, K:] = 0
    s = torch.randint(1, 4, (code.shape[1] // group, N), generator=g, device=DEV) * 2
    w4 = tw.Fp4(code[:, ::2] + 16 * code[:, 1::2], s.to(BF), K, group)
    return w4, w4.float().double()


def numbers(T, n, dtype, seed):
    """-3 to 3: sums of 2^17 of them times a value (36 at most) stay below 2^24."""
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randint(-3, 4, (T, n), generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("group", (32, 128))
def test_every_row_counts_once(N, K, group):
    w4, w = whole(N, K, group, N + K)
    for dtype, tokens in ((BF, (1, 3, 16, 17, 32)), (F32, (1, 2, 5, 6, 10))):
        for T in tokens:
            print("[case] fp4_matmul_dx", T, N, K, group, dtype, flush=True)
            dy, t = numbers(T, N, dtype, T), tw.KernelTimer()
            got = tw.fp4_matmul_dx(dy, w4, out_dtype=F32, timing=t)
            want = dy.double() @ w
            assert float(want.abs().max()) < 2 ** 24
            assert "fp4_cols" in [name for name, _ in t.collect()]
            assert torch.equal(got.double(), want)
            assert torch.equal(tw.fp4_matmul_dx(dy, w4), want.float().to(BF))
