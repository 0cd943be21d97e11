"""Zeros of either sign in matrices of 4 bits: each keeps its sign, there and back."""
import pytest
import torch

import fp4_ref as ref
from activation_sparse_ffn_gemm_amd import _lib as tw
from test_gpu_fp4 import BF, DEV, F32, GROUPS, gen, same, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", (F32, BF))
@pytest.mark.parametrize("group", GROUPS)
def test_zeros_keep_their_sign(dtype, group):
    w = weights(37, 300, 5, dtype)
    w[torch.rand(37, 300, generator=gen(1)) < 0.3] = 0.0
    w[torch.rand(37, 300, generator=gen(2)) < 0.3] = -0.0
    w[3], w[4] = 0.0, -0.0  # groups of zeros
    w4 = tw.fp4_quant(w.to(DEV), group=group)
    same(w4, *ref.quant(w, group))
    for out in (F32, BF):
        back = tw.fp4_dequant(w4, out_dtype=out).cpu()
        assert torch.equal(back[w == 0], w[w == 0].to(out))
        assert torch.equal(back.signbit(), w.signbit())
