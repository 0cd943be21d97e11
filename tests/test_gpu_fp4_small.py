"""Products on weights in 4 bits of activations under 2^-100: what lies below 2^-126,
the smallest normal bfloat16 number, may be lost of each, and no more."""
import pytest
import torch

import fp4_ref as ref
from activation_sparse_ffn_gemm_amd import _lib as tw
from test_gpu_fp4 import BF, DEV, F32, quantised, within
from test_gpu_fp4_calls import acts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dx", (False, True))
@pytest.mark.parametrize("dtype", (F32, BF))
@pytest.mark.parametrize("ex", (-104, -115, -122, -130))
def test_small_activations(dx, dtype, ex):
    """Beside the sums' roundings (fp4_ref) an activation is off by at most 2^-126 in
    each of its three parts, a product or a sum that is itself that small by 2^-126
    more: (3 w + 1) 2^-126 a term."""
    N, K, group = 200, 256, 64
    w4, w = quantised(N, K, group, 3, scale=1.0)
    w = w.t() if dx else w
    for T in (1, 3, 16, 40, 200):
        x = (acts(T, w.shape[1], T).clamp(-1, 1).double() * 2.0 ** ex).to(dtype)
        call = tw.fp4_matmul_dx if dx else tw.fp4_matmul
        want, mag = ref.matmul(x, w)
        tol = ref.bound(mag, want, w.shape[1], F32)
        tol = tol + 2.0 ** -126 * (3 * w.abs().sum(1) + w.shape[1])
        within(call(x.to(DEV), w4, out_dtype=F32), want, tol)
