"""Products of many tokens on weights in 4 bits, compared exactly with 64 bits on whole
numbers: tiles of each size, each with its contraction whole and in joined parts."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
from test_gpu_fp4 import BF, F32
from test_gpu_fp4_dx_parts import numbers, whole

pytestmark = pytest.mark.gpu

# tokens, columns of the result, contraction (more blocks of 128 than the scales of 16
# are staged for, among them), group
SIZES = [(500, 5632, 130, 64), (333, 2811, 130, 128), (100, 1000, 2200, 32), (33, 2050, 8200, 32),
         (40, 301, 1000, 64), (333, 11008, 130, 128), (33, 33000, 130, 64), (333, 4100, 20000, 32),
         (40, 8200, 8200, 64), (200, 2811, 20000, 64), (200, 33000, 130, 64), (2048, 4100, 2300, 32),
         (500, 300, 20000, 128), (130, 5632, 8200, 32)]
ALL = {(tile, join) for tile in ("fp4_tile64", "fp4_tile128", "fp4_tile256")
       for join in (False, True)}


@pytest.mark.parametrize("dx", (False, True))
@pytest.mark.parametrize("dtype", (BF, F32))
def test_tiles_exact_on_integers(dx, dtype):
    call, seen = tw.fp4_matmul_dx if dx else tw.fp4_matmul, set()
    for T, n, k, group in SIZES:
        print("[case]", call.__name__, T, n, k, group, dtype, flush=True)
        w4, w = whole(k, n, group, n + k) if dx else whole(n, k, group, n + k)
        x, timer = numbers(T, k, dtype, T), tw.KernelTimer()
        got = call(x, w4, out_dtype=F32, timing=timer)
        want = x.double() @ (w if dx else w.t().contiguous())
        assert float(want.abs().max()) < 2 ** 24
        assert torch.equal(got.double(), want)
        names = [name for name, _ in timer.collect()]
        seen.add((next((m for m in names if "tile" in m), None), "fp4_join" in names))
        assert torch.equal(call(x, w4), want.float().to(BF))
    assert ALL <= seen, ALL - seen
