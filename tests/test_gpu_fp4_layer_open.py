"""The sparse layer on weights in 4 bits: a neuron whose gate is open counts, however
small its product of gate and up value is."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
from test_gpu_fp4 import BF, DEV, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", (1, 6, 17, 40, 64))
@pytest.mark.parametrize("dtype", (F32, BF))
@pytest.mark.parametrize("up", (9, 10, 0, 8))  # codes of -0.5, -1, 0 and -0
def test_open_gates_that_underflow(T, dtype, up):
    """g = 2^-76 and u = -2^-76 (or a zero): g u lies under the smallest float. A NaN of
    wd's row reaches y all the same, as 0 times NaN does."""
    # 64 tokens: gates and up products as tiles, a formed by a kernel of its own
    d, f, group, i = 2304 if T == 64 else 256, 2560 if T == 64 else 1024, 64, 137
    timer = tw.KernelTimer()
    x = torch.zeros(T, d, dtype=dtype, device=DEV)
    x[:, 0] = 2.0 ** -10

    def coded(code):  # one weight, at neuron i and column 0; scales 2^-66
        q = torch.zeros(f, d // 2, dtype=torch.uint8, device=DEV)
        q[i, 0] = code
        return tw.Fp4(q, torch.full((d // group, f), 2.0 ** -66, dtype=BF, device=DEV), d, group)

    wd = coded(0)
    wd.scale[1, i] = float("nan")  # columns 64 to 127
    y = tw.fp4_decode_fwd(x, coded(2), coded(up), wd, timing=timer)
    assert y[:, 64:128].isnan().all()
    assert not y[:, :64].any() and not y[:, 128:].any()
    assert ("fp4_act" in [name for name, _ in timer.collect()]) == (T == 64)
    # the same neuron closed, by a gate of zero and one below
    for gate in (0, 10):
        y = tw.fp4_decode_fwd(x, coded(gate), coded(up), wd)
        assert not y.any()
