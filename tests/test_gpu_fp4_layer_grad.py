"""The sparse layer's gradient for its input through frozen weights in 4 bits, as a
program composes it from the products and their gradients: against the formula in 64
bits and against differences, on whole numbers, exactly."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw
from test_gpu_fp4 import BF, DEV, F32

pytestmark = pytest.mark.gpu


def whole(f, d, group, seed):
    """Weights -1, 0 and 1, most of them 0: (Fp4, float64 values), on the GPU."""
    g = torch.Generator(DEV).manual_seed(seed)
    w = torch.randint(-6, 7, (f, d), generator=g, device=DEV)
    w = torch.where(w.abs() == 6, w.sign(), 0 * w)
    w[:, ::group] = 6  # a group's largest: its scale is 1, codes are exact
    w4 = tw.fp4_quant(w.float(), group=group)
    assert torch.equal(w4.float(), w.float())
    return w4, w.double()


@pytest.mark.parametrize("T", (1, 9, 40, 64))
@pytest.mark.parametrize("d,f,group", [(256, 512, 64), (320, 1280, 128), (192, 384, 32)])
@pytest.mark.parametrize("dtype", (F32, BF))
def test_gradient_of_the_layer(T, d, f, group, dtype):
    (wg4, wg), (wu4, wu), (wd4, wd) = (whole(f, d, group, i) for i in range(3))
    g = torch.Generator(DEV).manual_seed(T)
    # few columns of x and dy are not zero: every sum stays a whole number below 2^24
    x, dy = (torch.zeros(T, d, device=DEV, dtype=dtype) for _ in range(2))
    x[:, 1:9] = torch.randint(-2, 3, (T, 8), generator=g, device=DEV).to(dtype)
    dy[:, 3:7] = torch.randint(-2, 3, (T, 4), generator=g, device=DEV).to(dtype)
    y = tw.fp4_decode_fwd(x, wg4, wu4, wd4)
    gate, up = (tw.fp4_matmul(x, w, out_dtype=F32) for w in (wg4, wu4))
    da = tw.fp4_matmul(dy, wd4, out_dtype=F32)
    open_ = gate > 0
    dx = (tw.fp4_matmul_dx(da * up * open_, wg4, out_dtype=F32) +
          tw.fp4_matmul_dx(da * torch.relu(gate), wu4, out_dtype=F32))

    xd = x.double().requires_grad_()
    want = (torch.relu(xd @ wg.t().contiguous()) * (xd @ wu.t().contiguous())) @ wd
    assert torch.equal(y.double(), want)
    (want * dy.double()).sum().backward()
    assert float(xd.grad.abs().max()) < 2 ** 24 and bool(xd.grad.any())
    assert torch.equal(dx.double(), xd.grad)
    # Along a line, the gates held open or closed as they are, the loss is of second
    # degree: its central difference is the gradient's product with the line.
    e = torch.zeros(T, d, device=DEV)
    e[:, 1:9] = torch.randint(-1, 2, (T, 8), generator=g, device=DEV).float()
    step = 1.0 / 1024

    def loss(s):
        p = x.float() + s * step * e
        gs, us = (tw.fp4_matmul(p, w, out_dtype=F32).double() for w in (wg4, wu4))
        a = torch.where(open_, gs, 0 * gs) * us
        return (a * da.double()).sum()
    diff = (loss(1) - loss(-1)) / (2 * step)
    assert float(diff) == float((dx.double() * e.double()).sum())
