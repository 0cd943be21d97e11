"""8-bit matrices with a NaN or an infinity in a block: every value that the
block stands for is NaN, the other blocks are as if it were not there, and the
codes past the columns are zeros all the same."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF, E4 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


def _rows(T, d, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, d), generator=g)


def _bytes(m):
    return m.q.cpu().view(torch.uint8)


# widths whose rows fill their lanes, end inside them, end inside a chunk of
# eight, and take two chunks a lane
@pytest.mark.parametrize("d", [128, 256, 300, 384, 1001, 2048, 8200])
@pytest.mark.parametrize("residual", [False, True], ids=["x", "x+res"])
def test_norm_gain(d, residual):
    """A NaN of the gain, and an infinity of it times a zero, in one column."""
    print("[case] norm to 8 bits, gain not finite", d, residual, flush=True)
    T = 21
    x, res = _rows(T, d, 1), _rows(T, d, 2).to(BF)
    bad = {d - 1: NAN, d // 2: INF}
    for j in bad:
        x[3, j] = 0
        res[3, j] = 0
    gain = 1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(3))
    dirty = gain.clone()
    for j, v in bad.items():
        dirty[j] = v
    args = dict(residual=res.to(DEV) if residual else None, out_dtype=E4)
    got = tw.rmsnorm_fwd(x.to(DEV), dirty.to(DEV), **args)[0]
    clean = tw.rmsnorm_fwd(x.to(DEV), gain.to(DEV), **args)[0]
    torch.cuda.synchronize()
    v, blocks = got.float().cpu(), {j // 128 for j in bad}
    for b in range(-(-d // 128)):
        part = v[:, 128 * b:min(d, 128 * b + 128)]
        if b in blocks:
            assert part.isnan().all(), b
        else:
            cut = slice(128 * b, 128 * b + 128)
            assert torch.equal(_bytes(got)[:, cut], _bytes(clean)[:, cut])
            assert torch.equal(got.scale[b], clean.scale[b])
    assert not _bytes(got)[:, d:].any()


@pytest.mark.parametrize("d", [300, 384, 1001, 2047, 8200])
@pytest.mark.parametrize("value", [NAN, INF, -INF], ids=str)
def test_norm_codes_past_the_columns(d, value):
    T = 9
    x = _rows(T, d, 1)
    x[2, d - 1] = x[5, 0] = value
    n = tw.rmsnorm_fwd(x.to(DEV), torch.ones(d, device=DEV), out_dtype=E4)[0]
    torch.cuda.synchronize()
    v = n.float().cpu()
    assert v[2, (d - 1) // 128 * 128:].isnan().all() and v[5, :128].isnan().all()
    assert v[[0, 1, 3, 4, 6, 7, 8]].isfinite().all()
    assert not _bytes(n)[:, d:].any()


@pytest.mark.parametrize("layout", ["rows", "cols", "both"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("R,C", [(1, 1), (3, 7), (129, 133), (200, 300), (250, 1001)])
def test_quant_codes_past_the_edges(R, C, dtype, block_rows, layout):
    """Not finite in the last block of both directions and in the first."""
    print("[case] quantised edges", R, C, dtype, block_rows, layout, flush=True)
    x = _rows(R, C, 1).to(dtype)
    x[R - 1, C - 1], x[0, 0], x[R // 2, C // 2] = INF, NAN, -INF
    o, t = tw.fp8_quant(x.to(DEV), block_rows=block_rows, layout=layout)
    torch.cuda.synchronize()
    for m, src in ((o, x), (t, x.t())):
        if m is None:
            continue
        rows, cols = src.shape
        v = m.float().cpu()
        bad = torch.zeros(src.shape, dtype=torch.bool)
        for i, j in (~src.isfinite()).nonzero().tolist():
            i0, j0 = i // block_rows * block_rows, j // 128 * 128
            bad[i0:i0 + block_rows, j0:j0 + 128] = True
        assert v[bad].isnan().all() and v[~bad].isfinite().all()
        assert not _bytes(m)[:, cols:].any()
