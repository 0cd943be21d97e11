"""The workspace of the 8-bit product: a call asks for what its own sums and
scales need, whatever the others of these sizes take."""
import pytest
import torch

from activation_sparse_ffn_gemm_amd import _lib as tw

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("M,N,K", [(300, 1000, 8192), (130, 1000, 16384), (300, 1024, 16384)])
def test_a_call_asks_for_its_own_workspace(M, N, K):
    """At these sizes fast sums split the contraction further than full sums,
    which take no parts at the first two."""
    print("[case] fp8_matmul workspace", M, N, K, flush=True)
    g = torch.Generator().manual_seed(1)
    a, b = (tw.fp8_quant(torch.randint(-2, 3, (r, K), generator=g).float().to(DEV))[0]
            for r in (M, N))
    most = tw.fp8_matmul_workspace_bytes(M, N, K)
    want = tw.fp8_matmul(a, b, out_dtype=torch.float32)
    out = torch.empty(M, N, device=DEV)
    args = [tw._pack_fp8(m.rows, K, 1, m.q.data_ptr(), m.scale.data_ptr()) for m in (a, b)]
    args.append(tw._pack_mat(M, N, N, tw.TWELL_F32, out.data_ptr()))
    ws = torch.empty(most, dtype=torch.uint8, device=DEV)

    def call(sums, nbytes):
        out.fill_(float("nan"))
        return tw.load().twell_fp8_matmul(*args, sums, ws.data_ptr() if nbytes else None, nbytes,
                                          None, torch.cuda.current_stream().cuda_stream)

    def least(sums):  # in partial results of M x N
        for parts in range(33):
            rc = call(sums, parts * M * N * 4)
            if rc != tw.E_WORKSPACE:
                torch.cuda.synchronize()
                assert rc == 0 and torch.allclose(out, want, rtol=1e-3, atol=1e-2)
                return parts

    full, fast = least(tw.SUMS_F32), least(tw.SUMS_FP8)
    assert full < fast and max(full, fast) * M * N * 4 == most
    if fast > 1:
        assert call(tw.SUMS_FP8, fast * M * N * 4 - 1) == tw.E_WORKSPACE
    # the Python call takes such a workspace, and names one that is too small
    small = ws[:full * M * N * 4]
    got = tw.fp8_matmul(a, b, out_dtype=torch.float32, workspace=small if full else None)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(tw.TwellError, match="workspace"):
        tw.fp8_matmul(a, b, fast_sums=True, workspace=ws[:fast * M * N * 4 - 16])
