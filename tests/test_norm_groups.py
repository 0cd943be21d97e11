"""How the norm's backward spreads its rows over workgroups, seen through its
workspace: one row of partial sums for each (CPU only)."""
import pytest

from activation_sparse_ffn_gemm_amd import _lib as tw


def _lanes(d):
    n = 16
    while n < 1024 and 8 * n < d:
        n *= 2
    return n


def _rows(d):
    """(threads of a workgroup, rows that it takes in a turn)."""
    lanes = _lanes(d)
    threads = 1024 if lanes <= 64 or lanes == 1024 else 512
    return threads, threads // lanes


def _groups(T, d):
    need = tw.load().twell_rmsnorm_bwd_workspace_bytes(T, d)
    assert need % (4 * d) == 0
    return need // (4 * d)


@pytest.mark.parametrize("d", [1, 64, 256, 500, 512, 513, 1024, 1100, 2048, 2304, 4096, 5000,
                               8192, 16384])
def test_groups(d):
    threads, rows = _rows(d)
    for turns in [*range(1, 1300), 1535, 1536, 1537, 2048, 3000, 8192, 12345]:
        for T in {turns * rows, (turns - 1) * rows + 1}:
            n = _groups(T, d)
            if turns <= 2:
                assert n == 1, (T, n)  # no second launch
                continue
            most = -(-turns // n)  # the turns of the workgroup that has most
            assert 1 < n <= 512 and most * n >= turns  # every row has its turn
            cap = 512 if threads == 512 and 8 * turns > 3 * d else 256
            if cap == 512 and turns > 1024:
                assert n == 512, (T, n)
            else:  # even: as few turns as the cap allows, and no workgroup too many
                assert n <= cap and most == -(-turns // cap), (T, n)
                assert n == -(-turns // most), (T, n)
    assert _groups(0, d) == 0
