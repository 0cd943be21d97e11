"""How the gradient of few tokens through weights in 4 bits spreads W's rows over
workgroups, on the CPU: the plan that the library takes, gone through step by step
as its kernel does, and seen through the call's workspace."""
import os
import shutil
import subprocess

import pytest

from activation_sparse_ffn_gemm_amd import _lib as tw

CSRC = os.path.join(tw.PKG, "csrc")

# Every row of W in exactly one step of one part: a step takes CN * sets rows from
# its first one on, as far as the matrix goes.
SWEEP = r"""
#include <algorithm>
#include <cstdio>
#include <vector>
#include "fp4_plan.hpp"

int main()
{
    long long plans = 0;
    std::vector<unsigned char> seen;
    auto check = [&](int N, int nkb) {
        const ColsPlan p = cols_plan(N, nkb);
        const int step = FP4_CN * p.sets;
        bool ok = p.parts >= 1 && p.per >= 1 && (p.sets == 1 || p.sets == 2) &&
                  (p.parts == 1 || p.parts * nkb <= 256);
        // by 32 rows, a wave's: every step is of whole waves
        seen.assign((N + 31) / 32, 0);
        for (int part = 0; ok && part < p.parts; ++part) {
            const int lo = part * p.per, hi = std::min(lo + p.per, N);
            ok = lo < N || N == 0;
            for (int n0 = lo; n0 < hi; n0 += step)
                for (int n = n0; n < n0 + step && n < N; n += 32)
                    ok = ok && !seen[n / 32]++;
        }
        for (unsigned char s : seen)
            ok = ok && s == 1;
        if (!ok) {
            std::printf("N %d nkb %d: parts %d per %d sets %d\n", N, nkb, p.parts, p.per, p.sets);
            return false;
        }
        ++plans;
        return true;
    };
    for (int nkb = 1; nkb <= 300; ++nkb)
        for (int N = 0; N <= 16640; N = N < 1100 ? N + 1 : N + (nkb % 2 ? 128 : 251))
            if (!check(N, nkb))
                return 1;
    for (int nkb : {1, 2, 3, 7, 16, 18, 32, 33, 44, 85, 127, 128, 129, 255, 256, 1 << 16})
        for (int N : {20000, 32768, 65535, 65537, 100000, 1 << 20, (1 << 21) - 1, 1 << 21})
            if (!check(N, nkb))
                return 1;
    std::printf("%lld plans\n", plans);
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_every_row_belongs_to_one_part(tmp_path):
    src, exe = tmp_path / "sweep.cpp", tmp_path / "sweep"
    src.write_text(SWEEP)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split()[0]) > 300000


@pytest.mark.parametrize("T", (1, 16, 32))
def test_parts_through_the_workspace(T):
    """The partial sums, float32 rows padded to whole blocks: parts of whole sets of 256
    rows."""
    def parts(N, K):
        kp = -(-K // 128) * 128
        pack = -(-(T * (-(-N // 128) * 128) * 2) // 256) * 256
        need = tw.fp4_matmul_dx_workspace_bytes(tw.TWELL_BF16, T, N, K)
        return max(1, (need - pack) // (T * kp * 4))
    assert parts(256, 4096) == parts(6144, 32768) == 1
    assert parts(1024, 1024) == 4    # 256 rows each
    assert parts(6144, 2304) == 12   # 512
    assert parts(6144, 4096) == 8    # 768
    assert parts(14336, 4096) == 8   # 1792
    assert parts(2816, 5632) == 4    # 768
