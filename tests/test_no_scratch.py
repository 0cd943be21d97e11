"""No kernel of the norm spills registers to memory: its rows are read once and
the bandwidth is theirs. The source is compiled to assembly here and the
kernels' own descriptions are read."""
import os
import re
import subprocess

import pytest

from activation_sparse_ffn_gemm_amd import build

CSRC = os.path.join(build.PKG, "csrc")


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not installed")
def test_norm_kernels_use_no_scratch(tmp_path):
    asm = str(tmp_path / "rmsnorm.s")
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-I", os.path.join(build.ROOT, "include"),
                        "-I", CSRC, "--offload-device-only", "-S",
                        os.path.join(CSRC, "rmsnorm.hip"), "-o", asm],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    with open(asm) as f:
        kernels = re.findall(r"\.amdhsa_kernel (\S+)(.*?)\.end_amdhsa_kernel", f.read(), re.S)
    assert len(kernels) > 40
    spills = {name: int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", body)[1])
              for name, body in kernels}
    assert not any(spills.values()), {n: b for n, b in spills.items() if b}
