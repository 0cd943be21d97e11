"""The host code of the calls on weights in 4 bits under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: the sources that those calls reach, and the
others that the library needs to link, are compiled with the sanitizers on the host
pass only and linked with ``tests/sanitize/abi_fp4.cpp``, none of whose calls is
launched. A sanitizer report aborts the run, which fails the test."""
import glob
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import CSRC, HIPCC, HOST_SAN, ROOT, SAN, SAN_ENV, _run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_fp4_host_code_under_asan_ubsan(tmp_path):
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    flags = ["--offload-arch=gfx950", "-std=c++17", "-O1", "-g", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *HOST_SAN, *inc]
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))

    def compile_one(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, *flags, "-c", src, "-o", obj])
        return obj

    with ThreadPoolExecutor(min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    drv = str(tmp_path / "abi_fp4.o")
    _run([HIPCC, "-std=c++17", "-O1", "-g", *HOST_SAN, *inc,
          "-c", os.path.join(SAN, "abi_fp4.cpp"), "-o", drv])
    exe = str(tmp_path / "abi_fp4")
    _run([HIPCC, "--offload-arch=gfx950", *HOST_SAN, drv, *objs, "-o", exe])
    r = _run([exe], env={**os.environ, **SAN_ENV}, timeout=300)
    assert "abi_fp4 ok" in r.stdout
