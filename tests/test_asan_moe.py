"""The mixture-of-experts entry points' host code under AddressSanitizer, without a GPU (dry run)."""

import os
import subprocess

import pytest

from conftest import ROOT
from test_asan_host import CLANG, CSRC, HIPCC, INC, _run

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                                reason="needs the ROCm compilers")


def test_moe_host_code_under_address_sanitizer(tmp_path):
    san = ["-fsanitize=address", "-fno-omit-frame-pointer", "-g", "-O1", "-fPIC"]
    api, drv, exe = (str(tmp_path / n) for n in ("api.o", "driver.o", "moe_driver"))
    _run([HIPCC, "--offload-arch=gfx950", "-std=c++17", f"-I{INC}", f"-I{CSRC}",
          *[a for f in san for a in ("-Xarch_host", f)], "-c", os.path.join(CSRC, "api_moe.hip"), "-o", api])
    _run([CLANG, "-std=c++17", *san, f"-I{INC}", "-c", os.path.join(ROOT, "tests", "asan", "moe_driver.cpp"), "-o", drv])
    _run([CLANG, "-fsanitize=address", api, drv, "-o", exe, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout + r.stderr
    assert "AddressSanitizer" not in r.stderr, r.stderr
