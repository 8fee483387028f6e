"""The attention and cache entry points' host code under AddressSanitizer, without a GPU (dry run)."""

import os
import subprocess

import pytest

from conftest import ROOT
from test_asan_host import CLANG, CSRC, HIPCC, INC, _run

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)),
                                reason="needs the ROCm compilers")


def test_attn_host_code_under_address_sanitizer(tmp_path):
    san = ["-fsanitize=address", "-fno-omit-frame-pointer", "-g", "-O1", "-fPIC"]
    api, drv, exe = (str(tmp_path / n) for n in ("api.o", "driver.o", "attn_driver"))
    _run([HIPCC, "--offload-arch=gfx950", "-std=c++17", f"-I{INC}", f"-I{CSRC}",
          *[a for f in san for a in ("-Xarch_host", f)], "-c", os.path.join(CSRC, "api_attn.hip"), "-o", api])
    _run([CLANG, "-std=c++17", *san, f"-I{INC}", "-c", os.path.join(ROOT, "tests", "asan", "attn_driver.cpp"), "-o", drv])
    _run([CLANG, "-fsanitize=address", api, drv, "-o", exe, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout + r.stderr
    assert "AddressSanitizer" not in r.stderr, r.stderr


def test_attn_workspace_sizes_under_sanitizers(tmp_path):
    """The real size arithmetic (only the launchers' host code is compiled: no device code, no HIP runtime)."""
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-g", "-O1", "-fPIC"]
    objs, binaries = [], []
    for name in ("api_attn", "attn_decode", "attn_decode_rows", "attn_prefill", "kv_cache"):
        objs.append(str(tmp_path / f"{name}.o"))
        _run([HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-std=c++17", f"-I{INC}", f"-I{CSRC}",
              *[a for f in san for a in ("-Xarch_host", f)], "-c", os.path.join(CSRC, f"{name}.hip"), "-o", objs[-1]])
        undefined = _run(["nm", "-u", objs[-1]]).stdout.split()
        binaries += [f"-Wl,--defsym={s}=0" for s in undefined if s.startswith("__hip_fatbin")]      # the device code
    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "sizes_driver")
    _run([CLANG, "-std=c++17", *san, f"-I{INC}", "-c", os.path.join(ROOT, "tests", "asan", "attn_sizes_driver.cpp"), "-o", drv])
    _run([CLANG, "-fsanitize=address,undefined", *objs, drv, *binaries, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr
