"""The 8-bit path's host layer (validation, planning, workspace sizes) under
AddressSanitizer and UndefinedBehaviorSanitizer, host code only, as
test_host_sanitize.py does for the rest of the C ABI.  CPU only."""

import os
import subprocess

import pytest

from test_host_sanitize import BUILD, CLANG, HERE, HIPCC, PKG, ROOT, SAN, _have_toolchain


@pytest.mark.skipif(not _have_toolchain(), reason="needs hipcc, ROCm clang and the library's objects (build())")
def test_fp8_host_layer_under_sanitizers(tmp_path):
    objs = [os.path.join(BUILD, f) for f in sorted(os.listdir(BUILD)) if f.endswith(".o") and f != "hxq_fp8_api.o"]
    assert objs, "no library objects: run build() first"
    api, exe = str(tmp_path / "hxq_fp8_api_san.o"), str(tmp_path / "fp8_host_sanitize")
    host_san = [a for f in SAN for a in ("-Xarch_host", f)]
    for cmd in ([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature",
                 "-Xclang", "-packed-fp32-ops", *host_san, "-c", os.path.join(PKG, "csrc", "hxq_fp8_api.cpp"), "-o", api],
                [CLANG, "-O1", "-g", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"),
                 os.path.join(HERE, "fp8_host_sanitize_driver.cpp"), api, *objs, "-L/opt/rocm/lib", "-lamdhip64",
                 "-Wl,-rpath,/opt/rocm/lib", "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "checks ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
