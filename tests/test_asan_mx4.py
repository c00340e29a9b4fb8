"""The host code of the MX4 entry points under AddressSanitizer and
UndefinedBehaviorSanitizer: a copy of the library with the host pass
instrumented, driven by tests/asan/host_mx4_check.c (device code never runs
here)."""
import os
import shutil

import pytest

from conftest import ROOT
from test_asan_host import CLANG, SAN, _run, _torch_lib


@pytest.mark.skipif(shutil.which("hipcc") is None or not os.path.exists(CLANG),
                    reason="needs hipcc and the ROCm clang")
def test_mx4_host_code_under_asan_and_ubsan(tmp_path):
    pkg = os.path.join(ROOT, "w2a8_gemv_amd")
    srcs = sorted(os.path.join(pkg, "csrc", f) for f in os.listdir(os.path.join(pkg, "csrc"))
                  if f.endswith(".hip"))
    tlib = _torch_lib()
    lib = str(tmp_path / "libw2a8_asan.so")
    _run(["hipcc", "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-shared", *SAN,
          "-ffp-contract=off", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
          "-I", os.path.join(ROOT, "include"), "-I", os.path.join(pkg, "csrc"), *srcs,
          "-L", tlib, "-Wl,-rpath," + tlib, "-lamdhip64", "-o", lib])
    exe = str(tmp_path / "host_mx4_check")
    _run([CLANG, *SAN, "-fsanitize=address,undefined", "-I", os.path.join(ROOT, "include"),
          os.path.join(ROOT, "tests", "asan", "host_mx4_check.c"),
          "-L", str(tmp_path), "-lw2a8_asan", "-Wl,-rpath," + str(tmp_path),
          "-L", tlib, "-Wl,-rpath," + tlib, "-lamdhip64", "-lpthread", "-o", exe])
    env = dict(os.environ)
    env["ASAN_OPTIONS"] = "detect_leaks=1:abort_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    env["HIP_VISIBLE_DEVICES"] = ""
    res = _run([exe], env=env, timeout=300)
    assert "host MX4 checks passed" in res.stdout
