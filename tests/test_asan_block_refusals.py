"""Argument checks of the device entry points of w2a8_block.h under
AddressSanitizer and UndefinedBehaviorSanitizer, one mistake at a time: their host
sources with the host pass instrumented, driven by tests/asan/host_block_refusals.c
(device code never runs here)."""
import os
import shutil

import pytest

from conftest import ROOT
from test_asan_host import CLANG, SAN, _run, _torch_lib


@pytest.mark.skipif(shutil.which("hipcc") is None or not os.path.exists(CLANG),
                    reason="needs hipcc and the ROCm clang")
def test_block_refusals_under_asan_and_ubsan(tmp_path):
    pkg = os.path.join(ROOT, "w2a8_gemv_amd")
    srcs = [os.path.join(pkg, "csrc", f) for f in ("host_block.hip", "host.hip", "rmsnorm.hip", "w4a8.hip", "moe.hip",
                                                   "gemm.hip", "gemm_ring.hip", "gemv.hip", "gemv_ring.hip",
                                                   "linear_ring.hip", "quant.hip")]
    tlib = _torch_lib()
    lib = str(tmp_path / "libw2a8_asan.so")
    _run(["hipcc", "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-shared", *SAN,
          "-ffp-contract=off", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
          "-I", os.path.join(ROOT, "include"), "-I", os.path.join(pkg, "csrc"), *srcs,
          "-L", tlib, "-Wl,-rpath," + tlib, "-lamdhip64", "-o", lib])
    exe = str(tmp_path / "host_block_refusals")
    _run([CLANG, *SAN, "-fsanitize=address,undefined", "-I", os.path.join(ROOT, "include"),
          os.path.join(ROOT, "tests", "asan", "host_block_refusals.c"),
          "-L", str(tmp_path), "-lw2a8_asan", "-Wl,-rpath," + str(tmp_path),
          "-L", tlib, "-Wl,-rpath," + tlib, "-lamdhip64", "-lpthread", "-o", exe])
    env = dict(os.environ)
    env["ASAN_OPTIONS"] = "detect_leaks=1:abort_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    env["HIP_VISIBLE_DEVICES"] = ""
    res = _run([exe], env=env, timeout=300)
    assert "host block refusals passed" in res.stdout
