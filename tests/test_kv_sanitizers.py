"""The key-value cache's host code (argument validation and planning) under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: built with g++
(host code only), the kernel launchers replaced by stand-ins."""
import os
import shutil

import pytest

H = pytest.importorskip("test_host_sanitizers", reason="needs the host sanitizer build's files")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_kv_validation_under_sanitizers():
    exe = os.path.join(H.OUT, "kv_validation")
    csrc = os.path.join(H.ROOT, "block_quantized_amd", "csrc")
    cmd = ["g++", "-std=c++17", *H.FLAGS, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", os.path.join(csrc, "kv.cpp"),
           os.path.join(csrc, "qmm.cpp"), os.path.join(H.SAN, "abi_stubs.cpp"), os.path.join(H.SAN, "kv_stubs.cpp"),
           os.path.join(H.SAN, "kv_driver.cpp")]
    assert "kv validation ok" in H._build_and_run(cmd, exe)
