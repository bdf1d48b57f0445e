"""The host code behind drafted tokens and logits under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: built with g++ (host code only), the
kernel launchers replaced by stand-ins."""
import os
import shutil

import pytest

H = pytest.importorskip("test_host_sanitizers", reason="needs the host sanitizer build's files")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_draft_validation_under_sanitizers():
    exe = os.path.join(H.OUT, "draft_validation")
    csrc = os.path.join(H.ROOT, "block_quantized_amd", "csrc")
    cmd = ["g++", "-std=c++17", *H.FLAGS, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           *[os.path.join(csrc, f) for f in ("kv.cpp", "kv_draft.cpp", "logits.cpp", "qmm.cpp")],
           *[os.path.join(H.SAN, f) for f in ("abi_stubs.cpp", "kv_stubs.cpp", "draft_stubs.cpp", "draft_driver.cpp")]]
    assert "draft validation ok" in H._build_and_run(cmd, exe)
