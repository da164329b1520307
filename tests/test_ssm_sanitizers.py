"""AddressSanitizer + UndefinedBehaviorSanitizer build of the host code of the
state space scan, its convolution and the draft verification (CPU only):
kda_ssm_abi.hip compiled as plain C++ with stub kernel launchers that check
every plan (tests/sanitize/ssm_abi_main.cpp)."""
import os
import shutil

import pytest

_san = pytest.importorskip("test_sanitizers")   # (absent where only GPU tests are)
ROOT, SAN, _build_and_run = _san.ROOT, _san.SAN, _san._build_and_run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_ssm_abi_host_code_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "ssm_abi_san")
    cmd = ["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"),
           "-I" + os.path.join(ROOT, "gated_delta_rule_amd", "csrc"),
           "-x", "c++", os.path.join(ROOT, "gated_delta_rule_amd", "csrc", "kda_ssm_abi.hip"),
           "-x", "c++", os.path.join(ROOT, "tests", "sanitize", "ssm_abi_main.cpp"), "-o", exe]
    assert "all checks passed" in _build_and_run(cmd, exe)
