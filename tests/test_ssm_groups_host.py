"""Workspaces of the scan's backward pass that hold some of its groups of
heads, on the host under AddressSanitizer and UndefinedBehaviorSanitizer (CPU
only): every array of every launch lies within the workspace
(tests/sanitize/ssm_groups_main.cpp)."""
import os
import shutil

import pytest

_san = pytest.importorskip("test_sanitizers")   # (absent where only GPU tests are)
ROOT, SAN, _build_and_run = _san.ROOT, _san.SAN, _san._build_and_run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_backward_workspace_of_some_groups(tmp_path):
    exe = str(tmp_path / "ssm_groups_san")
    cmd = ["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"),
           "-I" + os.path.join(ROOT, "gated_delta_rule_amd", "csrc"),
           "-x", "c++", os.path.join(ROOT, "gated_delta_rule_amd", "csrc", "kda_ssm_abi.hip"),
           "-x", "c++", os.path.join(ROOT, "tests", "sanitize", "ssm_groups_main.cpp"), "-o", exe]
    assert "all checks passed" in _build_and_run(cmd, exe)
