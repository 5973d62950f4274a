"""Leave for large dynamic LDS is asked for on every device of a process (host
code with stand-ins for HIP: no GPU needed)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_leave_is_per_device(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    exe = str(tmp_path / "smem_check")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(ROOT, "weight_only_bit_dequant_amd", "csrc"), "-I", "/opt/rocm/include",
                        os.path.join(ROOT, "tests", "host_abi", "smem_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
