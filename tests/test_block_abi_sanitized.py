"""The block-scaled operators' host code under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU): the ABI host sources are built with g++
and stub launchers, and the operators' CPU ABI tests run against that library
in a child process with the ASan runtime preloaded."""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HOST = os.path.join(ROOT, "tests", "host_abi")
CSRC = os.path.join(ROOT, "weight_only_bit_dequant_amd", "csrc")


def test_block_host_code_is_sanitizer_clean(tmp_path):
    asan = "" if shutil.which("g++") is None else subprocess.run(
        ["g++", "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("g++ with AddressSanitizer is not available")
    lib = str(tmp_path / "libwq_block_hostcheck.so")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", "/opt/rocm/include", "-x", "c++",
           *[os.path.join(CSRC, f) for f in ("wq_api.hip", "wq_plan.cpp", "wq_block_api.hip")],
           *[os.path.join(HOST, f) for f in ("stub_launchers.cpp", "stub_block_launchers.cpp")], "-o", lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-6000:]
    env = dict(os.environ, WQ_LIB=lib, LD_PRELOAD=asan,
               # the interpreter itself is not instrumented: leak checking would report its own allocations
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    # (the Python checks are torch's and not this library's; their C++ exceptions do not pass a preloaded ASan, which
    # looks for __cxa_throw before libstdc++ is loaded)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-k", "not python_checks",
                        os.path.join(ROOT, "tests", "test_block_abi_cpu.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-6000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-6000:]
    assert " passed" in out
