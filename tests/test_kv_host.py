"""How the key/value-cache entry points cut large calls into launches: csrc/mx_kv_api.cpp built by the host
compiler, undefined behaviour trapped, over stand-ins for the device launchers (tests/host_sanitizer/kv_driver.cpp).
CPU only."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "microscaling_fp4_weight_amd", "csrc")
HIP_INCLUDE = "/opt/rocm/include"


def test_launches_of_large_calls(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(os.path.join(HIP_INCLUDE, "hip", "hip_runtime.h")):
        pytest.skip("needs g++ and the HIP headers")
    exe = str(tmp_path / "kv_driver")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-g", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
                        "-I", HIP_INCLUDE, "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "mx_kv_api.cpp"),
                        os.path.join(ROOT, "tests", "host_sanitizer", "kv_driver.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "all " in r.stdout, (r.stdout + r.stderr)[-4000:]
