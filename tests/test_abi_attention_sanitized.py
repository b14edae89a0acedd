"""The attention block's ABI layer (abi_attention.cpp) built for the host with
AddressSanitizer and UndefinedBehaviorSanitizer (g++, host code only) and driven by
tests/csrc/abi_attention_sanitize.cpp with stubbed launchers.  No GPU."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
HIP_INCLUDE = "/opt/rocm/include"


def test_attention_abi_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")):
        pytest.skip("g++ or the HIP headers not found")
    csrc = os.path.join(ROOT, "blockwise_fp8_gemm_act_amd", "csrc")
    exe = str(tmp_path / "abi_attention_sanitize")
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
                    "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE, "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "abi_attention.cpp"), os.path.join(HERE, "csrc", "abi_attention_sanitize.cpp"), "-o", exe],
                   check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "abi under sanitizers: ok" in res.stdout
