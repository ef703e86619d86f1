"""The 8-bit and expert entry points' validation and planning under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU:
tests/host/i8_fuzz.cpp drives them with a few hundred thousand argument sets
against stubs of the launchers."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.mark.skipif(not os.path.exists(CLANG), reason="no clang++ with sanitizers")
def test_i8_validation_under_sanitizers(tmp_path):
    exe = tmp_path / "i8_fuzz"
    cmd = [CLANG, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "tiled_dense_gemm_fp16_amd", "csrc"),
           "-x", "c++", os.path.join(ROOT, "tiled_dense_gemm_fp16_amd", "csrc", "gemm_f16_i8_api.cpp"),
           os.path.join(ROOT, "tests", "host", "i8_fuzz.cpp"), "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.stdout[-2000:], run.stderr[-4000:])
    assert " 0 failed checks" in run.stdout
