"""The 4-bit entry points' validation at the ends of every argument's range,
on the CPU: under AddressSanitizer and UndefinedBehaviorSanitizer
(tests/host/q4_extremes.cpp), and by the statuses of the built library."""
import os
import subprocess

import pytest
import torch

import tiled_dense_gemm_fp16_amd as g
from test_host_q4 import INVALID, NO_DEVICE, SIZE, append, attention, cache_struct, read

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.mark.skipif(not os.path.exists(CLANG), reason="no clang++ with sanitizers")
def test_no_argument_overflows_validation(tmp_path):
    exe = tmp_path / "q4_extremes"
    cmd = [CLANG, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "tiled_dense_gemm_fp16_amd", "csrc"),
           "-x", "c++", os.path.join(ROOT, "tiled_dense_gemm_fp16_amd", "csrc", "gemm_f16_q4_api.cpp"),
           os.path.join(ROOT, "tests", "host", "q4_extremes.cpp"), "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.stdout[-2000:], run.stderr[-4000:])
    assert " 0 failed checks" in run.stdout


def test_caches_no_memory_holds_are_refused():
    # each dimension within its own limit, the bytes beyond 2^63, 2^64 (wrapping to 0) and an address space
    for over in (dict(pages=1 << 30, heads=4096, page_size=1 << 16, head_dim=256), dict(pages=1 << 30, heads=2048, page_size=1 << 16),
                 dict(pages=1 << 30, heads=4096, page_size=1 << 16, head_dim=256, group=32), dict(pages=1 << 30, heads=4096, page_size=1 << 15)):
        for call in (append, read, attention):
            assert call(cache_struct(**over), max_pages=2) == SIZE, (over, call.__name__)


def test_strides_and_tables_no_memory_holds_are_refused():
    far = 1 << 62
    for bad in (dict(ks=far), dict(vs=far), dict(qs=far), dict(ks=far, vs=far, qs=far), dict(positions=far), dict(positions=(1 << 63) - 1)):
        assert append(**bad) == SIZE, bad
    assert attention(qs=far) == SIZE
    assert append(ks=-far) == INVALID and attention(qs=-far) == INVALID
    if not torch.cuda.is_available():                      # rows far apart are none of this
        assert append(ks=1 << 34) == NO_DEVICE and attention(qs=1 << 34) == NO_DEVICE

