"""No kernel of the 4-bit operators keeps registers in scratch memory: the
metadata that the compiler writes for each kernel, read from a listing made of
the sources here."""
import os
import re
import subprocess

import pytest

from tiled_dense_gemm_fp16_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")

SOURCES = [s for s in build.SOURCES if "gemm_f16_q4" in s and s.endswith(".hip")]


@pytest.mark.parametrize("source", SOURCES, ids=[os.path.basename(s) for s in SOURCES])
def test_no_kernel_spills(source, tmp_path):
    listing = tmp_path / "kernels.s"
    res = subprocess.run([build.HIPCC, *build.FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "-x", "hip", "--cuda-device-only", "-S",
                          source, "-o", str(listing)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    found = re.findall(r"\.name:\s+(\S+)\n(?:(?!\.name:).)*?\.private_segment_fixed_size:\s+(\d+)", listing.read_text(), re.S)
    kernels = {name: int(size) for name, size in found if name.startswith("_Z")}
    assert len(kernels) >= 6
    assert not {name: size for name, size in kernels.items() if size}
