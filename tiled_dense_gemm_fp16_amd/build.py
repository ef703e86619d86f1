"""Compile the gfx950 GEMM library (libgemm_f16.so) in-tree with hipcc.

Each source file is compiled to an object of its own (in parallel; the tile
kernel is instantiated per layout in separate files), then the objects are
linked into the shared library.
"""
import concurrent.futures
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgemm_f16.so")
SOURCES = [os.path.join(CSRC, f) for f in (
    "gemm_f16_api.cpp", "gemm_f16_kernels.hip", "gemm_f16_nn.hip", "gemm_f16_nt.hip", "gemm_f16_tn.hip",
    "gemm_f16_tt.hip", "gemm_f16_sparse.hip", "gemm_f16_q4_api.cpp", "gemm_f16_q4_weights.hip", "gemm_f16_q4_tile.hip",
    "gemm_f16_q4_cache.hip", "gemm_f16_q4_attention.hip", "gemm_f16_i8_api.cpp", "gemm_f16_i8_rows.hip", "gemm_f16_i8_stream.hip",
    "gemm_f16_i8_tile.hip", "gemm_f16_route.hip")]
# what each kind of source includes (for incremental builds)
HOST_DEPS = [os.path.join(CSRC, f) for f in ("gemm_f16_internal.h", "gemm_f16_tuned.inc", "gemm_f16_q4_format.h",
                                             "gemm_f16_i8_internal.h")] + \
    [os.path.join(INCLUDE, f) for f in ("gemm_f16.h", "gemm_f16_q4.h", "gemm_f16_i8.h")]
KERNEL_DEPS = [os.path.join(CSRC, f) for f in ("gemm_f16_internal.h", "gemm_f16_tile.h", "gemm_f16_q4_format.h",
                                               "gemm_f16_i8_internal.h", "gemm_f16_i8_device.h")]
# the Python modules that marshal the 4-bit and the 8-bit entry points' tensors
BINDING = os.path.join(PKG, "_q4_binding.so")
I8_BINDING = os.path.join(PKG, "_i8_binding.so")
BINDINGS = {BINDING: os.path.join(CSRC, "q4_binding.cpp"), I8_BINDING: os.path.join(CSRC, "i8_binding.cpp")}
BINDING_DEPS = [os.path.join(CSRC, "binding.h")] + [os.path.join(INCLUDE, f) for f in ("gemm_f16.h", "gemm_f16_q4.h", "gemm_f16_i8.h")]
PROBE_LIB = os.path.join(PKG, "libgemm_f16_probe.so")
PROBE_SOURCES = [os.path.join(CSRC, "mfma_probe.hip")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "-O3", "-std=c++17", "-fPIC",
    "--offload-arch=gfx950",
    # keep hipcc from forming packed fp32 instructions on its own
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def build(verbose: bool = False, extra_flags=None, jobs: int | None = None, incremental: bool = False) -> str:
    """Compile libgemm_f16.so, the Python modules of its 4-bit and 8-bit entry points and
    the measurement probe libgemm_f16_probe.so next to this file; return the GEMM library's path.  ``incremental`` reuses an
    object newer than its source and every shared header (same flags
    assumed); by default everything is compiled."""
    os.makedirs(OBJDIR, exist_ok=True)
    jobs = jobs or min(len(SOURCES) + len(PROBE_SOURCES) + len(BINDINGS), max(1, (os.cpu_count() or 4) - 1), 8)
    units = [(src, LIB) for src in SOURCES] + [(src, PROBE_LIB) for src in PROBE_SOURCES]
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as pool:
        bindings = {to: pool.submit(_compile_binding, src, verbose, incremental) for to, src in BINDINGS.items()}
        objs = list(pool.map(lambda u: _compile(u[0], verbose, extra_flags, incremental), units))
    _link([o for o, (_, lib) in zip(objs, units) if lib == LIB], LIB, verbose)
    _link([o for o, (_, lib) in zip(objs, units) if lib == PROBE_LIB], PROBE_LIB, verbose)
    for to, obj in bindings.items():
        _link_binding(obj.result(), to, verbose)
    return LIB


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr.strip():
        # the host pass does not know the packed-fp32 feature flag; that warning is harmless
        lines = [ln for ln in res.stderr.splitlines() if "packed-fp32-ops" not in ln]
        if lines:
            print("\n".join(lines), flush=True)


def _compile(src, verbose, extra_flags, incremental=False):
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    if incremental and os.path.exists(obj):
        deps = HOST_DEPS if src.endswith(".cpp") else KERNEL_DEPS
        newest = max(os.path.getmtime(p) for p in [src, *deps])
        if os.path.getmtime(obj) > newest:
            return obj
    _run([HIPCC, *FLAGS, *(extra_flags or []), "-I", INCLUDE, "-I", CSRC, "-x", "hip", "-c", src, "-o", obj],
         verbose)
    return obj


def _link(objs, lib, verbose):
    tmp = lib + ".tmp"
    _run([HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", *objs, "-o", tmp], verbose)
    os.replace(tmp, lib)


def _compile_binding(source, verbose, incremental):
    """A Python module, host code against torch's and Python's headers."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    obj = os.path.join(OBJDIR, os.path.basename(source) + ".o")
    if incremental and os.path.exists(obj):
        newest = max(os.path.getmtime(p) for p in (source, *BINDING_DEPS))
        if os.path.getmtime(obj) > newest:
            return obj
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(HIPCC)))
    # (torch's and the system's headers are not ours to warn about)
    system = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(rocm, "include")]
    _run([HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-D__HIP_PLATFORM_AMD__",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
          *[flag for path in system for flag in ("-isystem", path)], "-c", source, "-o", obj], verbose)
    return obj


def _link_binding(obj, binding, verbose):
    import torch

    tmp = binding + ".tmp"
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    _run([HIPCC, "-shared", "-fPIC", obj, "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L", libs,
          "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-o", tmp], verbose)
    os.replace(tmp, binding)


if __name__ == "__main__":
    print(build(verbose=True))
