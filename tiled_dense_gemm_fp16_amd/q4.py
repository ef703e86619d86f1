"""Products with 4-bit operands (include/gemm_f16_q4.h): weights held as 4-bit
codes with a scale and a zero point per group, made by :func:`q4_compress`,
read back by :func:`q4_expand` and multiplied by :func:`gemm_q4`.

Argument marshalling only, as in the package's other entry points: tensors
give memory, torch's current stream is the default stream, and nothing falls
back to the CPU.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import _EPILOGUES, CONFIG_AUTO, SUCCESS, GemmError, Plan, _check_gpu_2d, lib

_i64, _vp, _int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int

GROUPS = (32, 64, 128)


class Q4Matrix(NamedTuple):
    """An n x k matrix held in 4 bits: int32 tensors of the dwords and group
    words that include/gemm_f16_q4.h describes."""
    codes: object    # int32 [ceil(n / 16), ceil(k / 128), 4, 16, 4]
    words: object    # int32 [ceil(n / 16), ceil(k / 128), 16, 128 / group]
    n: int
    k: int
    group: int


def _buffer_shapes(n, k, group):
    nb, kb = -(-n // 16), -(-k // 128)
    return (nb, kb, 4, 16, 4), (nb, kb, 16, 128 // group)


def _check_group(group):
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group!r}")


def _check_buffer(t, name, dtype, shape, device=None):
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _check_matrix(w, device=None):
    import torch

    if not isinstance(w, Q4Matrix):
        raise ValueError("w must be a Q4Matrix (as q4_compress returns)")
    _check_group(w.group)
    codes, words = _buffer_shapes(w.n, w.k, w.group)
    _check_buffer(w.codes, "w.codes", torch.int32, codes, device)
    _check_buffer(w.words, "w.words", torch.int32, words, w.codes.device)


def _stream(stream, device):
    import torch

    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream or None


def _call(device, what, fn, *args):
    import torch

    with torch.cuda.device(device):
        st = fn(*args)
    if st != SUCCESS:
        raise GemmError(st, what)


def q4_compress(w, group: int = 128, symmetric: bool = False, stream=None) -> Q4Matrix:
    """w (n x k float16 GPU tensor) rounded to 4-bit codes with a scale and a
    zero point for every ``group`` neighbours of a row (``symmetric``: zero
    point 8, largest magnitude at code 7 from it)."""
    import torch

    _check_gpu_2d(w, "w", torch.float16)
    _check_group(group)
    n, k = w.shape
    codes, words = _buffer_shapes(n, k, group)
    codes = torch.empty(codes, dtype=torch.int32, device=w.device)
    words = torch.empty(words, dtype=torch.int32, device=w.device)
    _call(w.device, "gemm_f16_q4_compress", lib().gemm_f16_q4_compress, n, k, group, int(bool(symmetric)),
          w.data_ptr() or None, codes.data_ptr() or None, words.data_ptr() or None, _stream(stream, w.device))
    return Q4Matrix(codes, words, n, k, group)


def q4_expand(w: Q4Matrix, out=None, stream=None):
    """The n x k float16 matrix that ``w`` stands for, each value rounded once."""
    import torch

    _check_matrix(w)
    device = w.codes.device
    if out is None:
        out = torch.empty((w.n, w.k), dtype=torch.float16, device=device)
    else:
        _check_buffer(out, "out", torch.float16, (w.n, w.k), device)
    _call(device, "gemm_f16_q4_expand", lib().gemm_f16_q4_expand, w.n, w.k, w.group, w.codes.data_ptr() or None,
          w.words.data_ptr() or None, out.data_ptr() or None, _stream(stream, device))
    return out


def gemm_q4(a, w: Q4Matrix, epilogue: str = "none", out=None, config: int = CONFIG_AUTO, stream=None,
            alpha: float = 1.0):
    """C = epi(alpha * (a @ w^T)) for a (m x k float16) and a 4-bit n x k
    matrix: the product of a layer whose weights are held in 4 bits.  Sums are
    fp32 and rounded once; one row reads each code once."""
    import torch

    if epilogue not in _EPILOGUES:
        raise ValueError(f"epilogue must be one of {sorted(_EPILOGUES)}, got {epilogue!r}")
    _check_gpu_2d(a, "a", torch.float16)
    _check_matrix(w, a.device)
    m, k = a.shape
    if k != w.k:
        raise ValueError(f"inner dimensions differ: a is {tuple(a.shape)}, w is {w.n} x {w.k}")
    if out is None:
        out = torch.empty((m, w.n), dtype=torch.float16, device=a.device)
    else:
        _check_buffer(out, "out", torch.float16, (m, w.n), a.device)
    _call(a.device, "gemm_f16_q4", lib().gemm_f16_q4, m, w.n, k, w.group, a.data_ptr() or None,
          w.codes.data_ptr() or None, w.words.data_ptr() or None, out.data_ptr() or None, float(alpha),
          _EPILOGUES[epilogue], config, _stream(stream, a.device))
    return out


def plan_q4(m: int, n: int, k: int, group: int = 128, config: int = CONFIG_AUTO) -> dict:
    """How gemm_f16_q4 would run this shape (host logic only)."""
    p = Plan()
    st = lib().gemm_f16_plan_q4(m, n, k, group, config, ctypes.byref(p))
    if st != SUCCESS:
        raise GemmError(st, "gemm_f16_plan_q4")
    return p.as_dict()


def q4_num_configs() -> int:
    return int(lib().gemm_f16_q4_num_configs())


def q4_config_name(config: int) -> str | None:
    s = lib().gemm_f16_q4_config_name(int(config))
    return s.decode() if s is not None else None
