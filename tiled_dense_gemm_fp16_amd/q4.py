"""Products with 4-bit operands (include/gemm_f16_q4.h): weights held as 4-bit
codes with a scale and a zero point per group, made by :func:`q4_compress`,
read back by :func:`q4_expand` and multiplied by :func:`gemm_q4`; and a paged
key/value cache in the same codes, filled by :func:`q4_cache_append`, read
back by :func:`q4_cache_read` and attended to by :func:`attention_q4`.

Argument marshalling only, as in the package's other entry points: tensors
give memory, torch's current stream is the default stream, and nothing falls
back to the CPU.  A decode step makes many of these calls on small tensors, so
their checks are compiled (csrc/q4_binding.cpp); results made here belong to
the call's stream.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

from . import _EPILOGUES, BINDING_PATH, CONFIG_AUTO, SPLITS_AUTO, SUCCESS, GemmError, Plan, lib

_vp = ctypes.c_void_p

GROUPS = (32, 64, 128)
_module = None


def _binding():
    """The compiled marshalling module, built with the library."""
    global _module
    if _module is None:
        lib()
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"{BINDING_PATH} is missing: build the HIP library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        from . import _q4_binding
        _q4_binding.setup(Q4Matrix, Q4Cache, GemmError, torch._C._cuda_getCurrentRawStream)
        _module = _q4_binding
    return _module


def _call(name, stream, *args):
    """Call the compiled entry point on `stream`, or on torch's current one."""
    fn = getattr(_module or _binding(), name)
    if stream is None:
        return fn(*args, None)
    with torch.cuda.stream(stream):
        return fn(*args, stream.device.index)


def _check_group(group):
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group!r}")


# ---- weights --------------------------------------------------------------------

class Q4Matrix(NamedTuple):
    """An n x k matrix held in 4 bits: int32 tensors of the dwords and group
    words that include/gemm_f16_q4.h describes."""
    codes: object    # int32 [ceil(n / 16), ceil(k / 128), 4, 16, 4]
    words: object    # int32 [ceil(n / 16), ceil(k / 128), 16, 128 / group]
    n: int
    k: int
    group: int


def q4_compress(w, group: int = 128, symmetric: bool = False, stream=None) -> Q4Matrix:
    """w (n x k float16 GPU tensor) rounded to 4-bit codes with a scale and a
    zero point for every ``group`` neighbours of a row (``symmetric``: zero
    point 8, largest magnitude at code 7 from it)."""
    return _call("compress", stream, w, group, symmetric)


def q4_expand(w: Q4Matrix, out=None, stream=None):
    """The n x k float16 matrix that ``w`` stands for, each value rounded once."""
    return _call("expand", stream, w, out)


def gemm_q4(a, w: Q4Matrix, epilogue: str = "none", out=None, config: int = CONFIG_AUTO, stream=None,
            splits: int | None = None, workspace=None, alpha: float = 1.0):
    """C = epi(alpha * (a @ w^T)) for a (m x k float16) and a 4-bit n x k
    matrix: the product of a layer whose weights are held in 4 bits.  Sums are
    fp32 and rounded once; one row reads each code once.

    ``splits`` and ``workspace`` as in gemm(): None lets the planner split K
    when that pays, copy rows of odd length to aligned ones and, from 2048 rows
    with groups of 32 or 64, expand w for the dense product (2 n k bytes) unless its
    outputs are few, with a workspace from torch's caching allocator.  The expanded weights are rounded
    to float16 (infinite from 65520 on); in all other products they are exact.  1
    does none of it: every weight is used exactly, whatever the number of rows;
    None falls back to it where the allocator has no room for the workspace."""
    epi = _EPILOGUES.get(epilogue)
    if epi is None:
        raise ValueError(f"epilogue must be one of {sorted(_EPILOGUES)}, got {epilogue!r}")
    return _call("gemm", stream, a, w, epi, out, config, splits, workspace, alpha)


def plan_q4(m: int, n: int, k: int, group: int = 128, config: int = CONFIG_AUTO, splits: int | None = 1,
            A_ptr: int = 0) -> dict:
    """How gemm_f16_q4 would run this shape (host logic only); the pointer
    only matters for its alignment."""
    p = Plan()
    st = lib().gemm_f16_plan_q4(m, n, k, group, A_ptr or None, config, SPLITS_AUTO if splits is None else int(splits),
                                ctypes.byref(p))
    if st != SUCCESS:
        raise GemmError(st, "gemm_f16_plan_q4")
    return p.as_dict()


def q4_num_configs() -> int:
    return int(lib().gemm_f16_q4_num_configs())


def q4_config_name(config: int) -> str | None:
    s = lib().gemm_f16_q4_config_name(int(config))
    return s.decode() if s is not None else None


# ---- the paged key/value cache ------------------------------------------------

class Q4Cache(NamedTuple):
    """Keys and values in 4 bits: int32 tensors of the dwords and group words
    that include/gemm_f16_q4.h describes (q4_cache() makes them)."""
    k_codes: object    # int32 [pages, heads, page_size, head_dim / 8]
    k_words: object    # int32 [pages, heads, head_dim / group, page_size]
    v_codes: object    # int32 [pages, heads, page_size / 8, 16, head_dim / 16]
    v_words: object    # int32 [pages, heads, head_dim / group, page_size]
    group: int


class _CacheStruct(ctypes.Structure):
    """gemm_f16_q4_cache_t, for calls of the C entry points through lib()."""
    _fields_ = [("k_codes", _vp), ("k_words", _vp), ("v_codes", _vp), ("v_words", _vp), ("pages", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group", ctypes.c_int32)]


def q4_cache(pages: int, heads: int, page_size: int, head_dim: int, group: int = 64, device="cuda") -> Q4Cache:
    """An empty cache (zeros) of ``pages`` pages of ``page_size`` tokens."""
    _check_group(group)
    if head_dim not in (64, 128, 256) or group > head_dim:
        raise ValueError(f"head_dim must be 64, 128 or 256 and at least group, got {head_dim} and group {group}")
    if pages < 0 or heads < 1 or page_size < 8 or page_size % 8:
        raise ValueError("pages must be at least 0, heads at least 1 and page_size a positive multiple of 8")

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=device)

    words = (pages, heads, head_dim // group, page_size)
    return Q4Cache(zeros(pages, heads, page_size, head_dim // 8), zeros(*words),
                   zeros(pages, heads, page_size // 8, 16, head_dim // 16), zeros(*words), group)


def q4_cache_append(cache: Q4Cache, k, v, table, lengths, starts=None, q=None, cos=None, sin=None,
                    interleaved: bool = False, out=None, stream=None):
    """Append new tokens' keys and values (tokens x heads x head_dim float16,
    possibly slices of wider rows) to the cache, rotating keys on the way.

    ``table`` (int32, batch x max_pages) holds each sequence's pages,
    ``lengths`` (int32, batch) the tokens it has; ``starts`` (int32,
    batch + 1) the rows of k and v of each sequence, or None for one new
    token each.  ``cos`` and ``sin`` (float32, positions x rotary / 2) rotate
    keys and the queries ``q`` (tokens x q_heads x head_dim) by their
    positions; the rotated queries are returned (``out`` when given, which
    may be a contiguous ``q`` itself), None without ``q``.  ``lengths`` is
    left as it is.  See include/gemm_f16_q4.h for tokens out of range."""
    return _call("append", stream, cache, k, v, table, lengths, starts, q, cos, sin, interleaved, out)


def q4_cache_read(cache: Q4Cache, table, starts, total: int, first=None, stream=None):
    """(k, v), each total x heads x head_dim float16: rows starts[i] up to
    starts[i + 1] are sequence i's tokens from ``first[i]`` (int32; None: from
    the first one), each value rounded once.  Rows past starts[-1] are not
    written."""
    return _call("read", stream, cache, table, starts, total, first)


def plan_attention_q4(batch: int, q_heads: int, heads: int, head_dim: int, group: int, max_length: int,
                      splits: int | None = None) -> dict:
    """How gemm_f16_q4_attention would run (host logic only)."""
    p = Plan()
    st = lib().gemm_f16_plan_q4_attention(batch, q_heads, heads, head_dim, group, max_length,
                                          SPLITS_AUTO if splits is None else int(splits), ctypes.byref(p))
    if st != SUCCESS:
        raise GemmError(st, "gemm_f16_plan_q4_attention")
    return p.as_dict()


def attention_q4(q, cache: Q4Cache, table, lengths, scale: float | None = None, out=None, splits: int | None = None,
                 workspace=None, max_length: int | None = None, stream=None):
    """Attention of one query token of each sequence (q: batch x q_heads x
    head_dim float16, rows possibly strided) over its first ``lengths[i]``
    cached tokens; q_heads is a multiple of the cache's heads.  A length of 0
    gives zeros.  ``scale`` defaults to head_dim ** -0.5.

    ``splits``: None lets the planner divide long sequences over workgroups
    (``max_length``, what no length exceeds, helps it; default: what the table
    can hold).  A split needs a workspace of fp32 partial results:
    ``workspace`` (a contiguous GPU tensor used as scratch) or, when it is
    None, one taken from torch's caching allocator on ``stream``."""
    return _call("attention", stream, q, cache, table, lengths, scale, out, splits, workspace, max_length)
