"""Products with 4-bit operands (include/gemm_f16_q4.h): weights held as 4-bit
codes with a scale and a zero point per group, made by :func:`q4_compress`,
read back by :func:`q4_expand` and multiplied by :func:`gemm_q4`; and a paged
key/value cache in the same codes, filled by :func:`q4_cache_append`, read
back by :func:`q4_cache_read` and attended to by :func:`attention_q4`.

Argument marshalling only, as in the package's other entry points: tensors
give memory, torch's current stream is the default stream, and nothing falls
back to the CPU.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import _EPILOGUES, CONFIG_AUTO, SPLITS_AUTO, SUCCESS, GemmError, Plan, _check_gpu_2d, lib

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


_plans: dict = {}


def _planned(key):
    """(splits, workspace bytes) of a product, by shape, alignment and request."""
    hit = _plans.get(key)
    if hit is None:
        m, n, k, group, odd, config, splits = key
        p = plan_q4(m, n, k, group, config, splits, 2 if odd else 0)
        hit = (p["splits"], p["workspace_bytes"])
        if len(_plans) > 4096:
            _plans.clear()
        _plans[key] = hit
    return hit


def gemm_q4(a, w: Q4Matrix, epilogue: str = "none", out=None, config: int = CONFIG_AUTO, stream=None,
            splits: int | None = None, workspace=None, alpha: float = 1.0):
    """C = epi(alpha * (a @ w^T)) for a (m x k float16) and a 4-bit n x k
    matrix: the product of a layer whose weights are held in 4 bits.  Sums are
    fp32 and rounded once; one row reads each code once.

    ``splits`` and ``workspace`` as in gemm(): None lets the planner split K
    when that pays, with a workspace from torch's caching allocator."""
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
    if stream is None:
        stream = torch.cuda.current_stream(a.device)
    request = SPLITS_AUTO if splits is None else int(splits)
    size = 0
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.device != a.device:
            raise ValueError(f"workspace must be a contiguous tensor on {a.device}")
        size = workspace.numel() * workspace.element_size()
    elif m > 0 and w.n > 0:
        size = _planned((m, w.n, k, w.group, a.data_ptr() % 4 != 0, config, request))[1]
        if size:
            with torch.cuda.device(a.device), torch.cuda.stream(stream):
                workspace = torch.empty(size // 4, dtype=torch.float32, device=a.device)
    _call(a.device, "gemm_f16_q4", lib().gemm_f16_q4, m, w.n, k, w.group, a.data_ptr() or None,
          w.codes.data_ptr() or None, w.words.data_ptr() or None, out.data_ptr() or None, float(alpha),
          _EPILOGUES[epilogue], config, request, workspace.data_ptr() if size else None, size, stream.cuda_stream or None)
    return out


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
    """gemm_f16_q4_cache_t"""
    _fields_ = [("k_codes", _vp), ("k_words", _vp), ("v_codes", _vp), ("v_words", _vp), ("pages", _i64),
                ("heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group", ctypes.c_int32)]


def q4_cache(pages: int, heads: int, page_size: int, head_dim: int, group: int = 64, device="cuda") -> Q4Cache:
    """An empty cache (zeros) of ``pages`` pages of ``page_size`` tokens."""
    import torch

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


def _cache_struct(cache):
    """(gemm_f16_q4_cache_t, device, heads, head_dim) of a checked cache."""
    import torch

    if not isinstance(cache, Q4Cache):
        raise ValueError("cache must be a Q4Cache (as q4_cache returns)")
    _check_group(cache.group)
    t = cache.k_codes
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError("cache.k_codes must be a tensor of pages x heads x page_size x head_dim / 8")
    pages, heads, page_size, d = t.shape[0], t.shape[1], t.shape[2], 8 * t.shape[3]
    words = (pages, heads, d // cache.group, page_size)
    _check_buffer(t, "cache.k_codes", torch.int32, t.shape)
    _check_buffer(cache.k_words, "cache.k_words", torch.int32, words, t.device)
    _check_buffer(cache.v_codes, "cache.v_codes", torch.int32, (pages, heads, page_size // 8, 16, d // 16), t.device)
    _check_buffer(cache.v_words, "cache.v_words", torch.int32, words, t.device)
    s = _CacheStruct(t.data_ptr() or None, cache.k_words.data_ptr() or None, cache.v_codes.data_ptr() or None,
                     cache.v_words.data_ptr() or None, pages, heads, page_size, d, cache.group)
    return s, t.device, heads, d


def _check_ints(t, name, shape, device):
    import torch

    _check_buffer(t, name, torch.int32, shape, device)
    return t.data_ptr() or None


def _check_rows(t, name, heads, d, device):
    """(rows, row pitch) of a rows x heads x d float16 tensor whose heads are contiguous."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype != torch.float16 or t.dim() != 3 or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a 3-D float16 tensor on {device}")
    if t.shape[1] != heads or t.shape[2] != d:
        raise ValueError(f"{name} must be rows x {heads} x {d}, got {tuple(t.shape)}")
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"{name}'s heads must be contiguous in each row")
    rows = t.shape[0]
    return rows, (t.stride(0) if rows > 1 else heads * d)


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
    import torch

    s, device, heads, d = _cache_struct(cache)
    tokens, k_stride = _check_rows(k, "k", heads, d, device)
    v_rows, v_stride = _check_rows(v, "v", heads, d, device)
    if v_rows != tokens:
        raise ValueError(f"k has {tokens} rows and v {v_rows}")
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be an int32 tensor of batch x max_pages")
    batch, max_pages = table.shape
    if starts is None and tokens != batch:
        raise ValueError(f"without starts there is one row for each of the {batch} sequences, got {tokens}")
    table_p = _check_ints(table, "table", table.shape, device)
    lengths_p = _check_ints(lengths, "lengths", (batch,), device)
    starts_p = None if starts is None else _check_ints(starts, "starts", (batch + 1,), device)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    positions = rotary = 0
    cos_p = sin_p = None
    if cos is not None:
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise ValueError("cos must be a float32 tensor of positions x rotary / 2")
        positions, rotary = cos.shape[0], 2 * cos.shape[1]
        _check_buffer(cos, "cos", torch.float32, cos.shape, device)
        _check_buffer(sin, "sin", torch.float32, cos.shape, device)
        if rotary < 16 or rotary > d or rotary % 16 or not positions:
            raise ValueError(f"cos must have 8, 16, ... {d // 2} columns and a row at least, got {tuple(cos.shape)}")
        cos_p, sin_p = cos.data_ptr(), sin.data_ptr()
    q_p = out_p = None
    q_stride = q_heads = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.shape[1] < 1:
            raise ValueError("q must be a tensor of tokens x q_heads x head_dim")
        q_heads = q.shape[1]
        q_rows, q_stride = _check_rows(q, "q", q_heads, d, device)
        if q_rows != tokens:
            raise ValueError(f"q has {q_rows} rows and k {tokens}")
        if out is None:
            out = torch.empty((tokens, q_heads, d), dtype=torch.float16, device=device)
        else:
            _check_buffer(out, "out", torch.float16, (tokens, q_heads, d), device)
        q_p, out_p = q.data_ptr() or None, out.data_ptr() or None
        if not tokens:
            q_p = out_p = None
    elif out is not None:
        raise ValueError("out is for the rotated queries: give q")
    _call(device, "gemm_f16_q4_cache_append", lib().gemm_f16_q4_cache_append, ctypes.byref(s), batch, tokens, max_pages,
          k.data_ptr() or None, k_stride, v.data_ptr() or None, v_stride, table_p, lengths_p, starts_p, q_p, q_stride,
          out_p, q_heads, cos_p, sin_p, positions, rotary, int(bool(interleaved)), _stream(stream, device))
    return out


def q4_cache_read(cache: Q4Cache, table, starts, total: int, first=None, stream=None):
    """(k, v), each total x heads x head_dim float16: rows starts[i] up to
    starts[i + 1] are sequence i's tokens from ``first[i]`` (int32; None: from
    the first one), each value rounded once.  Rows past starts[-1] are not
    written."""
    import torch

    s, device, heads, d = _cache_struct(cache)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be an int32 tensor of batch x max_pages")
    batch, max_pages = table.shape
    table_p = _check_ints(table, "table", table.shape, device)
    starts_p = _check_ints(starts, "starts", (batch + 1,), device)
    first_p = None if first is None else _check_ints(first, "first", (batch,), device)
    if total < 0:
        raise ValueError("total must not be negative")
    k = torch.empty((total, heads, d), dtype=torch.float16, device=device)
    v = torch.empty_like(k)
    _call(device, "gemm_f16_q4_cache_read", lib().gemm_f16_q4_cache_read, ctypes.byref(s), batch, total, max_pages,
          table_p, first_p, starts_p, k.data_ptr() or None, v.data_ptr() or None, _stream(stream, device))
    return k, v


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
    import torch

    s, device, heads, d = _cache_struct(cache)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor of batch x q_heads x head_dim")
    q_heads = q.shape[1]
    if q_heads < 1 or q_heads % heads:
        raise ValueError(f"q's heads must be a multiple of the cache's {heads}, got {q_heads}")
    batch, q_stride = _check_rows(q, "q", q_heads, d, device)
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[0] != batch:
        raise ValueError(f"table must be an int32 tensor of {batch} x max_pages")
    max_pages = table.shape[1]
    table_p = _check_ints(table, "table", table.shape, device)
    lengths_p = _check_ints(lengths, "lengths", (batch,), device)
    if out is None:
        out = torch.empty((batch, q_heads, d), dtype=torch.float16, device=device)
    else:
        _check_buffer(out, "out", torch.float16, (batch, q_heads, d), device)
    if max_length is not None and max_length < 0:
        raise ValueError("max_length must not be negative")
    if stream is None:
        stream = torch.cuda.current_stream(device)
    room = max_pages * s.page_size
    longest = room if not max_length else min(int(max_length), room)
    request = SPLITS_AUTO if splits is None else int(splits)
    if workspace is None:
        need = plan_attention_q4(batch, q_heads, heads, d, cache.group, longest, request)["workspace_bytes"]
        if need:
            with torch.cuda.device(device), torch.cuda.stream(stream):
                workspace = torch.empty(need // 4, dtype=torch.float32, device=device)
    elif not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call(device, "gemm_f16_q4_attention", lib().gemm_f16_q4_attention, ctypes.byref(s), batch, q_heads, max_pages,
          q.data_ptr() or None, q_stride, table_p, lengths_p, float(d ** -0.5 if scale is None else scale),
          out.data_ptr() or None, request, longest, workspace.data_ptr() or None if size else None, size,
          stream.cuda_stream or None)
    return out
