"""Products with 4-bit operands (include/gemm_f16_q4.h): weights held as 4-bit
codes with a scale and a zero point per group, made by :func:`q4_compress`,
read back by :func:`q4_expand` and multiplied by :func:`gemm_q4`; and a paged
key/value cache in the same codes, filled by :func:`q4_cache_append`, read
back by :func:`q4_cache_read` and attended to by :func:`attention_q4`.

Argument marshalling only, as in the package's other entry points: tensors
give memory, torch's current stream is the default stream, and nothing falls
back to the CPU.  A decode step makes many of these calls on small tensors, so
each argument is checked with a few attribute reads, and what was wrong is
worked out only when something was.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _EPILOGUES, CONFIG_AUTO, SPLITS_AUTO, SUCCESS, GemmError, Plan, lib

_i64, _vp = ctypes.c_int64, ctypes.c_void_p

GROUPS = (32, 64, 128)


def _check_group(group):
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group!r}")


def _device_of(t, name):
    """Index of the GPU that a tensor lies on."""
    index = t.get_device() if isinstance(t, torch.Tensor) else -1
    if index < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return index


def _buffer(t, name, dtype, shape, index):
    """Address of a contiguous tensor of this dtype and shape on GPU `index`."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return t.data_ptr() or None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    raise ValueError(f"{name} must be a contiguous tensor on cuda:{index}")


def _empty(shape, dtype, index, stream):
    """A new tensor that belongs to the call's stream: memory that another
    stream may still be using is not written to."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=index)
    if stream.device.index != index:
        raise ValueError(f"stream must be a stream of cuda:{index}")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=index)


def _output(out, shape, index, stream):
    """(tensor, address) of a caller's float16 output, or of a new one."""
    if out is None:
        out = _empty(shape, torch.float16, index, stream)
        return out, out.data_ptr() or None
    return out, _buffer(out, "out", torch.float16, shape, index)


def _workspace(workspace, need, index, stream):
    """(address, bytes) of a caller's workspace, or of one taken from torch's
    caching allocator on the call's stream, and what keeps it alive."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.get_device() != index:
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}")
        size = workspace.numel() * workspace.element_size()
        return (workspace.data_ptr() if size else None), size, workspace
    if not need:
        return None, 0, None
    t = _empty(need // 4, torch.float32, index, stream)
    return t.data_ptr(), need, t


def _call(index, stream, what, fn, *args):
    """Call a C entry point on GPU `index` and `stream` (its last argument)."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device.index == index:
        raw = stream.cuda_stream
    else:
        raise ValueError(f"stream must be a stream of cuda:{index}")
    if torch.cuda.current_device() == index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            st = fn(*args, raw)
    if st != SUCCESS:
        raise GemmError(st, what)


# ---- weights --------------------------------------------------------------------

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


def _matrix(w, index=None):
    """(device index, codes' address, words' address) of a checked matrix."""
    if not isinstance(w, Q4Matrix):
        raise ValueError("w must be a Q4Matrix (as q4_compress returns)")
    _check_group(w.group)
    if index is None:
        index = _device_of(w.codes, "w.codes")
    codes, words = _buffer_shapes(w.n, w.k, w.group)
    return index, _buffer(w.codes, "w.codes", torch.int32, codes, index), _buffer(w.words, "w.words", torch.int32, words, index)


def q4_compress(w, group: int = 128, symmetric: bool = False, stream=None) -> Q4Matrix:
    """w (n x k float16 GPU tensor) rounded to 4-bit codes with a scale and a
    zero point for every ``group`` neighbours of a row (``symmetric``: zero
    point 8, largest magnitude at code 7 from it)."""
    _check_group(group)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a 2-D float16 tensor")
    index = _device_of(w, "w")
    at = _buffer(w, "w", torch.float16, w.shape, index)
    n, k = w.shape
    codes, words = _buffer_shapes(n, k, group)
    codes, words = (_empty(shape, torch.int32, index, stream) for shape in (codes, words))
    _call(index, stream, "gemm_f16_q4_compress", lib().gemm_f16_q4_compress, n, k, group, 1 if symmetric else 0, at,
          codes.data_ptr() or None, words.data_ptr() or None)
    return Q4Matrix(codes, words, n, k, group)


def q4_expand(w: Q4Matrix, out=None, stream=None):
    """The n x k float16 matrix that ``w`` stands for, each value rounded once."""
    index, codes, words = _matrix(w)
    out, to = _output(out, (w.n, w.k), index, stream)
    _call(index, stream, "gemm_f16_q4_expand", lib().gemm_f16_q4_expand, w.n, w.k, w.group, codes, words, to)
    return out


_plans: dict = {}


def _planned(key, plan):
    """Workspace bytes of a call, by what decides them (shapes, an alignment and the request)."""
    need = _plans.get(key)
    if need is None:
        need = plan()["workspace_bytes"]
        if len(_plans) > 4096:
            _plans.clear()
        _plans[key] = need
    return need


def gemm_q4(a, w: Q4Matrix, epilogue: str = "none", out=None, config: int = CONFIG_AUTO, stream=None,
            splits: int | None = None, workspace=None, alpha: float = 1.0):
    """C = epi(alpha * (a @ w^T)) for a (m x k float16) and a 4-bit n x k
    matrix: the product of a layer whose weights are held in 4 bits.  Sums are
    fp32 and rounded once; one row reads each code once.

    ``splits`` and ``workspace`` as in gemm(): None lets the planner split K
    when that pays, with a workspace from torch's caching allocator."""
    epi = _EPILOGUES.get(epilogue)
    if epi is None:
        raise ValueError(f"epilogue must be one of {sorted(_EPILOGUES)}, got {epilogue!r}")
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise ValueError("a must be a 2-D float16 tensor")
    index = _device_of(a, "a")
    at = _buffer(a, "a", torch.float16, a.shape, index)
    _, codes, words = _matrix(w, index)
    m, k = a.shape
    n = w.n
    if k != w.k:
        raise ValueError(f"inner dimensions differ: a is {tuple(a.shape)}, w is {n} x {w.k}")
    out, to = _output(out, (m, n), index, stream)
    request = SPLITS_AUTO if splits is None else int(splits)
    need = 0
    if workspace is None and m and n:
        odd = (at or 0) % 4
        need = _planned(("gemm", m, n, k, w.group, odd == 0, config, request),
                        lambda: plan_q4(m, n, k, w.group, config, request, odd))
    ws, size, _keep = _workspace(workspace, need, index, stream)
    _call(index, stream, "gemm_f16_q4", lib().gemm_f16_q4, m, n, k, w.group, at, codes, words, to, alpha, epi, config,
          request, ws, size)
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


def _cache(cache):
    """(gemm_f16_q4_cache_t, device index) of a checked cache."""
    if not isinstance(cache, Q4Cache):
        raise ValueError("cache must be a Q4Cache (as q4_cache returns)")
    k_codes, k_words, v_codes, v_words, group = cache
    _check_group(group)
    if not isinstance(k_codes, torch.Tensor) or k_codes.dim() != 4:
        raise ValueError("cache.k_codes must be a tensor of pages x heads x page_size x head_dim / 8")
    index = _device_of(k_codes, "cache.k_codes")
    shape = k_codes.shape
    pages, heads, page_size, d = shape
    d *= 8
    words = (pages, heads, d // group, page_size)
    return _CacheStruct(_buffer(k_codes, "cache.k_codes", torch.int32, shape, index),
                        _buffer(k_words, "cache.k_words", torch.int32, words, index),
                        _buffer(v_codes, "cache.v_codes", torch.int32, (pages, heads, page_size // 8, 16, d // 16), index),
                        _buffer(v_words, "cache.v_words", torch.int32, words, index),
                        pages, heads, page_size, d, group), index


def _table(table, index, batch=None):
    """(address, batch, max_pages) of a page table."""
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or (batch is not None and table.shape[0] != batch):
        raise ValueError(f"table must be an int32 tensor of {'batch' if batch is None else batch} x max_pages")
    shape = table.shape
    return _buffer(table, "table", torch.int32, shape, index), shape[0], shape[1]


def _rows(t, name, heads, d, index, count=None):
    """(address, rows, row pitch) of a rows x heads x d float16 tensor whose heads are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float16 or t.dim() != 3 or t.get_device() != index:
        raise ValueError(f"{name} must be a 3-D float16 tensor on cuda:{index}")
    rows, h, e = t.shape
    if h != heads or e != d or (count is not None and rows != count):
        raise ValueError(f"{name} must be {'rows' if count is None else count} x {heads} x {d}, got {tuple(t.shape)}")
    pitch, head, one = t.stride()
    if one != 1 or (heads > 1 and head != d):
        raise ValueError(f"{name}'s heads must be contiguous in each row")
    return t.data_ptr() or None, rows, (pitch if rows > 1 else heads * d)


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
    s, index = _cache(cache)
    heads, d = s.heads, s.head_dim
    k_p, tokens, k_stride = _rows(k, "k", heads, d, index)
    v_p, _, v_stride = _rows(v, "v", heads, d, index, tokens)
    table_p, batch, max_pages = _table(table, index)
    if starts is None and tokens != batch:
        raise ValueError(f"without starts there is one row for each of the {batch} sequences, got {tokens}")
    lengths_p = _buffer(lengths, "lengths", torch.int32, (batch,), index)
    starts_p = None if starts is None else _buffer(starts, "starts", torch.int32, (batch + 1,), index)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    positions = rotary = 0
    cos_p = sin_p = None
    if cos is not None:
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise ValueError("cos must be a float32 tensor of positions x rotary / 2")
        shape = cos.shape
        positions, rotary = shape[0], 2 * shape[1]
        if rotary < 16 or rotary > d or rotary % 16 or not positions:
            raise ValueError(f"cos must have 8, 16, ... {d // 2} columns and a row at least, got {tuple(shape)}")
        cos_p = _buffer(cos, "cos", torch.float32, shape, index)
        sin_p = _buffer(sin, "sin", torch.float32, shape, index)
    q_p = out_p = None
    q_stride = q_heads = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.shape[1] < 1:
            raise ValueError("q must be a tensor of tokens x q_heads x head_dim")
        q_heads = q.shape[1]
        q_p, _, q_stride = _rows(q, "q", q_heads, d, index, tokens)
        out, out_p = _output(out, (tokens, q_heads, d), index, stream)
    elif out is not None:
        raise ValueError("out is for the rotated queries: give q")
    _call(index, stream, "gemm_f16_q4_cache_append", lib().gemm_f16_q4_cache_append, ctypes.byref(s), batch, tokens, max_pages,
          k_p, k_stride, v_p, v_stride, table_p, lengths_p, starts_p, q_p, q_stride, out_p, q_heads, cos_p, sin_p, positions,
          rotary, 1 if interleaved else 0)
    return out


def q4_cache_read(cache: Q4Cache, table, starts, total: int, first=None, stream=None):
    """(k, v), each total x heads x head_dim float16: rows starts[i] up to
    starts[i + 1] are sequence i's tokens from ``first[i]`` (int32; None: from
    the first one), each value rounded once.  Rows past starts[-1] are not
    written."""
    s, index = _cache(cache)
    table_p, batch, max_pages = _table(table, index)
    starts_p = _buffer(starts, "starts", torch.int32, (batch + 1,), index)
    first_p = None if first is None else _buffer(first, "first", torch.int32, (batch,), index)
    if total < 0:
        raise ValueError("total must not be negative")
    shape = (total, s.heads, s.head_dim)
    k, v = (_empty(shape, torch.float16, index, stream) for _ in range(2))
    _call(index, stream, "gemm_f16_q4_cache_read", lib().gemm_f16_q4_cache_read, ctypes.byref(s), batch, total, max_pages,
          table_p, first_p, starts_p, k.data_ptr() or None, v.data_ptr() or None)
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
    s, index = _cache(cache)
    heads, d = s.heads, s.head_dim
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor of batch x q_heads x head_dim")
    q_heads = q.shape[1]
    if q_heads < 1 or q_heads % heads:
        raise ValueError(f"q's heads must be a multiple of the cache's {heads}, got {q_heads}")
    q_p, batch, q_stride = _rows(q, "q", q_heads, d, index)
    table_p, _, max_pages = _table(table, index, batch)
    lengths_p = _buffer(lengths, "lengths", torch.int32, (batch,), index)
    out, out_p = _output(out, (batch, q_heads, d), index, stream)
    if max_length is not None and max_length < 0:
        raise ValueError("max_length must not be negative")
    room = max_pages * s.page_size
    longest = min(int(max_length), room) if max_length else room
    request = SPLITS_AUTO if splits is None else int(splits)
    need = 0
    if workspace is None:
        need = _planned(("attention", batch, q_heads, heads, d, cache.group, longest, request),
                        lambda: plan_attention_q4(batch, q_heads, heads, d, cache.group, longest, request))
    ws, size, _keep = _workspace(workspace, need, index, stream)
    _call(index, stream, "gemm_f16_q4_attention", lib().gemm_f16_q4_attention, ctypes.byref(s), batch, q_heads, max_pages, q_p,
          q_stride, table_p, lengths_p, d ** -0.5 if scale is None else scale, out_p, request, longest, ws, size)
    return out
