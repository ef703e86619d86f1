"""Products with 8-bit operands and routed experts (include/gemm_f16_i8.h).

Rows of float16 become integer codes with one scale each (a token's, or an
output channel's of a weight matrix) by :func:`i8_compress`, are read back by
:func:`i8_expand` and multiplied by :func:`gemm_i8`.  A layer of experts
chooses them with :func:`route`, sorts the chosen pairs with
:func:`expert_order`, multiplies each token with its experts' weights with
:func:`gemm_i8_experts` and adds up the results with :func:`expert_sum`::

    ids, weights = route(logits, top_k=8, score="sigmoid", bias=b, groups=8, top_groups=4)
    order = expert_order(ids, experts)
    h = gemm_i8_experts(i8_compress(x), w_up, order, epilogue="relu")     # tokens x 8 x n
    y = gemm_i8_experts(i8_compress(h), w_down, order)                    # a row for each pair
    out = expert_sum(y, weights)

Argument marshalling only, compiled (csrc/i8_binding.cpp) as for the 4-bit
entry points: tensors give memory, torch's current stream is the default
stream, results made here belong to the call's stream, and nothing falls
back to the CPU.  Inference only: results have no gradient.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

from . import _EPILOGUES, CONFIG_AUTO, I8_BINDING_PATH, SPLITS_AUTO, SUCCESS, GemmError, Plan, lib

_SCORES = {"softmax": 0, "sigmoid": 1}
_module = None


def _binding():
    """The compiled marshalling module, built with the library."""
    global _module
    if _module is None:
        lib()
        if not os.path.exists(I8_BINDING_PATH):
            raise RuntimeError(f"{I8_BINDING_PATH} is missing: build the HIP library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        from . import _i8_binding
        _i8_binding.setup(I8Matrix, ExpertOrder, GemmError, torch._C._cuda_getCurrentRawStream)
        _module = _i8_binding
    return _module


def _call(name, stream, *args):
    """Call the compiled entry point on `stream`, or on torch's current one."""
    fn = getattr(_module or _binding(), name)
    if stream is None:
        return fn(*args, None)
    with torch.cuda.stream(stream):
        return fn(*args, stream.device.index)


def _epilogue(name):
    epi = _EPILOGUES.get(name)
    if epi is None:
        raise ValueError(f"epilogue must be one of {sorted(_EPILOGUES)}, got {name!r}")
    return epi


# ---- rows in 8 bits -------------------------------------------------------------

class I8Matrix(NamedTuple):
    """Rows of ``k`` elements in 8 bits: element e of a row stands for its
    scale times its code.  (Products are faster where rows start on cache
    lines, as i8_compress's do from 65 elements on: a pitch of a multiple of 128.)"""
    codes: object    # int8 [..., rows, pitch], pitch a multiple of 16 and at least k; zeros from k to the next multiple of 16
    scales: object   # float32 [..., rows]
    k: int


def i8_compress(x, stream=None) -> I8Matrix:
    """x (... x rows x k float16 GPU tensor; rows may lie apart, as slices of
    wider ones do) rounded row by row to codes in -127..127 and a scale: the
    row's largest magnitude is 127.  NaN counts as 0, infinities as 65504."""
    return _call("compress", stream, x)


def i8_expand(x: I8Matrix, out=None, stream=None):
    """The float16 rows that ``x`` stands for, each value rounded once."""
    return _call("expand", stream, x, out)


def gemm_i8(a: I8Matrix, w: I8Matrix, epilogue: str = "none", out=None, config: int = CONFIG_AUTO, stream=None,
            splits: int | None = None, workspace=None, alpha: float = 1.0):
    """C = epi(alpha * (a @ w^T)), m x n float16, for 8-bit a (m x k) and w
    (n x k): a scale for each token and each output channel.  Sums of products
    of codes are exact; they are scaled in fp32 and rounded once.

    ``splits`` and ``workspace`` as in gemm(): None lets the planner split K
    when that pays, with a workspace from torch's caching allocator (or not,
    where it has no room for one).  Every configuration and split gives the
    same bits."""
    return _call("gemm", stream, a, w, _epilogue(epilogue), out, config, splits, workspace, alpha)


def plan_i8(m: int, n: int, k: int, config: int = CONFIG_AUTO, splits: int | None = 1) -> dict:
    """How gemm_f16_i8 would run this shape (host logic only)."""
    p = Plan()
    st = lib().gemm_f16_plan_i8(m, n, k, config, SPLITS_AUTO if splits is None else int(splits), ctypes.byref(p))
    if st != SUCCESS:
        raise GemmError(st, "gemm_f16_plan_i8")
    return p.as_dict()


def i8_num_configs() -> int:
    return int(lib().gemm_f16_i8_num_configs())


def i8_config_name(config: int) -> str | None:
    s = lib().gemm_f16_i8_config_name(int(config))
    return s.decode() if s is not None else None


# ---- routed experts ---------------------------------------------------------------

class ExpertOrder(NamedTuple):
    """The pairs token * top_k + slot by expert, as expert_order() makes it."""
    order: object    # int32 [tokens, top_k]: the pairs of expert 0, of expert 1, ..., of none
    starts: object   # int32 [experts + 1]: the place of each expert's first pair, and of the first pair of none


def route(logits, top_k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
          renormalise: bool = False, scale: float = 1.0, stream=None):
    """(ids, weights), int32 and float32 tokens x top_k: the experts that each
    token's logits (tokens x experts, float16 or float32) choose, the best
    first, equals in the order of their indexes.

    Scores are the softmax or sigmoid of the logits.  What is compared is
    score + ``bias`` (float32, one for each expert), in 64 bits; without a
    bias the logits, whose order is that of the scores also where these round
    to the same number.  With ``groups`` blocks of experts only those of the
    ``top_groups`` blocks whose two largest score + bias (score, without one)
    have the largest sum take part.  Weights are the chosen
    experts' scores without bias, divided by their sum with ``renormalise``,
    times ``scale``.  An expert whose logit or bias is NaN or -inf is never
    chosen; where none is left the id is -1 and the weight 0."""
    kind = _SCORES.get(score)
    if kind is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return _call("route", stream, logits, top_k, kind, bias, groups, top_groups, renormalise, scale)


def expert_order(ids, experts: int, stream=None) -> ExpertOrder:
    """The pairs of ``ids`` (int32 tokens x top_k) sorted by expert, those of
    one expert in ascending order; ids outside of 0 .. experts - 1 come last."""
    return _call("order", stream, ids, experts)


def gemm_i8_experts(a: I8Matrix, w: I8Matrix, order: ExpertOrder, epilogue: str = "none", out=None,
                    config: int = CONFIG_AUTO, stream=None, alpha: float = 1.0):
    """tokens x top_k x n float16: epi(alpha * (row @ w[expert]^T)) for each
    pair of ``order``, zeros for the pairs of no expert.  ``w`` holds experts x
    n rows; ``a`` one row for each token (which its top_k pairs share) or one
    for each pair (tokens x top_k x k, as the first product's result has);
    its codes are limited to 2 GiB, so more tokens take several calls, each
    with the order of its own ids.  Computed as by gemm_i8, bit for bit."""
    return _call("experts", stream, a, w, order, _epilogue(epilogue), out, config, alpha)


def plan_i8_experts(pairs: int, pairs_per_row: int, experts: int, n: int, k: int, config: int = CONFIG_AUTO) -> dict:
    """How gemm_f16_i8_experts would run (host logic only)."""
    p = Plan()
    st = lib().gemm_f16_plan_i8_experts(pairs, pairs_per_row, experts, n, k, config, ctypes.byref(p))
    if st != SUCCESS:
        raise GemmError(st, "gemm_f16_plan_i8_experts")
    return p.as_dict()


def expert_sum(y, weights, out=None, stream=None):
    """tokens x n float16: the sum over slots of weights[t][j] * y[t][j] (y:
    tokens x top_k x n float16, weights: tokens x top_k float32), in fp32 and
    in the order of the slots, rounded once."""
    return _call("sum", stream, y, weights, out)
