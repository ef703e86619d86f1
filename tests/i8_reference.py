"""What the 8-bit operators and the routing are checked against: numpy, 64 bits, from the definitions in
include/gemm_f16_i8.h."""
import numpy as np
import torch


def pitch(k):
    return -(-k // 16) * 16 if k <= 64 else -(-k // 128) * 128


def compress(x):
    """(codes, scales) of the rows of a float16 array, codes padded to pitch(k) columns.  127 x and m are exact
    in 64 bits, and a quotient of theirs that is no half keeps 2^-20 from one: the rounding is the definition's."""
    x = np.nan_to_num(np.asarray(x).astype(np.float64), nan=0.0, posinf=65504.0, neginf=-65504.0)
    m = np.abs(x).max(-1, initial=0.0)
    q = np.rint(127.0 * x / np.where(m > 0, m, 1.0)[..., None])
    pad = [(0, 0)] * (x.ndim - 1) + [(0, pitch(x.shape[-1]) - x.shape[-1])]
    # (64 bits then 32: a double rounding is innocuous, 53 >= 2 * 24 + 2)
    return np.pad(q, pad).astype(np.int8), (m / 127.0).astype(np.float32)


def expand(codes, scales, k):
    return (codes[..., :k].astype(np.float64) * scales[..., None].astype(np.float64))


def product(a, sa, w, sw, alpha=1.0, relu=False):
    """alpha sa sw a w^T of integer codes: sums exact, the factor in 64 bits."""
    c = (a.astype(np.float64) @ w.astype(np.float64).T) * (np.float64(np.float32(alpha)) * sa.astype(np.float64))[:, None] * sw.astype(np.float64)
    return np.maximum(c, 0.0) if relu else c


def bound(c):
    """Largest error of a product: (alpha sa), times sw, the sum and their product are rounded to fp32, each off by 2^-24
    of the value at most (4 of them: 2^-22 with their squares), then once to binary16, half a step of the result."""
    c = np.abs(c) * (1.0 + 2.0 ** -22)
    return np.maximum(c * 2.0 ** -11, 2.0 ** -25) + c * 2.0 ** -22


def near(got, want):
    """Whether a float16 array is within bound() of a 64-bit one (beyond binary16: infinite)."""
    got = np.asarray(got).astype(np.float64)
    over = np.abs(want) >= 65520 * (1 + 2.0 ** -22)
    edge = (np.abs(want) >= 65504) & ~over          # either the largest number or infinity
    fine = np.abs(got - want) <= bound(want)
    return np.where(over, got == np.copysign(np.inf, want), fine | (edge & (np.abs(got) >= 65504) & (np.sign(got) == np.sign(want))))


def scores(logits, bias, kind):
    """(score, key, open) in 64 bits."""
    x = np.asarray(logits).astype(np.float64)
    b = np.zeros(x.shape[-1]) if bias is None else np.asarray(bias).astype(np.float64)
    with np.errstate(all="ignore"):
        can = (x > -np.inf) & (b > -np.inf)
        x = np.where(can, np.minimum(x, float(np.finfo(np.float32).max)), -np.inf)
        if kind == "softmax":
            most = x.max(-1, keepdims=True)
            e = np.where(can, np.exp(x - np.where(np.isfinite(most), most, 0.0)), 0.0)
            total = e.sum(-1, keepdims=True)
            s = np.where(total > 0, e / np.where(total > 0, total, 1.0), 0.0)
        else:
            s = np.where(can, 1.0 / (1.0 + np.exp(-x)), 0.0)
        return s, (x if bias is None else s + b), can


def route(logits, top_k, kind="softmax", bias=None, groups=1, top_groups=1, renormalise=False, scale=1.0):
    """(ids, weights in 64 bits), token by token."""
    s, key, can = scores(logits, bias, kind)
    with np.errstate(all="ignore"):
        value = s + (0.0 if bias is None else np.asarray(bias).astype(np.float64))
    tokens, experts = s.shape
    ids, weights = np.full((tokens, top_k), -1, np.int32), np.zeros((tokens, top_k))
    n = experts // groups
    for t in range(tokens):
        left = [e for e in range(experts) if can[t, e]]
        if groups > 1:
            best = {}
            for g in range(groups):
                v = sorted((value[t, e] for e in left if e // n == g), reverse=True)[:2]
                if v:
                    best[g] = sum(v)
            stay = sorted(best, key=lambda g: (-best[g], g))[:top_groups]
            left = [e for e in left if e // n in stay]
        chosen = sorted(left, key=lambda e: (-key[t, e], e))[:top_k]
        w = np.array([s[t, e] for e in chosen])
        if renormalise:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = w * np.float64(np.float32(scale))
    return ids, weights


def order(ids, experts):
    flat = np.asarray(ids).reshape(-1)
    bins = np.where((flat >= 0) & (flat < experts), flat, experts)
    return np.argsort(bins, kind="stable").astype(np.int32), np.searchsorted(np.sort(bins), np.arange(experts + 1)).astype(np.int32)


def host(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().numpy()
