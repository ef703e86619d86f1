"""The 4-bit format of include/gemm_f16_q4.h in plain numpy / torch on the CPU,
by the place of each element, and the operators' definitions in 64 bits.
Test infrastructure; shares no code with the library."""
import numpy as np
import torch

NIBBLE = np.array([0, 4, 1, 5, 2, 6, 3, 7])


def round_groups(x, group, symmetric=False):
    """(q, z, s) of the groups along x's last axis: float32 arithmetic as the header states it (each step is one
    correctly rounded operation, so the results are exact).  x: float32 array, last axis a multiple of group."""
    x = np.asarray(x, np.float32)
    g = np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf).reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        lo, hi = np.minimum(g.min(-1), np.float32(0)), np.maximum(g.max(-1), np.float32(0))
        wide = np.abs(np.maximum(hi, -lo) / np.float32(7) if symmetric else (hi - lo) / np.float32(15))   # never -0
        s = np.minimum(wide, np.float32(65504)).astype(np.float16).astype(np.float32)
        some = s > 0
        z = np.full_like(s, 8) if symmetric else np.clip(np.rint(np.where(some, -lo / s, 0)), 0, 15)
        q = np.where(some[..., None], np.rint(g / s[..., None]), 0)
    q = np.clip(q + z[..., None], 0, 15).reshape(x.shape)
    return q.astype(np.int64), z.astype(np.int64), s.astype(np.float16)


def words_of(s, z):
    return (s.view(np.uint16).astype(np.uint32) | (z.astype(np.uint32) << 16))


def scale_zero(words):
    words = np.asarray(words).astype(np.uint32)
    return (words & 0xFFFF).astype(np.uint16).view(np.float16).astype(np.float64), (words >> 16).astype(np.float64)


def pack_weights(w, group, symmetric=False):
    """codes and words (uint32 arrays in the header's order) of a float32 n x k matrix."""
    n, k = w.shape
    nb, kb = -(-n // 16), -(-k // 128)
    full = np.zeros((16 * nb, 128 * kb), np.float32)
    full[:n, :k] = w
    q, z, s = round_groups(full, group, symmetric)
    codes = np.zeros((nb, kb, 4, 16, 4), np.uint32)
    for i in range(16 * nb):
        for b in range(kb):
            for g in range(4):
                for j in range(4):
                    eight = q[i, 128 * b + 32 * j + 8 * g:][:8]
                    codes[i // 16, b, g, i % 16, j] = np.sum(eight.astype(np.uint32) << (4 * NIBBLE).astype(np.uint32))
    words = words_of(s, z).reshape(nb, 16, kb, 128 // group).transpose(0, 2, 1, 3)
    return codes, np.ascontiguousarray(words)


def unpack_weights(codes, words, n, k, group):
    """The float64 matrix that codes and words (tensors or arrays) stand for."""
    codes, words = np.asarray(codes).astype(np.int64) & 0xFFFFFFFF, np.asarray(words).astype(np.int64) & 0xFFFFFFFF
    i, x = np.arange(n)[:, None], np.arange(k)[None]
    dword = codes[i // 16, x // 128, x % 32 // 8, i % 16, x % 128 // 32]
    s, z = scale_zero(words[i // 16, x // 128, i % 16, x % 128 // group])
    return s * ((dword >> (4 * NIBBLE[x % 8]) & 15) - z)


def product(a, w, alpha=1.0, relu=False):
    """(C in 64 bits, the same sum of magnitudes) for float64 a and w."""
    c, size = a @ w.T * alpha, np.abs(a) @ np.abs(w).T * abs(alpha)
    return (np.maximum(c, 0) if relu else c), size


def half_steps(r):
    """Largest error of one rounding of r to binary16: half a step of r's binade, 2^-25 below the normals."""
    return np.maximum(np.abs(r) * 2.0 ** -11, 2.0 ** -25)


def host(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().numpy()


# ---- the paged cache ---------------------------------------------------------------------------------------------

def key_place(d, dim):
    """Dword of a token's row that holds element d."""
    b = min(dim, 128)
    return d // b * (b // 8) + d % 32 // 8 * (b // 32) + d % b // 32


class Cache:
    """A cache as plain arrays: codes and zero points and scales by [page, slot, head, d]."""

    def __init__(self, k_codes, k_words, v_codes, v_words, group):
        u = [np.asarray(x).astype(np.int64) & 0xFFFFFFFF for x in (k_codes, k_words, v_codes, v_words)]
        pages, heads, slots, d8 = u[0].shape
        dim = 8 * d8
        d, t = np.arange(dim), np.arange(slots)[:, None]
        self.group = group
        self.q = {"k": np.stack([u[0][:, :, :, key_place(i, dim)] >> (4 * NIBBLE[i % 8]) & 15 for i in d], -1).transpose(0, 2, 1, 3),
                  "v": (u[2][:, :, t // 8, d % 16, d // 16] >> (4 * NIBBLE[t % 8]) & 15).transpose(0, 2, 1, 3)}
        self.word = {"k": u[1].transpose(0, 3, 1, 2), "v": u[3].transpose(0, 3, 1, 2)}

    def values(self, which):
        """float64 [page, slot, head, d]"""
        s, z = scale_zero(self.word[which])
        return np.repeat(s, self.group, -1) * (self.q[which] - np.repeat(z, self.group, -1))


def rotate(x, cos, sin, interleaved):
    """float32 rotation of x [rows, heads, d] with cos, sin [rows, half]: every product and sum rounded by itself."""
    x = np.asarray(x, np.float32).copy()
    half = cos.shape[1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    c, s = cos[:, None].astype(np.float32), sin[:, None].astype(np.float32)
    p, q = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = p * c - q * s, q * c + p * s
    return x


def attention(q, k, v, scale):
    """(out, sum of p |v|, largest sum of magnitudes of a score) of one head's query q [d] over k, v [n, d], 64 bits."""
    if not len(k):
        return np.zeros_like(q), np.zeros_like(q)
    x = k @ q * scale
    p = np.exp(x - x.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v)
