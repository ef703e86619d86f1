"""CPU tests of the 4-bit operand entry points: exported symbols, buffer
sizes, refusals and plans (validation runs before any HIP call, so no kernel
is launched here), and the reference the GPU tests compare with."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import q4_reference as ref
import tiled_dense_gemm_fp16_amd as g

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_f16_q4.h")

FAKE = 1 << 40          # aligned, never dereferenced; buffers a GiB or more apart
INVALID, MISALIGNED, NO_DEVICE, SIZE = 1, 2, 3, 6


def at(i):
    return FAKE + (i << 36)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(g.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gemm_f16\w*)\s*\(", text))
    lib = ctypes.CDLL(g.LIB_PATH)
    for name in names:
        assert hasattr(lib, name), name
    assert set(g.Q4_SIGNATURES) == names


def test_buffer_sizes():
    h = g.lib()
    for n, k in [(0, 0), (1, 1), (16, 128), (17, 129), (5000, 4100)]:
        nb, kb = -(-n // 16), -(-k // 128)
        assert h.gemm_f16_q4_codes_bytes(n, k) == nb * kb * 1024
        for group in (32, 64, 128):
            assert h.gemm_f16_q4_words_bytes(n, k, group) == nb * kb * 16 * 4 * (128 // group)
    assert h.gemm_f16_q4_codes_bytes(-1, 4) == -1 and h.gemm_f16_q4_codes_bytes(1, (1 << 22) + 1) == -1
    assert h.gemm_f16_q4_words_bytes(16, 128, 48) == -1


def test_product_refusals():
    h = g.lib()

    def call(m=4, n=32, k=256, group=64, a=at(0), codes=at(1), words=at(2), c=at(3), epi=0, config=-1):
        return h.gemm_f16_q4(m, n, k, group, a, codes, words, c, 1.0, epi, config, None)

    for bad in (dict(m=-1), dict(n=-1), dict(k=-1), dict(group=16), dict(group=0), dict(a=None), dict(codes=None),
                dict(words=None), dict(c=None), dict(epi=2), dict(epi=-1), dict(config=g.q4_num_configs()), dict(config=-2),
                dict(c=at(0)), dict(c=at(1) + 64), dict(c=at(2)), dict(c=at(0) + 2 * 4 * 256 - 2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(a=at(0) + 1), dict(c=at(3) + 1), dict(codes=at(1) + 8), dict(words=at(2) + 4)):
        assert call(**bad) == MISALIGNED, bad
    for bad in (dict(m=1 << 31), dict(n=(1 << 22) + 1), dict(k=(1 << 22) + 1)):
        assert call(**bad) == SIZE, bad
    assert call(m=0, a=None, c=None) == 0 and call(n=0, codes=None, words=None, c=None) == 0
    if not torch.cuda.is_available():
        assert call() == NO_DEVICE and call(c=at(0) + 2 * 4 * 256) == NO_DEVICE


def test_compress_and_expand_refusals():
    h = g.lib()
    for fn in (lambda w, c, o, n=32, k=256, group=64: h.gemm_f16_q4_compress(n, k, group, 0, w, c, o, None),
               lambda w, c, o, n=32, k=256, group=64: h.gemm_f16_q4_expand(n, k, group, c, o, w, None)):
        assert fn(None, at(1), at(2)) == INVALID and fn(at(0), None, at(2)) == INVALID
        assert fn(at(0), at(1), None) == INVALID and fn(at(0), at(1), at(2), group=33) == INVALID
        assert fn(at(0), at(1), at(2), n=-1) == INVALID and fn(at(0), at(1), at(2), k=1 << 23) == SIZE
        assert fn(at(0) + 1, at(1), at(2)) == MISALIGNED and fn(at(0), at(1) + 4, at(2)) == MISALIGNED
        assert fn(at(1), at(1), at(2)) == INVALID and fn(at(2), at(1), at(2)) == INVALID
        assert fn(None, None, None, n=0) == 0
    assert h.gemm_f16_q4_compress(32, 256, 64, 0, at(0), at(1), at(1), None) == INVALID
    assert h.gemm_f16_q4_compress(32, 256, 64, 2, at(0), at(1), at(2), None) == INVALID


def test_plans():
    for c in range(g.q4_num_configs()):
        assert g.q4_config_name(c)
        for m, n, k in [(1, 16, 128), (5, 1000, 4100), (64, 8192, 8192), (2048, 5000, 300), (1, 1, 1 << 22)]:
            p = g.plan_q4(m, n, k, 64, config=c)
            assert p["config"] == c and p["lds_bytes"] <= 163840 and p["threads"] <= 1024
            assert p["tiles_m"] * p["block_m"] >= m and p["tiles_n"] * p["block_n"] >= n
            assert p["flops"] == 2.0 * m * n * k
    assert g.q4_config_name(-1) is None and g.q4_config_name(g.q4_num_configs()) is None
    for bad in (dict(m=-1), dict(group=31), dict(k=1 << 23), dict(config=99)):
        with pytest.raises(g.GemmError):
            g.plan_q4(**{**dict(m=1, n=16, k=128), **bad})


def test_binding_refusals():
    w = torch.zeros(16, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        g.q4_compress(w)                                   # not on the GPU
    with pytest.raises(ValueError):
        g.q4_compress(w, group=48)
    m = g.Q4Matrix(torch.zeros(1, 1, 4, 16, 4, dtype=torch.int32), torch.zeros(1, 1, 16, 1, dtype=torch.int32), 16, 128, 128)
    with pytest.raises(ValueError):
        g.gemm_q4(w, m)
    with pytest.raises(ValueError):
        g.q4_expand(m)
    with pytest.raises(ValueError):
        g.q4_expand((m.codes, m.words))


def test_reference_rounding_and_layout():
    # a group held exactly: codes 0..15 with scale 1/4 and zero point 5
    x = (np.arange(16) - 5) / 4.0
    w = np.tile(x, (3, 16)).astype(np.float32)
    for group in (32, 64, 128):
        q, z, s = ref.round_groups(w, group)
        assert (z == 5).all() and (s == 0.25).all() and (q == np.tile(np.arange(16), (3, 16))).all()
        codes, words = ref.pack_weights(w, group)
        assert np.array_equal(ref.unpack_weights(codes, words, 3, 256, group), w)
    # the header's dword of 0..7 and its place: row 2, k 168..175 = tile 1, j 1, g 1
    assert codes[0, 1, 1, 2, 1] == sum(int(v) << (4 * p) for v, p in zip((8, 9, 10, 11, 12, 13, 14, 15), ref.NIBBLE))
    # rounding is off by at most half a step of s (and of s's own rounding)
    x = np.random.default_rng(0).normal(size=(7, 256)).astype(np.float32)
    for group, symmetric in [(32, False), (128, True)]:
        q, z, s = ref.round_groups(x, group, symmetric)
        back = (s[..., None] * (q.reshape(7, -1, group) - z[..., None])).reshape(x.shape)
        step = np.repeat(s.astype(np.float64), group, -1)
        assert (np.abs(back - x) <= step * (0.5 + 16 * 2.0 ** -11 + (0.5 if not symmetric else 0))).all()
