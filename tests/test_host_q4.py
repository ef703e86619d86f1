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

    def call(m=4, n=32, k=256, group=64, a=at(0), codes=at(1), words=at(2), c=at(3), epi=0, config=-1,
             splits=1, ws=None, size=0):
        return h.gemm_f16_q4(m, n, k, group, a, codes, words, c, 1.0, epi, config, splits, ws, size, None)

    for bad in (dict(m=-1), dict(n=-1), dict(k=-1), dict(group=16), dict(group=0), dict(a=None), dict(codes=None),
                dict(words=None), dict(c=None), dict(epi=2), dict(epi=-1), dict(config=g.q4_num_configs()), dict(config=-2),
                dict(c=at(0)), dict(c=at(1) + 64), dict(c=at(2)), dict(c=at(0) + 2 * 4 * 256 - 2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(a=at(0) + 1), dict(c=at(3) + 1), dict(codes=at(1) + 8), dict(words=at(2) + 4)):
        assert call(**bad) == MISALIGNED, bad
    for bad in (dict(m=1 << 31), dict(n=(1 << 22) + 1), dict(k=(1 << 22) + 1)):
        assert call(**bad) == SIZE, bad
    # the tile configurations need A's rows 4-byte aligned; a split a workspace
    last = g.q4_num_configs() - 1            # expands W into the workspace
    assert [g.plan_q4(64, 32, 4096, 64, config=c)["direct_lds"] for c in range(last + 1)] == [0] * (last - 2) + [1] * 2 + [0]
    for c in (last - 2, last - 1):
        assert call(config=c, a=at(0) + 2) == INVALID and call(config=c, k=255) == INVALID
    assert call(config=last, splits=2) == INVALID and call(config=last) == 7
    assert call(config=last, ws=at(4), size=2 * 32 * 256 - 1) == 7
    assert call(config=last, ws=at(4) + 8, size=2 * 32 * 256) == MISALIGNED
    for p in (at(0), at(1), at(2), at(3)):
        assert call(config=last, ws=p, size=2 * 32 * 256) == INVALID
    for c in range(last):
        need = g.plan_q4(4, 32, 4096, 64, config=c, splits=3)["workspace_bytes"]
        assert need == 3 * 4 * 32 * 4
        assert call(config=c, k=4096, splits=3) == 7
        assert call(config=c, k=4096, splits=3, ws=at(4), size=need - 1) == 7
        assert call(config=c, k=4096, splits=3, ws=at(4) + 8, size=need) == MISALIGNED
        for p in (at(0), at(1), at(2), at(3)):
            assert call(config=c, k=4096, splits=3, ws=p, size=need) == INVALID
    assert call(splits=-1) == INVALID and call(splits=65) == INVALID and call(ws=None, size=8) == INVALID
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
    last = g.q4_num_configs() - 1
    assert g.q4_config_name(last) == "q4_expanded"
    for m, n, k in [(1, 16, 128), (2048, 5001, 301), (1, 1, 1 << 22)]:
        p = g.plan_q4(m, n, k, 64, config=last)
        assert p["config"] == last and p["splits"] == 1 and p["workspace_bytes"] == 2 * n * k and p["flops"] == 2.0 * m * n * k
    assert g.plan_q4(2048, 8192, 8192, 64, splits=None)["config"] == last
    assert g.plan_q4(2048, 8192, 8192, 64, splits=1)["workspace_bytes"] == 0
    assert g.plan_q4(2047, 8192, 8192, 64, splits=None)["config"] < last
    assert g.plan_q4(4096, 8192, 0, 64, splits=None)["workspace_bytes"] == 0
    for c in range(last):
        assert g.q4_config_name(c)
        for m, n, k in [(1, 16, 128), (5, 1000, 4100), (64, 8192, 8192), (2048, 5000, 300), (1, 1, 1 << 22)]:
            p = g.plan_q4(m, n, k, 64, config=c)
            assert p["config"] == c and p["splits"] == 1 and p["workspace_bytes"] == 0 and p["lds_bytes"] <= 163840 and p["threads"] <= 1024
            assert p["tiles_m"] * p["block_m"] >= m and p["tiles_n"] * p["block_n"] >= n
            assert p["flops"] == 2.0 * m * n * k
    for m in (1, 16, 17, 33, 100, 300, 2000):
        for n, k in [(16, 128), (1000, 4100), (8192, 8192), (64, 100000)]:
            p = g.plan_q4(m, n, k, 64, splits=None)
            assert p["splits"] * p["k_split"] >= k and (p["splits"] - 1) * p["k_split"] < k
            assert p["workspace_bytes"] == (p["splits"] * m * n * 4 if p["splits"] > 1 else 0)
            assert g.plan_q4(m, n, k, 64, splits=1, A_ptr=2)["direct_lds"] == 0
            odd = g.plan_q4(m, n, k, 64, splits=None, A_ptr=2)     # from 16 rows A is copied to aligned rows
            if m >= 16:
                wide = g.plan_q4(m, n, -(-k // 8) * 8, 64, splits=None)
                copy = -(-2 * m * -(-k // 8) * 8 // 256) * 256
                assert odd["workspace_bytes"] == wide["workspace_bytes"] + copy and odd["config"] == wide["config"]
            else:
                assert odd["direct_lds"] == 0
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


def cache_struct(**over):
    from tiled_dense_gemm_fp16_amd.q4 import _CacheStruct
    f = {**dict(k_codes=at(10), k_words=at(11), v_codes=at(12), v_words=at(13), pages=4, heads=2, page_size=16, head_dim=128,
                group=64), **over}
    return _CacheStruct(*(f[n] for n, _ in _CacheStruct._fields_))


BAD_CACHES = [dict(k_codes=None), dict(k_words=None), dict(v_codes=None), dict(v_words=None), dict(pages=-1), dict(heads=0),
              dict(page_size=0), dict(page_size=12), dict(page_size=-8), dict(head_dim=96), dict(head_dim=0), dict(group=16),
              dict(head_dim=64, group=128)]
LARGE_CACHES = [dict(heads=4097), dict(page_size=(1 << 16) + 8), dict(pages=(1 << 30) + 1)]


def append(cache=None, batch=3, tokens=6, max_pages=2, k=at(0), ks=256, v=at(1), vs=256, table=at(2), lengths=at(3),
           starts=at(4), q=at(5), qs=512, out=at(6), heads=4, cos=at(7), sin=at(8), positions=32, rotary=128, inter=0):
    c = cache_struct() if cache is None else cache
    return g.lib().gemm_f16_q4_cache_append(ctypes.byref(c), batch, tokens, max_pages, k, ks, v, vs, table, lengths, starts, q, qs,
                                            out, heads, cos, sin, positions, rotary, inter, None)


def read(cache=None, batch=3, tokens=6, max_pages=2, table=at(2), first=at(3), starts=at(4), k=at(0), v=at(1)):
    c = cache_struct() if cache is None else cache
    return g.lib().gemm_f16_q4_cache_read(ctypes.byref(c), batch, tokens, max_pages, table, first, starts, k, v, None)


def attention(cache=None, batch=3, heads=4, max_pages=2, q=at(0), qs=512, table=at(1), lengths=at(2), out=at(3), splits=1,
              max_length=0, ws=None, size=0, scale=0.1):
    c = cache_struct() if cache is None else cache
    return g.lib().gemm_f16_q4_attention(ctypes.byref(c), batch, heads, max_pages, q, qs, table, lengths, scale, out, splits,
                                         max_length, ws, size, None)


@pytest.mark.parametrize("call", [append, read, attention])
def test_cache_refusals(call):
    for bad in BAD_CACHES:
        assert call(cache_struct(**bad)) == INVALID, bad
    for bad in LARGE_CACHES:
        assert call(cache_struct(**bad)) == SIZE, bad
    for bad in (dict(k_codes=at(10) + 8), dict(v_words=at(13) + 4)):
        assert call(cache_struct(**bad)) == MISALIGNED, bad
    assert call(batch=-1) == INVALID and call(max_pages=-1) == INVALID and call(batch=(1 << 20) + 1) == SIZE
    assert call(max_pages=1 << 27) == SIZE and call(table=None) == INVALID and call(table=at(2) + 2) == MISALIGNED
    assert call(batch=0) == 0 or call is not attention
    if not torch.cuda.is_available():
        assert call() == NO_DEVICE


def test_append_refusals():
    for bad in (dict(tokens=-1), dict(starts=None), dict(k=None), dict(v=None), dict(lengths=None), dict(ks=255), dict(vs=0),
                dict(qs=511), dict(q=None), dict(out=None), dict(heads=0), dict(cos=None), dict(sin=None), dict(rotary=8),
                dict(rotary=24), dict(rotary=144), dict(rotary=0), dict(positions=-1), dict(inter=2),
                dict(cos=None, sin=None, rotary=16), dict(out=at(0)), dict(out=at(1)), dict(out=at(5), qs=520),
                dict(out=at(5) + 2), dict(out=at(10)), dict(out=at(7)), dict(out=at(2)), dict(k=at(12)), dict(q=at(13)),
                dict(cache=cache_struct(v_codes=at(10)))):
        assert append(**bad) == INVALID, bad
    for bad in (dict(k=at(0) + 1), dict(q=at(5) + 1), dict(lengths=at(3) + 2), dict(starts=at(4) + 1), dict(cos=at(7) + 2)):
        assert append(**bad) == MISALIGNED, bad
    assert append(tokens=(1 << 26) + 1) == SIZE and append(heads=4097, qs=4097 * 128) == SIZE
    assert append(tokens=0) == 0 and append(batch=0) == 0
    if not torch.cuda.is_available():
        assert append(out=at(5)) == NO_DEVICE and append(batch=6, starts=None) == NO_DEVICE
        assert append(q=None, out=None, cos=None, sin=None, rotary=0) == NO_DEVICE


def test_read_refusals():
    for bad in (dict(tokens=-1), dict(k=None), dict(v=None), dict(starts=None), dict(k=at(1)), dict(k=at(10)), dict(v=at(2)),
                dict(v=at(4)), dict(k=at(3))):
        assert read(**bad) == INVALID, bad
    for bad in (dict(k=at(0) + 8), dict(v=at(1) + 2), dict(first=at(3) + 1), dict(starts=at(4) + 2)):
        assert read(**bad) == MISALIGNED, bad
    assert read(tokens=(1 << 26) + 1) == SIZE and read(tokens=0) == 0
    if not torch.cuda.is_available():
        assert read(first=None) == NO_DEVICE


def test_attention_refusals():
    for bad in (dict(heads=0), dict(heads=3), dict(heads=-2), dict(q=None), dict(out=None), dict(lengths=None), dict(qs=511),
                dict(splits=-1), dict(splits=257), dict(max_length=-1), dict(size=-1), dict(ws=None, size=4), dict(out=at(0)),
                dict(out=at(11)), dict(out=at(1)), dict(out=at(2)), dict(cache=cache_struct(pages=0)),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert attention(**bad) == INVALID, bad
    for bad in (dict(q=at(0) + 8), dict(qs=516), dict(out=at(3) + 8), dict(lengths=at(2) + 1)):
        assert attention(**bad) == MISALIGNED, bad
    need = g.plan_attention_q4(3, 4, 2, 128, 64, 32, 2)["workspace_bytes"]
    assert need == 3 * 4 * 2 * (128 + 2) * 4
    assert attention(splits=2) == 7 and attention(splits=2, ws=at(4), size=need - 1) == 7
    assert attention(splits=2, ws=at(4) + 4, size=need) == MISALIGNED
    assert attention(splits=2, ws=at(3), size=need) == INVALID and attention(splits=2, ws=at(13), size=need) == INVALID
    if not torch.cuda.is_available():
        assert attention(splits=2, ws=at(4), size=need) == NO_DEVICE and attention(max_pages=0, table=None) == NO_DEVICE


def test_attention_plans():
    for batch, heads, length in [(1, 1, 1), (1, 8, 131000), (64, 8, 4096), (0, 4, 10), (1, 2, 0)]:
        p = g.plan_attention_q4(batch, heads, heads, 128, 64, length)
        assert 1 <= p["splits"] <= 256 and p["lds_bytes"] <= 163840
        assert p["workspace_bytes"] == (batch * heads * p["splits"] * 130 * 4 if p["splits"] > 1 else 0)
    assert g.plan_attention_q4(1, 8, 8, 128, 64, 131000)["splits"] > 1
    assert g.plan_attention_q4(1, 8, 8, 128, 64, 100)["splits"] == 1
    for bad in ((1, 5, 2, 128, 64, 100), (1 << 20, 4096, 4096, 128, 64, 100), (1 << 20, 4096, 1, 128, 64, 100)):
        with pytest.raises(g.GemmError):       # heads that do not divide; launches of 2^32 work items
            g.plan_attention_q4(*bad)
    with pytest.raises(g.GemmError):
        g.plan_q4((1 << 31) - 1, 1 << 22, 128, config=g.q4_num_configs() - 2)


def test_cache_binding_refusals():
    with pytest.raises(ValueError):
        g.q4_cache(4, 2, 12, 128, device="cpu")
    with pytest.raises(ValueError):
        g.q4_cache(4, 2, 16, 64, 128, device="cpu")
    c = g.q4_cache(4, 2, 16, 128, device="cpu")
    i = torch.zeros(1, 1, dtype=torch.int32)
    q = torch.zeros(1, 2, 128, dtype=torch.float16)
    for fn in (lambda: g.attention_q4(q, c, i, i[0]), lambda: g.q4_cache_append(c, q, q, i, i[0]),
               lambda: g.q4_cache_read(c, i, torch.zeros(2, dtype=torch.int32), 1)):
        with pytest.raises(ValueError):
            fn()                                           # not on the GPU


def test_reference_cache_layout():
    # one token's key and value, by hand: d = 70 of 128 is dword 2 * 4 + ... of block 0 (j = 2, g = 0, i = 6)
    assert ref.key_place(70, 128) == 2 and ref.key_place(40, 64) == 3 and ref.key_place(200, 256) == 16 + 1 * 4 + 2
    codes = np.zeros((1, 1, 8, 16), np.uint32)
    codes[0, 0, 5, 2] = 9 << (4 * 3)                       # value 6 of the eight is nibble 3
    values = np.zeros((1, 1, 1, 16, 8), np.uint32)
    values[0, 0, 0, 70 % 16, 70 // 16] = 11 << (4 * 6)     # token 5 of the eight is nibble 6
    words = np.full((1, 1, 2, 8), 0x3C00, np.uint32)       # scale 1, zero point 0
    c = ref.Cache(codes, words, values, words, 64)
    k, v = c.values("k"), c.values("v")
    assert k[0, 5, 0, 70] == 9 and k.sum() == 9 and v[0, 5, 0, 70] == 11 and v.sum() == 11


def test_binding_refuses_any_object():
    """Every argument of every entry point replaced by something else, one at a time and all at once: an exception, never
    a crash (all of them lack a GPU tensor)."""
    cache, i = g.q4_cache(4, 2, 16, 128, device="cpu"), torch.zeros(1, 1, dtype=torch.int32)
    q = torch.zeros(1, 2, 128, dtype=torch.float16)
    w = g.Q4Matrix(torch.zeros(1, 1, 4, 16, 4, dtype=torch.int32), torch.zeros(1, 1, 16, 1, dtype=torch.int32), 16, 128, 128)
    turn, n = torch.zeros(64, 64), torch.zeros(2, dtype=torch.int32)
    junk = [None, 3, -1, 2 ** 70, 1.5, "x", [], (), {}, object(), torch.zeros(()), torch.zeros(2, 3).to_sparse(),
            torch.zeros(3, 3, 3, dtype=torch.float16, device="meta"), q.transpose(0, 1), q.to(torch.bfloat16), w, cache,
            g.Q4Matrix(*"abcde"), g.Q4Matrix(w.codes, w.words, -5, 2 ** 62, 128), g.Q4Matrix(w.codes, w.words, 2 ** 62, 1, 32),
            g.Q4Cache(*"abcde"), g.Q4Cache(i, i, i, i, 64), tuple.__new__(g.Q4Matrix, (1,)), tuple.__new__(g.Q4Cache, ())]
    calls = [(g.q4_compress, [q[0]], {"group": 64, "symmetric": False}), (g.q4_expand, [w], {"out": q[0]}),
             (g.gemm_q4, [q[0], w], {"epilogue": "none", "out": q[0], "config": 0, "splits": 1, "workspace": q, "alpha": 1.0}),
             (g.q4_cache_append, [cache, q, q, i, i[0]], {"starts": n, "q": q, "cos": turn, "sin": turn, "interleaved": True,
                                                          "out": q}),
             (g.q4_cache_read, [cache, i, n, 1], {"first": i[0]}),
             (g.attention_q4, [q, cache, i, i[0]], {"scale": 1.0, "out": q, "splits": 2, "workspace": q, "max_length": 8})]
    refused = (ValueError, TypeError, OverflowError, RuntimeError)
    for fn, args, kw in calls:
        with pytest.raises(ValueError):
            fn(*args, **kw)
        for x in junk:
            for at in range(len(args)):
                with pytest.raises(refused):
                    fn(*args[:at], x, *args[at + 1:], **kw)
            for name in kw:
                with pytest.raises(refused):
                    fn(*args, **{**kw, name: x})
            with pytest.raises(refused):
                fn(*[x] * len(args))
