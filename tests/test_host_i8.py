"""CPU tests of the 8-bit and expert entry points: exported symbols, refusals and plans (validation runs before any HIP
call, so no kernel is launched here), and the reference the GPU tests compare with."""
import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import i8_reference as ref
import tiled_dense_gemm_fp16_amd as g

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_f16_i8.h")

FAKE = 1 << 40          # aligned, never dereferenced; buffers a GiB or more apart
INVALID, MISALIGNED, NO_DEVICE, SIZE, WORKSPACE = 1, 2, 3, 6, 7
NAN, INF = float("nan"), float("inf")


def at(i):
    return FAKE + (i << 36)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(g.LIB_PATH) or not os.path.exists(g.I8_BINDING_PATH):
        import __graft_entry__
        __graft_entry__.build()


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gemm_f16\w*)\s*\(", text))
    lib = ctypes.CDLL(g.LIB_PATH)
    for name in names:
        assert hasattr(lib, name), name
    assert set(g.I8_SIGNATURES) == names


def test_pitch():
    h = g.lib()
    for k in (0, 1, 16, 17, 64, 65, 128, 129, 4100, 131071):
        assert h.gemm_f16_i8_pitch(k) == ref.pitch(k)
    assert h.gemm_f16_i8_pitch(-1) == -1 and h.gemm_f16_i8_pitch(1 << 17) == -1


def test_rows_refusals():
    h = g.lib()

    def compress(rows=4, k=100, x=at(0), stride=100, codes=at(1), scales=at(2)):
        return h.gemm_f16_i8_compress(rows, k, x, stride, codes, scales, None)

    def expand(rows=4, k=100, x=at(0), pitch=112, codes=at(1), scales=at(2)):
        return h.gemm_f16_i8_expand(rows, k, codes, pitch, scales, x, None)

    for fn in (compress, expand):
        for bad in (dict(rows=-1), dict(k=-1), dict(x=None), dict(codes=None), dict(scales=None), dict(x=at(1)), dict(x=at(2)),
                    dict(x=at(1) + 4 * 112 - 2), dict(rows=1, x=at(1) + 110)):
            assert fn(**bad) == INVALID, bad
        for bad in (dict(x=at(0) + 1), dict(codes=at(1) + 8), dict(scales=at(2) + 2)):
            assert fn(**bad) == MISALIGNED, bad
        assert fn(rows=1 << 31) == SIZE and fn(k=1 << 17) == SIZE
        assert fn(rows=0, x=None, codes=None, scales=None) == 0
    assert compress(stride=99) == INVALID and compress(scales=at(1)) == INVALID
    assert compress(stride=1 << 60) == SIZE and compress(rows=1 << 30, stride=1 << 40) == SIZE
    assert expand(pitch=96) == INVALID and expand(pitch=120) == INVALID and expand(pitch=(1 << 22) + 16) == SIZE
    if not torch.cuda.is_available():
        assert compress() == NO_DEVICE and expand() == NO_DEVICE and expand(pitch=4096) == NO_DEVICE
        assert compress(rows=2, x=at(0), codes=at(0) + 400) == NO_DEVICE     # right behind


def test_product_refusals():
    h = g.lib()

    def call(m=4, n=32, k=250, a=at(0), ap=256, sa=at(1), w=at(2), wp=256, sw=at(3), c=at(4), epi=0, config=-1, splits=1, ws=None,
             size=0):
        return h.gemm_f16_i8(m, n, k, a, ap, sa, w, wp, sw, c, 1.0, epi, config, splits, ws, size, None)

    for bad in (dict(m=-1), dict(n=-1), dict(k=-1), dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(c=None), dict(epi=2),
                dict(epi=-1), dict(config=g.i8_num_configs()), dict(config=-2), dict(splits=-1), dict(splits=65), dict(ap=240),
                dict(wp=240), dict(ap=264), dict(wp=260), dict(c=at(0)), dict(c=at(1)), dict(c=at(2) + 64), dict(c=at(3)),
                dict(c=at(0) + 4 * 256 - 2), dict(ws=at(5), size=-1), dict(size=8)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(a=at(0) + 8), dict(w=at(2) + 4), dict(sa=at(1) + 2), dict(sw=at(3) + 1), dict(c=at(4) + 1)):
        assert call(**bad) == MISALIGNED, bad
    for bad in (dict(m=1 << 31), dict(n=(1 << 22) + 1), dict(k=1 << 17), dict(ap=(1 << 22) + 16), dict(wp=(1 << 22) + 16)):
        assert call(**bad) == SIZE, bad
    for c in range(g.i8_num_configs()):
        need = g.plan_i8(4, 32, 4096, config=c, splits=3)["workspace_bytes"]
        big = dict(config=c, k=4096, ap=4096, wp=4096, splits=3)
        assert need == 3 * 4 * 32 * 4
        assert call(**big) == WORKSPACE and call(**big, ws=at(5), size=need - 1) == WORKSPACE
        assert call(**big, ws=at(5) + 8, size=need) == MISALIGNED
        for p in (at(0), at(1), at(2), at(3), at(4)):
            assert call(**big, ws=p, size=need) == INVALID
        assert call(config=c, splits=2, n=(1 << 20) + 1, k=4096, ap=4096, wp=4096, ws=at(5), size=1 << 40) == SIZE
    assert call(m=0, a=None, sa=None, c=None) == 0 and call(n=0, w=None, sw=None, c=None) == 0
    if not torch.cuda.is_available():
        assert call() == NO_DEVICE and call(k=0, a=None, w=None) == NO_DEVICE and call(c=at(0) + 4 * 256) == NO_DEVICE


def test_route_refusals():
    h = g.lib()

    def call(t=4, e=64, k=6, x=at(0), half=0, stride=64, score=0, bias=None, groups=1, top=1, renorm=0, scale=1.0, ids=at(1), w=at(2)):
        return h.gemm_f16_route(t, e, k, x, half, stride, score, bias, groups, top, renorm, scale, ids, w, None)

    for bad in (dict(t=-1), dict(e=0), dict(k=0), dict(k=65), dict(e=5), dict(x=None), dict(ids=None), dict(w=None), dict(half=2),
                dict(score=2), dict(score=-1), dict(groups=0), dict(groups=5), dict(groups=4, top=5), dict(groups=4, top=0), dict(renorm=2),
                dict(scale=NAN), dict(scale=INF), dict(stride=63), dict(w=at(1)), dict(ids=at(0)), dict(w=at(0) + 4 * 64 * 4 - 4),
                dict(bias=at(1)), dict(bias=at(2))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(x=at(0) + 2), dict(x=at(0) + 1, half=1), dict(ids=at(1) + 2), dict(w=at(2) + 1), dict(bias=at(3) + 2)):
        assert call(**bad) == MISALIGNED, bad
    for bad in (dict(e=1025, stride=2000), dict(e=128, stride=128, k=65), dict(e=260, stride=260, groups=65), dict(t=1 << 25, k=1),
                dict(t=1 << 22, stride=1 << 50)):
        assert call(**bad) == SIZE, bad
    assert call(t=0, x=None, ids=None, w=None) == 0
    if not torch.cuda.is_available():
        assert call() == NO_DEVICE and call(half=1, x=at(0) + 2, bias=at(3), groups=8, top=4) == NO_DEVICE


def test_order_and_sum_refusals():
    h = g.lib()

    def order(p=24, e=8, ids=at(0), to=at(1), starts=at(2)):
        return h.gemm_f16_expert_order(p, e, ids, to, starts, None)

    for bad in (dict(p=-1), dict(e=0), dict(ids=None), dict(to=None), dict(starts=None), dict(to=at(0)), dict(starts=at(0) + 92),
                dict(starts=at(1))):
        assert order(**bad) == INVALID, bad
    for bad in (dict(ids=at(0) + 2), dict(to=at(1) + 1), dict(starts=at(2) + 2)):
        assert order(**bad) == MISALIGNED, bad
    assert order(p=1 << 25) == SIZE and order(e=1025) == SIZE

    def add(t=4, k=6, n=100, y=at(0), w=at(1), out=at(2)):
        return h.gemm_f16_expert_sum(t, k, n, y, w, out, None)

    for bad in (dict(t=-1), dict(k=-1), dict(n=-1), dict(y=None), dict(w=None), dict(out=None), dict(out=at(0)), dict(out=at(1))):
        assert add(**bad) == INVALID, bad
    for bad in (dict(y=at(0) + 1), dict(w=at(1) + 2), dict(out=at(2) + 1)):
        assert add(**bad) == MISALIGNED, bad
    assert add(n=(1 << 22) + 1) == SIZE and add(k=1025) == SIZE and add(t=1 << 25) == SIZE
    assert add(t=0, y=None, out=None) == 0 and add(n=0, y=None, out=None) == 0
    if not torch.cuda.is_available():
        assert order() == NO_DEVICE and order(p=0, ids=None, to=None) == NO_DEVICE
        assert add() == NO_DEVICE and add(k=0, y=None, w=None) == NO_DEVICE


def test_experts_refusals():
    h = g.lib()

    def call(p=24, per=6, e=8, n=32, k=250, a=at(0), ap=256, sa=at(1), w=at(2), wp=256, sw=at(3), order=at(4), starts=at(5), c=at(6),
             epi=0, config=-1):
        return h.gemm_f16_i8_experts(p, per, e, n, k, a, ap, sa, w, wp, sw, order, starts, c, 1.0, epi, config, None)

    for bad in (dict(p=-1), dict(per=0), dict(per=5), dict(e=0), dict(n=-1), dict(k=-1), dict(a=None), dict(sa=None), dict(w=None),
                dict(sw=None), dict(order=None), dict(starts=None), dict(c=None), dict(epi=2), dict(config=g.i8_num_configs()),
                dict(config=-2), dict(ap=240), dict(wp=264), dict(c=at(0)), dict(c=at(1)), dict(c=at(2) + 8 * 32 * 256 - 2), dict(c=at(3)),
                dict(c=at(4)), dict(c=at(5) + 32)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(a=at(0) + 8), dict(w=at(2) + 4), dict(sa=at(1) + 2), dict(sw=at(3) + 1), dict(order=at(4) + 2), dict(starts=at(5) + 1),
                dict(c=at(6) + 1)):
        assert call(**bad) == MISALIGNED, bad
    for bad in (dict(p=1 << 25, per=1), dict(e=1025), dict(n=(1 << 22) + 1), dict(k=1 << 17), dict(p=1 << 23, per=1),
                dict(ap=(1 << 22) + 16)):
        assert call(**bad) == SIZE, bad
    assert call(p=0) == 0 and call(n=0, w=None, sw=None, c=None) == 0
    if not torch.cuda.is_available():
        assert call() == NO_DEVICE and call(per=1) == NO_DEVICE and call(per=24) == NO_DEVICE


def test_plans():
    for c in range(g.i8_num_configs()):
        assert g.i8_config_name(c)
        for m, n, k in [(1, 16, 128), (5, 1000, 4100), (64, 8192, 8192), (2048, 5000, 300), (1, 1, 131071), (7, 5, 0)]:
            p = g.plan_i8(m, n, k, config=c)
            assert p["config"] == c and p["splits"] == 1 and p["workspace_bytes"] == 0
            assert p["lds_bytes"] <= 163840 - 4 * p["block_m"] and p["threads"] <= 1024
            assert p["tiles_m"] * p["block_m"] >= m and p["tiles_n"] * p["block_n"] >= n
            tiles = p["tiles_m"] * p["tiles_n"]
            if p["block_m"] * p["block_n"] == 256 * 256 and 0 < tiles % 256 <= 128:    # cut in four for a last round
                assert p["grid"] == tiles - tiles % 256 + 4 * 8 * -(-(tiles % 256) // 8)
            else:
                assert p["grid"] == tiles
            assert p["flops"] == 2.0 * m * n * k
        for splits in (None, 2, 7, 64):
            for m, n, k in [(16, 128, 4100), (300, 520, 8192), (3, 40, 130), (200, 300, 100000)]:
                p = g.plan_i8(m, n, k, config=c, splits=splits)
                assert p["splits"] * p["k_split"] >= k and (p["splits"] - 1) * p["k_split"] < k
                assert p["splits"] == 1 or p["k_split"] % p["block_k"] == 0
                assert p["workspace_bytes"] == (p["splits"] * m * n * 4 if p["splits"] > 1 else 0)
        for pairs, per, e, n, k in [(8, 8, 256, 2048, 4096), (512, 1, 256, 100, 100), (16384, 8, 64, 2048, 4096), (1, 1, 1, 1, 1)]:
            p = g.plan_i8_experts(pairs, per, e, n, k, config=c)
            counts = [pairs // e + (i < pairs % e) for i in range(e)]
            for split in (counts, [pairs], [1] * (min(pairs, e + 1) - 1) + [pairs - min(pairs, e + 1) + 1]):
                assert sum(-(-x // p["block_m"]) for x in split) <= p["tiles_m"]
            assert p["tiles_m"] <= pairs and p["grid"] >= p["tiles_m"] * p["tiles_n"]
    for m in (1, 2, 16, 17, 33, 64, 100, 300, 2000, 8192):
        for n, k in [(16, 128), (1000, 4100), (8192, 8192), (64, 100000), (28672, 8192)]:
            p = g.plan_i8(m, n, k, splits=None)
            assert p["splits"] * p["k_split"] >= k
    assert g.i8_config_name(-1) is None and g.i8_config_name(g.i8_num_configs()) is None
    # as many rows as a call may have: a tile that makes few enough workgroups
    assert g.plan_i8((1 << 31) - 1, 16, 64, splits=None)["block_m"] == 256
    assert g.plan_i8_experts((1 << 25) - 1, 1, 8, 4096, 64)["grid"] < 1 << 24
    for bad in (dict(m=-1), dict(k=1 << 17), dict(config=99), dict(splits=65)):
        with pytest.raises(g.GemmError):
            g.plan_i8(**{**dict(m=1, n=16, k=128), **bad})


def test_python_refusals_without_a_gpu():
    x = torch.zeros(4, 32, dtype=torch.float16)
    for bad in (lambda: g.i8_compress(x), lambda: g.i8_compress(x.float()), lambda: g.i8_compress(None), lambda: g.i8_compress(x[0]),
                lambda: g.i8_expand(x), lambda: g.gemm_i8(x, x), lambda: g.gemm_i8(x, x, epilogue="gelu"),
                lambda: g.route(x, 2), lambda: g.route(x, 2, score="top"), lambda: g.expert_order(x, 4),
                lambda: g.expert_sum(x, x), lambda: g.gemm_i8_experts(x, x, x),
                lambda: g.gemm_i8(g.I8Matrix(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4), 32), None)):
        with pytest.raises(ValueError):
            bad()


def test_reference_codes_against_rationals():
    gen = np.random.default_rng(5)
    x = gen.normal(size=(40, 24)).astype(np.float16)
    x[:, 1] = x[:, 0] / 2
    x[3] *= np.float16(2.0 ** -14)
    codes, scales = ref.compress(x)
    for row, c, s in zip(x, codes, scales):
        most = max(abs(Fraction(float(v))) for v in row)
        for v, q in zip(row, c):
            ratio = 127 * Fraction(float(v)) / most
            assert abs(ratio - int(q)) <= Fraction(1, 2) and (abs(ratio - int(q)) < Fraction(1, 2) or q % 2 == 0)
        assert abs(Fraction(float(s)) - most / 127) <= abs(most / 127) * Fraction(1, 1 << 24)
    assert (codes[:, 24:] == 0).all()


def test_reference_route_against_torch():
    x = torch.randn(50, 32, generator=torch.Generator().manual_seed(1)).double()
    ids, weights = ref.route(x.numpy(), 4, "softmax")
    want = torch.softmax(x, 1).topk(4)
    assert np.array_equal(ids, want[1].numpy()) and np.allclose(weights, want[0].numpy(), rtol=1e-14)
    ids, _ = ref.route(x.numpy(), 4, "sigmoid", groups=8, top_groups=3)
    best = torch.sigmoid(x).view(50, 8, 4).topk(2)[0].sum(-1).topk(3)[1]
    stay = torch.zeros(50, 8, dtype=torch.bool).scatter_(1, best, True).repeat_interleave(4, 1)
    assert np.array_equal(ids, x.masked_fill(~stay, -INF).topk(4)[1].numpy())
