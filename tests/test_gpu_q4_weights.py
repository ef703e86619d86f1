"""GPU tests of 4-bit weights: compression, expansion and the product.

Compression and expansion are sequences of single correctly rounded
operations, so they must equal tests/q4_reference.py bit for bit.

The product's error against 64 bits: one rounding to binary16 (half a step)
and fp32 sums.  A product a (q - z) is exact in fp32; it passes through at
most 32 additions inside one matrix instruction, at most 3 further ones of its
group, one per group of its wave's share of K, 8 across the waves, and the
products with s and alpha: D = 32 + 3 + K / group + 8 + 2 roundings, each of at
most 2^-23 of the sum of magnitudes (2^-24 for a rounding to nearest, twice
that in case the matrix unit truncates).  (A split adds fewer than it takes
off a wave's share.)  The configurations that round the weights to binary16
add half a step of each: 2^-11 of the sum of magnitudes (no weight here is
below binary16's normals); their sums run through the matrix unit alone, one
addition for every 32 of K in the place of one for every group.
"""
import numpy as np
import pytest
import torch

import q4_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weights(n, k, seed):
    return (torch.randn(n, k, generator=gen(seed)) * (1.0 + torch.rand(n, 1, generator=gen(seed + 1)))).to(torch.float16)


def bound(c, size, k, group, rounded=False):
    depth = 45 + -(-k // (32 if rounded else group))
    return ref.half_steps(c) * (1 + 2.0 ** -10) + (depth * 2.0 ** -23 + (2.0 ** -11 if rounded else 0.0)) * size


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("n,k", [(1, 1), (16, 128), (17, 129), (5, 300), (40, 1000), (33, 96)])
def test_compress_and_expand_bit_exact(n, k, group, symmetric):
    print(f"[q4] compress {n}x{k} group={group} symmetric={symmetric}", flush=True)
    w = weights(n, k, n + k)
    packed = g.q4_compress(w.to(DEV), group, symmetric=symmetric)
    back = g.q4_expand(packed)
    torch.cuda.synchronize()
    codes, words = ref.pack_weights(w.float().numpy(), group, symmetric)
    assert np.array_equal(ref.host(packed.words).view(np.uint32), words)
    assert np.array_equal(ref.host(packed.codes).view(np.uint32), codes)
    want = ref.unpack_weights(codes, words, n, k, group).astype(np.float16)
    assert np.array_equal(ref.host(back), want)


def test_compress_special_values():
    w = torch.zeros(16, 256, dtype=torch.float16)
    w[0, 3] = float("nan")
    w[0, 4] = 3.0
    w[1, 0], w[1, 1] = float("inf"), -2.0
    w[2, 7] = float("-inf")
    w[3, 0], w[3, 1] = 65504.0, -65504.0
    w[4, 0] = 2.0 ** -24          # the scale underflows to 0: the group is held as zeros
    w[5, :128] = 1.5              # one sign only
    w[6, :128] = -1.5
    w[7, :128] = -0.0
    w[8, :15] = torch.arange(15).to(torch.float16) + 0.5    # ties
    for symmetric in (False, True):
        packed = g.q4_compress(w.to(DEV), 128, symmetric=symmetric)
        back = ref.host(g.q4_expand(packed))
        codes, words = ref.pack_weights(w.float().numpy(), 128, symmetric)
        assert np.array_equal(ref.host(packed.words).view(np.uint32), words)
        assert np.array_equal(ref.host(packed.codes).view(np.uint32), codes)
        with np.errstate(over="ignore"):
            want = ref.unpack_weights(codes, words, 16, 256, 128).astype(np.float16)
        assert np.array_equal(back, want)


def test_compress_unaligned_source():
    buf = torch.empty(24 * 136 + 1, dtype=torch.float16, device=DEV)
    w = weights(24, 136, 3)
    at = buf[1:].view(24, 136)
    at.copy_(w)
    packed = g.q4_compress(at, 64)
    codes, words = ref.pack_weights(w.float().numpy(), 64)
    assert np.array_equal(ref.host(packed.codes).view(np.uint32), codes)
    out = torch.full((24 * 136 + 3,), 7.0, dtype=torch.float16, device=DEV)
    g.q4_expand(packed, out=out[1:-2].view(24, 136))
    want = ref.unpack_weights(codes, words, 24, 136, 64).astype(np.float16)
    assert np.array_equal(ref.host(out[1:-2]).reshape(24, 136), want)
    assert bool((out[:1] == 7).all()) and bool((out[-2:] == 7).all())


EXPANDED = g.q4_num_configs() - 1              # W expanded, then the dense product: no split of K
ROUNDED = (EXPANDED - 1, EXPANDED)             # the configurations that round the weights


def check(m, n, k, group, config=g.CONFIG_AUTO, epilogue="none", alpha=1.0, shift=0, seed=0, splits=None):
    a = torch.randn(m, k, generator=gen(seed + 5)).to(torch.float16)
    packed = g.q4_compress(weights(n, k, seed).to(DEV), group)
    room = torch.full((m * n + 2 * 64 + shift,), 9.0, dtype=torch.float16, device=DEV)
    out = room[64 + shift:64 + shift + m * n].view(m, n)
    buf = torch.empty(m * k + shift, dtype=torch.float16, device=DEV)
    ad = buf[shift:].view(m, k)
    ad.copy_(a)
    got = g.gemm_q4(ad, packed, epilogue=epilogue, out=out, config=config, alpha=alpha, splits=splits)
    torch.cuda.synchronize()
    print(f"[q4] product {m}x{n}x{k} group={group} config={config} epi={epilogue} alpha={alpha} shift={shift}", flush=True)
    w = ref.unpack_weights(ref.host(packed.codes), ref.host(packed.words), n, k, group)
    want, size = ref.product(a.double().numpy(), w, float(np.float32(alpha)), epilogue == "relu")
    err = np.abs(ref.host(got).astype(np.float64) - want)
    chosen = g.plan_q4(m, n, k, group, config, splits, ad.data_ptr())["config"]
    tol = bound(want, size, k, group, chosen in ROUNDED)
    assert (err <= tol).all(), (err / tol).max()
    assert bool((room[:64 + shift] == 9).all()) and bool((room[64 + shift + m * n:] == 9).all())


@pytest.mark.parametrize("config", range(g.q4_num_configs()))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 16, 128), (1, 100, 2048), (3, 33, 1000), (16, 16, 1024), (17, 70, 1030),
                                   (33, 48, 520), (64, 64, 256), (65, 40, 4100), (130, 264, 136)])
def test_every_config(config, group, m, n, k):
    if k % 2 and g.plan_q4(m, n, k + 1, group, config=config)["direct_lds"]:
        with pytest.raises(g.GemmError):                # rows of odd length: not for the tile configurations
            check(m, n, k, group, config=config)
        return
    check(m, n, k, group, config=config, seed=m + n + k)


@pytest.mark.parametrize("config", range(EXPANDED))
@pytest.mark.parametrize("m,n,k,splits", [(1, 16, 384, 3), (70, 140, 1030, 2), (64, 128, 4100, 7), (130, 300, 2048, 64),
                                          (129, 257, 132, 2), (300, 520, 514, None)])
def test_splits(config, m, n, k, splits):
    check(m, n, k, 32, config=config, splits=splits, epilogue="relu", alpha=0.7)
    check(m, n, k, 128, config=config, splits=splits)


@pytest.mark.parametrize("config", range(g.q4_num_configs()))
def test_last_chunk_keeps_to_its_row(config):
    # infinities at the start of every row: the row before ends inside a 16-byte chunk that holds them
    for k in (130, 132, 262, 646):
        a = torch.randn(70, k, generator=gen(k)).to(torch.float16)
        a[1::2, 0] = float("inf")
        packed = g.q4_compress(weights(48, k, k).to(DEV), 64)
        got = ref.host(g.gemm_q4(a.to(DEV), packed, config=config)).astype(np.float64)
        w = ref.unpack_weights(ref.host(packed.codes), ref.host(packed.words), 48, k, 64)
        want, size = ref.product(a[::2].double().numpy(), w)
        assert (np.abs(got[::2] - want) <= bound(want, size, k, 64, config in ROUNDED)).all()
        assert not np.isfinite(got[1::2]).any() or (w[:, 0] == 0).any()


@pytest.mark.parametrize("m,n,k", [(1, 1024, 1024), (2, 5000, 4100), (13, 256, 8192), (40, 600, 3000), (300, 300, 300),
                                   (70, 64, 9000), (520, 700, 1000), (3, 70, 16500), (300, 5000, 300), (40, 9000, 520)])
@pytest.mark.parametrize("epilogue,alpha", [("none", 1.0), ("relu", 0.125), ("none", -1.7)])
def test_automatic_choice(m, n, k, epilogue, alpha):
    check(m, n, k, 64, epilogue=epilogue, alpha=alpha)


@pytest.mark.parametrize("n,k,shift", [(520, 1024, 0), (33, 300, 0), (48, 129, 1), (1, 1, 0)])
def test_many_rows(n, k, shift):
    """From 2048 rows W is expanded into the workspace; not with splits=1."""
    chosen = [g.plan_q4(2050, n, k, 64, splits=s, A_ptr=2 * shift)["config"] for s in (None, 1)]
    assert chosen[0] == EXPANDED and chosen[1] < EXPANDED
    for splits in (None, 1):
        check(2050, n, k, 64, epilogue="relu", alpha=0.3, shift=shift, splits=splits)
    w = g.q4_compress(weights(n, k, 0).to(DEV), 64)
    a = torch.randn(2050, k, generator=gen(1)).to(torch.float16).to(DEV)
    want = g.gemm_q4(a, w, alpha=0.3)
    if k % 2 == 0:
        assert torch.equal(want, g.gemm(a, g.q4_expand(w), trans_b=True, alpha=0.3, splits=1))
    need = g.plan_q4(2050, n, k, 64, splits=None)["workspace_bytes"]
    room = torch.full((need + 32,), 85, dtype=torch.uint8, device=DEV)
    assert torch.equal(g.gemm_q4(a, w, alpha=0.3, workspace=room[16:-16]), want)
    assert bool((room[:16] == 85).all()) and bool((room[-16:] == 85).all())
    with pytest.raises(g.GemmError):
        g.gemm_q4(a, w, workspace=room[16:-17])


@pytest.mark.parametrize("m,n,k,shift", [(16, 40, 129, 0), (17, 264, 1001, 1), (40, 9000, 300, 1), (33, 48, 8193, 0), (300, 520, 2047, 0),
                                         (70, 300, 8, 1), (130, 16400, 33, 3), (20, 30, 1, 0), (9, 40, 4099, 0)])
def test_rows_of_odd_length(m, n, k, shift):
    """From 16 rows (8 over long K) A is copied to aligned rows; not with splits=1 or a configuration."""
    for group, splits in ((32, None), (128, None), (64, 1)):
        check(m, n, k, group, shift=shift, splits=splits, epilogue="relu", alpha=0.7)
    w = g.q4_compress(weights(n, k, 0).to(DEV), 64)
    a = torch.randn(m, k, generator=gen(1)).to(torch.float16).to(DEV)
    if k % 2:
        need = g.plan_q4(m, n, k, 64, splits=None)["workspace_bytes"]
        assert need >= 2 * m * k
        room = torch.full((need + 32,), 255, dtype=torch.uint8, device=DEV)          # NaN: all that is read was written
        assert torch.equal(g.gemm_q4(a, w, workspace=room[16:-16]), g.gemm_q4(a, w))
        assert bool((room[:16] == 255).all()) and bool((room[-16:] == 255).all())
    a[1::2] = float("inf")                            # rows do not reach into each other
    got, clean = g.gemm_q4(a, w), g.gemm_q4(torch.where(a.isinf(), torch.zeros_like(a), a), w)
    assert torch.equal(got[::2], clean[::2])


def test_unaligned_pointers():
    check(5, 40, 264, 32, shift=1)
    check(20, 40, 264, 128, shift=3)
    check(33, 40, 261, 64, shift=1)


def test_long_k():
    check(1, 20, 70000, 128)
    check(18, 20, 40000, 64)


def test_empty_and_zero_depth():
    packed = g.q4_compress(torch.zeros(8, 0, dtype=torch.float16, device=DEV))
    out = torch.full((3, 8), 5.0, dtype=torch.float16, device=DEV)
    g.gemm_q4(torch.zeros(3, 0, dtype=torch.float16, device=DEV), packed, out=out, alpha=-1.0)
    assert bool((out.view(torch.int16) == 0).all())
    packed = g.q4_compress(weights(8, 128, 1).to(DEV))
    assert g.gemm_q4(torch.zeros(0, 128, dtype=torch.float16, device=DEV), packed).shape == (0, 8)
    packed = g.q4_compress(torch.zeros(0, 128, dtype=torch.float16, device=DEV))
    assert g.gemm_q4(torch.zeros(2, 128, dtype=torch.float16, device=DEV), packed).shape == (2, 0)
    assert g.q4_expand(packed).shape == (0, 128)


def test_infinite_rows_stay_in_their_row():
    a = torch.ones(20, 256, dtype=torch.float16)
    a[3, 5] = float("inf")
    a[7, 200] = float("nan")
    packed = g.q4_compress(weights(40, 256, 2).to(DEV))
    got = ref.host(g.gemm_q4(a.to(DEV), packed))
    fine = np.ones(20, bool)
    fine[[3, 7]] = False
    assert np.isfinite(got[fine]).all()
    assert np.isnan(got[7]).all() and not np.isfinite(got[3]).any()
