"""GPU tests that the product with 4-bit weights uses s (q - z) exactly, whatever
the number of rows, in every configuration but the expanded one, which rounds
each weight to binary16 (and is chosen from 2048 rows with groups of 32 and 64
where the caller allows a workspace).

Rows of A hold 1 at one k and -1 at another.  s has 11 bits and q - z at most 4
and a sign, so a product has 15 bits; the two weights of a row's difference lie
within 8 binary exponents of each other, so every sum of the chain (products of
a group, groups, waves, parts) is exact in fp32 and the result is the exact
difference, rounded once: equality, no tolerance.  Rounding the weights first
changes most of the differences.
"""
import numpy as np
import pytest
import torch

import q4_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EXPANDED = g.q4_num_configs() - 1


def gen(seed):
    return torch.Generator().manual_seed(seed)


def setup(m, n, k, group, seed):
    """A of differences, packed weights, and the results as binary16."""
    # magnitudes in [1/2, 4): within a group of such values (hi - lo) / 15 lies in [1/30, 8/15], so s (q - z), a
    # multiple of s 2^-10 at most 15 s, stays within 2^-15 .. 8: 24 bits hold every difference
    w = (torch.rand(n, k, generator=gen(seed)) * 3.5 + 0.5) * torch.randint(0, 2, (n, k), generator=gen(seed + 1)).mul(2).sub(1)
    packed = g.q4_compress(w.to(torch.float16).to(DEV), group)
    rows = torch.arange(m)
    one = torch.randint(0, k, (m,), generator=gen(seed + 2))
    two = (one + 1 + torch.randint(0, k - 1, (m,), generator=gen(seed + 3))) % k
    a = torch.zeros(m, k, dtype=torch.float16)
    a[rows, one], a[rows, two] = 1.0, -1.0
    dense = ref.unpack_weights(ref.host(packed.codes), ref.host(packed.words), n, k, group)
    want = (dense[:, one.numpy()] - dense[:, two.numpy()]).T
    return a.to(DEV), packed, want.astype(np.float16), dense, (one.numpy(), two.numpy())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("config", range(EXPANDED))
def test_every_exact_config(config, group):
    for m, n, k in [(1, 70, 520), (70, 300, 1030), (200, 520, 256)]:
        print(f"[q4] exact config={config} group={group} {m}x{n}x{k}", flush=True)
        a, packed, want, _, _ = setup(m, n, k, group, m + config)
        for splits in (1, 2):
            assert np.array_equal(ref.host(g.gemm_q4(a, packed, config=config, splits=splits)), want)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 300, 384), (17, 300, 384), (40, 300, 1024), (130, 16500, 256), (1100, 6000, 384),
                                   (2050, 2100, 264), (2050, 40, 512), (2050, 64, 2056), (2500, 300, 4096)])
def test_automatic_choice_is_exact(m, n, k, group):
    a, packed, want, dense, (one, two) = setup(m, n, k, group, m)
    assert np.array_equal(ref.host(g.gemm_q4(a, packed, splits=1)), want)
    if g.plan_q4(m, n, k, group, splits=None)["config"] < EXPANDED:
        assert np.array_equal(ref.host(g.gemm_q4(a, packed)), want)
    else:                                       # the one choice that rounds: not below 2048 rows nor with groups of 128
        assert m >= 2048 and group < 128
        rounded = dense.astype(np.float16).astype(np.float64)
        got = ref.host(g.gemm_q4(a, packed))
        assert np.array_equal(got, (rounded[:, one] - rounded[:, two]).T.astype(np.float16))
        assert not np.array_equal(got, want)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_scales_whose_largest_value_passes_binary16(group):
    # a group of 0 .. 65504 is held with s = 4368, whose 15 s is 65520; its sums are finite for any number of rows
    n, k = 2100, 256
    w = torch.rand(n, k, generator=gen(1)).mul(0.01).to(torch.float16)
    w[:, :group] = 0.0
    w[:, 3], w[:, 5] = 65504.0, 1000.0
    packed = g.q4_compress(w.to(DEV), group)
    dense = ref.unpack_weights(ref.host(packed.codes), ref.host(packed.words), n, k, group)
    assert dense[0, 3] == 65520.0
    for m in (1, 40, 200, 1100, 2050):
        a = torch.zeros(m, k, dtype=torch.float16)
        a[:, 3] = 2.0 ** -10
        a[:, 5] = 1.0
        want = (dense[:, 3] * 2.0 ** -10 + dense[:, 5])[None].repeat(m, 0).astype(np.float16)
        for splits in (1, None):
            if splits == 1 or g.plan_q4(m, n, k, group, splits=splits)["config"] < EXPANDED:
                assert np.array_equal(ref.host(g.gemm_q4(a.to(DEV), packed, splits=splits)), want), (m, splits)


def test_no_room_for_the_expanded_weights():
    """A product whose automatic workspace the allocator cannot give runs without one."""
    m, n, k = 2048, 16384, 16384
    assert g.plan_q4(m, n, k, 64, splits=None)["workspace_bytes"] == 2 * n * k
    packed = g.q4_compress(torch.randn(n, k, generator=torch.Generator(DEV).manual_seed(0), device=DEV, dtype=torch.float16), 64)
    a = torch.randn(m, k, generator=torch.Generator(DEV).manual_seed(1), device=DEV, dtype=torch.float16)
    want, out = g.gemm_q4(a, packed, splits=1), torch.empty(m, n, dtype=torch.float16, device=DEV)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) / total)
        assert torch.equal(g.gemm_q4(a, packed, out=out), want)
        with pytest.raises(torch.OutOfMemoryError):           # asked for, so not replaced
            g.gemm_q4(a, packed, out=out, config=EXPANDED)
        assert torch.equal(g.gemm_q4(a[:64], packed, out=out[:64]), g.gemm_q4(a[:64], packed))
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert not torch.equal(g.gemm_q4(a, packed), want)        # with room for them the weights are rounded
