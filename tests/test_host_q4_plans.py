"""CPU tests of the choices that gemm_f16_plan_q4 makes for many rows: which
products round their weights, and that one more row does not leave the card
idle."""
import pytest

import tiled_dense_gemm_fp16_amd as g

EXPANDED = g.q4_num_configs() - 1          # rounds each weight to binary16; all other configurations use it exactly


@pytest.mark.parametrize("group", [32, 64, 128])
def test_weights_are_rounded_only_where_it_is_said(group):
    for m in (1, 16, 33, 65, 300, 2047, 2048, 8192):
        for n, k in [(16, 128), (300, 4100), (8192, 8192), (28672, 8192), (4096, 4095)]:
            assert g.plan_q4(m, n, k, group, splits=1)["config"] < EXPANDED
            assert g.plan_q4(m, n, k, group, splits=1)["workspace_bytes"] == 0
            if m < 2048 or group == 128:
                p = g.plan_q4(m, n, k, group, splits=None)
                assert p["config"] < EXPANDED and p["workspace_bytes"] < 2 * n * k + (p["splits"] > 1) * 2 ** 40 + 2 * m * (k + 256)
    assert g.plan_q4(2048, 8192, 8192, group, splits=None)["config"] == (EXPANDED if group < 128 else EXPANDED - 1)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", [1, 16, 64, 128, 256, 512])
@pytest.mark.parametrize("k", [2048, 8192, 16384])
def test_few_outputs_over_a_long_k_keep_the_split(n, k, group):
    """At 2048 rows as at 2047: a few columns of tiles fill the card only with K split, which the dense product never does."""
    below, at = (g.plan_q4(m, n, k, group, splits=None) for m in (2047, 2048))
    assert at["config"] == below["config"] < EXPANDED and at["splits"] == below["splits"]
    assert at["grid"] >= (128 if k == 2048 else 192)
    for m in (3000, 4000):
        if m * -(-n // 64) * 64 < 1 << 21:
            p = g.plan_q4(m, n, k, group, splits=None)
            assert p["config"] < EXPANDED and p["grid"] >= 128
    assert g.plan_q4(2048, 2048, k, 64, splits=None)["config"] == EXPANDED
