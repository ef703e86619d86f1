"""CPU tests of what the plans of the 8-bit products say about a launch."""
import os

import pytest

import tiled_dense_gemm_fp16_amd as g


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(g.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
def test_lds_bytes(config):
    """Stages of 128 bytes of k a row, a factor for each row and a scale for each column; over experts each row's pair, too.
    The kernel for few rows: the sums (4 int32 a lane) of each of its 8 waves."""
    for m, n, k, splits in [(1, 16, 128, 1), (300, 520, 4100, 1), (4200, 4096, 300, 1), (4096, 4096, 300, 1), (300, 520, 4100, 4)]:
        p = g.plan_i8(m, n, k, config=config, splits=splits)
        e = g.plan_i8_experts(m * 8, 8, 16, n, k, config=config)
        assert (p["block_m"], p["block_n"], p["stages"]) == (e["block_m"], e["block_n"], e["stages"])
        bm, bn = p["block_m"], p["block_n"]
        if p["direct_lds"]:
            want = p["stages"] * (bm + bn) * 128 + 4 * (bm + bn)
            assert p["lds_bytes"] == want and e["lds_bytes"] == want + 4 * bm <= 163840
        else:
            assert p["lds_bytes"] == e["lds_bytes"] == 8 * 64 * 16


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
@pytest.mark.parametrize("n,vec", [(40, 8), (44, 4), (42, 1), (41, 1)])
def test_vec_c(config, n, vec):
    """Elements for each store of C, were it 16-byte aligned: rows of C start where N lets them.  A split's sum stores four
    at most, and the kernel for few rows one at a time."""
    whole = g.plan_i8(300, n, 4100, config=config)
    assert whole["vec_c"] == (vec if whole["direct_lds"] else 1)
    split = g.plan_i8(300, n, 4100, config=config, splits=4)
    assert split["splits"] == 4 and split["vec_c"] == min(vec, 4)
    experts = g.plan_i8_experts(600, 2, 16, n, 4100, config=config)
    assert experts["vec_c"] == (vec if experts["direct_lds"] else 1)
