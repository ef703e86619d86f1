"""GPU tests of the product with 4-bit weights where other tests do not reach:
rows that hold an infinity, and more rows than one launch's grid holds; and of
appends that share a page."""
import numpy as np
import pytest
import torch

import q4_reference as ref
import tiled_dense_gemm_fp16_amd as g
from test_gpu_q4_weights import DEV, bound, gen, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("config", range(g.q4_num_configs()))
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_every_column_sees_an_infinity_of_its_row(config, value):
    # a weight of 0 gives NaN, any other an infinity: no result of such a row is finite
    for k, at in ((130, 0), (130, 129), (262, 255), (646, 645), (1032, 517)):
        a = torch.randn(70, k, generator=gen(k)).to(torch.float16)
        a[1::2, at] = value
        packed = g.q4_compress(weights(48, k, k).to(DEV), 64)
        got = ref.host(g.gemm_q4(a.to(DEV), packed, config=config))
        print(f"[q4] config={config} k={k} {value} at {at}", flush=True)
        assert not np.isfinite(got[1::2]).any()
        assert np.isfinite(got[::2]).all()


@pytest.mark.parametrize("splits", [1, 2])
def test_more_rows_than_a_grid_holds(splits):
    """16 x 65535 rows fill the second dimension of the first launch; the others come in a second one."""
    edge = 16 * 65535
    m, n, k = edge + 17, 3, 130
    r = torch.Generator(DEV).manual_seed(1)
    a = torch.randn(m, k, generator=r, device=DEV).to(torch.float16)
    packed = g.q4_compress(weights(n, k, 3).to(DEV), 64)
    dense = ref.unpack_weights(ref.host(packed.codes), ref.host(packed.words), n, k, 64)
    room = torch.full((m * n + 64,), 9.0, dtype=torch.float16, device=DEV)
    got = room[32:-32].view(m, n)
    g.gemm_q4(a, packed, config=0, splits=splits, alpha=0.5, out=got)
    torch.cuda.synchronize()
    assert bool((room[:32] == 9).all()) and bool((room[-32:] == 9).all())
    for rows in (slice(0, 4096), slice(edge - 4096, m)):
        want, size = ref.product(a[rows].cpu().double().numpy(), dense, 0.5)
        assert (np.abs(ref.host(got[rows]).astype(np.float64) - want) <= bound(want, size, k, 64)).all()
    wide = torch.as_tensor(dense, device=DEV)
    worst = 0.0
    for i in range(0, m, 1 << 18):                         # every row, by a looser common bound
        want = a[i:i + (1 << 18)].double() @ wide.t().contiguous() * 0.5
        worst = max(worst, (got[i:i + (1 << 18)].double() - want).abs().max().item())
    assert worst < 2.0 ** -5                               # half a step of results below 128, and fp32's part of it


def test_appends_to_granules_of_one_page():
    """Two sequences, and one sequence whose table names the page twice, append to neighbouring granules of a page: each slot
    holds what it would hold alone."""
    from test_gpu_q4_cache import check_append
    check_append(128, 64, 32, [0, 8, 16], [8, 5, 3], table=[[0], [0], [0]], positions=32)
    check_append(64, 32, 32, [8], [24], table=[[3, 3]], positions=64, heads=3)
    check_append(256, 128, 16, [4, 8], [4, 8], table=[[5], [5]], positions=16)
