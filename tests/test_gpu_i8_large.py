"""GPU tests of the 8-bit and expert operators where rows pass a launch's and elements 32 bits."""
import numpy as np
import pytest
import torch

import i8_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("rows,k,stride", [((1 << 21) + 5, 16, 16), ((1 << 22) + 3, 5, 7), ((1 << 21) + 1, 70, 70)])
def test_compress_in_several_launches(rows, k, stride):
    """A launch takes 2^21 rows: those on both sides of its end, and all of them as in calls of fewer rows."""
    print(f"[i8] compress {rows}x{k} stride={stride}", flush=True)
    x = torch.randn(rows, stride, generator=torch.Generator(DEV).manual_seed(rows), device=DEV).to(torch.float16)[:, :k]
    got = g.i8_compress(x)
    for at in (0, (1 << 21) - 3, (1 << 22) - 3, rows - 4):
        codes, scales = ref.compress(ref.host(x[at:at + 6]))
        assert np.array_equal(ref.host(got.codes[at:at + 6]), codes) and np.array_equal(ref.host(got.scales[at:at + 6]), scales)
    for at in range(0, rows, 1 << 20):
        part = g.i8_compress(x[at:at + (1 << 20)])
        assert torch.equal(got.codes[at:at + (1 << 20)], part.codes) and torch.equal(got.scales[at:at + (1 << 20)], part.scales)
    back = g.i8_expand(got)
    assert torch.equal(back[-9:], g.i8_expand(g.i8_compress(x[-9:])))


@pytest.mark.parametrize("n", [65536, 65540, 65537])
def test_results_of_more_than_2_to_31_elements(n):
    """The last pairs of the experts' products, of an expert and of none, and their sum."""
    k, pairs, experts = 16, 32768 + 48, 3
    gen = torch.Generator(DEV).manual_seed(n)
    a = g.I8Matrix(torch.randint(-127, 128, (pairs, k), generator=gen, dtype=torch.int8, device=DEV),
                   torch.rand(pairs, generator=gen, device=DEV) * 1e-2, k)
    w = g.I8Matrix(torch.randint(-127, 128, (experts, n, k), generator=gen, dtype=torch.int8, device=DEV),
                   torch.rand(experts, n, generator=gen, device=DEV) * 1e-2, k)
    ids = torch.randint(0, experts, (pairs, 1), generator=gen, dtype=torch.int32, device=DEV)
    ids[-48:] = experts - 1
    ids[-16:] = -1
    order = g.expert_order(ids, experts)
    ac, sa = ref.host(a.codes[-48:-16]), ref.host(a.scales[-48:-16])
    want = ref.product(ac, sa, ref.host(w.codes[-1]), ref.host(w.scales[-1]))
    first = None
    for config in (1, 3, g.i8_num_configs() - 1, g.CONFIG_AUTO):
        print(f"[experts] {pairs} pairs n={n} config={config}", flush=True)
        out = torch.full((pairs, 1, n), 5.0, dtype=torch.float16, device=DEV)
        g.gemm_i8_experts(a, w, order, out=out, config=config)
        assert ref.near(ref.host(out[-48:-16, 0]), want).all() and bool((out[-16:] == 0).all())
        first = out if first is None else first
        assert torch.equal(out, first)
    with pytest.raises(g.GemmError):       # more workgroups of 512 threads than a launch's 32 bits of work items
        g.gemm_i8_experts(a, w, order, out=out, config=0)
    del out
    y = first.view(pairs // 8, 8, n)
    weights = torch.rand(pairs // 8, 8, generator=gen, device=DEV)
    got = g.expert_sum(y, weights)
    assert torch.equal(got[-6:], g.expert_sum(y[-6:].contiguous(), weights[-6:].contiguous()))


def test_logits_beyond_32_bits():
    base = torch.empty((1 << 31) + 100, dtype=torch.float16, device=DEV)
    x = base.as_strided((3, 64), (1 << 30, 1), 20)
    x.copy_(torch.randn(3, 64, generator=torch.Generator(DEV).manual_seed(1), device=DEV))
    ids, weights = g.route(x, 6, score="sigmoid")
    want = g.route(x.contiguous(), 6, score="sigmoid")
    assert torch.equal(ids, want[0]) and torch.equal(weights, want[1])


@pytest.mark.parametrize("experts", [5, 1000])
def test_order_of_the_most_pairs(experts):
    pairs = (1 << 25) - 1
    print(f"[route] order of {pairs} pairs over {experts}", flush=True)
    ids = torch.randint(-1, experts + 1, (pairs, 1), generator=torch.Generator(DEV).manual_seed(experts), dtype=torch.int32, device=DEV)
    got = g.expert_order(ids, experts)
    bins = torch.where((ids >= 0) & (ids < experts), ids, experts).view(-1)
    in_order, want = torch.sort(bins, stable=True)
    assert torch.equal(got.order.view(-1), want.to(torch.int32))
    starts = torch.searchsorted(in_order, torch.arange(experts + 1, dtype=torch.int32, device=DEV))
    assert torch.equal(got.starts, starts.to(torch.int32))
