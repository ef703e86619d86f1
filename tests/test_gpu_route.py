"""GPU tests of the choice of experts and the order of the pairs: ids and orders are whole numbers and have to be equal;
a weight is a 64-bit value rounded once to fp32 (2^-24 of it; 2^-22 leaves room for exp and sums in another order)."""
import numpy as np
import pytest
import torch

import i8_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = float("inf")


def check(logits, top_k, score="softmax", bias=None, **kw):
    print(f"[route] {tuple(logits.shape)} {logits.dtype} top_k={top_k} {score} bias={bias is not None} {kw}", flush=True)
    ids, weights = g.route(logits.to(DEV), top_k, score=score, bias=None if bias is None else bias.to(DEV), **kw)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32
    want_ids, want = ref.route(logits.numpy(), top_k, score, None if bias is None else bias.numpy(), **kw)
    assert np.array_equal(ref.host(ids), want_ids)
    assert (np.abs(ref.host(weights) - want) <= np.abs(want) * 2.0 ** -22 + 2.0 ** -149).all()
    return ids, weights


def draw(tokens, experts, dtype, seed):
    return (1.5 * torch.randn(tokens, experts, generator=torch.Generator().manual_seed(seed))).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (3, 8, 2), (5, 8, 8), (7, 40, 6), (9, 64, 6), (4, 65, 3), (6, 128, 8),
                                                  (11, 160, 6), (13, 256, 8), (5, 257, 10), (3, 512, 64), (6, 1000, 8), (2, 1024, 64)])
def test_plain(tokens, experts, top_k, score, dtype):
    for renormalise in (False, True):
        check(draw(tokens, experts, dtype, tokens + experts), top_k, score, renormalise=renormalise, scale=2.5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups,top_k", [(8, 8, 3, 3), (40, 4, 2, 6), (64, 8, 1, 8), (160, 8, 3, 6), (256, 8, 4, 8),
                                                             (256, 64, 5, 8), (1024, 16, 4, 10), (60, 12, 4, 8), (256, 1, 1, 8), (9, 3, 2, 4)])
def test_bias_and_groups(experts, groups, top_groups, top_k, score, dtype):
    x = draw(33, experts, dtype, experts + groups)
    bias = 0.3 * torch.randn(experts, generator=torch.Generator().manual_seed(1))
    check(x, top_k, score, bias, groups=groups, top_groups=top_groups, renormalise=True, scale=2.5)
    check(x, top_k, score, None, groups=groups, top_groups=top_groups)
    check(x, top_k, score, torch.zeros(experts), groups=groups, top_groups=top_groups)


def test_ties_go_to_the_lowest_index():
    for experts in (8, 64, 100, 256, 700):
        for dtype in (torch.float16, torch.float32):
            x = torch.randint(-2, 3, (20, experts), generator=torch.Generator().manual_seed(experts)).to(dtype)
            x[0] = 0
            x[1, ::2] = -0.0
            x[1, 1::2] = 0.0
            bias = torch.zeros(experts)
            for score in ("softmax", "sigmoid"):
                check(x, 7, score)
                check(x, 7, score, bias)
                if experts % 4 == 0:
                    check(x, 7, score, bias, groups=4, top_groups=2)
                    check(x, 7, score, groups=4, top_groups=2)


def test_far_logits_keep_their_order():
    """Sigmoids of far logits are all 1, and softmaxes all 0, but in 64 bits or beyond: without bias the logits decide."""
    x = torch.tensor([[50.0, 60.0, 40.0, 55.0, -800.0, -900.0, -850.0, 700.0], [-65504.0, 65504.0, 1e4, -1e4, 0.0, 3.0, 2e4, 3e4],
                      [-3e38, 3e38, 1e38, -1e38, 0.0, 1e-38, -1e-38, 1e-45]])
    for score in ("softmax", "sigmoid"):
        for k in (1, 5, 8):
            check(x, k, score)
            check(x, k, score, renormalise=True)


@pytest.mark.parametrize("experts", [8, 64, 256])
def test_closed_experts(experts):
    x = draw(12, experts, torch.float32, 3)
    x[0] = -INF                               # nobody's token
    x[1] = float("nan")
    x[2, 2:] = -INF                           # two experts left
    x[3, 1] = float("nan")
    x[4, 0] = INF
    x[5, 3], x[5, 5] = INF, INF
    x[6, :experts // 2] = -INF
    x[7] = torch.finfo(torch.float32).min
    x[8] = INF
    bias = 0.2 * torch.randn(experts, generator=torch.Generator().manual_seed(2))
    bias[1], bias[2], bias[6] = -INF, float("nan"), INF
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            for t in (x, x.to(torch.float16)):
                check(t, 4, score, renormalise=renormalise)
                check(t, 4, score, bias, renormalise=renormalise)
                for groups, top in ((2, 1), (4, 2), (8, 3)):
                    check(t, 4, score, groups=groups, top_groups=top, renormalise=renormalise)
                    check(t, 4, score, bias, groups=groups, top_groups=top, renormalise=renormalise)
    ids, weights = g.route(x.to(DEV), 4, bias=bias.to(DEV))
    order = g.expert_order(ids, experts)
    assert order.starts[experts] <= 4 * 12 - 8 and sorted(ref.host(order.order).reshape(-1)) == list(range(48))


def test_rows_apart():
    base = draw(50, 80, torch.float16, 9)
    ids, weights = g.route(base.to(DEV)[3:40:2, 5:69], 6)
    want = g.route(base[3:40:2, 5:69].contiguous().to(DEV), 6)
    assert torch.equal(ids, want[0]) and torch.equal(weights, want[1])


def test_many_tokens():
    x = draw(20000, 64, torch.float16, 4)
    ids, weights = g.route(x.to(DEV), 6)
    best = torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :6].to(torch.int32)
    assert torch.equal(ids.cpu(), best)
    p = torch.softmax(x.double(), 1).gather(1, best.long())
    assert ((weights.cpu() - p).abs() <= p * 2.0 ** -22).all()


@pytest.mark.parametrize("tokens,top_k,experts", [(0, 3, 5), (1, 1, 1), (1, 8, 256), (7, 3, 5), (64, 8, 256), (100, 6, 64), (1000, 2, 8),
                                                  (3001, 7, 40), (8192, 6, 64), (20000, 8, 1024), (70000, 4, 3)])
def test_order(tokens, top_k, experts):
    print(f"[route] order {tokens}x{top_k} of {experts}", flush=True)
    gen = torch.Generator().manual_seed(tokens + experts)
    ids = torch.randint(-1, experts + 1, (tokens, top_k), generator=gen, dtype=torch.int32)
    ids[tokens // 2:] = torch.where(torch.rand(tokens - tokens // 2, top_k, generator=gen) < 0.5, experts // 2, ids[tokens // 2:])
    order = g.expert_order(ids.to(DEV), experts)
    want, starts = ref.order(ids.numpy(), experts)
    assert order.order.shape == (tokens, top_k) and np.array_equal(ref.host(order.order).reshape(-1), want)
    assert np.array_equal(ref.host(order.starts), starts)


def test_order_of_any_ids():
    ids = torch.tensor([[-2 ** 31, 2 ** 31 - 1, -1, 5, 4, 0]], dtype=torch.int32)
    order = g.expert_order(ids.to(DEV), 5)
    assert ref.host(order.order).tolist() == [[5, 4, 0, 1, 2, 3]] and ref.host(order.starts).tolist() == [0, 1, 1, 1, 1, 2]
