"""GPU tests of the 8-bit and expert operators: what is refused, offsets beyond 32 bits, seeded random cases, and calls that
share their buffers."""
import numpy as np
import pytest
import torch

import i8_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def codes(*shape):
    return torch.randint(-127, 128, shape, dtype=torch.int8, device=DEV)


def test_refusals():
    a, w = g.I8Matrix(codes(4, 64), torch.ones(4, device=DEV), 60), g.I8Matrix(codes(8, 64), torch.ones(8, device=DEV), 60)
    experts = g.I8Matrix(codes(3, 8, 64), torch.ones(3, 8, device=DEV), 60)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    order = g.expert_order(ids, 3)
    x, y = torch.zeros(4, 60, dtype=torch.float16, device=DEV), torch.zeros(4, 2, 8, dtype=torch.float16, device=DEV)
    logits = torch.zeros(4, 12, device=DEV)
    ones = torch.ones(4, 2, device=DEV)
    half = dict(dtype=torch.float16, device=DEV)
    bad = [
        lambda: g.gemm_i8(a, w._replace(k=59)), lambda: g.gemm_i8(a._replace(codes=a.codes[:, :48]), w),
        lambda: g.gemm_i8(a._replace(codes=a.codes.t()), w), lambda: g.gemm_i8(a._replace(codes=a.codes[:, :32]), w),
        lambda: g.gemm_i8(a._replace(scales=a.scales[:3]), w), lambda: g.gemm_i8(a._replace(scales=a.scales.double()), w),
        lambda: g.gemm_i8(a._replace(codes=a.codes.float()), w), lambda: g.gemm_i8(a._replace(scales=a.scales.cpu()), w),
        lambda: g.gemm_i8(a._replace(k=-1), w), lambda: g.gemm_i8(a, experts), lambda: g.gemm_i8(a, x), lambda: g.gemm_i8(a, w, epilogue="max"),
        lambda: g.gemm_i8(a, w, out=torch.empty(4, 9, **half)), lambda: g.gemm_i8(a, w, out=torch.empty(4, 8, device=DEV)),
        lambda: g.gemm_i8(a, w, out=torch.empty(8, 4, **half).t()), lambda: g.gemm_i8(a, w, workspace=torch.empty(4)),
        lambda: g.i8_compress(x.t()), lambda: g.i8_compress(x[:1].expand(4, 60)), lambda: g.i8_compress(x.float()), lambda: g.i8_compress(x[0]),
        lambda: g.i8_compress(torch.zeros(4, 6, 10, **half).transpose(0, 1)), lambda: g.i8_compress(torch.zeros(1, 131072, **half)),
        lambda: g.i8_expand(a, out=torch.empty(4, 64, **half)),
        lambda: g.route(logits, 0), lambda: g.route(logits, 13), lambda: g.route(logits, 2, groups=5), lambda: g.route(logits, 2, groups=3, top_groups=4),
        lambda: g.route(logits, 2, bias=torch.zeros(11, device=DEV)), lambda: g.route(logits, 2, bias=torch.zeros(12, **half)),
        lambda: g.route(logits.double(), 2), lambda: g.route(logits[0], 2), lambda: g.route(logits.t(), 2), lambda: g.route(logits[:1].expand(4, 12), 2),
        lambda: g.route(torch.zeros(2, 1025, device=DEV), 2), lambda: g.route(torch.zeros(2, 0, device=DEV), 1), lambda: g.route(logits, 2, score="max"),
        lambda: g.expert_order(ids.long(), 3), lambda: g.expert_order(ids, 0), lambda: g.expert_order(ids, 1025), lambda: g.expert_order(ids.t(), 3),
        lambda: g.gemm_i8_experts(a, w, order), lambda: g.gemm_i8_experts(a._replace(k=59), experts, order), lambda: g.gemm_i8_experts(a, experts, ids),
        lambda: g.gemm_i8_experts(a, experts, g.expert_order(ids, 4)), lambda: g.gemm_i8_experts(a, experts, g.expert_order(ids[:3].contiguous(), 3)),
        lambda: g.gemm_i8_experts(a, experts, order._replace(order=order.order.reshape(-1))),
        lambda: g.gemm_i8_experts(a, experts, order, out=torch.empty(8, 8, **half)),
        lambda: g.expert_sum(y, ones.half()), lambda: g.expert_sum(y, ones[:, :1]), lambda: g.expert_sum(y[..., :4], ones), lambda: g.expert_sum(y[0], ones),
        lambda: g.expert_sum(y, ones, out=torch.empty(4, 9, **half)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            print(f"[i8] refusal {i}", flush=True)
            call()
    out = torch.empty(4, 8, **half)
    refused = [
        lambda: g.gemm_i8(a, w, config=g.i8_num_configs()), lambda: g.gemm_i8(a, w, splits=65),
        lambda: g.gemm_i8(g.I8Matrix(codes(4 * 64 + 1)[1:].view(4, 64), a.scales, 60), w), lambda: g.route(logits, 2, scale=float("nan")),
        lambda: g.expert_sum(y, ones, out=y.view(-1)[:32].view(4, 8)), lambda: g.gemm_i8(a, w, out=a.codes.view(torch.float16).view(-1)[:32].view(4, 8)),
        lambda: g.gemm_i8_experts(a, experts, order, config=99),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(g.GemmError):
            print(f"[i8] refusal by the library {i}", flush=True)
            call()
    g.gemm_i8(a, w, out=out)


def test_a_matrix_with_itself_and_shared_outputs():
    x = g.i8_compress(torch.randn(70, 200, generator=torch.Generator().manual_seed(1)).to(torch.float16).to(DEV))
    got = ref.host(g.gemm_i8(x, x))
    c, s = ref.host(x.codes), ref.host(x.scales)
    assert ref.near(got, ref.product(c, s, c, s)).all() and np.array_equal(got, got.T)
    out = torch.empty(70, 70, dtype=torch.float16, device=DEV)
    for _ in range(3):            # the same output again, each call after the one before
        g.gemm_i8(x, x, out=out, splits=1)
        g.gemm_i8(x, x, out=out, epilogue="relu")
        g.gemm_i8(x, x, out=out)
    assert np.array_equal(ref.host(out), got)
    # the same expert in several slots of a token
    w = g.I8Matrix(codes(3, 24, 256), torch.rand(3, 24, device=DEV) * 1e-3, 200)
    ids = torch.tensor([[2, 2, 0]] * 70, dtype=torch.int32, device=DEV)
    y = g.gemm_i8_experts(x, w, g.expert_order(ids, 3))
    assert torch.equal(y[:, 0], y[:, 1]) and torch.equal(y[:, 0], g.gemm_i8(x, g.I8Matrix(w.codes[2], w.scales[2], 200)))


def test_offsets_beyond_32_bits():
    """Weights of 5 GB, results of 5 GB, rows of 5 GB: the last ones are right."""
    k, n = 8192, 700000
    w = torch.zeros(n, k, dtype=torch.int8, device=DEV)
    w[-300:] = codes(300, k)
    a, scales = codes(3, k), torch.rand(n, device=DEV) * 1e-4
    want = ref.product(ref.host(a), np.ones(3, np.float32), ref.host(w[-300:]), ref.host(scales[-300:]))
    for config in range(g.i8_num_configs()):
        got = g.gemm_i8(g.I8Matrix(a, torch.ones(3, device=DEV), k), g.I8Matrix(w, scales, k), config=config)
        assert ref.near(ref.host(got[:, -300:]), want).all() and bool((got[:, :-300] == 0).all())
    order = g.expert_order(torch.tensor([[6999], [0], [6999]], dtype=torch.int32, device=DEV) % 1000, 1000)
    for config in range(g.i8_num_configs()):
        got = g.gemm_i8_experts(g.I8Matrix(a, torch.ones(3, device=DEV), k), g.I8Matrix(w.view(1000, 700, k), scales.view(1000, 700), k), order,
                                config=config)
        assert ref.near(ref.host(got[[0, 2], 0, -300:]), want[[0, 2]]).all() and bool((got[1] == 0).all())
    del w, got
    m, n = 70000, 40000
    a, w = g.I8Matrix(codes(m, 16), torch.ones(m, device=DEV), 16), g.I8Matrix(codes(n, 16), torch.full((n,), 1e-3, device=DEV), 16)
    for config in (5, g.i8_num_configs() - 1):
        got = g.gemm_i8(a, w, config=config)
        at = slice(m - 260, m)
        want = ref.product(ref.host(a.codes[at]), np.ones(260, np.float32), ref.host(w.codes), np.full(n, 1e-3, np.float32))
        assert ref.near(ref.host(got[at]), want).all()
    x = got.view(-1)[:70000 * 39999].view(70000, 39999)          # rows of odd length
    packed = g.i8_compress(x)
    c, s = ref.compress(ref.host(x[-5:]))
    assert np.array_equal(ref.host(packed.codes[-5:]), c) and np.array_equal(ref.host(packed.scales[-5:]), s)
    back = g.i8_expand(packed)
    assert torch.equal(back[-5:], g.i8_expand(g.i8_compress(x[-5:].contiguous())))


@pytest.mark.parametrize("seed", range(40))
def test_random_products(seed):
    rng = np.random.default_rng(seed)
    m, n, k = (int(np.exp(rng.uniform(0, np.log(top)))) for top in (700, 1500, 5000))
    config, splits = int(rng.integers(-1, g.i8_num_configs())), [None, 1, 2, 3, 7][rng.integers(5)]
    alpha, relu, shift = float(rng.choice([1.0, -0.3, 2.5])), bool(rng.integers(2)), int(rng.integers(0, 5))
    print(f"[i8] random {seed}: {m}x{n}x{k} config={config} splits={splits} shift={shift}", flush=True)
    ap, wp = (-(-k // 16) * 16 + 16 * int(rng.integers(0, 9)) for _ in range(2))
    ac, wc = (np.pad(rng.integers(-128, 128, (r, k), dtype=np.int8), ((0, 0), (0, p - k))) for r, p in ((m, ap), (n, wp)))
    sa, sw = (np.exp2(rng.uniform(-14, -4, r)).astype(np.float32) for r in (m, n))
    room = torch.full((m * n + 16 + shift,), 9.0, dtype=torch.float16, device=DEV)
    out = room[8 + shift:8 + shift + m * n].view(m, n)
    a, w = (g.I8Matrix(torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV), k) for c, s in ((ac, sa), (wc, sw)))
    g.gemm_i8(a, w, epilogue="relu" if relu else "none", alpha=alpha, out=out, config=config, splits=splits)
    assert ref.near(ref.host(out), ref.product(ac[:, :k], sa, wc[:, :k], sw, alpha, relu)).all()
    assert bool((room[:8 + shift] == 9).all()) and bool((room[8 + shift + m * n:] == 9).all())


@pytest.mark.parametrize("seed", range(30))
def test_random_routing(seed):
    rng = np.random.default_rng(1000 + seed)
    groups = int(rng.choice([1, 1, 2, 4, 8, 16]))
    experts = groups * int(rng.integers(1, 1 + min(64, 1024 // groups)))
    top_k, tokens = int(rng.integers(1, min(experts, 12) + 1)), int(rng.integers(1, 60))
    top_groups = int(rng.integers(1, groups + 1))
    dtype = [torch.float16, torch.float32][rng.integers(2)]
    x = torch.from_numpy(rng.normal(size=(tokens, experts)) * rng.choice([0.5, 2.0, 20.0])).to(dtype)
    x[torch.from_numpy(rng.random((tokens, experts)) < rng.choice([0.0, 0.1, 0.8]))] = -float("inf")
    bias = torch.from_numpy(rng.normal(size=experts) * 0.3).float() if rng.integers(2) else None
    score, renormalise = ["softmax", "sigmoid"][rng.integers(2)], bool(rng.integers(2))
    print(f"[route] random {seed}: {tokens}x{experts} top_k={top_k} groups={groups}/{top_groups} {score} bias={bias is not None}", flush=True)
    ids, weights = g.route(x.to(DEV), top_k, score=score, bias=None if bias is None else bias.to(DEV), groups=groups, top_groups=top_groups,
                           renormalise=renormalise, scale=2.0)
    want_ids, want = ref.route(x.numpy(), top_k, score, None if bias is None else bias.numpy(), groups, top_groups, renormalise, 2.0)
    assert np.array_equal(ref.host(ids), want_ids)
    assert (np.abs(ref.host(weights) - want) <= want * 2.0 ** -22 + 2.0 ** -149).all()
    order = g.expert_order(ids, experts)
    places, starts = ref.order(want_ids, experts)
    assert np.array_equal(ref.host(order.order).reshape(-1), places) and np.array_equal(ref.host(order.starts), starts)
