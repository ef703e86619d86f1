"""GPU tests of the experts' products, and of a layer made of all the operators."""
import numpy as np
import pytest
import torch

import i8_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def held(lead, k, seed):
    gen = np.random.default_rng(seed)
    codes = np.zeros((*lead, -(-k // 16) * 16), np.int8)
    codes[..., :k] = gen.integers(-127, 128, (*lead, k), dtype=np.int8)
    scales = np.exp2(gen.uniform(-12, -6, lead)).astype(np.float32)
    return g.I8Matrix(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), k), codes[..., :k], scales


def some_ids(tokens, top_k, experts, seed, skew=False):
    """Distinct experts of each token; a tenth of the tokens have none, and one slot in ten."""
    gen = np.random.default_rng(seed)
    like = gen.random((tokens, experts)) + (np.arange(experts) < max(1, experts // 8)) * (0.8 if skew else 0.0)
    ids = np.argsort(-like, 1)[:, :top_k].astype(np.int32)
    ids[gen.random(tokens) < 0.1] = -1
    ids[gen.random(ids.shape) < 0.1] = experts + 3
    return ids


def expected(ids, experts, ac, sa, wc, sw, alpha, relu):
    tokens, top_k = ids.shape
    out = np.zeros((tokens, top_k, wc.shape[1]))
    per = tokens * top_k // ac.shape[0]
    for t in range(tokens):
        for j in range(top_k):
            e = ids[t, j]
            if 0 <= e < experts:
                r = (t * top_k + j) // per
                out[t, j] = ref.product(ac[r:r + 1], sa[r:r + 1], wc[e], sw[e], alpha, relu)[0]
    return out


def check(tokens, top_k, experts, n, k, per_pair=False, config=g.CONFIG_AUTO, epilogue="none", alpha=1.0, shift=0, skew=False):
    print(f"[experts] {tokens}x{top_k} of {experts} n={n} k={k} per_pair={per_pair} config={config} shift={shift}", flush=True)
    ids = some_ids(tokens, top_k, experts, tokens + n, skew)
    a, ac, sa = held((tokens, top_k) if per_pair else (tokens,), k, 1)
    w, wc, sw = held((experts, n), k, 2)
    order = g.expert_order(torch.from_numpy(ids).to(DEV), experts)
    size = tokens * top_k * n
    room = torch.full((size + 128 + shift,), 9.0, dtype=torch.float16, device=DEV)
    out = room[64 + shift:64 + shift + size].view(tokens, top_k, n)
    assert g.gemm_i8_experts(a, w, order, epilogue=epilogue, out=out, config=config, alpha=alpha) is out
    want = expected(ids, experts, ac.reshape(-1, k), sa.reshape(-1), wc, sw, alpha, epilogue == "relu")
    assert ref.near(ref.host(out), want).all()
    assert bool((room[:64 + shift] == 9).all()) and bool((room[64 + shift + size:] == 9).all())
    return out


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
@pytest.mark.parametrize("tokens,top_k,experts,n,k", [(1, 1, 1, 1, 1), (1, 8, 16, 64, 256), (5, 2, 8, 33, 100), (40, 4, 6, 70, 300),
                                                      (64, 3, 70, 48, 520), (130, 2, 3, 136, 130), (300, 2, 2, 264, 272), (33, 8, 130, 40, 64),
                                                      (600, 1, 1, 300, 64), (20, 5, 1024, 16, 32)])
def test_every_config(config, tokens, top_k, experts, n, k):
    top_k = min(top_k, experts)
    for per_pair in (False, True):
        check(tokens, top_k, experts, n, k, per_pair, config, epilogue="relu" if per_pair else "none", alpha=0.7)


@pytest.mark.parametrize("tokens,top_k,experts,n,k", [(1, 8, 256, 512, 1024), (64, 8, 64, 256, 512), (500, 4, 16, 300, 500), (1500, 2, 4, 260, 130),
                                                      (100, 6, 40, 64, 4100)])
def test_automatic_choice(tokens, top_k, experts, n, k):
    check(tokens, top_k, experts, n, k, skew=True)
    check(tokens, top_k, experts, n, k, per_pair=True, epilogue="relu")


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
@pytest.mark.parametrize("n,shift", [(40, 1), (40, 2), (40, 4), (44, 0), (42, 0), (41, 0)])
def test_alignment(config, n, shift):
    check(20, 3, 5, n, 80, config=config, shift=shift)


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
def test_as_the_dense_product_bit_for_bit(config):
    """All tokens to one expert, and each to its own."""
    a, w = held((70,), 300, 3)[0], held((5, 130), 300, 4)[0]
    for e in (0, 4):
        ids = torch.full((70, 1), e, dtype=torch.int32, device=DEV)
        got = g.gemm_i8_experts(a, w, g.expert_order(ids, 5), config=config, alpha=0.3)
        assert torch.equal(got[:, 0], g.gemm_i8(a, g.I8Matrix(w.codes[e], w.scales[e], 300), alpha=0.3))


@pytest.mark.parametrize("tokens,experts,n", [(2048, 4, 4100), (2000, 3, 4096), (3000, 5, 2056), (2300, 2, 3500)])
def test_last_round_in_quarters(tokens, experts, n):
    """More tiles of 256 x 256 than CUs: whatever the counts, the last round (and what is cut of it) misses no row."""
    a, w = held((tokens,), 200, 3)[0], held((experts, n), 200, 4)[0]
    for seed in range(6):
        order = g.expert_order(torch.from_numpy(some_ids(tokens, 2, experts, seed, skew=seed % 2 == 1)).to(DEV), experts)
        got, want = (torch.full((tokens, 2, n), 5.0, dtype=torch.float16, device=DEV) for _ in range(2))
        g.gemm_i8_experts(a, w, order, out=got, config=g.i8_num_configs() - 1, alpha=0.3)
        g.gemm_i8_experts(a, w, order, out=want, config=6, alpha=0.3)
        assert torch.equal(got, want)


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
def test_no_expert_and_empty(config):
    a, w = held((9,), 64, 3)[0], held((4, 40), 64, 4)[0]
    out = torch.full((9, 2, 40), 5.0, dtype=torch.float16, device=DEV)
    g.gemm_i8_experts(a, w, g.expert_order(torch.full((9, 2), -1, dtype=torch.int32, device=DEV), 4), out=out, config=config)
    assert bool((out == 0).all())
    for tokens, top_k in ((0, 3), (3, 0)):
        none = held((tokens,), 64, 1)[0]
        ids = torch.zeros(tokens, top_k, dtype=torch.int32, device=DEV)
        assert g.gemm_i8_experts(none, w, g.expert_order(ids, 4), config=config).shape == (tokens, top_k, 40)
    order = g.expert_order(torch.zeros(9, 2, dtype=torch.int32, device=DEV), 4)
    assert g.gemm_i8_experts(a, held((4, 0), 64, 4)[0], order, config=config).shape == (9, 2, 0)
    zero = g.i8_compress(torch.zeros(4, 40, 0, dtype=torch.float16, device=DEV))
    out.fill_(5.0)
    g.gemm_i8_experts(g.i8_compress(torch.zeros(9, 0, dtype=torch.float16, device=DEV)), zero, order, out=out, config=config)
    assert bool((out.view(torch.int16) == 0).all())


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
def test_orders_that_are_none(config):
    """Places out of range are skipped, starts out of range clamped, and rows that no place names left as they were."""
    a, ac, sa = held((6,), 64, 3)
    w, wc, sw = held((2, 24), 64, 4)
    order = torch.tensor([[0, 5], [99, -1], [3, 2], [1, 2 ** 31 - 1], [-2 ** 31, 4], [12, 6]], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 5, 12], dtype=torch.int32, device=DEV)
    out = torch.full((6, 2, 24), 5.0, dtype=torch.float16, device=DEV)
    g.gemm_i8_experts(a, w, g.ExpertOrder(order, starts), out=out, config=config)
    got = ref.host(out).reshape(12, 24)
    flat = ref.host(order).reshape(-1)
    named = np.zeros(12, bool)
    for i, p in enumerate(flat):
        if 0 <= p < 12:
            named[p] = True
            e = 0 if i < 5 else 1
            assert ref.near(got[p], ref.product(ac[p // 2:p // 2 + 1], sa[p // 2:p // 2 + 1], wc[e], sw[e])[0]).all()
    assert (got[~named] == 5).all() and not named.all()
    for bad in ([-7, 2 ** 31 - 1, 12], [12, 0, 12], [5, 3, 1], [100, 200, -300]):
        out.fill_(5.0)
        g.gemm_i8_experts(a, w, g.ExpertOrder(order, torch.tensor(bad, dtype=torch.int32, device=DEV)), out=out, config=config)
        assert bool(out.isfinite().all())


def layer(x, logits, bias, w_up, w_down, top_k):
    ids, weights = g.route(logits, top_k, score="sigmoid", bias=bias, groups=4, top_groups=2, renormalise=True, scale=2.5)
    order = g.expert_order(ids, logits.shape[1])
    h = g.gemm_i8_experts(g.i8_compress(x), w_up, order, epilogue="relu")
    return g.expert_sum(g.gemm_i8_experts(g.i8_compress(h), w_down, order), weights)


def layer_inputs(tokens, experts, d, n, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, d, generator=gen).to(torch.float16).to(DEV)
    logits = torch.randn(tokens, experts, generator=gen).to(DEV)
    if tokens > 2:
        logits[2] = -float("inf")             # a padded token
    bias = (0.1 * torch.randn(experts, generator=gen)).to(DEV)
    w_up = g.i8_compress((torch.randn(experts, n, d, generator=gen) * d ** -0.5).to(torch.float16).to(DEV))
    w_down = g.i8_compress((torch.randn(experts, d, n, generator=gen) * n ** -0.5).to(torch.float16).to(DEV))
    return x, logits, bias, w_up, w_down


@pytest.mark.parametrize("tokens", [1, 7, 64, 300])
def test_layer(tokens):
    """All of it, step by step against 64 bits, each step from what the one before gave."""
    x, logits, bias, w_up, w_down = layer_inputs(tokens, 16, 200, 136, tokens)
    ids, weights = g.route(logits, 4, score="sigmoid", bias=bias, groups=4, top_groups=2, renormalise=True, scale=2.5)
    want_ids, want_w = ref.route(ref.host(logits), 4, "sigmoid", ref.host(bias), 4, 2, True, 2.5)
    assert np.array_equal(ref.host(ids), want_ids) and (np.abs(ref.host(weights) - want_w) <= want_w * 2.0 ** -22).all()
    order = g.expert_order(ids, 16)
    xq = g.i8_compress(x)
    h = g.gemm_i8_experts(xq, w_up, order, epilogue="relu")
    wu = (ref.host(w_up.codes)[..., :200], ref.host(w_up.scales))
    assert ref.near(ref.host(h), expected(want_ids, 16, ref.host(xq.codes)[:, :200], ref.host(xq.scales), *wu, 1.0, True)).all()
    hq = g.i8_compress(h)
    y = g.gemm_i8_experts(hq, w_down, order)
    wd = (ref.host(w_down.codes)[..., :136], ref.host(w_down.scales))
    hc, hs = ref.host(hq.codes)[..., :136].reshape(-1, 136), ref.host(hq.scales).reshape(-1)
    assert ref.near(ref.host(y), expected(want_ids, 16, hc, hs, *wd, 1.0, False)).all()
    out = g.expert_sum(y, weights)
    if tokens > 2:
        assert bool((out[2] == 0).all()) and bool((ids[2] == -1).all())
    assert torch.equal(out, layer(x, logits, bias, w_up, w_down, 4))


def test_layer_captured_and_replayed():
    """A captured layer follows its inputs: tokens, logits and with them every count."""
    one, two = layer_inputs(40, 16, 200, 136, 1), layer_inputs(40, 16, 200, 136, 2)
    x, logits = one[0].clone(), one[1].clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer(x, logits, *one[2:], 4)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = layer(x, logits, *one[2:], 4)
    for i in range(6):
        now = two if i % 2 else one
        x.copy_(now[0])
        logits.copy_(now[1] if i < 4 else now[1].flip(1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer(x, logits, *one[2:], 4))


def test_layers_on_two_streams():
    cases = [layer_inputs(50, 16, 200, 136, i) for i in (1, 2)]
    want = [layer(*c, 4) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(*cases[i], 4))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in got[i])
    # an explicit stream
    x, logits, bias, w_up, w_down = cases[0]
    s = streams[0]
    ids, weights = g.route(logits, 4, score="sigmoid", bias=bias, groups=4, top_groups=2, renormalise=True, scale=2.5, stream=s)
    order = g.expert_order(ids, 16, stream=s)
    h = g.gemm_i8_experts(g.i8_compress(x, stream=s), w_up, order, epilogue="relu", stream=s)
    out = g.expert_sum(g.gemm_i8_experts(g.i8_compress(h, stream=s), w_down, order, stream=s), weights, stream=s)
    s.synchronize()
    assert torch.equal(out, want[0])
