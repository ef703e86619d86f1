"""GPU tests of the 8-bit product: sums of codes are exact, so all that is off is i8_reference.bound()."""
import numpy as np
import pytest
import torch

import i8_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def held(rows, k, seed, pitch=None):
    """(device I8Matrix, host codes, host scales) of random rows, some of them zero."""
    gen = np.random.default_rng(seed)
    codes = np.zeros((rows, pitch or -(-k // 16) * 16), np.int8)
    codes[:, :k] = gen.integers(-127, 128, (rows, k), dtype=np.int8)
    scales = np.exp2(gen.uniform(-12, -6, rows)).astype(np.float32)
    if rows > 3:
        scales[3] = 0
    return g.I8Matrix(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), k), codes, scales


def check(m, n, k, config=g.CONFIG_AUTO, epilogue="none", alpha=1.0, shift=0, splits=None, a_pitch=None, w_pitch=None):
    print(f"[i8] product {m}x{n}x{k} config={config} epi={epilogue} alpha={alpha} shift={shift} splits={splits}", flush=True)
    a, ac, sa = held(m, k, m + k, a_pitch)
    w, wc, sw = held(n, k, n + 7 * k, w_pitch)
    room = torch.full((m * n + 128 + shift,), 9.0, dtype=torch.float16, device=DEV)
    out = room[64 + shift:64 + shift + m * n].view(m, n)
    assert g.gemm_i8(a, w, epilogue=epilogue, out=out, config=config, alpha=alpha, splits=splits) is out
    want = ref.product(ac[:, :k], sa, wc[:, :k], sw, alpha, epilogue == "relu")
    assert ref.near(ref.host(out), want).all()
    assert bool((room[:64 + shift] == 9).all()) and bool((room[64 + shift + m * n:] == 9).all())
    return out


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 16, 128), (1, 100, 2048), (3, 33, 1000), (16, 16, 1024), (17, 70, 1030),
                                   (33, 48, 520), (64, 64, 256), (65, 40, 4100), (130, 264, 136), (257, 300, 100), (300, 520, 700)])
def test_every_config(config, m, n, k):
    check(m, n, k, config=config)


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
@pytest.mark.parametrize("m,n,k,splits", [(1, 16, 600, 3), (70, 140, 1030, 2), (16, 128, 4100, 7), (130, 300, 2048, 64),
                                          (129, 257, 1000, 2), (300, 520, 514, None), (5, 33, 9000, 4)])
def test_splits(config, m, n, k, splits):
    whole = check(m, n, k, config=config, splits=1, epilogue="relu", alpha=0.7)
    assert torch.equal(check(m, n, k, config=config, splits=splits, epilogue="relu", alpha=0.7), whole)


@pytest.mark.parametrize("m,n,k", [(1, 1024, 1024), (2, 5000, 4100), (13, 256, 8192), (40, 600, 3000), (300, 300, 300), (70, 64, 9000),
                                   (520, 700, 1000), (3, 70, 16500), (300, 5000, 300), (40, 9000, 520), (1, 12000, 300), (2050, 1030, 64)])
@pytest.mark.parametrize("epilogue,alpha", [("none", 1.0), ("relu", 0.125), ("none", -1.7)])
def test_automatic_choice(m, n, k, epilogue, alpha):
    check(m, n, k, epilogue=epilogue, alpha=alpha)


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
def test_every_config_gives_the_same_bits(config):
    for m, n, k in [(16, 70, 1000), (70, 136, 3000)]:
        a, w = held(m, k, 1)[0], held(n, k, 2)[0]
        want = g.gemm_i8(a, w, config=0, splits=1, alpha=0.3)
        for splits in (1, 2, 5, None):
            assert torch.equal(g.gemm_i8(a, w, config=config, splits=splits, alpha=0.3), want)


@pytest.mark.parametrize("m,n", [(4200, 4096), (4100, 4104), (4100, 4100), (4353, 4301), (2100, 8000), (4096, 4096)])
def test_last_round_in_quarters(m, n):
    """More tiles of 256 x 256 than CUs by a few: the last ones are cut in four."""
    last = g.i8_num_configs() - 1
    p = g.plan_i8(m, n, 300, config=last)
    assert p["block_m"] == p["block_n"] == 256
    print(f"[i8] {m}x{n} tiles={p['tiles_m'] * p['tiles_n']} grid={p['grid']}", flush=True)
    a, w = held(m, 300, 1)[0], held(n, 300, 2)[0]
    room = torch.full((m * n + 128,), 9.0, dtype=torch.float16, device=DEV)
    got = g.gemm_i8(a, w, config=last, alpha=0.3, epilogue="relu", out=room[64:-64].view(m, n))
    assert torch.equal(got, g.gemm_i8(a, w, config=6, alpha=0.3, epilogue="relu"))
    assert bool((room[:64] == 9).all()) and bool((room[-64:] == 9).all())


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
def test_pitches_and_alignment(config):
    check(20, 40, 100, config=config, a_pitch=256, w_pitch=128)
    check(20, 40, 100, config=config, a_pitch=112, w_pitch=4096)
    for shift in (1, 2, 4):
        check(33, 48, 261, config=config, shift=shift)
    check(33, 44, 261, config=config)


@pytest.mark.parametrize("config", range(g.i8_num_configs()))
def test_largest_sums(config):
    k = 131071
    codes = torch.full((2, 131072), -128, dtype=torch.int8, device=DEV)
    codes[:, k:] = 0
    ones = torch.tensor([2.0 ** -16, 2.0 ** -20], device=DEV)
    got = ref.host(g.gemm_i8(g.I8Matrix(codes, ones, k), g.I8Matrix(codes, torch.ones(2, device=DEV), k), config=config, splits=1))
    assert ref.near(got, 16384.0 * k * np.array([[2.0 ** -16] * 2, [2.0 ** -20] * 2])).all()
    split = g.gemm_i8(g.I8Matrix(codes, ones, k), g.I8Matrix(codes, torch.ones(2, device=DEV), k), config=config, splits=9)
    assert np.array_equal(ref.host(split), got)


def test_scales_of_any_size():
    """Scales far from 1 whose product is a finite fp32 number; results beyond binary16 are infinite, tiny ones 0."""
    a, ac, _ = held(6, 64, 3)
    w, wc, _ = held(8, 64, 4)
    sa = np.array([1e30, 1e-30, 1e-38, 1.0, 0.0, -2.5], np.float32)
    sw = np.array([1e-30, 1e30, 1e-3, 0.0, 1e5, -1e-2, 1e-36, 3e37], np.float32)
    with np.errstate(over="ignore"):
        fits = np.isfinite(np.float32(sa)[:, None] * np.float32(sw))
    got = ref.host(g.gemm_i8(a._replace(scales=torch.from_numpy(sa).to(DEV)), w._replace(scales=torch.from_numpy(sw).to(DEV))))
    want = ref.product(ac[:, :64], sa, wc[:, :64], sw)
    assert ref.near(got, want)[fits].all()


def test_bad_scales_stay_in_their_row_and_column():
    a, ac, sa = held(20, 256, 5)
    w, wc, sw = held(40, 256, 6)
    sa[3], sw[7] = np.nan, np.inf
    got = ref.host(g.gemm_i8(a._replace(scales=torch.from_numpy(sa).to(DEV)), w._replace(scales=torch.from_numpy(sw).to(DEV))))
    assert np.isnan(got[3]).all()
    rows, cols = np.arange(20) != 3, np.arange(40) != 7
    assert ref.near(got[rows][:, cols], ref.product(ac[rows], sa[rows], wc[cols], sw[cols])).all()
    assert not np.isfinite(got[rows][:, 7]).any()


def test_empty_and_zero_depth():
    zero = g.i8_compress(torch.zeros(8, 0, dtype=torch.float16, device=DEV))
    zero = zero._replace(scales=torch.full((8,), -3.0, device=DEV))
    out = torch.full((3, 8), 5.0, dtype=torch.float16, device=DEV)
    a = g.i8_compress(torch.zeros(3, 0, dtype=torch.float16, device=DEV))._replace(scales=torch.ones(3, device=DEV))
    for config in (g.CONFIG_AUTO, *range(g.i8_num_configs())):
        out.fill_(5.0)
        g.gemm_i8(a, zero, out=out, alpha=2.0, config=config)
        assert bool((out.view(torch.int16) == 0).all())
    w = held(8, 128, 1)[0]
    assert g.gemm_i8(held(0, 128, 1)[0], w).shape == (0, 8)
    assert g.gemm_i8(w, held(0, 128, 1)[0]).shape == (8, 0)


def test_workspace():
    a, w = held(64, 4096, 1)[0], held(512, 4096, 2)[0]
    want = g.gemm_i8(a, w, splits=1)
    need = g.plan_i8(64, 512, 4096, splits=4)["workspace_bytes"]
    assert need == 4 * 64 * 512 * 4
    room = torch.full((need + 32,), 85, dtype=torch.uint8, device=DEV)
    assert torch.equal(g.gemm_i8(a, w, splits=4, workspace=room[16:-16]), want)
    assert bool((room[:16] == 85).all()) and bool((room[-16:] == 85).all())
    with pytest.raises(g.GemmError):
        g.gemm_i8(a, w, splits=4, workspace=room[16:-17])


def test_compressed_product_is_near_the_dense_one():
    """A whole use: activations and weights compressed here; each factor is off by half a code's step at most."""
    gen = torch.Generator().manual_seed(11)
    x, w = torch.randn(33, 1000, generator=gen).to(torch.float16), torch.randn(70, 1000, generator=gen).to(torch.float16)
    xq, wq = g.i8_compress(x.to(DEV)), g.i8_compress(w.to(DEV))
    got = ref.host(g.gemm_i8(xq, wq)).astype(np.float64)
    dx, dw = ref.host(xq.scales).astype(np.float64)[:, None] / 2, ref.host(wq.scales).astype(np.float64)[:, None] / 2
    xd, wd = x.double().numpy(), w.double().numpy()
    most = np.abs(xd).sum(1)[:, None] * dw.T + dx * np.abs(wd).sum(1)[None] + 1000 * dx * dw.T
    assert (np.abs(got - xd @ wd.T) <= most * (1 + 2.0 ** -20) + ref.bound(xd @ wd.T) + most * 2.0 ** -10).all()


def test_splits_captured_and_replayed():
    """Two captured products with workspaces of their own, replayed with eager ones of other inputs between."""
    one, two = ((held(70, 2000, s), held(300, 2000, s + 1)) for s in (1, 3))
    want = [g.gemm_i8(a[0], w[0], splits=4) for a, w in (one, two)]
    (a, _, _), (w, _, _) = one
    codes, scales = a.codes.clone(), a.scales.clone()
    mine, s, graphs = g.I8Matrix(codes, scales, a.k), torch.cuda.Stream(), []
    for config in (3, 6):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = g.gemm_i8(mine, w, splits=4, config=config)
        graphs.append((graph, out))
    other = g.gemm_i8(two[0][0], w, splits=4)
    for i in range(6):
        now = (one, two)[i % 2][0][0]
        codes.copy_(now.codes)
        scales.copy_(now.scales)
        for graph, out in graphs:
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, other if i % 2 else want[0])
            assert torch.equal(g.gemm_i8(two[0][0], two[1][0], splits=4), want[1])
