"""GPU tests of rows in 8 bits: codes and scales are the definition's bit for bit."""
import numpy as np
import pytest
import torch

import i8_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def rows(r, k, seed):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(r, k, generator=gen) * torch.exp(2 * torch.randn(r, 1, generator=gen))).to(torch.float16)


def same(x, packed):
    codes, scales = ref.compress(ref.host(x))
    assert np.array_equal(ref.host(packed.codes), codes) and np.array_equal(ref.host(packed.scales), scales)
    assert packed.k == x.shape[-1]
    # one rounding of the product to fp32 and one to binary16
    want = ref.expand(codes, scales, packed.k)
    got = ref.host(g.i8_expand(packed)).astype(np.float64)
    assert (np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -11, 2.0 ** -25) * (1 + 2.0 ** -12)).all()


@pytest.mark.parametrize("r,k", [(1, 1), (3, 15), (5, 16), (17, 17), (33, 100), (16, 255), (9, 256), (7, 257), (4, 1000), (6, 2048),
                                 (3, 2049), (5, 4100), (2, 8192), (3, 8200), (2, 28672), (1, 131071)])
def test_rows(r, k):
    print(f"[i8] compress {r}x{k}", flush=True)
    x = rows(r, k, r + k)
    same(x, g.i8_compress(x.to(DEV)))


def test_quotients_next_to_a_half():
    # every binary16 in (0, 1] under the largest magnitudes 1, 1 + 2^-10, ...: with m = 1 the code of 1/2 is a tie
    bits = np.arange(1, 0x3C01, dtype=np.uint16)
    x = bits.view(np.float16)
    for most in (1.0, 1.0009765625, 1.5, 1.984375, 1.9990234375):
        x2 = torch.from_numpy(np.concatenate([x, -x, [np.float16(most)]])[None])
        same(x2, g.i8_compress(x2.to(DEV)))
    half = torch.tensor([[2.0 * v, v, -v, 3 * v / 2] for v in (2.0 ** -24, 2.0 ** -20, 1.0, 100.0)], dtype=torch.float16)
    packed = g.i8_compress(half.to(DEV))
    same(half, packed)
    assert ref.host(packed.codes)[2, 1] == 64 and ref.host(packed.codes)[2, 2] == -64      # 63.5 to the even code


def test_special_values():
    x = torch.zeros(8, 40, dtype=torch.float16)
    x[0, 3], x[0, 4] = float("nan"), 3.0
    x[1, 0], x[1, 1] = float("inf"), -2.0
    x[2, 7] = float("-inf")
    x[3, 0], x[3, 39] = 65504.0, -65504.0
    x[4, 0] = 2.0 ** -24
    x[5] = -0.0
    x[6] = float("nan")
    same(x, g.i8_compress(x.to(DEV)))


@pytest.mark.parametrize("shift,stride", [(1, 137), (0, 200), (3, 131), (8, 144)])
def test_rows_apart_and_unaligned(shift, stride):
    base = rows(1, 24 * stride + 16, 5)[0].to(DEV)
    x = base[shift:shift + 24 * stride].view(24, stride)[:, :130]
    same(x.cpu(), g.i8_compress(x))
    same(x[3:4].cpu(), g.i8_compress(x[3:4]))
    cube = base[shift:shift + 24 * stride].view(4, 6, stride)[:, :, 1:100]
    packed = g.i8_compress(cube)
    assert packed.codes.shape == (4, 6, 128)
    same(cube.cpu(), packed)
    out = torch.full((24 * 130 + 9,), 7.0, dtype=torch.float16, device=DEV)
    g.i8_expand(g.i8_compress(x), out=out[1:-8].view(24, 130))
    assert torch.equal(out[1:-8].view(24, 130), g.i8_expand(g.i8_compress(x)))
    assert bool((out[:1] == 7).all()) and bool((out[-8:] == 7).all())


def test_nothing_beside_the_codes_is_written():
    for r, k in [(3, 17), (4, 65), (5, 300), (2, 4100)]:
        x = rows(r, k, 1).to(DEV)
        pitch = ref.pitch(k)
        room = torch.full((r * pitch + 64,), 77, dtype=torch.int8, device=DEV)
        scales = torch.full((r + 2,), 7.0, device=DEV)
        st = g.lib().gemm_f16_i8_compress(r, k, x.data_ptr(), k, room[32:].data_ptr(), scales[1:].data_ptr(),
                                          torch.cuda.current_stream().cuda_stream)
        assert st == 0
        codes, want = ref.compress(ref.host(x))
        assert np.array_equal(ref.host(room[32:-32]).reshape(r, pitch), codes) and np.array_equal(ref.host(scales[1:-1]), want)
        assert bool((room[:32] == 77).all()) and bool((room[-32:] == 77).all()) and scales[0] == 7 and scales[-1] == 7


def test_wide_pitch_and_empty():
    x = rows(5, 40, 3)
    codes, scales = ref.compress(ref.host(x))
    wide = np.full((5, 96), 55, np.int8)
    wide[:, :48] = codes
    back = g.i8_expand(g.I8Matrix(torch.from_numpy(wide).to(DEV), torch.from_numpy(scales).to(DEV), 40))
    assert torch.equal(back, g.i8_expand(g.i8_compress(x.to(DEV))))
    for shape in [(0, 8), (3, 0), (0, 0), (2, 0, 5)]:
        packed = g.i8_compress(torch.zeros(shape, dtype=torch.float16, device=DEV))
        assert packed.scales.shape == shape[:-1] and bool((packed.scales == 0).all())
        assert g.i8_expand(packed).shape == shape


def test_expand_of_any_codes():
    codes = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).view(1, 256).repeat(4, 1).to(DEV)
    scales = torch.tensor([1.0, 2.0 ** -24, 1000.0, -0.37], device=DEV)
    got = ref.host(g.i8_expand(g.I8Matrix(codes, scales, 250))).astype(np.float64)
    want = ref.expand(ref.host(codes), ref.host(scales), 250)
    assert ref.near(got, want).all()


@pytest.mark.parametrize("t,j,n", [(1, 1, 1), (3, 8, 100), (64, 8, 4096), (5, 2, 33), (2, 3, 7), (300, 6, 1000), (4, 64, 24)])
def test_expert_sum(t, j, n):
    gen = torch.Generator().manual_seed(t * j + n)
    y = torch.randn(t, j, n, generator=gen).to(torch.float16)
    w = torch.rand(t, j, generator=gen)
    room = torch.full((t * n + 10,), 9.0, dtype=torch.float16, device=DEV)
    out = room[5:-5].view(t, n)
    assert g.expert_sum(y.to(DEV), w.to(DEV), out=out) is out
    want = (y.double() * w.double()[..., None]).sum(1).numpy()
    # j multiply-adds in fp32, each off by 2^-24 of a partial sum, then one rounding to binary16
    size = (y.double().abs() * w.double()[..., None]).sum(1).numpy()
    err = np.abs(ref.host(out).astype(np.float64) - want)
    assert (err <= np.maximum(np.abs(want) * 2.0 ** -11, 2.0 ** -25) * (1 + 2.0 ** -10) + j * 2.0 ** -23 * size).all()
    assert bool((room[:5] == 9).all()) and bool((room[-5:] == 9).all())
    assert torch.equal(g.expert_sum(y.to(DEV), w.to(DEV)), out)


def test_expert_sum_empty():
    out = g.expert_sum(torch.zeros(3, 0, 20, dtype=torch.float16, device=DEV), torch.zeros(3, 0, device=DEV))
    assert out.shape == (3, 20) and bool((out == 0).all())
    assert g.expert_sum(torch.zeros(0, 4, 20, dtype=torch.float16, device=DEV), torch.zeros(0, 4, device=DEV)).shape == (0, 20)
