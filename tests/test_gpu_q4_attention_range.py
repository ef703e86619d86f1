"""GPU tests of attention over 4-bit values whose scales differ widely between
groups of d, between tokens and from step to step: an output's accuracy must
come from its own group's products p s, whatever stands beside it.

The bound per element is that of test_gpu_q4_cache.py but for two parts.  A
score's error is counted with its own token's weight: with relative errors o of
the probabilities, sum p v / sum p is off by at most sum p o |v| + sum p o sum p |v|,
and a token without weight adds nothing however large its score.  The other part
comes from rounding P' = p s below binary16's normals.  P' enters with an
absolute error under 2^-24, times a code difference of at most 15, for each of
n tokens.  The largest P' of a group of d is at least 2^3 (groups within 8 bits
of the largest one share its power of two, which puts that at 2^11 or more; a group
further below is lifted until its own is at least 2^10), so relative to the
group's own largest p s, m, the error is at most n 15 2^-27 m < n 2^-23 m.
"""
import numpy as np
import pytest
import torch

import q4_reference as ref
import tiled_dense_gemm_fp16_amd as g
from test_gpu_q4_cache import KINDS, arrays, gen, i32, make_table, noise_cache

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SMALL, TINY, ONE, LARGE = 2.0 ** -14, 2.0 ** -24, 1.0, 4096.0     # 15 x 4096 is below binary16's largest


def attend(cache, tab, lengths, q, scale, got, page, exact=False):
    """Every head's output against the definition, with each group's own largest p s in its bound.  Returns how many
    elements are large against their bound.  exact: scores have no error."""
    c = arrays(cache)
    keys, values = c.values("k"), c.values("v")
    ks, kz = ref.scale_zero(c.word["k"])
    size = np.repeat(ks, c.group, -1) * (c.q["k"] + np.repeat(kz, c.group, -1) + 128)
    vs = np.repeat(ref.scale_zero(c.word["v"])[0], c.group, -1)
    heads, dim = values.shape[2:]
    ratio, checked = q.shape[1] // heads, 0
    for b, n in enumerate(lengths):
        pos = np.array([t for t in range(n) if tab[b][t // page] >= 0], dtype=np.int64)
        if not len(pos):
            assert (got[b] == 0).all()
            continue
        at = np.array(tab[b])[pos // page]
        for h in range(q.shape[1]):
            k, v, w, s = (x[at, pos % page, h // ratio] for x in (keys, values, size, vs))
            x = k @ q[b, h] * scale
            p = np.exp(x - x.max())
            p /= p.sum()
            want, mass, most = p @ v, p @ np.abs(v), (p[:, None] * s).max(0)
            off = (dim / 32 + 40) * 2.0 ** -23 * abs(scale) * 1.4427 * (w @ np.abs(q[b, h])) * (not exact) + 2.0 ** -21   # of p
            eps = 2.0 ** -20 + (96 + len(pos) / 16) * 2.0 ** -23
            tol = (ref.half_steps(want) * (1 + 2.0 ** -10) + (p * off) @ np.abs(v) + (p @ off + eps) * mass +
                   len(pos) * 2.0 ** -23 * most)
            err = np.abs(got[b, h].astype(np.float64) - want)
            assert (err <= tol).all(), (b, h, n, (err / tol).max())
            checked += int((np.abs(want) > 64 * tol).sum())
    return checked


def set_scales(cache, scales):
    """v_words with these scales (broadcast to [pages, heads, groups, slots]) and zero point 7."""
    s = torch.as_tensor(scales, dtype=torch.float32).expand(cache.v_words.shape)
    cache.v_words.copy_((s.to(torch.float16).contiguous().view(torch.int16).to(torch.int32) & 0xFFFF) | 7 << 16)


def run(cache, tab, lengths, q_heads, page, scale=None, splits=None, spread=1.0, seed=0):
    dim = cache.k_codes.shape[3] * 8
    q = (torch.randn(len(lengths), q_heads, dim, generator=gen(seed)) * spread).to(torch.float16)
    got = g.attention_q4(q.to(DEV), cache, i32(tab), i32(lengths), scale=scale, splits=splits)
    torch.cuda.synchronize()
    return attend(cache, tab, lengths, q.double().numpy(), dim ** -0.5 if scale is None else scale, ref.host(got), page)


WIDE = 16384       # room for as many tokens makes steps of several blocks where few heads share a cache head


@pytest.mark.parametrize("dim,group", [k for k in KINDS if k[0] > k[1]])
@pytest.mark.parametrize("ratio", [2, 8, 16])
def test_groups_with_scales_of_their_own(dim, group, ratio):
    lengths, page = [1, 40, 300, 90], 16
    tab = make_table(lengths, page, 64, 1, WIDE // page)
    for turn in range(4):
        cache = noise_cache(64, 2, page, dim, group, turn)
        size = ([LARGE, SMALL, ONE, TINY, 300.0, 2.0 ** -8, 2.0 ** -19, 2.0 ** -3] * 2)[turn:turn + dim // group]
        set_scales(cache, torch.tensor(size)[:, None])
        print(f"[q4] range dim={dim} group={group} ratio={ratio} turn={turn}", flush=True)
        for splits in (1, 2):
            checked = run(cache, tab, lengths, 2 * ratio, page, splits=splits, seed=turn)
            assert checked > 0


@pytest.mark.parametrize("dim,group", KINDS)
@pytest.mark.parametrize("ratio", [2, 8, 16])
@pytest.mark.parametrize("where", [0, 33, 89])
def test_a_large_token_without_weight(dim, group, ratio, where):
    """One token's values are large, its score is so low that it does not count; the others are small."""
    page, lengths = 16, [90]
    tab = make_table(lengths, page, 8, 1, WIDE // page)
    cache = noise_cache(8, 1, page, dim, group, 3)
    cache.k_words.zero_()                                          # scores 0 ...
    scales = torch.full((8, 1, 1, page), SMALL)
    scales[tab[0][where // page], ..., where % page] = LARGE
    set_scales(cache, scales)
    cache.k_words[tab[0][where // page], ..., where % page] = 0x3C00   # ... but this one's: codes times 1
    cache.k_codes[tab[0][where // page], :, where % page] = -1         # (15 everywhere)
    q = torch.full((1, ratio, dim), -1.0, dtype=torch.float16)
    for splits in (1, 3):
        got = g.attention_q4(q.to(DEV), cache, i32(tab), i32(lengths), scale=8.0 / dim, splits=splits)     # e^-120
        checked = attend(cache, tab, lengths, q.double().numpy(), 8.0 / dim, ref.host(got), page)
        assert checked > 0


@pytest.mark.parametrize("dim,group", KINDS)
@pytest.mark.parametrize("ratio", [1, 6, 16])
def test_scales_of_any_size(dim, group, ratio):
    """Scales from 0 and 2^-24 to 4096 at random for every token and group, flat and sharp scores."""
    lengths, page = [3, 33, 128, 400], 24
    tab = make_table(lengths, page, 40, 1, WIDE // page)
    for seed in range(4):
        cache = noise_cache(40, 2, page, dim, group, seed)
        r = gen(seed + 9)
        size = 2.0 ** torch.randint(-24, 13, cache.v_words.shape, generator=r).float()
        size[torch.rand(cache.v_words.shape, generator=r) < 0.1] = 0.0
        set_scales(cache, size)
        for spread in (0.1, 1.0, 8.0):
            run(cache, tab, lengths, 2 * ratio, page, spread=spread, seed=seed, splits=1 + seed % 3)


@pytest.mark.parametrize("rising", [True, False])
def test_scales_that_move_with_the_scores(rising):
    """Scores along the sequence rise (or fall) by many powers of two while scales fall (or rise), and tokens of scale 0 stand
    before all others."""
    dim, group, page, n = 128, 64, 16, 512
    tab = make_table([n], page, 32, 1, WIDE // page)
    cache = noise_cache(32, 1, page, dim, group, 5)
    order = torch.arange(n) if rising else torch.arange(n).flip(0)
    cache.k_codes.fill_(-1)
    cache.k_words.zero_()
    size = torch.zeros(32, 1, 1, page)
    for t in range(n):
        p, slot = tab[0][t // page], t % page
        s = torch.tensor(order[t].item() * 2.0 ** -9).to(torch.float16)          # key = 15 s everywhere
        cache.k_words[p, ..., slot] = int(s.view(torch.int16)) & 0xFFFF
        size[p, ..., slot] = 0.0 if t < 20 else 2.0 ** (12 - 36 * order[t].item() / n)
    set_scales(cache, size)
    q = torch.full((1, 4, dim), 1.0, dtype=torch.float16)
    for scale in (1.0 / 64, 1.0 / 16):                              # 15 x 128 x scale: e^30, e^120 from end to end
        for splits in (1, 2, None):
            got = g.attention_q4(q.to(DEV), cache, i32(tab), i32([n]), scale=scale, splits=splits)
            attend(cache, tab, [n], q.double().numpy(), scale, ref.host(got), page)


@pytest.mark.parametrize("dim,group", KINDS)
@pytest.mark.parametrize("ratio", [1, 8, 16])
@pytest.mark.parametrize("power", [16, 20, 23, 24, 26, 30, 36])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(dim, group, ratio, power, sign):
    """Scores up to 2^36: the tokens with the largest one share the weight, all others are far behind.

    Every element of a key is s times a code difference, of a query 1 or -1, so that a token's score is dim times a small
    integer times a power of two, exact in fp32, equal for equal tokens and at least 2^13 apart for others; the output is
    the mean of the first ones' values."""
    page, lengths, order = 16, [200, 33, 1], gen(power)
    tab = make_table(lengths, page, 24, 1, WIDE // page)
    cache = noise_cache(24, 1, page, dim, group, power)
    steps = torch.randint(9, 16, (24, page), generator=order) - 8          # 1 .. 7
    cache.k_codes.copy_(((steps + 8) * 0x11111111 - (1 << 32)).to(torch.int32)[:, None, :, None].expand(cache.k_codes.shape))
    unit = 2.0 ** (power - 3) / dim                                         # scores: steps times unit times dim
    key = min(unit, 2.0 ** 12)
    cache.k_words.fill_((int(torch.tensor(key).to(torch.float16).view(torch.int16)) & 0xFFFF) | 8 << 16)
    q = torch.full((3, ratio, dim), float(sign), dtype=torch.float16)
    scale = unit / key
    for splits in (1, 2, 5):
        got = g.attention_q4(q.to(DEV), cache, i32(tab), i32(lengths), scale=scale, splits=splits)
        checked = attend(cache, tab, lengths, q.double().numpy(), scale, ref.host(got), page, exact=True)
        assert checked > 0


@pytest.mark.parametrize("dim,group", KINDS)
@pytest.mark.parametrize("ratio", [1, 4, 8, 16])
def test_scales_of_any_size_in_whole_pages(dim, group, ratio):
    """As test_scales_of_any_size, in pages that hold whole blocks of tokens, with pages left out and empty sequences."""
    lengths, page = [3, 0, 65, 128, 500, 31], 64
    for seed in range(4):
        tab = make_table(lengths, page, 24, seed, WIDE // page if seed % 2 else None)
        tab[4][2] = tab[3][0] = -1
        cache = noise_cache(24, 2, page, dim, group, seed)
        r = gen(seed + 19)
        size = 2.0 ** torch.randint(-24, 13, cache.v_words.shape, generator=r).float()
        size[torch.rand(cache.v_words.shape, generator=r) < 0.1] = 0.0
        set_scales(cache, size)
        for spread in (0.3, 4.0):
            run(cache, tab, lengths, 2 * ratio, page, spread=spread, seed=seed, splits=(1, 2, 5, None)[seed])


def test_far_scores_stay_in_their_head():
    """A head whose scores pass 2^23, and one with groups far apart, do not change a bit of the heads beside them."""
    for width, ratio in ((32, 4), (1024, 4), (1024, 8)):
        cache = noise_cache(100, 2, 16, 128, 64, 0)
        lengths = [90, 300, 40, 500]
        table = i32(make_table(lengths, 16, 100, 0, width))
        q = torch.randn(4, 2 * ratio, 128, generator=gen(1)).to(torch.float16).to(DEV)
        want = g.attention_q4(q, cache, table, i32(lengths))
        odd = q.clone()
        odd[1, 3] *= 2.0 ** 14
        odd[2, ratio + 1] *= -2.0 ** 12
        scale = 128 ** -0.5
        got = g.attention_q4(odd, cache, table, i32(lengths), scale=scale)
        keep = torch.ones(4, 2 * ratio, dtype=torch.bool, device=DEV)
        keep[1, 3] = keep[2, ratio + 1] = False
        assert torch.equal(got[keep], want[keep]) and bool(got.isfinite().all())
        huge = q.clone()
        huge[0, 0], huge[3, 2 * ratio - 1] = 60000.0, -60000.0
        got = g.attention_q4(huge, cache, table, i32(lengths), scale=1000.0)
        want = g.attention_q4(q, cache, table, i32(lengths), scale=1000.0)
        keep = torch.ones(4, 2 * ratio, dtype=torch.bool, device=DEV)
        keep[0, 0] = keep[3, 2 * ratio - 1] = False
        assert torch.equal(got[keep], want[keep]) and bool(got.isfinite().all())
