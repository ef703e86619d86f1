"""GPU tests of the 4-bit paged cache: append (with rotation), read and
attention of single tokens, against tests/q4_reference.py.

Append and read are sequences of single correctly rounded operations and must
equal the reference bit for bit; everything not appended to must stay as it was.

Attention's error against 64 bits, per element of the output: one rounding to
binary16 (half a step), and relative to sum_t p |v|:
* the probabilities: a score passes through at most D / 32 + 40 roundings of
  2^-23 of X = scale log2(e) max_t sum_d |q_d| s (code + z + 128), the size of the
  terms that are added (codes enter with 64 on top, which is taken off again), then exp2 and a subtraction, 2^-21; both in numerator
  and denominator, hence twice;
* P' split into two parts, 2^-20;
* additions: 32 in a matrix instruction, 2 for each block of 32 tokens, 64 for
  the joins of waves and parts, 2^-23 each;
and P' rounded below binary16's normals, at 2^-24 where the largest is at
least 2^12 / 2^3 (the slack before it is rescaled): 15 n 2^-33 max s, n 2^-29 max s.
"""
import numpy as np
import pytest
import torch

import q4_reference as ref
import tiled_dense_gemm_fp16_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KINDS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def noise_cache(pages, heads, page, dim, group, seed):
    """A cache full of arbitrary codes and finite words."""
    c = g.q4_cache(pages, heads, page, dim, group, DEV)
    r = gen(seed)
    for codes, words in ((c.k_codes, c.k_words), (c.v_codes, c.v_words)):
        codes.copy_(torch.randint(-2 ** 31, 2 ** 31, codes.shape, generator=r).to(torch.int32))
        s = (torch.rand(words.shape, generator=r) * 0.3 + 0.01).to(torch.float16).view(torch.int16).to(torch.int32)
        words.copy_(s | torch.randint(0, 16, words.shape, generator=r).to(torch.int32) << 16)
    return c


def clone(c):
    return g.Q4Cache(*(t.clone() for t in c[:4]), c.group)


def arrays(c):
    return ref.Cache(*(ref.host(t) for t in c[:4]), c.group)


def make_table(needs, page, pages, seed, width=None):
    """Shuffled pages for sequences that hold `needs` tokens."""
    order = iter(torch.randperm(pages, generator=gen(seed)).tolist())
    width = width or max(1, max(-(-n // page) for n in needs))
    return [[next(order) if i * page < n else -1 for i in range(width)] for n in needs]


def rotation(positions, rotary):
    f = 10000.0 ** (-np.arange(rotary // 2) * 2.0 / rotary)
    a = np.arange(positions)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def check_append(dim, group, page, past, new, heads=2, q_heads=4, rotary=None, interleaved=False, bad=(), table=None,
                 positions=None, single=False, fused=True, tail=0, in_place=False, seed=0):
    pages, batch = 60, len(past)
    totals = [max(p, 0) + n for p, n in zip(past, new)]
    rows = sum(new) + tail
    tab = make_table(totals, page, pages, seed) if table is None else table
    for b, i, value in bad:
        tab[b][i] = value
    cache = noise_cache(pages, heads, page, dim, group, seed)
    before = arrays(cache)
    qkv = (torch.randn(rows, q_heads + 2 * heads, dim, generator=gen(seed + 1)) * 2).to(torch.float16).to(DEV)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    host = [ref.host(t).astype(np.float32) for t in (q, k, v)]
    rotary = dim if rotary is None else rotary
    positions = len(tab[0]) * page if positions is None else positions
    cos, sin = rotation(positions, rotary) if rotary else (None, None)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    out = q if in_place else torch.full((rows, q_heads, dim), 3.0, dtype=torch.float16, device=DEV)
    print(f"[q4] append dim={dim} group={group} page={page} past={past} new={new}", flush=True)
    got = g.q4_cache_append(cache, k, v, i32(tab), i32(past), starts=None if single else i32(starts), q=q,
                            cos=None if cos is None else torch.tensor(cos, device=DEV),
                            sin=None if sin is None else torch.tensor(sin, device=DEV), interleaved=interleaved, out=out)
    torch.cuda.synchronize()
    assert got is out
    after = arrays(cache)
    want_out = host[0].astype(np.float16) if in_place else np.full((rows, q_heads, dim), 3.0, np.float16)
    for b in range(batch):
        for j in range(new[b]):
            r, pos = starts[b] + j, past[b] + j
            ok = 0 <= pos < len(tab[b]) * page and (not rotary or pos < positions) and 0 <= tab[b][pos // page] < pages
            want_out[r] = 0
            if not ok:
                continue
            turn = (lambda x: ref.rotate(x[r:r + 1], cos[pos:pos + 1], sin[pos:pos + 1], interleaved)[0]) if rotary else (lambda x: x[r])
            want_out[r] = turn(host[0]).astype(np.float16)
            p, s = tab[b][pos // page], pos % page
            for name, x in (("k", turn(host[1])), ("v", host[2][r])):
                cq, z, sc = ref.round_groups(x, group)
                before.q[name][p, s], before.word[name][p, s] = cq, ref.words_of(sc, z)
    for name in ("k", "v"):
        assert np.array_equal(after.word[name], before.word[name]), name
        assert np.array_equal(after.q[name], before.q[name]), name
    assert np.array_equal(ref.host(got), want_out)


@pytest.mark.parametrize("dim,group", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_ragged(dim, group, interleaved):
    check_append(dim, group, 16, [0, 5, 8, 31, 40], [3, 1, 17, 0, 9], interleaved=interleaved)


@pytest.mark.parametrize("page", [8, 24, 64])
def test_append_one_token_each(page):
    for past in ([0, 1, 7, 8, 9, 15, 23, 24], [40, 39, 38, 37, 36, 35, 34, 33]):
        check_append(128, 64, page, past, [1] * 8, single=True)
        check_append(64, 32, page, past, [1] * 8, single=False)


def test_append_partial_and_no_rotation():
    check_append(128, 32, 16, [3, 20], [11, 2], rotary=64)
    check_append(128, 32, 16, [3, 20], [11, 2], rotary=16, interleaved=True)
    check_append(256, 128, 16, [3, 20], [11, 2], rotary=0)


def test_append_contiguous_and_in_place():
    check_append(128, 64, 16, [3, 20, 0], [11, 2, 5], fused=False, in_place=True)
    check_append(64, 64, 16, [3, 20, 0], [11, 2, 5], fused=False, in_place=True, interleaved=True)


def test_append_heads():
    check_append(64, 32, 16, [2, 9], [4, 13], heads=1, q_heads=1)
    check_append(64, 32, 16, [2, 9], [4, 13], heads=3, q_heads=15)


def test_append_out_of_range():
    # pages that are missing or outside the pool, positions past the table's end, before 0 and past the rotation's rows
    check_append(128, 64, 16, [10, 20, 0], [20, 9, 5], bad=[(0, 1, -1), (1, 1, 60), (2, 0, 2 ** 31 - 1)])
    check_append(128, 64, 16, [10, -20, -4], [40, 15, 9], table=[[0, 1], [2, 3], [4, 5]])
    check_append(128, 64, 16, [10, 0], [20, 30], positions=25)
    check_append(128, 64, 16, [2 ** 31 - 3, 0], [5, 1], table=[[0], [1]])


def test_append_rows_of_no_sequence():
    check_append(64, 32, 8, [0, 5], [3, 9], tail=7)


def test_append_many_sequences():
    new = [i % 3 for i in range(150)]
    table = [[i % 40] for i in range(150)]
    # sequences sharing pages write different slots, whole granules apart
    past = [8 * (i // 40) for i in range(150)]
    check_append(64, 64, 64, past, new, heads=1, q_heads=1, table=table, positions=64)


@pytest.mark.parametrize("dim,group", KINDS)
@pytest.mark.parametrize("page", [8, 24])
def test_read(dim, group, page):
    lengths, first = [0, 5, 31, 50], [0, 3, 8, 17]
    cache = noise_cache(30, 3, page, dim, group, 5)
    tab = make_table(lengths, page, 30, 6)
    tab[3][1] = -1
    whole = arrays(cache)
    for begin in (None, first):
        starts, want = [0], {"k": [], "v": []}
        for b, n in enumerate(lengths):
            f = begin[b] if begin else 0
            n = max(0, n - f)
            starts.append(starts[-1] + n)
            for pos in range(f, f + n):
                p = tab[b][pos // page]
                for name in want:
                    want[name].append(whole.values(name)[p, pos % page] if p >= 0 else np.zeros((3, dim)))
        k, v = g.q4_cache_read(cache, i32(tab), i32(starts), starts[-1], first=None if begin is None else i32(begin))
        torch.cuda.synchronize()
        assert np.array_equal(ref.host(k), np.stack(want["k"]).astype(np.float16))
        assert np.array_equal(ref.host(v), np.stack(want["v"]).astype(np.float16))
    assert all(np.array_equal(arrays(cache).q[n], whole.q[n]) for n in ("k", "v"))


def attend(cache, tab, lengths, q, scale, got, page):
    """Compare every head's output with the definition over the tokens whose pages exist."""
    c = arrays(cache)
    values = {n: c.values(n) for n in ("k", "v")}
    s, z = ref.scale_zero(c.word["k"])
    size = np.repeat(s, c.group, -1) * (c.q["k"] + np.repeat(z, c.group, -1) + 128)
    top = ref.scale_zero(c.word["v"])[0].max()
    heads, dim = values["k"].shape[2:]
    ratio = q.shape[1] // heads
    for b, n in enumerate(lengths):
        n = min(max(n, 0), len(tab[b]) * page)
        pos = np.array([p for p in range(n) if 0 <= tab[b][p // page] < values["k"].shape[0]], dtype=np.int64)
        p = np.array(tab[b])[pos // page]
        for h in range(q.shape[1]):
            k, v, w = (x[p, pos % page, h // ratio] for x in (values["k"], values["v"], size))
            want, mass = ref.attention(q[b, h], k, v, scale)
            X = abs(scale) * 1.4427 * (w @ np.abs(q[b, h])).max() if len(pos) else 0.0
            eps = 2 * ((dim / 32 + 40) * 2.0 ** -23 * X + 2.0 ** -21) + 2.0 ** -20 + (96 + len(pos) / 16) * 2.0 ** -23
            tol = ref.half_steps(want) * (1 + 2.0 ** -10) + eps * mass + len(pos) * 2.0 ** -29 * top
            err = np.abs(got[b, h].astype(np.float64) - want)
            assert (err <= tol).all(), (b, h, n, (err / tol).max())


def check_attention(dim, group, page, lengths, q_heads, heads, pages=64, splits=None, scale=None, bad=(), width=None,
                    max_length=None, seed=0, spread=1.0):
    cache = noise_cache(pages, heads, page, dim, group, seed)
    tab = make_table(lengths, page, pages, seed, width)
    for b, i, value in bad:
        tab[b][i] = value
    q = (torch.randn(len(lengths), q_heads, dim, generator=gen(seed + 3)) * spread).to(torch.float16)
    room = torch.full((len(lengths) * q_heads * dim + 32,), 9.0, dtype=torch.float16, device=DEV)
    out = room[16:-16].view(len(lengths), q_heads, dim)
    print(f"[q4] attention dim={dim} group={group} page={page} lengths={lengths} heads={q_heads}/{heads} splits={splits}",
          flush=True)
    g.attention_q4(q.to(DEV), cache, i32(tab), i32(lengths), scale=scale, out=out, splits=splits, max_length=max_length)
    torch.cuda.synchronize()
    attend(cache, tab, lengths, q.double().numpy(), dim ** -0.5 if scale is None else scale, ref.host(out), page)
    assert bool((room[:16] == 9).all()) and bool((room[-16:] == 9).all())


@pytest.mark.parametrize("dim,group", KINDS)
@pytest.mark.parametrize("q_heads,heads", [(2, 2), (8, 2)])
def test_attention_kinds(dim, group, q_heads, heads):
    check_attention(dim, group, 16, [1, 0, 7, 33, 64, 100], q_heads, heads)


@pytest.mark.parametrize("ratio", [1, 3, 15, 16, 17, 40])
def test_attention_ratios(ratio):
    check_attention(64, 32, 8, [5, 40], 2 * ratio, 2)


@pytest.mark.parametrize("page", [8, 24, 40, 256])
@pytest.mark.parametrize("splits", [None, 1, 3, 7])
def test_attention_pages_and_splits(page, splits):
    check_attention(128, 64, page, [0, 1, 31, 32, 33, 200, 257], 4, 1, pages=110, splits=splits)


def steps(dim, group, lengths, q_heads, heads, room, splits=None):
    """Tokens of a wave's step: several blocks where few heads share the columns and the table has room for many tokens."""
    return g.plan_attention_q4(len(lengths), q_heads, heads, dim, group, room, splits)["block_n"]


@pytest.mark.parametrize("dim,group", KINDS)
@pytest.mark.parametrize("ratio", [1, 2, 3, 4, 5, 7, 8])
def test_attention_blocks_side_by_side(dim, group, ratio):
    lengths, width = [1, 0, 7, 33, 64, 100, 129, 300, 31, 128], 1024
    want = 64 if ratio > 4 or dim == 256 else 128
    assert steps(dim, group, lengths, 2 * ratio, 2, 16 * width) == want
    check_attention(dim, group, 16, lengths, 2 * ratio, 2, width=width, pages=80, splits=1)
    check_attention(dim, group, 16, lengths, 2 * ratio, 2, width=width, pages=80, splits=2, seed=1)


@pytest.mark.parametrize("page", [8, 24, 32, 40, 256])
@pytest.mark.parametrize("splits", [None, 3, 9])
@pytest.mark.parametrize("ratio", [3, 6])
def test_attention_blocks_side_by_side_pages(page, splits, ratio):
    lengths, width = [0, 1, 95, 96, 97, 127, 160, 257, 700, 33], 16384 // page
    assert steps(128, 64, lengths, 2 * ratio, 2, page * width) == (128 if ratio == 3 else 64)
    check_attention(128, 64, page, lengths, 2 * ratio, 2, pages=210, splits=splits, width=width)


@pytest.mark.parametrize("ratio", [2, 8])
def test_attention_blocks_side_by_side_scores(ratio):
    # sharp, negative and constant scores; parts that are joined by one team and by several; strided queries
    kw = dict(q_heads=2 * ratio, heads=2, pages=100, width=1024)
    lengths = [90, 300, 0, 500]
    assert steps(128, 64, lengths, 2 * ratio, 2, 16384) == (128 if ratio == 2 else 64)
    check_attention(128, 64, 16, lengths, spread=20.0, splits=2, **kw)
    check_attention(128, 64, 16, lengths, scale=-0.3, splits=8, **kw)
    check_attention(128, 64, 16, lengths, scale=0.0, splits=9, **kw)
    cache = noise_cache(100, 2, 16, 128, 64, 0)
    table = i32(make_table(lengths, 16, 100, 0, 1024))
    wide = torch.randn(4, 4 * ratio, 128, generator=gen(1)).to(torch.float16).to(DEV)
    part = wide[:, ratio:3 * ratio]
    assert torch.equal(g.attention_q4(part, cache, table, i32(lengths)), g.attention_q4(part.contiguous(), cache, table, i32(lengths)))


def test_attention_infinite_queries_stay_in_their_head():
    for width, ratio in ((32, 4), (1024, 4), (1024, 8)):
        cache = noise_cache(100, 2, 16, 128, 64, 0)
        lengths = [90, 300, 40, 500]
        table = i32(make_table(lengths, 16, 100, 0, width))
        q = torch.randn(4, 2 * ratio, 128, generator=gen(1)).to(torch.float16).to(DEV)
        want = g.attention_q4(q, cache, table, i32(lengths))
        odd = q.clone()
        odd[1, 3, 5] = float("inf")
        odd[2, ratio + 1, 7] = float("nan")
        got = g.attention_q4(odd, cache, table, i32(lengths))
        assert not got[1, 3].isfinite().any() and not got[2, ratio + 1].isfinite().any()
        keep = torch.ones(4, 2 * ratio, dtype=torch.bool, device=DEV)
        keep[1, 3] = keep[2, ratio + 1] = False
        assert torch.equal(got[keep], want[keep])


def test_attention_blocks_side_by_side_pages_left_out():
    for page, bad in ((16, [(0, 0, -1), (0, 3, 64), (1, 7, -2), (2, 1, 2 ** 31 - 1)]), (64, [(0, 1, -1), (1, 0, 64), (2, 0, -9)])):
        for ratio in (2, 8):
            for splits in (1, 2):
                lengths = [200, 140, 30] + [5] * 9
                assert steps(128, 64, lengths, 2 * ratio, 2, 16384) == (128 if ratio == 2 else 64)
                check_attention(128, 64, page, lengths, 2 * ratio, 2, bad=bad, splits=splits, width=16384 // page)


def test_attention_blocks_side_by_side_ignores_what_lies_behind():
    # infinite and NaN scales behind the length, in the same blocks and in pages of nobody
    for ratio in (4, 8):
        cache = noise_cache(8, 2, 16, 64, 32, 1)
        tab = torch.full((64, 1024), -1, dtype=torch.int32)
        tab[0, :3], tab[1, 0] = torch.tensor([3, 5, 1], dtype=torch.int32), 0
        tab[0, 3], tab[1, 1] = 2, 4                   # pages behind the last token
        lengths = i32([37, 9] + [0] * 62)
        assert steps(64, 32, lengths, 2 * ratio, 2, 16384) == 512 // ratio
        q = torch.randn(64, 2 * ratio, 64, generator=gen(1)).to(torch.float16).to(DEV)
        want = g.attention_q4(q, cache, tab.to(DEV), lengths).clone()
        junk = clone(cache)
        for words in (junk.k_words, junk.v_words):
            for page, slot in ((1, 5), (0, 9)):
                words[page, ..., slot:] = torch.tensor([0x7FFF7C00, 0xFFFF7E00 - 2 ** 32], dtype=torch.int32, device=DEV).repeat(
                    8)[:16 - slot]
            for page in (2, 4, 6, 7):
                words[page] = -1
        assert torch.equal(g.attention_q4(q, junk, tab.to(DEV), lengths), want)
        assert bool((want[2:] == 0).all()) and bool(want[:2].isfinite().all())


def test_attention_long():
    check_attention(128, 128, 64, [3000, 20], 4, 2, pages=70)
    check_attention(64, 64, 16, [6000], 1, 1, pages=400, splits=256)
    check_attention(256, 64, 128, [5000], 2, 1, pages=48, max_length=1)


def test_attention_peaked_and_scaled():
    check_attention(128, 64, 16, [90, 300], 4, 2, spread=20.0)
    check_attention(128, 64, 16, [90, 300], 4, 2, scale=-0.3)
    check_attention(128, 64, 16, [90, 300], 4, 2, scale=0.0)


def test_attention_pages_left_out_and_lengths_out_of_range():
    check_attention(128, 64, 16, [60, 40, 30], 4, 2, bad=[(0, 1, -1), (1, 0, 64), (2, 0, -5), (2, 1, -1)], splits=1)
    check_attention(128, 64, 16, [60, 40, 30], 4, 2, bad=[(0, 1, -1), (1, 0, 64), (2, 0, -5), (2, 1, -1)], splits=2)
    cache = noise_cache(8, 2, 16, 128, 64, 0)
    q = torch.randn(3, 4, 128, generator=gen(1)).to(torch.float16)
    tab = [[0, 1], [2, 3], [4, 5]]
    out = g.attention_q4(q.to(DEV), cache, i32(tab), i32([1000, -7, 2 ** 31 - 1]))
    attend(cache, tab, [32, 0, 32], q.double().numpy(), 128 ** -0.5, ref.host(out), 16)


def test_attention_ignores_what_lies_behind_the_last_token():
    # infinite and NaN scales and zero points beyond 15 behind the length and in pages of nobody
    for splits in (1, 2):
        cache = noise_cache(8, 1, 16, 64, 32, 1)
        tab, lengths = [[3, 5, 1], [0, -1, -1]], [37, 9]
        q = torch.randn(2, 3, 64, generator=gen(1)).to(torch.float16).to(DEV)
        want = g.attention_q4(q, cache, i32(tab), i32(lengths), splits=splits).clone()
        junk = clone(cache)
        for words in (junk.k_words, junk.v_words):
            for page, slot in ((1, 5), (0, 9)):
                words[page, ..., slot:] = torch.tensor([0x7FFF7C00, 0xFFFF7E00 - 2 ** 32], dtype=torch.int32, device=DEV).repeat(
                    8)[:16 - slot]
            for page in (2, 4, 6, 7):
                words[page] = -1
        junk.k_codes[2] = -1
        got = g.attention_q4(q, junk, i32(tab), i32(lengths), splits=splits)
        assert torch.equal(got, want)


def test_attention_small_scales():
    # scales down to binary16's smallest, next to large ones, in one group's tokens
    cache = noise_cache(8, 1, 16, 64, 32, 1)
    s = torch.tensor([2.0 ** -24, 2.0 ** -14, 1.0, 300.0] * 4).to(torch.float16).view(torch.int16).to(torch.int32).to(DEV)
    cache.v_words.copy_(s.expand(cache.v_words.shape) | 7 << 16)
    q = torch.randn(2, 3, 64, generator=gen(1)).to(torch.float16)
    tab, lengths = [[3, 5, 1], [0, -1, -1]], [37, 1]
    out = g.attention_q4(q.to(DEV), cache, i32(tab), i32(lengths))
    attend(cache, tab, lengths, q.double().numpy(), 0.125, ref.host(out), 16)
    cache.v_words.copy_((cache.v_words & -65536) | 1)          # every scale 2^-24
    out = g.attention_q4(q.to(DEV), cache, i32(tab), i32(lengths))
    attend(cache, tab, lengths, q.double().numpy(), 0.125, ref.host(out), 16)


def test_attention_strided_queries():
    cache = noise_cache(8, 2, 16, 128, 64, 0)
    wide = torch.randn(3, 12, 128, generator=gen(1)).to(torch.float16).to(DEV)
    tab, lengths = i32([[0, 1], [2, 3], [4, 5]]), i32([20, 5, 32])
    assert torch.equal(g.attention_q4(wide[:, 2:6], cache, tab, lengths),
                       g.attention_q4(wide[:, 2:6].contiguous(), cache, tab, lengths))


def test_decode_steps_match_one_prompt():
    # appending token by token gives the cache that one prompt gives, and attention over both is the same
    heads, dim, page, n = 2, 128, 24, 61
    k, v = (torch.randn(n, heads, dim, generator=gen(i)).to(torch.float16).to(DEV) for i in (1, 2))
    cos, sin = (torch.tensor(x, device=DEV) for x in rotation(72, dim))
    tab = i32([[2, 0, 1]])
    whole, step = (g.q4_cache(3, heads, page, dim, 64, DEV) for _ in range(2))
    g.q4_cache_append(whole, k, v, tab, i32([0]), starts=i32([0, n]), cos=cos, sin=sin)
    length = i32([0])
    for t in range(n):
        g.q4_cache_append(step, k[t:t + 1], v[t:t + 1], tab, length, cos=cos, sin=sin)
        length += 1
    assert all(torch.equal(a, b) for a, b in zip(whole[:4], step[:4]))
    q = torch.randn(1, 4, dim, generator=gen(3)).to(torch.float16).to(DEV)
    assert torch.equal(g.attention_q4(q, whole, tab, length), g.attention_q4(q, step, tab, length))
