"""GPU tests of the 4-bit operators used together: the projections, the cache
and the attention of a decoding layer, run eagerly, captured and replayed, on
other streams and with workspaces of the caller.

Each stage of a step is compared with the 64-bit definition at what the stage
before it gave, so that each is held to its own bound: the product's and the
attention's as derived in test_gpu_q4_weights.py and test_gpu_q4_cache.py, and
equality for the cache.  Replays must equal the eager results bit for bit:
every sum has a fixed order.
"""
import numpy as np
import pytest
import torch

import q4_reference as ref
import tiled_dense_gemm_fp16_amd as g
from test_gpu_q4_cache import arrays, attend, clone, gen, i32, make_table, noise_cache, rotation
from test_gpu_q4_weights import ROUNDED, bound, weights

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


class Layer:
    """The attention half of a decoding layer: one projection to queries, keys
    and values, the cache, attention, one projection back."""

    def __init__(self, batch, hidden, q_heads, heads, dim, page, width, group, cache_group, seed=0):
        self.q_heads, self.heads, self.dim, self.page, self.batch = q_heads, heads, dim, page, batch
        rows = (q_heads + 2 * heads) * dim
        self.w_in = g.q4_compress((weights(rows, hidden, seed) * hidden ** -0.5).to(DEV), group)
        self.w_out = g.q4_compress((weights(hidden, q_heads * dim, seed + 2) * (q_heads * dim) ** -0.5).to(DEV), group)
        pages = batch * width
        self.cache = noise_cache(pages, heads, page, dim, cache_group, seed)
        self.tab = make_table([width * page] * batch, page, pages, seed, width)
        self.table = i32(self.tab)
        self.angles = rotation(width * page, dim)
        self.cos, self.sin = (torch.tensor(t, device=DEV) for t in self.angles)

    def step(self, x, lengths, split=None, parts=None, workspaces=(None, None), stream=None):
        """One token of each sequence; lengths grows by one. (all stages' results)"""
        at, out = workspaces
        qkv = g.gemm_q4(x, self.w_in, splits=split, workspace=at, stream=stream).view(self.batch, -1, self.dim)
        q, k, v = qkv.split([self.q_heads, self.heads, self.heads], 1)
        q = g.q4_cache_append(self.cache, k, v, self.table, lengths, q=q, cos=self.cos, sin=self.sin, stream=stream)
        lengths += 1
        o = g.attention_q4(q, self.cache, self.table, lengths, splits=parts, workspace=out, stream=stream)
        y = g.gemm_q4(o.view(self.batch, -1), self.w_out, splits=split, workspace=at, stream=stream)
        return qkv, q, o, y

    def check_product(self, a, w, got):
        m, k = a.shape
        dense = ref.unpack_weights(ref.host(w.codes), ref.host(w.words), w.n, w.k, w.group)
        want, size = ref.product(a.cpu().double().numpy(), dense)
        tol = bound(want, size, w.k, w.group, g.plan_q4(m, w.n, k, w.group, splits=None)["config"] in ROUNDED)
        assert (np.abs(ref.host(got).reshape(m, -1).astype(np.float64) - want) <= tol).all()

    def check_step(self, x, past, before, results):
        """Every stage of a step from `past` tokens over the cache's arrays `before`."""
        qkv, q, o, y = results
        after = arrays(self.cache)
        self.check_product(x, self.w_in, qkv)
        new = ref.host(qkv).astype(np.float32)
        cos, sin = (t[past] for t in self.angles)
        turned = ref.rotate(new[:, :self.q_heads + self.heads], cos, sin, False)
        assert np.array_equal(ref.host(q), turned[:, :self.q_heads].astype(np.float16))
        for b, n in enumerate(past):
            p, s = self.tab[b][n // self.page], n % self.page
            for name, rows in (("k", turned[b, self.q_heads:]), ("v", new[b, self.q_heads + self.heads:])):
                codes, z, scale = ref.round_groups(rows, before.group)
                before.q[name][p, s], before.word[name][p, s] = codes, ref.words_of(scale, z)
        for name in ("k", "v"):
            assert np.array_equal(after.q[name], before.q[name]) and np.array_equal(after.word[name], before.word[name])
        attend(self.cache, self.tab, [n + 1 for n in past], q.cpu().double().numpy(), self.dim ** -0.5, ref.host(o), self.page)
        self.check_product(o.view(self.batch, -1), self.w_out, y)


def copies(tensors):
    return [t.clone() for t in tensors]


@pytest.mark.parametrize("batch,hidden,q_heads,heads,dim,page,width,group,cache_group", [
    (1, 512, 8, 2, 64, 16, 40, 128, 64),         # one sequence, in parts
    (3, 520, 4, 4, 128, 24, 3, 64, 32),          # ragged hidden size, pages that end inside a block
    (5, 264, 6, 1, 256, 8, 12, 32, 128),         # one key head
    (48, 256, 4, 2, 64, 32, 2, 128, 32),         # a batch for the tile products
])
def test_decoding_steps(batch, hidden, q_heads, heads, dim, page, width, group, cache_group):
    layer = Layer(batch, hidden, q_heads, heads, dim, page, width, group, cache_group)
    past = torch.randint(0, width * page - 3, (batch,), generator=gen(batch)).tolist()
    past[0] = width * page - 3                   # the last step fills this sequence's pages
    lengths = i32(past)
    x = torch.randn(batch, hidden, generator=gen(9)).to(torch.float16).to(DEV)
    for i in range(3):
        print(f"[q4] step {i} batch={batch} hidden={hidden} heads={q_heads}/{heads} dim={dim}", flush=True)
        before = arrays(layer.cache)
        results = layer.step(x, lengths)
        torch.cuda.synchronize()
        layer.check_step(x, [n + i for n in past], before, results)
        x = results[-1]
    assert lengths.tolist() == [n + 3 for n in past]


def test_prompt_then_decoding():
    # a ragged batch of prompts through the same weights and pages, then single tokens
    layer = Layer(3, 256, 4, 2, 64, 16, 6, 64, 64)
    new = [37, 0, 5]
    starts = i32([0, 37, 37, 42])
    x = torch.randn(42, 256, generator=gen(3)).to(torch.float16).to(DEV)
    lengths = i32([0, 0, 0])
    qkv = g.gemm_q4(x, layer.w_in).view(42, -1, 64)
    layer.check_product(x, layer.w_in, qkv)
    g.q4_cache_append(layer.cache, qkv[:, 4:6], qkv[:, 6:], layer.table, lengths, starts=starts, cos=layer.cos, sin=layer.sin)
    k, v = g.q4_cache_read(layer.cache, layer.table, starts, 42)
    rows = ref.host(qkv).astype(np.float32)
    at = np.concatenate([np.arange(n) for n in new])
    keys = ref.rotate(rows[:, 4:6], *(t[at] for t in layer.angles), False)
    for got, want in ((k, keys), (v, rows[:, 6:])):
        codes, z, scale = ref.round_groups(want, 64)
        want = scale[..., None].astype(np.float64) * (codes.reshape(*z.shape, 64) - z[..., None])
        assert np.array_equal(ref.host(got), want.reshape(42, 2, 64).astype(np.float16))
    lengths += i32(new)
    for i in range(2):
        before = arrays(layer.cache)
        results = layer.step(x[:3], lengths)
        layer.check_step(x[:3], [n + i for n in new], before, results)


@pytest.mark.parametrize("split,parts", [(None, None), (2, 3), (1, 1)])
def test_captured_steps(split, parts):
    """A step captured once and replayed for the next tokens, with eager work
    and synchronisations between: each replay equals the eager step."""
    layer = Layer(2, 512, 8, 2, 64, 16, 20, 128, 64)
    start = clone(layer.cache)
    x = torch.randn(2, 512, generator=gen(1)).to(torch.float16).to(DEV)
    lengths = i32([30, 250])
    eager = []
    for _ in range(4):
        eager.append(copies(layer.step(x, lengths, split, parts)))
    end = copies(layer.cache[:4])
    for t, s in zip(layer.cache[:4], start[:4]):
        t.copy_(s)
    lengths.copy_(i32([30, 250]))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        results = layer.step(x, lengths, split, parts)
    other = Layer(3, 264, 4, 2, 64, 8, 8, 64, 32, seed=5)
    other_x = torch.randn(3, 264, generator=gen(2)).to(torch.float16).to(DEV)
    for want in eager:
        for t in results:
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results, want))
        other.step(other_x, i32([3, 0, 20]), 2, 2)         # eager split work between the replays
        torch.cuda.synchronize()
    assert lengths.tolist() == [34, 254]
    assert all(torch.equal(a, b) for a, b in zip(layer.cache[:4], end))
    del graph


def test_two_graphs_with_a_workspace_each():
    """Two captured steps with workspaces of the caller, replayed in turn and at the same time."""
    layers = [Layer(2, 512, 8, 2, 64, 16, 20, 128, 64, seed=i) for i in (0, 7)]
    x = torch.randn(2, 512, generator=gen(1)).to(torch.float16).to(DEV)
    rooms = [(torch.empty(2 * 2 * 768 * 4, dtype=torch.uint8, device=DEV),
              torch.empty(2 * 8 * 3 * 66 * 4, dtype=torch.uint8, device=DEV)) for _ in layers]
    start, lengths = i32([30, 250]), [i32([30, 250]) for _ in layers]
    eager = [copies(layer.step(x, i32([30, 250]), 2, 3)) for layer in layers]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in layers]
    for layer, room, n, s in zip(layers, rooms, lengths, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            torch.add(start, 0, out=n)
            outs.append(layer.step(x, n, 2, 3, room))
        graphs.append(graph)
    for _ in range(3):
        for out in outs:
            for t in out:
                t.fill_(7.0)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for out, want in zip(outs, eager):
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        x.add_(0.0)                                          # eager work between the replays
        torch.cuda.synchronize()
    del graphs


def test_streams():
    """torch's current stream by default, `stream` when it is given."""
    layer = Layer(2, 512, 8, 2, 64, 16, 20, 128, 64)
    start = clone(layer.cache)
    x = torch.randn(2, 512, generator=gen(1)).to(torch.float16).to(DEV)
    want = copies(layer.step(x, i32([30, 250]), 2, 3))
    side = torch.cuda.Stream()
    for given in (False, True):
        for t, s in zip(layer.cache[:4], start[:4]):
            t.copy_(s)
        lengths = i32([30, 250])
        side.wait_stream(torch.cuda.current_stream())
        if not given:
            with torch.cuda.stream(side):
                got = layer.step(x, lengths, 2, 3)
        else:
            qkv = g.gemm_q4(x, layer.w_in, splits=2, stream=side).view(2, -1, 64)
            q, k, v = qkv.split([8, 2, 2], 1)
            q = g.q4_cache_append(layer.cache, k, v, layer.table, lengths, q=q, cos=layer.cos, sin=layer.sin, stream=side)
            with torch.cuda.stream(side):
                lengths += 1
            o = g.attention_q4(q, layer.cache, layer.table, lengths, splits=3, stream=side)
            got = qkv, q, o, g.gemm_q4(o.view(2, -1), layer.w_out, splits=2, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()


def test_weights_on_a_stream():
    w = weights(100, 300, 4).to(DEV)
    want = g.q4_compress(w, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = g.q4_compress(w, 64, stream=side)
    back = g.q4_expand(got, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.words, want.words)
    assert torch.equal(back, g.q4_expand(want))
    torch.cuda.synchronize()


def test_workspaces():
    layer = Layer(2, 512, 8, 2, 64, 16, 20, 128, 64)
    x = torch.randn(2, 512, generator=gen(1)).to(torch.float16).to(DEV)
    lengths = i32([31, 251])
    q = torch.randn(2, 8, 64, generator=gen(2)).to(torch.float16).to(DEV)
    product, attention = g.gemm_q4(x, layer.w_in, splits=2), g.attention_q4(q, layer.cache, layer.table, lengths, splits=3)
    need = g.plan_q4(2, 768, 512, 128, splits=2)["workspace_bytes"], g.plan_attention_q4(2, 8, 2, 64, 64, 320, 3)["workspace_bytes"]
    assert need == (2 * 2 * 768 * 4, 2 * 8 * 3 * 66 * 4)
    calls = (lambda ws: g.gemm_q4(x, layer.w_in, splits=2, workspace=ws),
             lambda ws: g.attention_q4(q, layer.cache, layer.table, lengths, splits=3, workspace=ws))
    for call, size, want in zip(calls, need, (product, attention)):
        room = torch.full((size + 32,), 85, dtype=torch.uint8, device=DEV)     # exactly what it needs, and guards
        assert torch.equal(call(room[16:-16]), want)
        assert bool((room[:16] == 85).all()) and bool((room[-16:] == 85).all())
        room.fill_(255)                                                         # NaN: nothing is read before it is written
        assert torch.equal(call(room[16:-16]), want)
        for bad in (room[16:-17], room[8:], room[:0]):                          # short, misaligned, none
            with pytest.raises(g.GemmError):
                call(bad)
        with pytest.raises(ValueError):
            call(torch.empty(size, dtype=torch.uint8))
    room = torch.full((64,), 85, dtype=torch.uint8, device=DEV)                 # one that a whole run leaves alone
    whole = g.attention_q4(q, layer.cache, layer.table, lengths, splits=1)
    assert torch.equal(g.attention_q4(q, layer.cache, layer.table, lengths, splits=1, workspace=room), whole)
    assert torch.equal(g.gemm_q4(x, layer.w_in, splits=1, workspace=room), g.gemm_q4(x, layer.w_in, splits=1))
    assert bool((room == 85).all())
    torch.cuda.synchronize()


def test_repeated_calls_are_bitwise_equal():
    for m, n, k, splits in ((1, 1000, 4096, 4), (40, 520, 2048, 3), (300, 264, 1024, None)):
        w = g.q4_compress(weights(n, k, m).to(DEV), 64)
        a = torch.randn(m, k, generator=gen(m)).to(torch.float16).to(DEV)
        want = g.gemm_q4(a, w, splits=splits)
        assert all(torch.equal(g.gemm_q4(a, w, splits=splits), want) for _ in range(5))
    cache = noise_cache(120, 2, 16, 128, 64, 0)
    table, lengths = i32(make_table([900, 700], 16, 120, 0)), i32([900, 700])
    q = torch.randn(2, 4, 128, generator=gen(1)).to(torch.float16).to(DEV)
    want = g.attention_q4(q, cache, table, lengths)
    assert all(torch.equal(g.attention_q4(q, cache, table, lengths), want) for _ in range(5))


def test_sequences_share_pages():
    # a common beginning held once: two rows of the table name the same pages
    cache = noise_cache(6, 2, 16, 128, 64, 0)
    tab, lengths = [[0, 1, 2], [0, 1, 3], [0, 1, -1]], [40, 47, 32]
    q = torch.randn(3, 4, 128, generator=gen(1)).to(torch.float16)
    out = g.attention_q4(q.to(DEV), cache, i32(tab), i32(lengths))
    attend(cache, tab, lengths, q.double().numpy(), 128 ** -0.5, ref.host(out), 16)


@pytest.mark.parametrize("dim,page", [(256, 64), (64, 24)])
def test_offsets_beyond_32_bits(dim, page):
    """Pages whose codes lie beyond 2^32 bytes (their count times a page's bytes), the last of them used."""
    heads, group = 8, 64
    pages = (1 << 32) // (heads * page * dim // 2) + 3
    cache = g.q4_cache(pages, heads, page, dim, group, DEV)
    assert cache.k_codes.numel() * 4 > 1 << 32
    tab = [[pages - 1, 0], [1, pages - 2]]
    n = page + 3
    k, v = (torch.randn(2 * n, heads, dim, generator=gen(i)).to(torch.float16).to(DEV) for i in (1, 2))
    starts = i32([0, n, 2 * n])
    g.q4_cache_append(cache, k, v, i32(tab), i32([0, 0]), starts=starts)
    small = g.q4_cache(4, heads, page, dim, group, DEV)
    near = i32([[3, 0], [1, 2]])
    g.q4_cache_append(small, k, v, near, i32([0, 0]), starts=starts)
    for a, b in zip(cache[:4], small[:4]):
        assert all(torch.equal(a[p], b[s]) for p, s in ((pages - 1, 3), (0, 0), (1, 1), (pages - 2, 2)))
    for a, b in zip(g.q4_cache_read(cache, i32(tab), starts, 2 * n), g.q4_cache_read(small, near, starts, 2 * n)):
        assert torch.equal(a, b)
    q = torch.randn(2, 16, dim, generator=gen(3)).to(torch.float16).to(DEV)
    lengths = i32([n, n])
    assert torch.equal(g.attention_q4(q, cache, i32(tab), lengths), g.attention_q4(q, small, near, lengths))


def test_refusals():
    layer = Layer(2, 256, 4, 2, 64, 16, 4, 64, 64)
    c, table, lengths = layer.cache, layer.table, i32([5, 9])
    x = torch.zeros(2, 256, dtype=torch.float16, device=DEV)
    q, kv = torch.zeros(2, 4, 64, dtype=torch.float16, device=DEV), torch.zeros(2, 2, 64, dtype=torch.float16, device=DEV)
    w = layer.w_in
    before = copies(c[:4])
    values = [lambda: g.gemm_q4(x.float(), w), lambda: g.gemm_q4(x[0], w), lambda: g.gemm_q4(x[:, :128].contiguous(), w),
              lambda: g.gemm_q4(x.t(), w), lambda: g.gemm_q4(x.cpu(), w), lambda: g.gemm_q4(x, w, epilogue="tanh"),
              lambda: g.gemm_q4(x, w, out=q), lambda: g.gemm_q4(x, w._replace(codes=w.codes[1:])),
              lambda: g.gemm_q4(x, w._replace(group=32)), lambda: g.gemm_q4(x, w._replace(words=w.words.cpu())),
              lambda: g.q4_compress(x[:, ::2]), lambda: g.q4_compress(x, 48), lambda: g.q4_expand(w, out=x),
              lambda: g.attention_q4(q[:, :3], c, table, lengths), lambda: g.attention_q4(q[:1], c, table, lengths),
              lambda: g.attention_q4(q, c, table, lengths.long()), lambda: g.attention_q4(q, c, table.long(), lengths),
              lambda: g.attention_q4(q, c, table, lengths, max_length=-1), lambda: g.attention_q4(q, c, table.t(), lengths),
              lambda: g.attention_q4(q.transpose(1, 2).contiguous().transpose(1, 2), c, table, lengths),
              lambda: g.attention_q4(q, c._replace(k_words=c.k_words[:1]), table, lengths),
              lambda: g.attention_q4(q, c._replace(group=32), table, lengths),
              lambda: g.attention_q4(q, c, table, lengths, out=kv),
              lambda: g.q4_cache_append(c, kv, kv[:1], table, lengths), lambda: g.q4_cache_append(c, kv[:1], kv[:1], table, lengths),
              lambda: g.q4_cache_append(c, q, q, table, lengths), lambda: g.q4_cache_append(c, kv, kv, table, lengths, cos=layer.cos),
              lambda: g.q4_cache_append(c, kv, kv, table, lengths, out=q), lambda: g.q4_cache_append(c, kv, kv, table, lengths[:1]),
              lambda: g.q4_cache_append(c, kv, kv, table, lengths, cos=layer.cos[:, :4], sin=layer.sin[:, :4]),
              lambda: g.q4_cache_append(c, kv, kv, table, lengths, cos=layer.cos, sin=layer.sin[:-1]),
              lambda: g.q4_cache_append(c, kv, kv, table, lengths, starts=lengths),
              lambda: g.q4_cache_read(c, table, lengths, 2), lambda: g.q4_cache_read(c, table, i32([0, 1, 2]), -1),
              lambda: g.q4_cache_read(c, table, i32([0, 1, 2]), 2, first=i32([0]))]
    for i, call in enumerate(values):
        with pytest.raises(ValueError):
            call()
            print(f"[q4] call {i} was not refused", flush=True)
    statuses = [lambda: g.gemm_q4(x, w, config=99), lambda: g.gemm_q4(x, w, splits=-3), lambda: g.gemm_q4(x, w, splits=65),
                lambda: g.attention_q4(q, c, table, lengths, scale=float("nan")), lambda: g.attention_q4(q, c, table, lengths, splits=257),
                lambda: g.attention_q4(q, c, table, lengths, out=q)]
    for call in statuses:
        with pytest.raises(g.GemmError):
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(c[:4], before))


def test_nothing_to_do():
    none = torch.empty(0, 128, dtype=torch.float16, device=DEV)
    w = g.q4_compress(none, 64)
    assert g.q4_expand(w).shape == (0, 128)
    a = torch.ones(3, 128, dtype=torch.float16, device=DEV)
    assert g.gemm_q4(a, w).shape == (3, 0)
    assert g.gemm_q4(none, g.q4_compress(a, 64)).shape == (0, 3)
    assert g.gemm_q4(a[:, :0], g.q4_compress(a[:, :0], 64)).tolist() == [[0.0] * 3] * 3
    cache = g.q4_cache(0, 2, 16, 64, 32, DEV)
    table, lengths = torch.empty(2, 0, dtype=torch.int32, device=DEV), i32([7, 0])
    rows = torch.ones(2, 2, 64, dtype=torch.float16, device=DEV)
    assert bool((g.attention_q4(rows, cache, table, lengths) == 0).all())
    q = g.q4_cache_append(cache, rows, rows, table, lengths, q=rows)
    assert bool((q == 0).all())                      # no page: rotated queries of tokens that are not appended are zeros
    k, v = g.q4_cache_read(cache, table, i32([0, 1, 2]), 2)
    assert bool((k == 0).all()) and bool((v == 0).all())
    some = noise_cache(2, 2, 16, 64, 32, 0)
    empty = torch.empty(0, 3, dtype=torch.int32, device=DEV)
    assert g.attention_q4(rows[:0], some, empty, lengths[:0]).shape == (0, 2, 64)
    assert g.q4_cache_append(some, rows[:0], rows[:0], empty, lengths[:0], q=rows[:0]).shape == (0, 2, 64)
    assert g.q4_cache_read(some, empty, i32([0]), 0)[0].shape == (0, 2, 64)


def test_threads():
    """Calls from several threads at once, each on a stream of its own."""
    import threading

    w = g.q4_compress(weights(520, 4096, 1).to(DEV), 64)
    cache, table, lengths = noise_cache(120, 2, 16, 128, 64, 0), i32(make_table([900, 700], 16, 120, 0)), i32([900, 700])
    a = [torch.randn(2 + i, 4096, generator=gen(i)).to(torch.float16).to(DEV) for i in range(4)]
    q = [torch.randn(2, 4, 128, generator=gen(i)).to(torch.float16).to(DEV) for i in range(4)]
    want = [(g.gemm_q4(x, w, splits=3), g.attention_q4(y, cache, table, lengths, splits=5)) for x, y in zip(a, q)]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                got = g.gemm_q4(a[i], w, splits=3), g.attention_q4(q[i], cache, table, lengths, splits=5)
                if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                    failed.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
