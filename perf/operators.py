"""The 4-bit operand operators, case by case: what a user's program holds, the call it makes, the same in elementary
torch operations, and the definition in 64 bits.

A 4-bit operand is held in groups of 32, 64 or 128 neighbours along the contraction (weights) or the head dimension
(cache).  A group has one 32-bit word: a binary16 scale s in the low half and an integer zero point z in 0..15 in the
high half; a code q in 0..15 stands for s (q - z).  Eight codes share a dword: code i of the eight sits in nibble
NIBBLE[i].  The three orders of the dwords:

* weights W (N x K), padded to whole tiles of 16 rows by 128 k: codes[N/16][K/128][4 g][16 n][4 j] holds row n of the
  tile, k = 32 j + 8 g + 0..7 of the tile; words[N/16][K/128][16 n][128/group].
* cached keys: codes[page][head][token][D/8], in every block of min(D, 128) the dword of d = 32 j + 8 g + 0..7 at
  g (block / 32) + j; words[page][head][D/group][token].
* cached values: codes[page][head][token / 8][d % 16][d / 16], a dword holding 8 successive tokens of one d; words as
  for the keys.
"""
import math

import torch

own = False   # True: run() calls the library's operators; False: it computes their plain form

NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)


# ---- cases -----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token through a small projection: the call's own latency
        {"name": "gemm_1x1024x1024", "op": "gemm", "m": 1, "n": 1024, "k": 1024, "group": 128, "relu": False, "alpha": 1.0},
        # one token through the MLP projection of the benchmark's large workload: the weights' bytes
        {"name": "gemm_1x28672x8192", "op": "gemm", "m": 1, "n": 28672, "k": 8192, "group": 128, "relu": False, "alpha": 1.0},
        # a few sequences decoded together, sizes that fill no tile, the finest groups, scale and ReLU
        {"name": "gemm_13x5000x4100", "op": "gemm", "m": 13, "n": 5000, "k": 4100, "group": 32, "relu": True, "alpha": 0.125},
        # a serving batch of single tokens
        {"name": "gemm_64x8192x8192", "op": "gemm", "m": 64, "n": 8192, "k": 8192, "group": 64, "relu": False, "alpha": 1.0},
        # a prompt of 2048 tokens through the same weights: matrix-core work
        {"name": "gemm_2048x8192x8192", "op": "gemm", "m": 2048, "n": 8192, "k": 8192, "group": 128, "relu": False, "alpha": 1.0},
        # compressing one layer's weights and reading back what they stand for
        {"name": "compress_8192x8192", "op": "compress", "n": 8192, "k": 8192, "group": 128, "symmetric": False},
        # ... of sizes that fill no tile, symmetric codes, the finest groups
        {"name": "compress_5000x4100", "op": "compress", "n": 5000, "k": 4100, "group": 32, "symmetric": True},
        # one new token of each of 64 short sequences into the paged cache, rotated on the way
        {"name": "append_64x1", "op": "append", "batch": 64, "new": 1, "past": 60, "q_heads": 32, "heads": 8, "dim": 128,
         "group": 64, "page": 16, "interleaved": False},
        # prompts of different lengths behind a cached prefix, one call
        {"name": "append_prompts", "op": "append", "batch": 5, "new": 1021, "past": 37, "q_heads": 32, "heads": 8, "dim": 128,
         "group": 128, "page": 24, "interleaved": True},
        # one sequence with a short past: latency
        {"name": "attention_1x100", "op": "attention", "batch": 1, "length": 100, "q_heads": 8, "heads": 8, "dim": 64,
         "group": 32, "page": 16},
        # a serving batch of ragged lengths, grouped heads
        {"name": "attention_32x4096", "op": "attention", "batch": 32, "length": 4096, "q_heads": 32, "heads": 8, "dim": 128,
         "group": 64, "page": 64},
        # one long context
        {"name": "attention_1x131000", "op": "attention", "batch": 1, "length": 131000, "q_heads": 64, "heads": 8, "dim": 128,
         "group": 128, "page": 256},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "compress", "append", "attention", "attention"])
    if op == "gemm":
        k, n = _log(rng, 64, 16384), _log(rng, 16, 28672)
        n = min(n, 28672 * 8192 // k)
        m = min(_log(rng, 1, 2048), max(1, 2048 * 8192 * 8192 // (n * k)))
        if rng.random() < 0.5:
            k = max(64, k // 64 * 64)
        return {"op": op, "m": m, "n": n, "k": k, "group": rng.choice([32, 64, 128]), "relu": rng.random() < 0.3,
                "alpha": rng.choice([1.0, 0.125, 1.7])}
    if op == "compress":
        n, k = _log(rng, 16, 8192), _log(rng, 64, 8192)
        return {"op": op, "n": n, "k": k, "group": rng.choice([32, 64, 128]), "symmetric": rng.random() < 0.5}
    dim, heads = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    page = rng.choice([8, 16, 24, 64, 128, 256])
    if op == "append":
        batch = _log(rng, 1, 64)
        q_heads = heads * rng.choice([1, 4, 8])
        new = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 2600 * 48 * 128 // (batch * (q_heads + 2 * heads) * dim)))
        return {"op": op, "batch": batch, "new": new, "past": rng.randint(0, 90), "q_heads": q_heads, "heads": heads,
                "dim": dim, "group": group, "page": page, "interleaved": rng.random() < 0.5}
    batch = _log(rng, 1, 64)
    length = _log(rng, 1, min(131000, 131000 * 8 * 96 // (batch * heads * dim)))
    return {"op": op, "batch": batch, "length": length, "q_heads": heads * rng.choice([1, 3, 4, 8, 16]),
            "heads": heads, "dim": dim, "group": group, "page": page}


# ---- quantisation and the storage orders -----------------------------------------------------------------------------

def _quantise(x, group, symmetric):
    """Codes, zero points and binary16 scales of x's groups along its last dimension (float32, a multiple of group)."""
    g = torch.nan_to_num(x, nan=0.0, posinf=math.inf, neginf=-math.inf).reshape(*x.shape[:-1], x.shape[-1] // group, group)
    if symmetric:
        s = g.abs().amax(-1) / torch.tensor(7.0, device=x.device)   # a tensor: division, not a product with 1/7
    else:
        lo, hi = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
        s = (hi - lo) / torch.tensor(15.0, device=x.device)
    s = s.clamp(max=65504.0).to(torch.float16).to(torch.float32)
    z = torch.full_like(s, 8.0) if symmetric else torch.round(torch.where(s > 0, -lo / s, torch.zeros_like(s))).clamp(0, 15)
    q = torch.where(s[..., None] > 0, torch.round(g / s[..., None]), torch.zeros_like(g))   # halves go to the even code
    q = (q + z[..., None]).clamp(0, 15)
    return q.reshape(x.shape).to(torch.int32), z.to(torch.int32), s.to(torch.float16)


def _words(s, z):
    return (s.contiguous().view(torch.int16).to(torch.int32) & 0xFFFF) | (z << 16)


def _scale_zero(words):
    s = (words & 0xFFFF).to(torch.int16).view(torch.float16).to(torch.float32)
    return s, ((words >> 16) & 0xFFFF).to(torch.float32)


def _join(eight):
    """Dwords of the eight codes along the last dimension."""
    at = torch.tensor([4 * p for p in NIBBLE], device=eight.device, dtype=torch.int32)
    return (eight << at).sum(-1, dtype=torch.int32)


def _split(dwords):
    at = torch.tensor([4 * p for p in NIBBLE], device=dwords.device, dtype=torch.int32)
    return (dwords[..., None] >> at) & 15


def _quantise_weights(w, group, symmetric):
    """_quantise of a matrix padded with zeros to whole 16 x 128 tiles."""
    n, k = w.shape
    return _quantise(torch.nn.functional.pad(w.to(torch.float32), (0, -k % 128, 0, -n % 16)), group, symmetric)


def _pack_weights(q, z, s):
    n, k = q.shape
    codes = _join(q.view(n // 16, 16, k // 128, 4, 4, 8).permute(0, 2, 4, 1, 3, 5)).contiguous()
    words = _words(s, z).view(n // 16, 16, k // 128, -1).permute(0, 2, 1, 3).contiguous()
    return codes, words


def _weights(codes, words, n, k):
    """The float32 matrix that a packed one stands for."""
    nb, kb = codes.shape[:2]
    q = _split(codes).permute(0, 3, 1, 4, 2, 5).reshape(16 * nb, 128 * kb)
    s, z = (t.permute(0, 2, 1, 3).reshape(16 * nb, -1) for t in _scale_zero(words))
    per = q.shape[1] // s.shape[1]
    w = (q.view(16 * nb, -1, per) - z[..., None]) * s[..., None]
    return w.reshape(16 * nb, 128 * kb)[:n, :k]


def _key_order(q):
    """Codes [..., D] in storage order [..., D / 8, 8]."""
    d = q.shape[-1]
    b = min(d, 128)
    return q.reshape(*q.shape[:-1], d // b, b // 32, 4, 8).transpose(-3, -2).reshape(*q.shape[:-1], d // 8, 8)


def _pack_cache(x, group):
    """Codes and words [pages, slots, heads, ...] of float32 keys or values [pages, slots, heads, D], as plain integers."""
    q, z, s = _quantise(x, group, False)
    return q, _words(s, z)


def _store_keys(q, words):
    return _join(_key_order(q)).transpose(1, 2).contiguous(), words.permute(0, 2, 3, 1).contiguous()


def _store_values(q, words):
    p, slots, h, d = q.shape
    codes = _join(q.view(p, slots // 8, 8, h, d // 16, 16).permute(0, 3, 1, 5, 4, 2))
    return codes.contiguous(), words.permute(0, 2, 3, 1).contiguous()


def _load_keys(codes, words):
    """Codes [pages, slots, heads, D] and words [pages, slots, heads, D / group] of stored keys."""
    p, h, slots, d8 = codes.shape
    d = 8 * d8
    b = min(d, 128)
    q = _split(codes).view(p, h, slots, d // b, 4, b // 32, 8).transpose(4, 5).reshape(p, h, slots, d)
    return q.transpose(1, 2), words.permute(0, 3, 1, 2)


def _load_values(codes, words):
    p, h, s8, _, d16 = codes.shape
    q = _split(codes).permute(0, 2, 5, 1, 4, 3).reshape(p, 8 * s8, h, 16 * d16)
    return q, words.permute(0, 3, 1, 2)


def _values_of(q, words):
    s, z = _scale_zero(words)
    d = q.shape[-1]
    g = q.reshape(*q.shape[:-1], s.shape[-1], d // s.shape[-1])
    return ((g - z[..., None]) * s[..., None]).reshape(q.shape)


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _spread(count, most, least):
    """`count` lengths between least and most, the largest among them."""
    return [most if i == 0 else least + (most - least) * ((i * 7919) % 1000) // 1000 for i in range(count)]


def _lengths(case):
    """(past, new) tokens of each sequence of an append, lengths of an attention's sequences (one empty in larger batches)."""
    b = case["batch"]
    if case["op"] == "append":
        return _spread(b, case["past"], 0), _spread(b, case["new"], 1)
    lengths = _spread(b, case["length"], 1)
    if b >= 4:
        lengths[b // 2] = 0
    return lengths


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, totals, page):
    """Pages of a shuffled pool for each sequence; entries past a sequence's last page are -1."""
    need = [-(-t // page) for t in totals]
    pages = max(1, sum(need))
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(totals), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = ids[at:at + c]
        at += c
    return pages, table


def _tokens(g, *shape):
    """Keys or values: normal, with a few channels of larger size, as projections give them."""
    x = _randn(g, *shape)
    return x * (1.0 + 3.0 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.05))


def prepare(case, seed):
    g, c = _gen(seed), case
    if c["op"] == "gemm":
        q, z, s = _quantise_weights(_randn(g, c["n"], c["k"]) / math.sqrt(c["k"]), c["group"], False)
        codes, words = _pack_weights(q, z, s)
        return {"case": c, "a": _randn(g, c["m"], c["k"]).to(torch.float16), "codes": codes, "words": words}
    if c["op"] == "compress":
        return {"case": c, "w": (_randn(g, c["n"], c["k"]) / math.sqrt(c["k"])).to(torch.float16)}
    h, d, page = c["heads"], c["dim"], c["page"]
    if c["op"] == "append":
        past, new = _lengths(c)
        totals = [p + n for p, n in zip(past, new)]
        pages, table = _table(g, totals, page)
        starts, all_starts = [0], [0]
        for n, t in zip(new, totals):
            starts.append(starts[-1] + n)
            all_starts.append(all_starts[-1] + t)
        t = starts[-1]
        # one projection's output, of which queries, keys and values are strided views
        qkv = torch.cat([_tokens(g, t, c["q_heads"], d), _tokens(g, t, h, d), _tokens(g, t, h, d)], 1).to(torch.float16)
        f = torch.arange(d // 2, dtype=torch.float64, device="cuda") * (-2.0 * math.log(10000.0) / d)
        angle = torch.arange(table.shape[1] * page, dtype=torch.float64, device="cuda")[:, None] * torch.exp(f)
        kc, kw = _store_keys(*_pack_cache(_tokens(g, pages, page, h, d), c["group"]))
        vc, vw = _store_values(*_pack_cache(_tokens(g, pages, page, h, d), c["group"]))
        return {"case": c, "q": qkv[:, :c["q_heads"]], "k": qkv[:, c["q_heads"]:-h], "v": qkv[:, -h:], "kc": kc, "kw": kw,
                "vc": vc, "vw": vw, "table": table, "past": _i32(past), "starts": _i32(starts), "all": _i32(all_starts),
                "total": all_starts[-1], "cos": angle.cos().to(torch.float32), "sin": angle.sin().to(torch.float32)}
    lengths = _lengths(c)
    pages, table = _table(g, lengths, page)
    kc, kw = _store_keys(*_pack_cache(_tokens(g, pages, page, h, d), c["group"]))
    vc, vw = _store_values(*_pack_cache(_tokens(g, pages, page, h, d), c["group"]))
    return {"case": c, "q": _randn(g, c["batch"], c["q_heads"], d).to(torch.float16), "kc": kc, "kw": kw, "vc": vc, "vw": vw,
            "table": table, "lengths": _i32(lengths)}


# ---- one pass --------------------------------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _plain_gemm(st):
    c = st["case"]
    out = (st["a"].to(torch.float32) @ _weights(st["codes"], st["words"], c["n"], c["k"]).t()) * c["alpha"]
    return (out.clamp(min=0.0) if c["relu"] else out).to(torch.float16)


def _plain_compress(st):
    c = st["case"]
    q, z, s = _quantise_weights(st["w"], c["group"], c["symmetric"])
    v = _values_of(q, _words(s, z))[:c["n"], :c["k"]].to(torch.float16)
    return v


def _rows(starts, total):
    """Sequence and index in it of each of `total` packed rows."""
    row = torch.arange(total, device=starts.device, dtype=torch.int32)
    seq = torch.searchsorted(starts, row, right=True) - 1
    return seq, row - starts[seq]


def _rotate(x, cos, sin, interleaved):
    x = x.to(torch.float32)
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).reshape(x.shape)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(st):
    c = st["case"]
    page, group = c["page"], c["group"]
    seq, i = _rows(st["starts"], st["q"].shape[0])
    pos = st["past"][seq] + i
    at = st["table"][seq, pos // page].long(), (pos % page).long()
    cos, sin = st["cos"][pos], st["sin"][pos]
    seq, i = _rows(st["all"], st["total"])
    back = st["table"][seq, i // page].long(), (i % page).long()
    found = []
    for stored, x in (((st["kc"], st["kw"]), _rotate(st["k"], cos, sin, c["interleaved"])), ((st["vc"], st["vw"]), st["v"])):
        q, words = (_load_values if found else _load_keys)(*stored)
        nq, nwords = _pack_cache(x.to(torch.float32), group)
        q, words = q.clone(), words.clone()
        q[at], words[at] = nq, nwords
        found.append(_values_of(q[back], words[back]).to(torch.float16))
    return {"q": _rotate(st["q"], cos, sin, c["interleaved"]).to(torch.float16), "k": found[0], "v": found[1]}


def _plain_attention(st):
    c = st["case"]
    h, d, page = c["heads"], c["dim"], c["page"]
    b, most = st["table"].shape[0], st["table"].shape[1] * page
    ids = st["table"].clamp(min=0).long()
    k = _values_of(*_load_keys(st["kc"], st["kw"]))[ids].reshape(b, most, h, d)
    v = _values_of(*_load_values(st["vc"], st["vw"]))[ids].reshape(b, most, h, d)
    q = st["q"].to(torch.float32).view(b, h, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * d ** -0.5
    there = torch.arange(most, device=x.device) < st["lengths"][:, None]
    x = x.masked_fill(~there[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return torch.matmul(p, v.transpose(1, 2).contiguous()).view(b, -1, d).to(torch.float16)


_run_plain = {"gemm": _plain_gemm, "compress": _plain_compress, "append": _plain_append, "attention": _plain_attention}


def _own_gemm(st):
    import tiled_dense_gemm_fp16_amd as ops
    c = st["case"]
    w = ops.Q4Matrix(st["codes"], st["words"], c["n"], c["k"], c["group"])
    return ops.gemm_q4(st["a"], w, epilogue="relu" if c["relu"] else "none", alpha=c["alpha"])


def _own_compress(st):
    import tiled_dense_gemm_fp16_amd as ops
    return ops.q4_expand(ops.q4_compress(st["w"], st["case"]["group"], symmetric=st["case"]["symmetric"]))


def _own_append(st):
    import tiled_dense_gemm_fp16_amd as ops
    c = st["case"]
    cache = ops.Q4Cache(st["kc"], st["kw"], st["vc"], st["vw"], c["group"])
    q = ops.q4_cache_append(cache, st["k"], st["v"], st["table"], st["past"], starts=st["starts"], q=st["q"], cos=st["cos"],
                            sin=st["sin"], interleaved=c["interleaved"])
    k, v = ops.q4_cache_read(cache, st["table"], st["all"], st["total"])
    return {"q": q, "k": k, "v": v}


def _own_attention(st):
    import tiled_dense_gemm_fp16_amd as ops
    cache = ops.Q4Cache(st["kc"], st["kw"], st["vc"], st["vw"], st["case"]["group"])
    return ops.attention_q4(st["q"], cache, st["table"], st["lengths"])


_run_own = {"gemm": _own_gemm, "compress": _own_compress, "append": _own_append, "attention": _own_attention}


# ---- what a pass cannot do without -----------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "gemm":
        held = c["n"] * c["k"] / 2 + 4 * c["n"] * -(-c["k"] // c["group"])
        return {"bytes": held + 2 * c["m"] * (c["n"] + c["k"]), "flops": 2 * c["m"] * c["n"] * c["k"]}
    if c["op"] == "compress":
        held = c["n"] * c["k"] / 2 + 4 * c["n"] * -(-c["k"] // c["group"])
        return {"bytes": 4 * c["n"] * c["k"] + held, "flops": 8 * c["n"] * c["k"]}
    token = c["heads"] * (c["dim"] + 8 * c["dim"] // c["group"])    # a token's keys and values as held, in bytes
    if c["op"] == "append":
        past, new = _lengths(c)
        new, total = sum(new), sum(past) + sum(new)
        moved = new * (4 * c["heads"] * c["dim"] + 4 * c["q_heads"] * c["dim"] + token + 4 * c["dim"])
        return {"bytes": moved + total * (token + 4 * c["heads"] * c["dim"]),
                "flops": new * c["dim"] * (3 * c["q_heads"] + 10 * c["heads"]) + 4 * total * c["heads"] * c["dim"]}
    total = sum(_lengths(c))
    return {"bytes": total * token + 4 * c["batch"] * c["q_heads"] * c["dim"], "flops": 4 * total * c["q_heads"] * c["dim"]}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------------

def _nibble(dwords, i):
    """Code i (0..7, a tensor of indices like dwords) of each dword."""
    shift = torch.tensor(NIBBLE, device=dwords.device)[i] * 4
    return (dwords.long() & 0xFFFFFFFF) >> shift & 15


def _meaning(code, word):
    word = word.long() & 0xFFFFFFFF
    scale = (word & 0xFFFF).to(torch.int32).to(torch.int16).view(torch.float16).double()
    return scale * (code - (word >> 16)).double()


def _exact_weights(codes, words, rows, k, group):
    """Rows `rows` of the matrix, by each element's place."""
    n, kk = rows[:, None], torch.arange(k, device=codes.device)[None]
    t = kk % 128
    dword = codes.reshape(-1)[(((n // 16 * codes.shape[1] + kk // 128) * 4 + t % 32 // 8) * 16 + n % 16) * 4 + t // 32]
    word = words.reshape(-1)[((n // 16 * codes.shape[1] + kk // 128) * 16 + n % 16) * (128 // group) + t // group]
    return _meaning(_nibble(dword, t % 8), word)


def _exact_codes(x, group, symmetric):
    """Values that x's groups are held as (x in 64 bits, whole groups)."""
    g = x.unflatten(-1, (-1, group))
    if symmetric:
        s, top = g.abs().amax(-1, keepdim=True) / 7, None
    else:
        bottom, top = g.amin(-1, keepdim=True).clamp(max=0), g.amax(-1, keepdim=True).clamp(min=0)
        s = (top - bottom) / 15
    s = s.half().double()
    over = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.full_like(s, 8) if symmetric else (-bottom / over).round().clamp(0, 15) * (s > 0)
    return (((g / over).round() + z).clamp(0, 15) - z).mul(s).flatten(-2)


def _exact_turn(x, pos, cos, sin, interleaved):
    x, half = x.double(), x.shape[-1] // 2
    first = torch.arange(half, device=x.device) * 2 if interleaved else torch.arange(half, device=x.device)
    second = first + 1 if interleaved else first + half
    c, s = cos[pos].double()[:, None], sin[pos].double()[:, None]
    out = torch.empty_like(x)
    out[..., first] = x[..., first] * c - x[..., second] * s
    out[..., second] = x[..., second] * c + x[..., first] * s
    return out


def _exact_cached(st, b, count):
    """Keys and values [count, heads, D] that the cache holds for sequence b's first tokens."""
    c = st["case"]
    h, d, page, group = c["heads"], c["dim"], c["page"], c["group"]
    pos = torch.arange(count, device="cuda")
    p, t = st["table"][b].long()[pos // page][:, None, None], (pos % page)[:, None, None]
    head, x = torch.arange(h, device="cuda")[:, None], torch.arange(d, device="cuda")
    wide = min(d, 128)
    place = x // wide * (wide // 8) + x % 32 // 8 * (wide // 32) + x % wide // 32
    keys = st["kc"].reshape(-1)[((p * h + head) * page + t) * (d // 8) + place]
    values = st["vc"].reshape(-1)[((p * h + head) * (page // 8) + t // 8) * 2 * 8 * (d // 16) + x % 16 * (d // 16) + x // 16]
    word = ((p * h + head) * (d // group) + x // group) * page + t
    k = _meaning(_nibble(keys, x % 8), st["kw"].reshape(-1)[word])
    return k, _meaning(_nibble(values, t % 8), st["vw"].reshape(-1)[word])


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "gemm":
        a, parts = st["a"].double(), []
        for n0 in range(0, c["n"], 2048):
            w = _exact_weights(st["codes"], st["words"], torch.arange(n0, min(c["n"], n0 + 2048), device="cuda"), c["k"], c["group"])
            parts.append(a @ w.t().contiguous())
        out = torch.cat(parts, 1) * c["alpha"]
        return out.clamp(min=0) if c["relu"] else out
    if c["op"] == "compress":
        x = torch.nn.functional.pad(st["w"].double(), (0, -c["k"] % c["group"]))
        return _exact_codes(x, c["group"], c["symmetric"])[:, :c["k"]]
    if c["op"] == "append":
        past, new = _lengths(c)
        qs, ks, vs, at = [], [], [], 0
        for b in range(c["batch"]):
            rows, pos = slice(at, at + new[b]), torch.arange(past[b], past[b] + new[b], device="cuda")
            k, v = _exact_cached(st, b, past[b])
            turned = _exact_turn(st["k"][rows], pos, st["cos"], st["sin"], c["interleaved"])
            ks += [k, _exact_codes(turned, c["group"], False)]
            vs += [v, _exact_codes(st["v"][rows].double(), c["group"], False)]
            qs.append(_exact_turn(st["q"][rows], pos, st["cos"], st["sin"], c["interleaved"]))
            at += new[b]
        return {"q": torch.cat(qs), "k": torch.cat(ks), "v": torch.cat(vs)}
    out = torch.zeros(c["batch"], c["q_heads"], c["dim"], dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c)):
        if n:
            k, v = _exact_cached(st, b, n)
            q = st["q"][b].double().view(c["heads"], -1, c["dim"])
            x = q @ k.permute(1, 2, 0).contiguous() / math.sqrt(c["dim"])
            out[b] = (torch.softmax(x, -1) @ v.transpose(0, 1).contiguous()).reshape(-1, c["dim"])
    return out
