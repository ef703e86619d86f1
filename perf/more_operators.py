"""The 8-bit operators and the routed experts, case by case: what a user's program holds, the call it makes, the same in
elementary torch operations, and the definition in 64 bits.

An 8-bit matrix holds each row (a token, or an output channel of a weight matrix) as integer codes in -127..127 and one
scale: for a row's largest magnitude m, code = 127 x / m rounded to the nearest integer (halves to the even one) and
scale = m / 127 in binary32; a row of zeros has scale 0.  Rows are padded with zero codes to a multiple of 16.

Routing: score = softmax or sigmoid of a token's logits; what is compared is score + bias; with groups, the groups whose
two best such values have the largest sum stay, and the top_k best experts in them are chosen, best first, ties to the
lowest index.  Weights are the chosen experts' scores without bias, divided by their sum or not, times a factor.
A token x top_k pair of index p = token * top_k + slot belongs to the expert ids[token][slot], or to none (-1); `order`
lists the pairs by expert, those of none last, each expert's in ascending order, and starts[e] says where expert e begins.
"""
import math

import torch

own = False   # True: run() calls the library's operators; False: it computes their plain form


# ---- cases -----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token through a small projection: the call's own latency
        {"name": "gemm_i8_1x1024x1024", "op": "gemm", "m": 1, "n": 1024, "k": 1024, "relu": False, "alpha": 1.0},
        # one token through the MLP projection of the benchmark's large workload: the weights' bytes
        {"name": "gemm_i8_1x28672x8192", "op": "gemm", "m": 1, "n": 28672, "k": 8192, "relu": False, "alpha": 1.0},
        # a serving batch of single tokens
        {"name": "gemm_i8_64x8192x8192", "op": "gemm", "m": 64, "n": 8192, "k": 8192, "relu": False, "alpha": 1.0},
        # a prompt, sizes that fill no tile, scale and ReLU
        {"name": "gemm_i8_1000x5000x4100", "op": "gemm", "m": 1000, "n": 5000, "k": 4100, "relu": True, "alpha": 0.125},
        # the benchmark's headline size: matrix-core work
        {"name": "gemm_i8_8192x8192x8192", "op": "gemm", "m": 8192, "n": 8192, "k": 8192, "relu": False, "alpha": 1.0},
        # a few tokens of an odd width to codes, and what the codes stand for
        {"name": "compress_i8_13x4100", "op": "compress", "rows": 13, "k": 4100},
        # a prompt's activations, or a layer's weights
        {"name": "compress_i8_8192x8192", "op": "compress", "rows": 8192, "k": 8192},
        # a serving batch of single tokens over many experts in groups, biased for balance
        {"name": "route_64x256", "op": "route", "tokens": 64, "experts": 256, "top_k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "renormalise": True, "scale": 2.5, "half": False},
        # a prompt over fewer experts
        {"name": "route_8192x64", "op": "route", "tokens": 8192, "experts": 64, "top_k": 6, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renormalise": False, "scale": 1.0, "half": True},
        # one token through its 8 experts: the first product of their layer
        {"name": "experts_1of256", "op": "experts", "tokens": 1, "experts": 256, "top_k": 8, "n": 2048, "k": 4096,
         "per_pair": False, "relu": True, "alpha": 1.0, "masked": False},
        # a serving batch, about two tokens for each expert: the second product, its rows one for each pair
        {"name": "experts_64of256", "op": "experts", "tokens": 64, "experts": 256, "top_k": 8, "n": 4096, "k": 2048,
         "per_pair": True, "relu": False, "alpha": 1.0, "masked": True},
        # a prompt, hundreds of tokens for each expert
        {"name": "experts_2048of64", "op": "experts", "tokens": 2048, "experts": 64, "top_k": 8, "n": 2048, "k": 4096,
         "per_pair": False, "relu": True, "alpha": 1.0, "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "compress", "route", "experts", "experts"])
    if op == "gemm":
        k, n = _log(rng, 64, 16384), _log(rng, 16, 28672)
        n = min(n, 28672 * 8192 // k)
        m = min(_log(rng, 1, 8192), max(1, 8192 ** 3 // (n * k)))
        if rng.random() < 0.5:
            k = max(64, k // 64 * 64)
        return {"op": op, "m": m, "n": n, "k": k, "relu": rng.random() < 0.3, "alpha": rng.choice([1.0, 0.125, 1.7])}
    if op == "compress":
        rows = _log(rng, 1, 8192)
        return {"op": op, "rows": rows, "k": _log(rng, 64, min(28672, 8192 * 8192 // rows))}
    experts = rng.choice([8, 16, 40, 64, 128, 160, 256, 384])
    top_k = rng.randint(1, min(experts, 10))
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        top_groups = rng.randint(-(-top_k * groups // experts), groups)
        return {"op": op, "tokens": _log(rng, 1, 8192 * 64 // experts), "experts": experts, "top_k": top_k,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": top_groups, "renormalise": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]),
                "half": rng.random() < 0.5}
    most = 2 ** 31 // experts
    n = _log(rng, 16, 8192)
    k = min(_log(rng, 64, 8192), max(64, most // n))
    tokens = min(_log(rng, 1, 4096), max(1, 2048 * 8 * 2048 * 4096 // (top_k * n * k)))
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "n": n, "k": k, "per_pair": rng.random() < 0.5,
            "relu": rng.random() < 0.5, "alpha": rng.choice([1.0, 0.125]), "masked": rng.random() < 0.5}


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, k):
    """Normal, with a few channels of larger size, and rows of different size."""
    return _randn(g, rows, k) * (1.0 + 5.0 * (torch.rand(k, generator=g, device="cuda") < 0.01)) * torch.exp(_randn(g, rows, 1) * 0.5)


def _quantise(x):
    """Codes (padded) and scales of the rows of x (binary16)."""
    x = torch.nan_to_num(x.to(torch.float64), nan=0.0, posinf=65504.0, neginf=-65504.0)   # 64 bits: quotients next to a half
    most = x.abs().amax(-1)
    over = torch.where(most > 0, most, torch.ones_like(most))
    codes = torch.round(127.0 * x / over[..., None]).to(torch.int8)
    return torch.nn.functional.pad(codes, (0, -x.shape[-1] % 16)), (most / 127.0).to(torch.float32)


def _held_weights(g, *shape):
    """Codes and scales of random weights, one scale for each row of the last dimension."""
    k = shape[-1]
    codes = torch.zeros(*shape[:-1], k + -k % 16, dtype=torch.int8, device="cuda")
    parts = codes.view(-1, codes.shape[-1])
    for r in range(0, parts.shape[0], 65536):
        part = _randn(g, min(65536, parts.shape[0] - r), k)
        parts[r:r + 65536, :k] = (part * 30.0).round_().clamp_(-127, 127).to(torch.int8)
    scales = torch.rand(shape[:-1], generator=g, device="cuda", dtype=torch.float32) + 0.5
    return codes, scales / (30.0 * math.sqrt(k))


def _some_ids(g, c):
    """Distinct experts for each token, some of them more popular; with `masked`, tokens of no expert among them."""
    t, e = c["tokens"], c["experts"]
    liking = _randn(g, t, e) + 0.5 * _randn(g, e)
    ids = torch.sort(liking, dim=-1, descending=True, stable=True)[1][:, :c["top_k"]].to(torch.int32)
    if c["masked"]:
        ids[torch.arange(t, device="cuda") % 9 == 4] = -1
    return ids.contiguous()


def _order(ids, experts):
    flat = ids.reshape(-1)
    keys = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    order = torch.sort(keys, dim=0, stable=True)[1].to(torch.int32)
    starts = (keys[None] < torch.arange(experts + 1, device=ids.device, dtype=torch.int32)[:, None]).sum(1, dtype=torch.int32)
    return order.view(ids.shape), starts


def prepare(case, seed):
    g, c = _gen(seed), case
    if c["op"] == "gemm":
        a, sa = _quantise(_activations(g, c["m"], c["k"]).to(torch.float16))
        w, sw = _held_weights(g, c["n"], c["k"])
        return {"case": c, "a": a, "sa": sa, "w": w, "sw": sw}
    if c["op"] == "compress":
        return {"case": c, "x": _activations(g, c["rows"], c["k"]).to(torch.float16)}
    if c["op"] == "route":
        t, e = c["tokens"], c["experts"]
        logits = 1.5 * _randn(g, t, e) + 0.5 * _randn(g, e)
        bias = 0.1 * _randn(g, e) if c["bias"] else None
        return {"case": c, "logits": logits.to(torch.float16 if c["half"] else torch.float32), "bias": bias}
    ids = _some_ids(g, c)
    order, starts = _order(ids, c["experts"])
    rows = c["tokens"] * (c["top_k"] if c["per_pair"] else 1)
    a, sa = _quantise(_activations(g, rows, c["k"]).to(torch.float16))
    w, sw = _held_weights(g, c["experts"], c["n"], c["k"])
    weights = torch.rand(ids.shape, generator=g, device="cuda", dtype=torch.float32)
    weights = weights / weights.sum(-1, keepdim=True) * (ids >= 0)
    return {"case": c, "a": a, "sa": sa, "w": w, "sw": sw, "ids": ids, "order": order, "starts": starts, "weights": weights}


# ---- one pass --------------------------------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _values(codes, scales):
    return codes.to(torch.float32) * scales[..., None]


def _plain_gemm(st):
    c = st["case"]
    out = (_values(st["a"], st["sa"]) @ _values(st["w"], st["sw"]).t()) * c["alpha"]
    return (out.clamp(min=0.0) if c["relu"] else out).to(torch.float16)


def _plain_compress(st):
    codes, scales = _quantise(st["x"])
    return _values(codes, scales)[:, :st["case"]["k"]].to(torch.float16)


def _plain_route(st):
    c = st["case"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    x = st["logits"].to(torch.float64)      # scores that are compared: next to a border 32 bits lose the order
    if c["score"] == "softmax":
        x = torch.exp(x - x.amax(-1, keepdim=True))
        score = x / x.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    key = score + st["bias"].to(torch.float64) if c["bias"] else score
    if c["groups"] > 1:
        best = torch.sort(key.view(t, c["groups"], -1), dim=-1, descending=True)[0][..., :2].sum(-1)
        first = torch.sort(best, dim=-1, descending=True, stable=True)[1][:, :c["top_groups"]]
        stay = torch.zeros(t, c["groups"], dtype=torch.bool, device=x.device).scatter_(1, first, True)
        key = key.masked_fill(~stay.repeat_interleave(e // c["groups"], 1), -math.inf)
    ids = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :k]
    weights = torch.gather(score, 1, ids)
    if c["renormalise"]:
        weights = weights / weights.sum(-1, keepdim=True)
    ids = ids.to(torch.int32)
    order, starts = _order(ids, e)
    return {"ids": ids, "weights": (weights * c["scale"]).to(torch.float32), "order": order, "starts": starts}


def _plain_experts(st):
    c = st["case"]
    order, per = st["order"].reshape(-1).long(), 1 if c["per_pair"] else c["top_k"]
    y = torch.zeros(order.shape[0], c["n"], dtype=torch.float16, device=order.device)
    starts = st["starts"].tolist()
    for e in range(c["experts"]):
        pairs = order[starts[e]:starts[e + 1]]
        if starts[e + 1] > starts[e]:
            out = (_values(st["a"][pairs // per], st["sa"][pairs // per]) @ _values(st["w"][e], st["sw"][e]).t()) * c["alpha"]
            y[pairs] = (out.clamp(min=0.0) if c["relu"] else out).to(torch.float16)
    y = y.view(c["tokens"], c["top_k"], c["n"])
    return {"y": y, "out": (y.to(torch.float32) * st["weights"][..., None]).sum(1).to(torch.float16)}


_run_plain = {"gemm": _plain_gemm, "compress": _plain_compress, "route": _plain_route, "experts": _plain_experts}


def _own_gemm(st):
    import tiled_dense_gemm_fp16_amd as ops
    c = st["case"]
    return ops.gemm_i8(ops.I8Matrix(st["a"], st["sa"], c["k"]), ops.I8Matrix(st["w"], st["sw"], c["k"]),
                       epilogue="relu" if c["relu"] else "none", alpha=c["alpha"])


def _own_compress(st):
    import tiled_dense_gemm_fp16_amd as ops
    return ops.i8_expand(ops.i8_compress(st["x"]))


def _own_route(st):
    import tiled_dense_gemm_fp16_amd as ops
    c = st["case"]
    ids, weights = ops.route(st["logits"], c["top_k"], score=c["score"], bias=st["bias"], groups=c["groups"],
                             top_groups=c["top_groups"], renormalise=c["renormalise"], scale=c["scale"])
    order = ops.expert_order(ids, c["experts"])
    return {"ids": ids, "weights": weights, "order": order.order, "starts": order.starts}


def _own_experts(st):
    import tiled_dense_gemm_fp16_amd as ops
    c = st["case"]
    y = ops.gemm_i8_experts(ops.I8Matrix(st["a"], st["sa"], c["k"]), ops.I8Matrix(st["w"], st["sw"], c["k"]),
                            ops.ExpertOrder(st["order"], st["starts"]), epilogue="relu" if c["relu"] else "none",
                            alpha=c["alpha"])
    return {"y": y, "out": ops.expert_sum(y, st["weights"])}


_run_own = {"gemm": _own_gemm, "compress": _own_compress, "route": _own_route, "experts": _own_experts}


# ---- what a pass cannot do without -----------------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m + n) * (k + 4) + 2 * m * n, "flops": 2 * m * n * k}
    if c["op"] == "compress":
        return {"bytes": c["rows"] * (5 * c["k"] + 4), "flops": 4 * c["rows"] * c["k"]}
    pairs = c["tokens"] * c["top_k"]
    if c["op"] == "route":
        each = 2 if c["half"] else 4
        return {"bytes": c["tokens"] * c["experts"] * each + 12 * pairs + 4 * c["experts"] * (1 + c["bias"]),
                "flops": 4 * c["tokens"] * c["experts"]}
    if c["masked"]:
        pairs -= c["top_k"] * ((c["tokens"] + 4) // 9)
    # experts that some token chose, were all equally popular
    chosen = c["experts"] * (1.0 - (1.0 - c["top_k"] / c["experts"]) ** (pairs // c["top_k"]))
    rows = pairs if c["per_pair"] else pairs // c["top_k"]
    outputs = c["tokens"] * c["n"] * (c["top_k"] + 1)
    return {"bytes": chosen * c["n"] * (c["k"] + 4) + rows * (c["k"] + 4) + 2 * outputs + 8 * c["tokens"] * c["top_k"],
            "flops": 2 * pairs * c["n"] * (c["k"] + 1)}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------------

def _exact_product(a, sa, w, sw, alpha, relu):
    """alpha sa sw sum_k a w for integer codes, whose sums are exact in 64 bits."""
    parts = [a.double() @ w[n:n + 4096].double().t().contiguous() for n in range(0, w.shape[0], 4096)]
    out = torch.cat(parts, 1) * sa.double()[:, None] * sw.double() * alpha
    return out.clamp(min=0) if relu else out


def _exact_route(c, st):
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    logits = st["logits"].double()
    score = torch.softmax(logits, -1) if c["score"] == "softmax" else torch.sigmoid(logits)
    key = score + st["bias"].double() if c["bias"] else score.clone()

    def first_best(values):
        """Index of each row's largest value, the first of equals."""
        index = torch.arange(values.shape[1], device="cuda").expand_as(values)
        return torch.where(values == values.max(-1, keepdim=True)[0], index, values.shape[1]).min(-1)[0]

    rows, n = torch.arange(t, device="cuda"), e // c["groups"]
    if c["groups"] > 1:
        per = key.view(t, c["groups"], n).clone()
        top = per.max(-1)[0]
        if n > 1:
            per.view(t * c["groups"], n)[torch.arange(t * c["groups"], device="cuda"), first_best(per.view(-1, n))] = -math.inf
            top = top + per.max(-1)[0]
        stay = torch.zeros(t, c["groups"], dtype=torch.bool, device="cuda")
        for _ in range(c["top_groups"]):
            at = first_best(top)
            stay[rows, at] = True
            top[rows, at] = -math.inf
        key = torch.where(stay[:, torch.arange(e, device="cuda") // n], key, -math.inf)
    ids = torch.empty(t, k, dtype=torch.int32, device="cuda")
    for j in range(k):
        at = first_best(key)
        ids[:, j] = at.to(torch.int32)
        key[rows, at] = -math.inf
    weights = torch.stack([score[rows, ids[:, j].long()] for j in range(k)], 1)
    if c["renormalise"]:
        weights = weights / weights.sum(-1, keepdim=True)
    flat = ids.reshape(-1).long()
    place = torch.argsort(flat * flat.numel() + torch.arange(flat.numel(), device="cuda"))
    starts = torch.cat([flat.new_zeros(1), torch.cumsum(torch.bincount(flat, minlength=e), 0)])
    return {"ids": ids, "weights": weights * c["scale"], "order": place.to(torch.int32).view(t, k), "starts": starts.to(torch.int32)}


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "gemm":
        return _exact_product(st["a"], st["sa"], st["w"], st["sw"], c["alpha"], c["relu"])
    if c["op"] == "compress":
        x = st["x"].double()
        step = x.abs().max(-1, keepdim=True)[0] / 127
        ratio = 127 * x / torch.where(step > 0, 127 * step, 1.0)
        low = torch.floor(ratio)
        up = (ratio - low > 0.5) | ((ratio - low == 0.5) & (low % 2 != 0))
        return (low + up) * step
    if c["op"] == "route":
        return _exact_route(c, st)
    ids, per = st["ids"].reshape(-1), 1 if c["per_pair"] else c["top_k"]
    y = torch.zeros(ids.shape[0], c["n"], dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.tolist()) - {-1}):
        pairs = torch.nonzero(ids == e)[:, 0]
        rows = torch.div(pairs, per, rounding_mode="floor")
        y[pairs] = _exact_product(st["a"][rows], st["sa"][rows], st["w"][e], st["sw"][e], c["alpha"], c["relu"])
    y = y.view(c["tokens"], c["top_k"], c["n"])
    return {"y": y, "out": (y * st["weights"].double()[..., None]).sum(1)}
