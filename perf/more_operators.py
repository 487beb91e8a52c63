"""Measured cases of a decode step's other half: moe.route, moe.experts and sampling.sample.

Where a model's feed-forward is a mixture of experts, route chooses each token's experts and experts runs them on 4-bit
or ternary weights; sample turns the vocabulary projection's logits into the next tokens.

``run`` computes an operator in plain torch (32-bit sums; 64-bit scores and probabilities where a whole number hangs on
them) or, with ``own``, calls this library.  ``exact`` evaluates the definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def _route(name, **over):
    return {"name": name, "op": "route", "tokens": 1, "hidden": 2048, "experts": 128, "top_k": 8, "act": "f32",
            "kind": "bf16", "scoring": "softmax", "bias": False, "renormalize": True, "scale": 1.0, **over}


def _experts(name, **over):
    return {"name": name, "op": "experts", "tokens": 1, "hidden": 2048, "inter": 768, "experts": 128, "top_k": 8,
            "act": "f32", "fmt": "q4", "group": 128, "residual": False, **over}


def _sample(name, **over):
    return {"name": name, "op": "sample", "rows": 1, "vocab": 32000, "kind": "f32", "mixed": False, "masked": False,
            "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, **over}


def listed():
    return [
        # The router of one decoding sequence: pure latency.
        _route("route_token"),
        # A decode batch of a wide model: sigmoid scores, a balancing bias for the choice, scaled weights.
        _route("route_batch_sigmoid", tokens=64, hidden=7168, experts=256, act="bf16", kind="f32", scoring="sigmoid",
               bias=True, scale=2.5),
        # A prompt of an odd length through a router of an odd number of experts, weights as they come.
        _route("route_prompt", tokens=4099, hidden=4096, experts=60, top_k=4, act="f16", kind="f16",
               renormalize=False),
        # One sequence decoding, many small 4-bit experts: latency and a few megabytes.
        _experts("experts_token_q4"),
        # One sequence decoding, two of eight large ternary experts, onto the residual stream.
        _experts("experts_token_tq2", hidden=4096, inter=11008, experts=8, top_k=2, fmt="tq2", residual=True),
        # A handful of sequences (or a short draft), bf16 activations, small groups.
        _experts("experts_few_q4", tokens=7, inter=640, experts=64, top_k=6, act="bf16", group=32),
        # A decode batch that touches nearly every expert.
        _experts("experts_batch_q4", tokens=64, group=64, residual=True),
        # The largest batch, ternary.
        _experts("experts_batch_tq2", tokens=128, hidden=4096, inter=1408, experts=64, top_k=6, act="bf16", fmt="tq2",
                 residual=True),
        # The usual truncations on a small vocabulary, one row.
        _sample("sample_token", temperature=0.7, top_k=50, top_p=0.95),
        # Nucleus alone over a large vocabulary, one row.
        _sample("sample_nucleus", vocab=131072, top_p=0.9),
        # A serving batch whose requests differ in every setting, some of them greedy; bf16 logits tie; an odd vocabulary.
        _sample("sample_batch_mixed", rows=64, vocab=128255, kind="bf16", mixed=True, masked=True),
        # A large batch of plain draws with the least likely tokens cut.
        _sample("sample_many", rows=256, vocab=151936, min_p=0.02),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "sample"])
    if op == "route":
        experts = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        c = _route("", tokens=_log(rng, 1, 4096), hidden=8 * _log(rng, 64, 896), experts=experts,
                   top_k=rng.choice([1, 2, 4, 6, 8]), act=rng.choice(["f32", "f16", "bf16"]),
                   kind=rng.choice(["f32", "f16", "bf16"]), scoring=rng.choice(["softmax", "sigmoid"]),
                   bias=rng.random() < 0.5, renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
        c["tokens"] = max(1, min(c["tokens"], 1000000000 // (c["hidden"] * experts)))
    elif op == "experts":
        experts = rng.choice([8, 16, 32, 60, 64, 128])
        c = _experts("", tokens=_log(rng, 1, 128), hidden=128 * _log(rng, 4, 32), inter=128 * _log(rng, 2, 64),
                     experts=experts, top_k=rng.choice([1, 2, 4, 6, 8]), act=rng.choice(["f32", "f32", "f16", "bf16"]),
                     fmt=rng.choice(["q4", "tq2"]), group=rng.choice([32, 64, 128]), residual=rng.random() < 0.5)
        c["inter"] = max(128, min(c["inter"], 600000000 // (3 * c["hidden"] * experts) // 128 * 128))
        c["tokens"] = max(1, min(c["tokens"], 13000000000 // (6 * c["top_k"] * c["hidden"] * c["inter"])))
    else:
        c = _sample("", rows=_log(rng, 1, 256), vocab=_log(rng, 2000, 160000), kind=rng.choice(["f32", "f16", "bf16"]),
                    mixed=rng.random() < 0.4, masked=rng.random() < 0.3, temperature=rng.choice([0.6, 0.8, 1.0, 1.3]),
                    top_k=rng.choice([0, 0, 20, 50, 1000]), top_p=rng.choice([1.0, 0.8, 0.95]),
                    min_p=rng.choice([0.0, 0.0, 0.05]))
    del c["name"]
    return c


def _q4_weight(experts, n, k, group, g):
    codes = torch.randint(0, 256, (experts, n, k // 2), device=DEV, generator=g, dtype=torch.uint8)
    scales = (torch.rand(experts, n, k // group, device=DEV, generator=g) + 0.5) * (0.2 / math.sqrt(k))
    return codes, scales.to(torch.float16)


def _tq2_weight(experts, n, k, g):
    """Blocks of 34 bytes: 128 codes 0, 1, 2 (four to a byte), then a binary16 scale; [experts, n, k / 128, 34]."""
    four = torch.tensor([a | b << 2 | c << 4 | d << 6 for a in range(3) for b in range(3) for c in range(3)
                         for d in range(3)], dtype=torch.uint8, device=DEV)
    blocks = torch.empty(experts, n, k // 128, 34, dtype=torch.uint8, device=DEV)
    for e in range(experts):
        pick = torch.randint(0, 81, (n, k // 128, 32), device=DEV, generator=g, dtype=torch.uint8)
        blocks[e, ..., :32] = four[pick.int()]
        d = (torch.rand(n, k // 128, 1, device=DEV, generator=g) + 0.5) * (1.2 / math.sqrt(k))
        blocks[e, ..., 32:] = d.to(torch.float16).view(torch.uint8)
    return blocks


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "sample":
        return _prepare_sample(case, s, g)
    tokens, hidden, experts, k = case["tokens"], case["hidden"], case["experts"], case["top_k"]
    act = TYPES[case["act"]]
    s["x"] = torch.randn(tokens, hidden, device=DEV, generator=g).to(act)
    if case["op"] == "route":
        s["weight"] = (torch.randn(experts, hidden, device=DEV, generator=g) * (1.5 / math.sqrt(hidden))).to(TYPES[case["kind"]])
        s["bias"] = torch.randn(experts, device=DEV, generator=g) * 0.05 if case["bias"] else None
        s["weights"] = torch.empty(tokens, k, device=DEV)
        s["ids"] = torch.empty(tokens, k, device=DEV, dtype=torch.int32)
        return s
    n, inter = 2 * case["inter"], case["inter"]
    if case["fmt"] == "q4":
        s["gate_up"] = _q4_weight(experts, n, hidden, case["group"], g)
        s["down"] = _q4_weight(experts, hidden, inter, case["group"], g)
    else:
        s["gate_up"], s["down"] = _tq2_weight(experts, n, hidden, g), _tq2_weight(experts, hidden, inter, g)
        if own:  # a program keeps the resident layout
            from gemv_tq2_g128_amd import tq2
            s["gate_up"] = tq2.reformat_aos_to_soa(s["gate_up"].flatten(), experts * n, hidden)
            s["down"] = tq2.reformat_aos_to_soa(s["down"].flatten(), experts * hidden, inter)
    score = torch.randn(tokens, experts, device=DEV, generator=g)
    top, ids = torch.topk(score, k, dim=1)
    s["ids"], s["weights"] = ids.to(torch.int32), torch.softmax(top, 1)
    s["residual"] = torch.randn(tokens, hidden, device=DEV, generator=g).to(act) if case["residual"] else None
    s["out"] = torch.empty(tokens, hidden, device=DEV, dtype=act)
    return s


def _prepare_sample(case, s, g):
    rows, vocab = case["rows"], case["vocab"]
    # A bulk of unlikely tokens and a few favourites, as many and as far above it as the row is sure of itself.
    logits = torch.randn(rows, vocab, device=DEV, generator=g) * 2.0
    liked = torch.randint(0, vocab, (rows, 24), device=DEV, generator=g)
    sure = torch.rand(rows, 1, device=DEV, generator=g) * 10.0 + 4.0
    logits.scatter_(1, liked, sure + torch.randn(rows, 24, device=DEV, generator=g) * 2.0)
    if case["masked"]:  # a padded vocabulary, and tokens that a grammar forbids
        logits[:, vocab - vocab // 50:] = -math.inf
        logits[:, 7:vocab:97] = -math.inf
    s["logits"] = logits.to(TYPES[case["kind"]])
    s["u"] = torch.rand(rows, device=DEV, generator=g)
    for name in ("temperature", "top_k", "top_p", "min_p"):
        s[name] = case[name]
    if case["mixed"]:
        def choice(values, dtype=torch.float32):
            at = torch.randint(0, len(values), (rows,), device=DEV, generator=g)
            return torch.tensor(values, device=DEV, dtype=dtype)[at]
        s["temperature"] = choice([0.0, 0.3, 0.7, 1.0, 1.5])
        s["top_k"] = choice([0, 0, 1, 20, 50, 1000], torch.int32)
        s["top_p"] = choice([1.0, 0.9, 0.95, 0.5])
        s["min_p"] = choice([0.0, 0.0, 0.05, 0.2])
    s["ids"] = torch.empty(rows, device=DEV, dtype=torch.int32)
    s["logprob"] = torch.empty(rows, device=DEV)
    return s


def run(s):
    return {"route": _run_route, "experts": _run_experts, "sample": _run_sample}[s["case"]["op"]](s)


def _run_route(s):
    case = s["case"]
    if own:
        from gemv_tq2_g128_amd import moe
        weights, ids = moe.route(s["x"], s["weight"], case["top_k"], bias=s["bias"], scoring=case["scoring"],
                                 renormalize=case["renormalize"], scale=case["scale"], weights=s["weights"],
                                 ids=s["ids"])
        return {"weights": weights, "ids": ids}
    score = torch.matmul(s["x"].double(), s["weight"].double().t())
    if case["scoring"] == "softmax":
        p = torch.exp(score - score.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-score))
    # Both keep the order of the scores, which lie further apart than the probabilities.
    by = p + s["bias"].double() if case["bias"] else score
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :case["top_k"]]
    weights = torch.gather(p, 1, ids)
    if case["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    return {"weights": (weights * case["scale"]).float(), "ids": ids.to(torch.int32)}


def _values(case, weight, e):
    """Expert e's weights in 32 bits; e an index tensor of one element or a number."""
    pick = (lambda t: t.index_select(0, e)[0]) if isinstance(e, torch.Tensor) else (lambda t: t[e])
    if case["fmt"] == "q4":
        codes, scales = pick(weight[0]), pick(weight[1]).float()
        w = torch.stack((codes & 15, codes >> 4), -1).flatten(1).float() - 8.0
        return (w.unflatten(1, (-1, case["group"])) * scales[..., None]).flatten(1)
    blocks = pick(weight)
    shift = torch.arange(0, 8, 2, device=DEV, dtype=torch.uint8)
    w = ((blocks[..., :32, None] >> shift) & 3).flatten(2).float() - 1.0
    return (w * blocks[..., 32:].contiguous().view(torch.float16).float()).flatten(1)


def _ffn(case, s, x, e):
    y = torch.matmul(x, _values(case, s["gate_up"], e).t())
    gate, up = y[:, :case["inter"]], y[:, case["inter"]:]
    return torch.matmul(gate / (1.0 + torch.exp(-gate)) * up, _values(case, s["down"], e).t())


def _run_experts(s):
    case = s["case"]
    if own:
        from gemv_tq2_g128_amd import moe
        return moe.experts(s["x"], s["gate_up"], s["down"], s["ids"], s["weights"], experts=case["experts"],
                           residual=s["residual"], out=s["out"])
    x, ids = s["x"].float(), s["ids"].long()
    y = torch.zeros_like(x) if s["residual"] is None else s["residual"].float()
    if ids.numel() <= 16:  # few of the experts: each chosen one by itself
        for t in range(case["tokens"]):
            for j in range(case["top_k"]):
                part = _ffn(case, s, x[t:t + 1], ids[t, j:j + 1]) * s["weights"][t, j]
                y = torch.cat((y[:t], y[t:t + 1] + part, y[t + 1:]))
    else:
        share = torch.zeros(case["tokens"], case["experts"], device=DEV).scatter_add_(1, ids, s["weights"])
        for e in range(case["experts"]):
            y = y + _ffn(case, s, x, e) * share[:, e:e + 1]
    return y.to(s["x"].dtype)


def _column(v, rows):
    return v.double()[:, None] if isinstance(v, torch.Tensor) else torch.full((rows, 1), float(v), dtype=torch.float64,
                                                                              device=DEV)


def _run_sample(s):
    if own:
        from gemv_tq2_g128_amd import sampling
        sampling.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                        min_p=s["min_p"], out=s["ids"], logprob=s["logprob"])
        return {"ids": s["ids"], "logprob": s["logprob"]}
    rows, vocab = s["logits"].shape
    heat, most, share, least = (_column(s[n], rows) for n in ("temperature", "top_k", "top_p", "min_p"))
    value, index = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    e = torch.exp((value - value[:, :1]) / torch.where(heat > 0, heat, 1.0))
    rank = torch.arange(vocab, device=DEV)
    e = torch.where((e >= least) & ((rank < most) | (most <= 0)), e, 0.0)
    upto = torch.cumsum(e, 1)
    run_ = (upto - e < share * upto[:, -1:]) | (share >= 1)      # in front of these the share is not reached
    mass = torch.where(run_, upto, 0.0).amax(1, keepdim=True)
    at = (upto <= _column(s["u"], rows) * mass).sum(1, keepdim=True)
    at = torch.where(heat > 0, at, 0)
    logprob = torch.where(heat > 0, torch.log(torch.gather(e, 1, at) / mass), 0.0)
    return {"ids": torch.gather(index, 1, at)[:, 0].to(torch.int32), "logprob": logprob[:, 0].float()}


def work(case):
    """Bytes and operations of one pass."""
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * SIZE[case["kind"]] + case["rows"] * (28 if case["mixed"] else 12), "flops": n}
    tokens, hidden, experts, k = case["tokens"], case["hidden"], case["experts"], case["top_k"]
    if case["op"] == "route":
        return {"bytes": hidden * (tokens * SIZE[case["act"]] + experts * SIZE[case["kind"]]) + 8 * tokens * k,
                "flops": 2 * tokens * experts * hidden}
    # Experts that a batch touches, each token choosing k different ones of them at random.
    touched = experts * (1.0 - (1.0 - k / experts) ** tokens)
    bits = 4.0 + 16.0 / case["group"] if case["fmt"] == "q4" else 2.125
    moved = touched * 3 * hidden * case["inter"] * bits / 8 + tokens * (
        hidden * SIZE[case["act"]] * (3 if case["residual"] else 2) + 8 * k)
    return {"bytes": int(moved), "flops": 6 * tokens * k * hidden * case["inter"]}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"route": _exact_route, "experts": _exact_experts, "sample": _exact_sample}[case["op"]](case, s)


def _exact_route(case, s):
    score = torch.empty(case["tokens"], case["experts"], dtype=torch.float64, device=DEV)
    w = s["weight"].double()
    for lo in range(0, case["tokens"], 256):
        score[lo:lo + 256] = (w @ s["x"][lo:lo + 256].double().t().contiguous()).t()
    p = torch.softmax(score, 1) if case["scoring"] == "softmax" else torch.special.expit(score)
    left = p + s["bias"].double() if case["bias"] else score.clone()
    ids = []
    for _ in range(case["top_k"]):
        best = (left == left.amax(1, keepdim=True)).to(torch.int32).argmax(1, keepdim=True)
        ids.append(best)
        left.scatter_(1, best, -math.inf)
    ids = torch.cat(ids, 1)
    weights = torch.take_along_dim(p, ids, 1)
    if case["renormalize"]:
        weights /= weights.sum(1, keepdim=True)
    return {"weights": weights * case["scale"], "ids": ids.to(torch.int32)}


def _exact_weight(case, weight, e, rows, cols):
    w = torch.empty(rows, cols, dtype=torch.float64, device=DEV)
    if case["fmt"] == "q4":
        codes, scales = weight[0][e], weight[1][e]
        w[:, 0::2], w[:, 1::2] = (codes % 16).double() - 8, (codes // 16).double() - 8
        return w * scales.double().repeat_interleave(case["group"], 1)
    blocks = weight[e]
    fields = w.view(rows, cols // 128, 32, 4)
    for i in range(4):
        fields[..., i] = (blocks[..., :32] // 4 ** i % 4).double() - 1
    d = blocks[..., 32:].contiguous().view(torch.float16).double()
    return (w.view(rows, cols // 128, 128) * d).view(rows, cols)


def _exact_experts(case, s):
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    inter, ids = case["inter"], s["ids"].tolist()
    for e in sorted({i for row in ids for i in row}):
        who = [(t, j) for t, row in enumerate(ids) for j, i in enumerate(row) if i == e]
        at = torch.tensor([t for t, _ in who], device=DEV)
        x = s["x"][at].double()
        both = x @ _exact_weight(case, s["gate_up"], e, 2 * inter, case["hidden"]).t().contiguous()
        h = torch.nn.functional.silu(both[:, :inter]) * both[:, inter:]
        o = h @ _exact_weight(case, s["down"], e, case["hidden"], inter).t().contiguous()
        y.index_add_(0, at, o * torch.stack([s["weights"][t, j] for t, j in who]).double()[:, None])
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_sample(case, s):
    out, logprob = [], []
    for r in range(case["rows"]):
        heat, most, share, least, u = (float(v[r]) if isinstance(v, torch.Tensor) else float(v) for v in (
            s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"]))
        row = s["logits"][r].double()
        order = torch.argsort(-row, stable=True)
        if heat <= 0:
            out.append(int(order[0]))
            logprob.append(0.0)
            continue
        if most > 0:
            order = order[:int(most)]
        z = (row[order] - row[order[0]]) / heat
        p = torch.exp(z)
        p = p[p >= least]
        if share < 1:
            total = torch.cumsum(p, 0)
            p = p[:int(torch.searchsorted(total, share * total[-1])) + 1]
        total = torch.cumsum(p, 0)
        at = min(int(torch.searchsorted(total, u * total[-1], right=True)), len(p) - 1)
        out.append(int(order[at]))
        logprob.append(float(z[at] - torch.log(total[-1])))
    return {"ids": torch.tensor(out, dtype=torch.int32, device=DEV),
            "logprob": torch.tensor(logprob, dtype=torch.float64, device=DEV)}
