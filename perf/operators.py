"""Measured cases of the attention-layer operators: kv_append, paged_attention and q4_gemv.

Together they are the attention half of a decoder layer around the library's quantised projections: 4-bit projections
give q, k and v; kv_append normalises and rotates q and k and stores k and v in a paged cache; paged_attention reads
that cache for the new tokens; a 4-bit projection adds its result to the residual stream.

``run`` computes an operator in plain torch (32-bit sums, 64-bit angles) or, with ``own``, calls this library.
``exact`` evaluates the definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
EPS = 1e-6


def _append(name, **over):
    return {"name": name, "op": "append", "batch": 1, "q_len": 1, "past": 1000, "q_heads": 32, "kv_heads": 8,
            "head_dim": 128, "rot": 128, "page": 16, "act": "f32", "cache": "f16", "axes": 1, "norm": True,
            "interleaved": False, **over}


def _attention(name, **over):
    return {"name": name, "op": "attention", "batch": 1, "q_len": 1, "kv_len": 1000, "ragged": False, "q_heads": 32,
            "kv_heads": 8, "head_dim": 128, "page": 16, "act": "f32", "cache": "f16", "window": 0, **over}


def _q4(name, **over):
    return {"name": name, "op": "q4", "m": 1, "n": 4096, "k": 4096, "group": 128, "residual": False, **over}


def listed():
    return [
        # One token of one sequence, f32 activations as the ternary GEMV gives them: pure latency.
        _append("append_token"),
        # A full decode batch into an 8-bit cache.
        _append("append_decode_e4m3", batch=256, past=2000, q_heads=64, act="bf16", cache="e4m3", page=32),
        # Prompts of images and text, rotated by time, height and width, ragged.
        _append("append_prompt_axes", batch=3, q_len=2731, past=0, axes=3, page=64),
        # A chunk of a model with as many key heads as query heads, partial rotation of neighbouring pairs.
        _append("append_chunk_pairs", batch=2, q_len=1025, past=513, q_heads=16, kv_heads=16, head_dim=64, rot=32,
                act="bf16", cache="bf16", norm=False, interleaved=True),
        # One sequence decoding early in its answer: latency again.
        _attention("attention_token", kv_len=1001),
        # A serving batch of sequences of all lengths.
        _attention("attention_decode", batch=64, kv_len=8192, ragged=True, act="bf16", cache="bf16"),
        # Few very long sequences over an 8-bit cache.
        _attention("attention_long_e4m3", batch=4, kv_len=131071, ragged=True, act="f16", cache="e4m3", page=64),
        # A chunk of a long prompt over what is cached of it.
        _attention("attention_chunk", q_len=512, kv_len=16895, act="f16", page=32),
        # Whole prompts at once, of different lengths.
        _attention("attention_prompt", batch=2, q_len=4096, kv_len=4096, ragged=True, act="bf16", cache="bf16",
                   page=64),
        # An attention projection of one token with its residual.
        _q4("q4_token", residual=True),
        # A feed-forward projection with an odd number of rows in small groups.
        _q4("q4_rows", n=11007, group=32),
        # The vocabulary of eight sequences.
        _q4("q4_vocabulary", m=8, n=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "q4"])
    if op == "q4":
        c = _q4("", m=rng.choice([1, 1, 1, 2, 3, 5, 8, 13]), n=_log(rng, 256, 65536), k=128 * _log(rng, 4, 96),
                group=rng.choice([32, 64, 128]), residual=rng.random() < 0.5)
        c["n"] = min(c["n"], (131072 * 4096) // c["k"])
    else:
        heads = rng.choice([(32, 8), (32, 8), (16, 16), (64, 8), (24, 4), (14, 2), (40, 8)])
        act, cache = rng.choice([("f32", "f16"), ("f32", "e4m3"), ("f16", "f16"), ("f16", "e4m3"), ("bf16", "bf16"),
                                 ("bf16", "e4m3")])
        common = dict(q_heads=heads[0], kv_heads=heads[1], head_dim=rng.choice([64, 96, 128, 128, 128, 256]),
                      page=rng.choice([16, 32, 64, 128]), act=act, cache=cache)
        if op == "append":
            tokens = _log(rng, 1, 8192)
            batch = min(tokens, _log(rng, 1, 256))
            c = _append("", batch=batch, q_len=tokens // batch, past=rng.randrange(0, 4096),
                        axes=rng.choice([1, 1, 3]), norm=rng.random() < 0.5, interleaved=rng.random() < 0.3, **common)
            c["rot"] = rng.choice([c["head_dim"], c["head_dim"], c["head_dim"] // 2])
        else:
            q_len = rng.choice([1, 1, 1, rng.randrange(2, 9), _log(rng, 16, 2048)])
            batch = _log(rng, 1, 64) if q_len < 16 else _log(rng, 1, 3)
            kv_len = q_len + _log(rng, 1, 16384 if q_len < 16 else 6000)
            pair = 2 * batch * heads[1] * common["head_dim"] * SIZE[cache]
            kv_len = max(q_len, min(kv_len, 600000000 // pair))
            q_len = max(1, min(q_len, 68000000000 // (batch * heads[0] * common["head_dim"] * kv_len)))
            c = _attention("", batch=batch, q_len=q_len, kv_len=kv_len, ragged=rng.random() < 0.7,
                           window=rng.choice([0, 0, 0, 1024]), **common)
    del c["name"]
    return c


def _lengths(case):
    """New tokens and cached tokens (those included) of each sequence. They belong to the case: any seed has the same."""
    def spread(least, longest):  # the first is the longest, the others lie all over the range
        return [longest if i == 0 else least + int((longest - least + 1) * (i * 0.6180339887 % 1.0))
                for i in range(case["batch"])]

    if case["op"] == "append":
        q_len = spread(1, case["q_len"])
        return q_len, [n + case["past"] for n in q_len]
    kv_len = spread((case["q_len"] + 1) // 2, case["kv_len"]) if case["ragged"] else [case["kv_len"]] * case["batch"]
    return [min(n, case["q_len"]) for n in kv_len], kv_len


def _pages(kv_len, page, gen):
    """Block table [batch, most] of a cache whose pages were handed out in no order, and the number of pages."""
    most = int((int(kv_len.max()) + page - 1) // page)
    pages = kv_len.numel() * most
    return torch.randperm(pages, generator=gen).to(torch.int32).reshape(kv_len.numel(), most), pages


def _cache(shape, kind, g):
    x = torch.randn(shape, device=DEV, generator=g, dtype=torch.float16)
    return (x * 8.0).to(TYPES[kind]) if kind == "e4m3" else x.to(TYPES[kind])


def _scales(case, g):
    if case["cache"] != "e4m3":
        return None, None
    s = torch.rand(2, case["kv_heads"], device=DEV, generator=g) * 0.05 + 0.1
    return s[0].contiguous(), s[1].contiguous()


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "q4":
        m, n, k = case["m"], case["n"], case["k"]
        s["codes"] = torch.randint(0, 256, (n, k // 2), device=DEV, generator=g, dtype=torch.uint8)
        s["scales"] = ((torch.rand(n, k // case["group"], device=DEV, generator=g) + 0.5) * 0.01).to(torch.float16)
        x = torch.randn(m, k, device=DEV, generator=g)
        s["x"] = x * torch.where(torch.rand(k, device=DEV, generator=g) < 0.01, 10.0, 1.0)  # some strong channels
        s["residual"] = torch.randn(m, n, device=DEV, generator=g) if case["residual"] else None
        s["out"] = torch.empty(m, n, device=DEV)
        return s
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    act = TYPES[case["act"]]
    q_len, kv_len = (torch.tensor(n, dtype=torch.int64) for n in _lengths(case))
    table, pages = _pages(kv_len, page, gen)
    tokens = int(q_len.sum())
    cu = torch.zeros(case["batch"] + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(q_len, 0)
    s["kv_len"] = kv_len.to(torch.int32).to(DEV)
    s["table"] = table.to(DEV)
    s["cu"] = None if case["q_len"] == 1 else cu.to(DEV)
    s["max_q"], s["max_kv"] = int(q_len.max()), int(kv_len.max())
    s["k_scale"], s["v_scale"] = _scales(case, g)
    if case["op"] == "append":
        # q, k and v are columns of one projection's output.
        qkv = torch.randn(tokens, (hq + 2 * hkv) * d, device=DEV, generator=g).to(act)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        s["q_out"] = torch.empty(tokens, hq, d, device=DEV, dtype=act)
        s["k_cache"] = torch.zeros(pages, hkv, page, d, device=DEV, dtype=torch.float16).to(TYPES[case["cache"]])
        s["v_cache"] = s["k_cache"].clone()
        half = case["rot"] // 2
        s["freqs"] = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        s["sections"] = s["positions"] = None
        if case["axes"] == 3:
            s["sections"] = (half - 2 * (3 * half // 8), 3 * half // 8, 3 * half // 8)
            s["positions"] = torch.randint(0, 4096, (3, tokens), device=DEV, generator=g, dtype=torch.int32)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = torch.rand(d, device=DEV, generator=g) + 0.5
            s["k_norm"] = torch.rand(d, device=DEV, generator=g) + 0.5
        return s
    s["q"] = (torch.randn(tokens, hq, d, device=DEV, generator=g) * 1.5).to(act)
    s["out"] = torch.empty(tokens, hq, d, device=DEV, dtype=act)
    shape = (pages, hkv, page, d)
    s["k_cache"], s["v_cache"] = _cache(shape, case["cache"], g), _cache(shape, case["cache"], g)
    return s


def run(s):
    return {"append": _run_append, "attention": _run_attention, "q4": _run_q4}[s["case"]["op"]](s)


def _owner(s, tokens):
    """Each new token's sequence and its place in that sequence's cache."""
    t = torch.arange(tokens, device=DEV)
    if s["cu"] is None:
        return t, s["kv_len"].long() - 1
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, s["kv_len"].long()[b] - (cu[b + 1] - t)


def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _rotated(x, cos, sin, interleaved):
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _stored(x, scale, dtype):
    if scale is not None:
        x = (x / scale[:, None]).clamp(-448.0, 448.0)
    return x.to(dtype)


def _run_append(s):
    case = s["case"]
    if own:
        from gemv_tq2_g128_amd import attn
        attn.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["kv_len"], s["table"], q=s["q"],
                       q_out=s["q_out"], cu_q=s["cu"], freqs=s["freqs"], positions=s["positions"],
                       sections=s["sections"], interleaved=case["interleaved"], q_norm=s["q_norm"],
                       k_norm=s["k_norm"], eps=EPS, k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    b, place = _owner(s, s["k"].shape[0])
    if s["positions"] is None:
        angle = place.double()[:, None] * s["freqs"]
    else:
        axis = torch.repeat_interleave(torch.arange(3, device=DEV), torch.tensor(s["sections"], device=DEV))
        angle = s["positions"].double()[axis].t() * s["freqs"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    s["q_out"].copy_(_rotated(_normed(s["q"], s["q_norm"]), cos, sin, case["interleaved"]))
    k = _rotated(_normed(s["k"], s["k_norm"]), cos, sin, case["interleaved"])
    page, off = s["table"].long()[b, place // case["page"]], place % case["page"]
    # Byte views: every cache type is moved as the bits it is.
    bits = torch.uint8 if case["cache"] == "e4m3" else torch.int16
    kind = TYPES[case["cache"]]
    s["k_cache"].view(bits)[page, :, off] = _stored(k, s["k_scale"], kind).view(bits)
    s["v_cache"].view(bits)[page, :, off] = _stored(s["v"].float(), s["v_scale"], kind).view(bits)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _run_attention(s):
    case = s["case"]
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    if own:
        from gemv_tq2_g128_amd import attn
        return attn.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["kv_len"], s["table"], cu_q=s["cu"],
                                    max_q=s["max_q"], max_kv=s["max_kv"], window=case["window"],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
    tokens, batch, rows = s["q"].shape[0], case["batch"], s["max_q"]
    b, place = _owner(s, tokens)
    first = torch.zeros_like(s["kv_len"]).long() if s["cu"] is None else s["cu"][:-1].long()
    t = torch.arange(tokens, device=DEV)
    row = torch.zeros_like(t) if s["cu"] is None else t - first[b]
    # Padded to the longest chunk and the longest cache; group * row query vectors share a key head.
    q = torch.zeros(batch, rows, hq, d, device=DEV)
    q[b, row] = s["q"].float()
    at = torch.full((batch, rows), -1, dtype=torch.int64, device=DEV)
    at[b, row] = place
    table = s["table"].long()
    k = s["k_cache"].float()[table].transpose(1, 2).flatten(2, 3)
    v = s["v_cache"].float()[table].transpose(1, 2).flatten(2, 3)
    q = q.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    scale = torch.full((hkv, 1, 1), 1.0 / math.sqrt(d), device=DEV)
    if s["k_scale"] is not None:
        scale = scale * s["k_scale"][:, None, None]
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * scale
    del k
    key = torch.arange(score.shape[-1], device=DEV)
    seen = key <= at[..., None]
    if case["window"]:
        seen = seen & (key > at[..., None] - case["window"])
    score = score.unflatten(2, (hq // hkv, rows)).masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp_(score - torch.where(top == float("-inf"), 0.0, top)).flatten(2, 3)
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    if s["v_scale"] is not None:
        o = o * s["v_scale"][:, None, None]
    o = o.unflatten(2, (hq // hkv, rows)).permute(0, 3, 1, 2, 4).reshape(batch, rows, hq, d)
    return o[b, row].to(s["q"].dtype)


def _run_q4(s):
    case = s["case"]
    if own:
        from gemv_tq2_g128_amd import q4
        return q4.gemv(s["codes"], s["scales"], s["x"], residual=s["residual"], out=s["out"])
    w = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).flatten(1).float() - 8.0
    w = (w.unflatten(1, (-1, case["group"])) * s["scales"].float()[..., None]).flatten(1)
    y = torch.matmul(s["x"], w.t())
    return y if s["residual"] is None else y + s["residual"]


def work(case):
    """Bytes and operations of one pass."""
    if case["op"] == "q4":
        m, n, k = case["m"], case["n"], case["k"]
        moved = n * k // 2 + 2 * n * (k // case["group"]) + 4 * m * (k + n * (2 if case["residual"] else 1))
        return {"bytes": moved, "flops": 2 * m * n * k}
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    a, c = SIZE[case["act"]], SIZE[case["cache"]]
    if case["op"] == "append":
        tokens = sum(_lengths(case)[0])
        return {"bytes": tokens * d * (2 * hq * a + 2 * hkv * (a + c)) + 12 * tokens * (case["axes"] == 3),
                "flops": 6 * tokens * (hq + hkv) * d}
    total = {"bytes": 0, "flops": 0}
    for q_len, n in zip(*_lengths(case)):
        seen, keys = n - (q_len - 1) / 2, n
        if case["window"]:
            seen, keys = min(seen, case["window"]), min(n, case["window"] + q_len - 1)
        total["bytes"] += 2 * q_len * hq * d * a + 2 * keys * hkv * d * c
        total["flops"] += 4 * q_len * hq * d * seen
    return total


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "q4":
        code = torch.empty(case["n"], case["k"], dtype=torch.int8, device=DEV)
        code[:, 0::2] = (s["codes"] % 16).to(torch.int8)
        code[:, 1::2] = (s["codes"] // 16).to(torch.int8)
        out = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
        for lo in range(0, case["n"], 16384):
            part = slice(lo, lo + 16384)
            d = s["scales"][part].double().repeat_interleave(case["group"], 1)
            out[:, part] = (((code[part].double() - 8) * d) @ s["x"].double().t().contiguous()).t()
        return out if s["residual"] is None else out + s["residual"].double()
    q_len, kv_len = _lengths(case)
    start = [0]
    for n in q_len:
        start.append(start[-1] + n)
    hkv, d, page = case["kv_heads"], case["head_dim"], case["page"]
    group = case["q_heads"] // hkv
    if case["op"] == "append":
        return _exact_append(case, s, q_len, kv_len, start)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    ks = torch.ones(hkv, device=DEV) if s["k_scale"] is None else s["k_scale"]
    vs = torch.ones(hkv, device=DEV) if s["v_scale"] is None else s["v_scale"]
    for b, (new, n) in enumerate(zip(q_len, kv_len)):
        ids = s["table"][b, :(n + page - 1) // page].long()
        here = slice(start[b], start[b] + new)
        place = torch.arange(n - new, n, device=DEV)
        keys = torch.arange(n, device=DEV)
        hidden = keys[None] > place[:, None]
        if case["window"]:
            hidden |= keys[None] <= place[:, None] - case["window"]
        for h in range(hkv):
            k = s["k_cache"][ids, h].double().reshape(-1, d)[:n] * ks[h].double()
            v = s["v_cache"][ids, h].double().reshape(-1, d)[:n] * vs[h].double()
            kt = k.t().contiguous()
            for j in range(h * group, (h + 1) * group):
                w = (s["q"][here, j].double().contiguous() @ kt) / math.sqrt(d)
                w[hidden] = -math.inf
                out[here, j] = torch.softmax(w, -1) @ v
    return out


def _exact_append(case, s, q_len, kv_len, start):
    half, page = case["rot"] // 2, case["page"]
    owner = [b for b, n in enumerate(q_len) for _ in range(n)]
    place = [kv_len[b] - q_len[b] + i for b, n in enumerate(q_len) for i in range(n)]
    owner, place = torch.tensor(owner, device=DEV), torch.tensor(place, device=DEV)
    angle = torch.empty(start[-1], half, dtype=torch.float64, device=DEV)
    at = 0
    for axis, width in enumerate(s["sections"] or (half,)):
        pos = place if s["positions"] is None else s["positions"][axis]
        angle[:, at:at + width] = pos.double()[:, None] * s["freqs"][at:at + width]
        at += width
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotate(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
        y = x.clone()
        real, imag = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else \
            (slice(0, half), slice(half, 2 * half))
        z = torch.complex(x[..., real].contiguous(), x[..., imag].contiguous()) * turn
        y[..., real], y[..., imag] = z.real, z.imag
        return y

    k, v = rotate(s["k"], s["k_norm"]), s["v"].double()
    if case["cache"] == "e4m3":
        k = (k / s["k_scale"].double()[:, None]).clamp(-448, 448)
        v = (v / s["v_scale"].double()[:, None]).clamp(-448, 448)
    ids, off = s["table"][owner, place // page].long(), place % page
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc[ids, :, off], vc[ids, :, off] = k, v
    return {"q": rotate(s["q"], s["q_norm"]), "k_cache": kc, "v_cache": vc}
