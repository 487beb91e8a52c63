"""GPU parity of tq2_paged_attention against softmax attention in float64.

Tolerance, per component, in units of S = sum_j p_j |v_j|:
* scores: f32 sums of at most 256 products whose operands are exact to 2^-22 (f32 q in two parts) or exact; a score's
  error is below (256 * 2^-24 + 2^-21) * A, A = scale * sum_i |q_i k_i|, and moves p_j by that much, relative, once
  against the sum and once in it: 2 * 1.6e-5 * max A.  That is a bound on every rounding falling the same way; the sums
  are of random signs, so their square root is allowed: 32 roundings of 2^-24 and the operands' 2^-21, times A and
  twice, 2 * (2e-6 + 5e-7) * A.
* the exponential, the rescalings and the sums over keys: 64 roundings of 2^-24, 4e-6.
* probabilities: two parts for f32 (2^-21); otherwise half a step of the products' type each, 2^-11 (binary16, also over
  e4m3) or 2^-8 (bfloat16).
* the output's own rounding: half a step.
"""

import math

import pytest

torch = pytest.importorskip("torch")
from tests import attn_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu

PAIRS = [("f32", "f16"), ("f32", "e4m3"), ("f16", "f16"), ("f16", "e4m3"), ("bf16", "bf16"), ("bf16", "e4m3")]


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    from gemv_tq2_g128_amd import attn as mod
    return mod


def make(seed, act="f32", cache="f16", q_len=(1, 1, 1), kv_len=(5, 16, 33), heads=(8, 2), dim=128, page=16,
         order="pages", spread=1.5):
    gen = torch.Generator().manual_seed(seed)
    hq, hkv = heads
    c = {"q_len": list(q_len), "kv_len": list(kv_len), "act": act, "cache": cache}
    c["q"] = (torch.randn(sum(q_len), hq, dim, generator=gen) * spread).to(R.DTYPES[act])
    c["table"], pages = R.block_table(c["kv_len"], page, gen)
    for n in "kv":
        x = torch.randn(pages, hkv, page, dim, generator=gen)
        x = (x * 8).to(R.DTYPES[cache]) if cache == "e4m3" else x.to(R.DTYPES[cache])
        if order == "tokens":
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        c[n] = x
        c[n + "_scale"] = torch.rand(hkv, generator=gen) * 0.05 + 0.1 if cache == "e4m3" else None
    return c


def cuda(t):
    return None if t is None else t.cuda()


def call(attn, c, **more):
    cu = None if all(n == 1 for n in c["q_len"]) else R.offsets(c["q_len"]).cuda()
    more.setdefault("max_q", max(c["q_len"]))
    more.setdefault("max_kv", max(0, *c["kv_len"]))
    q = c["q"].cuda() if more.get("q") is None else more["q"]
    more.pop("q", None)
    return attn.paged_attention(q, cuda(c["k"]), cuda(c["v"]), torch.tensor(c["kv_len"], dtype=torch.int32).cuda(),
                                cuda(c["table"]), cu_q=cu, k_scale=cuda(c["k_scale"]), v_scale=cuda(c["v_scale"]),
                                **more)


def tolerance(c, want, size, scale=None):
    d = c["q"].shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    k = c["k"].double().abs()
    if c["k_scale"] is not None:
        k = k * c["k_scale"].double()[None, :, None, None]
    k = torch.nan_to_num(k, nan=0.0, posinf=0.0)
    # |q . k| at its largest is below |q| |k|.
    top = scale * float(c["q"].double().norm(dim=-1).max() * k.norm(dim=-1).max())
    p = {"f32": 2.0 ** -21, "f16": 2.0 ** -11, "bf16": 2.0 ** -8 if c["cache"] == "bf16" else 2.0 ** -11}[c["act"]]
    rel = 2 * (2e-6 + 5e-7) * top + 4e-6 + p
    return rel * size + R.HALF[c["act"]] * (want.abs() + rel * size) + R.TINY[c["act"]]


def check(attn, c, label, window=0, scale=None, **more):
    out = call(attn, c, window=window, scale=scale, **more)
    torch.cuda.synchronize()
    want, size = R.attend(c["q"], c["k"], c["v"], c["q_len"], c["kv_len"], c["table"], window, scale, c["k_scale"],
                          c["v_scale"])
    err, tol = (out.double().cpu() - want).abs(), tolerance(c, want, size, scale)
    print(label, "worst err / tol %.3f" % float((err / tol).max()) if err.numel() else "", flush=True)
    assert bool((err <= tol).all()), label
    return out


@pytest.mark.parametrize("act,cache", PAIRS)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads", [(8, 2), (14, 2)])
def test_single_tokens(attn, act, cache, dim, heads):
    c = make(dim + heads[0], act, cache, kv_len=(1, 15, 16, 17, 31, 33, 64, 129, 300), q_len=[1] * 9, dim=dim,
             heads=heads)
    check(attn, c, "%s %s %d" % (act, cache, dim))


@pytest.mark.parametrize("act,cache", PAIRS)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_chunks(attn, act, cache, dim):
    """New tokens with and without a past, none, one and many, row tiles that end early."""
    c = make(dim, act, cache, q_len=(5, 0, 1, 40, 37, 130), kv_len=(5, 20, 9, 40, 200, 133), dim=dim, heads=(6, 2))
    check(attn, c, "%s %s %d" % (act, cache, dim))


@pytest.mark.parametrize("act,cache", PAIRS)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_prompts(attn, act, cache, dim):
    """Several blocks of rows, several parts of the keys, tiles of keys that end early and pages longer than a run."""
    c = make(dim + 1, act, cache, q_len=(513, 0, 1, 65, 300), kv_len=(1213, 20, 700, 65, 333), dim=dim, heads=(3, 1),
             page=32)
    check(attn, c, "%s %s %d" % (act, cache, dim))
    check(attn, c, "window %s %s %d" % (act, cache, dim), window=130)


@pytest.mark.parametrize("heads", [(1, 1), (16, 16), (32, 2), (24, 4), (40, 8), (5, 1)])
@pytest.mark.parametrize("q_len", [1, 3, 70])
def test_head_counts(attn, heads, q_len):
    c = make(heads[0], "f16", "f16", q_len=(q_len, q_len), kv_len=(q_len + 50, q_len), heads=heads, dim=64)
    check(attn, c, "%s %d" % (heads, q_len))


@pytest.mark.parametrize("page,order", [(16, "tokens"), (32, "pages"), (128, "tokens"), (1024, "pages")])
def test_pages_and_orders(attn, page, order):
    c = make(page, "bf16", "bf16", q_len=(1, 20, 3), kv_len=(400, 75, 3), page=page, order=order)
    check(attn, c, "page %d %s" % (page, order))


@pytest.mark.parametrize("window", [1, 7, 32, 100, 1000])
@pytest.mark.parametrize("q_len", [1, 6, 150])
def test_windows(attn, window, q_len):
    c = make(window, "f16", "f16", q_len=(q_len, 1, q_len), kv_len=(q_len + 300, 500, q_len), heads=(4, 2), dim=64)
    check(attn, c, "window %d" % window, window=window)


@pytest.mark.parametrize("act,cache", [("f32", "f16"), ("bf16", "e4m3"), ("bf16", "bf16")])
def test_long_caches(attn, act, cache):
    """Many parts of a sequence's keys, beside short sequences."""
    c = make(77, act, cache, q_len=(1, 1, 1), kv_len=(20011, 1, 4096), heads=(4, 1), page=64)
    check(attn, c, "long %s %s" % (act, cache))
    c = make(78, act, cache, q_len=(4, 2), kv_len=(9001, 2), heads=(4, 1), page=64)
    check(attn, c, "long chunk %s %s" % (act, cache))


def test_sizes_that_the_launch_was_not_shaped_for(attn):
    """max_q and max_kv too small or too large change nothing but rounding."""
    c = make(5, "f16", "f16", q_len=(70, 3, 1), kv_len=(900, 3, 41), heads=(4, 1), dim=64)
    for max_q, max_kv in ((1, 1), (1, 100000), (70, 0), (0, 900), (1000, 64), (None, None)):
        check(attn, c, "hints %s %s" % (max_q, max_kv), max_q=max_q, max_kv=max_kv)


@pytest.mark.parametrize("q_len", [1, 24])
def test_rows_that_see_nothing(attn, q_len):
    """Empty sequences, more new tokens than kv_len, lengths past the table, and pages that do not exist."""
    c = make(6, "f32", "f16", q_len=(q_len,) * 5, kv_len=(40,) * 5, heads=(4, 2), dim=64)
    c["kv_len"] = [0, -7, q_len // 2, 1000, 40]
    c["table"][4, 1] = -1
    c["table"][3, 0] = c["k"].shape[0]
    c["kv_len"][3] = 48 + q_len                 # the last rows lie past the table's 48 places
    out = check(attn, c, "empty")
    assert bool((out[:2 * q_len] == 0).all())
    c["table"][:] = -1
    assert bool((call(attn, c) == 0).all())


def test_rows_without_a_sequence(attn):
    c = make(8, "f32", "f16", q_len=(3, 4), kv_len=(10, 20), heads=(2, 1), dim=64)
    want, _ = R.attend(c["q"], c["k"], c["v"], [3, 4], [10, 20], c["table"])
    for cu, owned in (([0, 3, 90], range(0, 3)), ([0, 3, 3], range(0, 3)), ([-5, 3, 3], range(0, 3)),
                      ([0, 0, 0], range(0))):
        out = torch.full((7, 2, 64), 7.0, device="cuda")
        attn.paged_attention(c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), torch.tensor([10, 20]).int().cuda(),
                             c["table"].cuda(), cu_q=torch.tensor(cu, dtype=torch.int32).cuda(), out=out)
        for t in range(7):
            if t in owned:
                assert float((out[t].double().cpu() - want[t]).abs().max()) < 1e-4, (cu, t)
            elif t >= max(cu):
                assert bool((out[t] == 7.0).all()), (cu, t)


@pytest.mark.parametrize("act,cache", PAIRS)
@pytest.mark.parametrize("q_len", [1, 9, 150])
def test_masked_places_may_hold_anything(attn, act, cache, q_len):
    """Past the end, in front of the window and later in the chunk: NaN, infinities and the largest values there
    change no bit of rows that do not see them."""
    c = make(9, act, cache, q_len=(q_len, 2), kv_len=(q_len + 90, 50), heads=(4, 2), dim=96, page=32)
    window = 60
    out = check(attn, c, "clean", window=window)
    top = 448.0 if cache == "e4m3" else float(torch.finfo(R.DTYPES[cache]).max)
    odd = [float("nan"), top, -top] + ([] if cache == "e4m3" else [float("inf"), -float("inf")])
    for n in "kv":
        x = c[n].float()
        for b in range(2):
            room = c["table"].shape[1] * 32
            first = c["kv_len"][b] - c["q_len"][b]
            hidden = list(range(c["kv_len"][b], room)) + list(range(0, max(0, first - window + 1)))
            for i, at in enumerate(hidden):
                x[int(c["table"][b, at // 32]), :, at % 32, (i % 3)::3] = odd[i % len(odd)]
        c[n] = x.to(R.DTYPES[cache])
    assert torch.equal(call(attn, c, window=window), out)
    # The last new token of sequence 0 is seen by its own row alone.
    if q_len > 1:
        at = c["kv_len"][0] - 1
        c["v"] = c["v"].float()
        c["v"][int(c["table"][0, at // 32]), :, at % 32, 5] = float("nan")
        c["k"] = c["k"].float()
        c["k"][int(c["table"][0, at // 32]), :, at % 32, 3] = float("nan")
        c["v"], c["k"] = c["v"].to(R.DTYPES[cache]), c["k"].to(R.DTYPES[cache])
        got = call(attn, c, window=window)
        assert torch.equal(got[:q_len - 1], out[:q_len - 1]) and torch.equal(got[q_len:], out[q_len:])
        assert bool(got[q_len - 1].isnan().all())


@pytest.mark.parametrize("act,cache", [("f32", "f16"), ("f16", "f16"), ("bf16", "bf16")])
def test_infinite_values_that_are_seen(attn, act, cache):
    """They reach exactly the rows and components that see them, with their sign."""
    c = make(10, act, cache, q_len=(12,), kv_len=(40,), heads=(2, 1), dim=64)
    base = call(attn, c)
    page, off = int(c["table"][0, 2]), 33 % 16
    c["v"][page, 0, off, 7] = float("inf")
    c["v"][page, 0, off, 9] = -float("inf")
    out = call(attn, c).float()
    for t in range(12):
        see = 28 + t >= 33
        assert bool((out[t, :, 7] == float("inf")).all()) == see and bool((out[t, :, 9] == -float("inf")).all()) == see
    rest = [i for i in range(64) if i not in (7, 9)]
    assert torch.equal(out[:, :, rest], base.float()[:, :, rest])


@pytest.mark.parametrize("act,cache", [("f32", "f16"), ("f16", "f16"), ("bf16", "bf16")])
def test_large_scores(attn, act, cache):
    """One key takes all the weight, wherever it lies; scores far apart underflow to nothing."""
    c = make(11, act, cache, q_len=(1, 3), kv_len=(200, 77), heads=(4, 2), dim=64, spread=1.0)
    c["q"] = (c["q"].float() * 30).to(R.DTYPES[act])
    check(attn, c, "large", scale=1.0)


def test_magnitudes_of_f32_q(attn):
    """Rows of q sixty binary orders apart keep their accuracy; zeros give the mean."""
    c = make(12, "f32", "f16", q_len=(16,), kv_len=(80,), heads=(2, 1), dim=64)
    c["q"] *= torch.exp2(torch.linspace(-60, 3, 16))[:, None, None]
    c["q"][5] = 0
    check(attn, c, "magnitudes")


def test_in_place_columns_stream(attn):
    c = make(13, "f16", "f16", q_len=(1, 7, 30), kv_len=(70, 7, 90))
    want = call(attn, c)
    q = c["q"].cuda()
    assert torch.equal(call(attn, c, q=q, out=q), want)
    wide = torch.zeros(38, 12, 128, device="cuda", dtype=torch.float16)       # q is columns of a wider array
    wide[:, 2:10] = c["q"].cuda()
    held = torch.zeros(38, 20, 128, device="cuda", dtype=torch.float16)
    call(attn, c, q=wide[:, 2:10], out=held[:, 4:12])
    assert torch.equal(held[:, 4:12], want) and bool((held[:, :4] == 0).all()) and bool((held[:, 12:] == 0).all())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        other = call(attn, c)
    stream.synchronize()
    assert torch.equal(other, want)
    assert call(attn, make(14, "f16", "f16", q_len=(0,), kv_len=(4,))).shape == (0, 8, 128)


@pytest.mark.parametrize("q_len", [1, 40])
def test_graph_replays_match_eager(attn, q_len):
    c = make(15, "bf16", "bf16", q_len=(q_len, q_len), kv_len=(3000, 41), heads=(8, 2))
    want = call(attn, c)
    k, v, table = c["k"].cuda(), c["v"].cuda(), c["table"].cuda()
    q, lens, cu = c["q"].cuda(), torch.tensor(c["kv_len"]).int().cuda(), R.offsets(c["q_len"]).cuda()
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.paged_attention(q, k, v, lens, table, cu_q=cu, max_q=q_len, max_kv=3000, out=out)
    for replay in range(3):
        out.fill_(float("nan"))
        call(attn, c)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), replay


def test_append_then_attend(attn):
    """A sequence taken in by chunks gives what it gives at once, and the new entries are read back."""
    gen = torch.Generator().manual_seed(16)
    n, hq, hkv, d = 75, 4, 2, 64
    qkv = torch.randn(n, hq + 2 * hkv, d, generator=gen).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    freqs = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).cuda()
    table = torch.randperm(5, generator=gen).int().reshape(1, 5).cuda()

    def chunks(sizes):
        kc = torch.full((5, hkv, 16, d), float("nan"), device="cuda", dtype=torch.float16)
        vc = kc.clone()
        done, outs = 0, []
        for m in sizes:
            part = slice(done, done + m)
            done += m
            lens, cu = torch.tensor([done]).int().cuda(), torch.tensor([0, m]).int().cuda()
            turned = attn.kv_append(k[part], v[part], kc, vc, lens, table, q=q[part], cu_q=cu, freqs=freqs)
            outs.append(attn.paged_attention(turned, kc, vc, lens, table, cu_q=cu))
        return torch.cat(outs)

    whole = chunks([n])
    for sizes in ([1] * n, [30, 1, 44], [74, 1]):
        assert float((chunks(sizes) - whole).abs().max()) < 2e-5, sizes


def test_pages_far_apart(attn):
    """Pages beyond 2^32 elements: append and both forms of attention address them in 64 bits."""
    d, far = 64, (1 << 32) + 4096
    held = [torch.empty(far + 2048, dtype=torch.float16, device="cuda") for _ in range(2)]
    kc, vc = (t.as_strided((2, 1, 16, d), (far, 1024, 64, 1)) for t in held)
    near = [torch.empty(2, 1, 16, d, dtype=torch.float16, device="cuda") for _ in range(2)]
    gen = torch.Generator().manual_seed(17)
    n = 30
    q, k, v = (torch.randn(n, h, d, generator=gen).half().cuda() for h in (2, 1, 1))
    lens, cu = torch.tensor([n]).int().cuda(), torch.tensor([0, n]).int().cuda()
    table = torch.tensor([[1, 0]]).int().cuda()
    outs = []
    for a, b in ((kc, vc), near):
        attn.kv_append(k, v, a, b, lens, table, cu_q=cu)
        outs.append([attn.paged_attention(q, a, b, lens, table, cu_q=cu),
                     attn.paged_attention(q[-1:], a, b, lens, table)])
    assert torch.equal(kc[1, 0, 3], near[0][1, 0, 3]) and torch.equal(vc[0, 0, 13], near[1][0, 0, 13])
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_refusals_name_the_argument(attn):
    c = make(18, "f16", "f16")
    base = dict(q=c["q"].cuda(), k_cache=c["k"].cuda(), v_cache=c["v"].cuda(), kv_len=torch.tensor(c["kv_len"]).int().cuda(),
                table=c["table"].cuda())
    for over, match in ((dict(kv_len=base["kv_len"].long()), "kv_len must have dtype"),
                        (dict(table=base["table"].long()), "table must be an int32 matrix"),
                        (dict(table=base["table"].cpu()), "table must be a device tensor"),
                        (dict(kv_len=base["kv_len"][:2]), "kv_len must be contiguous with 3"),
                        (dict(cu_q=base["kv_len"]), "cu_q must be contiguous with 4"),
                        (dict(v_cache=base["v_cache"].bfloat16()), "must have one dtype"),
                        (dict(v_cache=base["v_cache"][:, :1]), "k_cache and v_cache must be"),
                        (dict(k_cache=base["k_cache"].transpose(2, 3), v_cache=base["v_cache"].transpose(2, 3)), "head_dim"),
                        (dict(out=base["q"].float()), "out must have dtype"),
                        (dict(out=base["q"][:2]), "out must be"),
                        (dict(k_scale=torch.ones(3, device="cuda")), "k_scale must be contiguous with 2")):
        with pytest.raises(ValueError, match=match):
            attn.paged_attention(**{**base, **over})
    with pytest.raises(TypeError, match="window must be an integer"):
        attn.paged_attention(**base, window="3")
    for over in (dict(window=-1), dict(scale=0.0), dict(k_scale=torch.ones(2, device="cuda")),
                 dict(q=base["q"].bfloat16())):
        with pytest.raises(RuntimeError, match="paged_attention"):
            attn.paged_attention(**{**base, **over})
    k = base["q"][:, :2]
    rest = (base["k_cache"], base["v_cache"], base["kv_len"], base["table"])
    for over, match in ((dict(q_out=base["q"]), "q_out without q"), (dict(freqs=torch.ones(64, device="cuda")), "freqs must have dtype"),
                        (dict(positions=torch.zeros(2, 3, device="cuda").int()), "one section for each"),
                        (dict(q=base["q"][0]), "q must be"), (dict(q_norm=torch.ones(64, device="cuda")), "q_norm must be contiguous")):
        with pytest.raises(ValueError, match=match):
            attn.kv_append(k, k, *rest, **over)
    with pytest.raises(ValueError, match="heads for this cache"):
        attn.kv_append(base["q"], base["q"], *rest)
    with pytest.raises(TypeError, match="sections must be"):
        attn.kv_append(k, k, *rest, positions=torch.zeros(3, device="cuda").int(), sections=7)
