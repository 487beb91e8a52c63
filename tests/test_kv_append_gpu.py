"""GPU parity of tq2_kv_append against the definition in float64.

Tolerance.  In f32, at most 24 roundings reach a component before its last one
(8 of a lane's squares, 5 of the tree, 2 of the root, all halved by the root,
2 products of the norm, 1 of a sine, 2 of the turn): 24 * 2^-24 (|a| + |b|) for
the pair (a, b).  Then one rounding to the stored type, half a step; 8-bit
values are divided by their scale first, one rounding more, which 24 covers.
Values that are only copied (v without a scale) are equal.
"""

import pytest

torch = pytest.importorskip("torch")
from tests import attn_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    from gemv_tq2_g128_amd import attn as mod
    return mod


def make(seed, act="f32", cache="f16", q_len=(1, 1, 1), kv_len=(5, 16, 33), heads=(4, 2), dim=128, rot=None, page=16,
         axes=1, norm=True, interleaved=False, far=0, order="pages"):
    """A case on the CPU: activations are columns of one array, as a fused projection gives them."""
    gen = torch.Generator().manual_seed(seed)
    hq, hkv = heads
    tokens = sum(q_len)
    rot = dim if rot is None else rot
    half = rot // 2
    c = {"q_len": list(q_len), "kv_len": list(kv_len), "interleaved": interleaved, "act": act, "cache": cache}
    qkv = (torch.randn(tokens, (hq + 2 * hkv) * dim, generator=gen) * 2).to(R.DTYPES[act])
    c["qkv"], c["heads"], c["dim"], c["page"], c["half"], c["order"] = qkv, heads, dim, page, half, order
    c["table"], c["pages"] = R.block_table(c["kv_len"], page, gen)
    c["freqs"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1)) if half else None
    c["positions"] = c["sections"] = None
    if axes > 1 or far:
        c["positions"] = torch.randint(0, far or 4096, (axes, tokens), generator=gen, dtype=torch.int32)
        cut = [half // 4, half // 4] if axes == 3 else [half // 3] if axes == 2 else []
        c["sections"] = tuple([half - sum(cut)] + cut)
    c["q_norm"] = torch.rand(dim, generator=gen) + 0.5 if norm else None
    c["k_norm"] = torch.rand(dim, generator=gen) + 0.5 if norm else None
    c["k_scale"] = torch.rand(hkv, generator=gen) * 0.05 + 0.01 if cache == "e4m3" else None
    c["v_scale"] = torch.rand(hkv, generator=gen) * 0.05 + 0.01 if cache == "e4m3" else None
    return c


def split(c, qkv):
    (hq, hkv), d = c["heads"], c["dim"]
    return (qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
            qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)))


def cuda(t):
    return None if t is None else t.cuda()


def caches(c, device):
    hkv, d = c["heads"][1], c["dim"]
    shape = (c["pages"], hkv, c["page"], d) if c["order"] == "pages" else (c["pages"], c["page"], hkv, d)
    k = torch.full(shape, 3.0, device=device, dtype=torch.float16).to(R.DTYPES[c["cache"]])
    v = k.clone()
    return (k, v) if c["order"] == "pages" else (k.transpose(1, 2), v.transpose(1, 2))


def call(attn, c, q_out=None, with_q=True, kv=None, qkv=None):
    q, k, v = split(c, c["qkv"].cuda() if qkv is None else qkv)
    kc, vc = caches(c, "cuda") if kv is None else kv
    cu = None if all(n == 1 for n in c["q_len"]) else R.offsets(c["q_len"]).cuda()
    out = attn.kv_append(k, v, kc, vc, torch.tensor(c["kv_len"], dtype=torch.int32).cuda(), cuda(c["table"]),
                         q=q if with_q else None, q_out=q_out, cu_q=cu, freqs=cuda(c["freqs"]),
                         positions=cuda(c["positions"]), sections=c["sections"], interleaved=c["interleaved"],
                         q_norm=cuda(c["q_norm"]) if with_q else None, k_norm=cuda(c["k_norm"]), eps=1e-6,
                         k_scale=cuda(c["k_scale"]), v_scale=cuda(c["v_scale"]))
    return out, kc, vc


def expected(c):
    """(value, bound's size) of q_out, k and v of each new token, before rounding."""
    q, k, v = (x.double() for x in split(c, c["qkv"]))
    at = R.places(c["q_len"], c["kv_len"])
    place = torch.tensor([n for _, n in at], dtype=torch.float64)
    half = c["half"]
    angle = torch.zeros(len(at), half, dtype=torch.float64)
    lo = 0
    for axis, n in enumerate(c["sections"] or (half,)):
        pos = place if c["positions"] is None else c["positions"][axis].double()
        if n:
            angle[:, lo:lo + n] = pos[:, None] * c["freqs"][lo:lo + n]
        lo += n
    q, q_size = R.rotate(R.normed(q, c["q_norm"], 1e-6), angle, half, c["interleaved"])
    k, k_size = R.rotate(R.normed(k, c["k_norm"], 1e-6), angle, half, c["interleaved"])
    return (q, q_size), (k, k_size), (v, v.abs())


def near(got, want, size, kind, scale=None, label=""):
    want = want.clone()
    if scale is not None:
        want, size = want / scale.double()[:, None], size / scale.double()[:, None]
    if kind == "e4m3":
        want = want.clamp(-448.0, 448.0)
    e32 = 24 * 2.0 ** -24 * size
    tol = e32 + R.HALF[kind] * (want.abs() + e32) + R.TINY[kind]
    err = (got.double().cpu() - want).abs()
    worst = float((err / tol).max()) if err.numel() else 0.0
    print(label, "worst err / tol %.3f" % worst, flush=True)
    assert bool((err <= tol).all()), label


def check(attn, c, label):
    out, kc, vc = call(attn, c)
    torch.cuda.synchronize()
    (q, qs), (k, ks), (v, vs) = expected(c)
    near(out, q, qs, c["act"], label=label + " q")
    kc, vc = kc.float().cpu(), vc.float().cpu()
    seen = torch.zeros(kc.shape[0], kc.shape[2], dtype=torch.bool)
    for t, (b, n) in enumerate(R.places(c["q_len"], c["kv_len"])):
        p = R.page_id(c["table"], c["pages"], c["page"], b, n)
        if p is None:
            continue
        seen[p, n % c["page"]] = True
        near(kc[p, :, n % c["page"]], k[t], ks[t], c["cache"], c["k_scale"], label + " k%d" % t)
        if c["cache"] == c["act"]:
            assert torch.equal(vc[p, :, n % c["page"]].double(), v[t])
        near(vc[p, :, n % c["page"]], v[t], vs[t], c["cache"], c["v_scale"], label + " v%d" % t)
    assert bool((kc.transpose(1, 2)[~seen] == 3.0).all()) and bool((vc.transpose(1, 2)[~seen] == 3.0).all())


@pytest.mark.parametrize("act,cache", [("f32", "f16"), ("f32", "e4m3"), ("f16", "f16"), ("f16", "e4m3"),
                                       ("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("dim,rot", [(64, 64), (96, 96), (96, 48), (128, 128), (128, 64), (128, 8), (192, 128),
                                     (256, 256), (256, 0)])
def test_types_and_heads(attn, act, cache, dim, rot):
    check(attn, make(dim + rot, act, cache, dim=dim, rot=rot), "%s %s %d %d" % (act, cache, dim, rot))


@pytest.mark.parametrize("heads", [(1, 1), (14, 2), (24, 4), (16, 16), (64, 8), (5, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_counts(attn, heads, interleaved):
    check(attn, make(heads[0], "bf16", "bf16", heads=heads, interleaved=interleaved), "heads %s" % (heads,))


@pytest.mark.parametrize("page,order", [(16, "tokens"), (32, "pages"), (128, "tokens")])
@pytest.mark.parametrize("axes", [1, 2, 3])
def test_ragged_chunks(attn, page, order, axes):
    """Sequences without new tokens, with one, and with chunks that cross pages."""
    c = make(page + axes, "f16", "f16", q_len=(0, 1, 37, 0, 18), kv_len=(9, 1, 70, 0, 18), page=page, axes=axes,
             order=order, norm=axes == 2)
    check(attn, c, "page %d axes %d" % (page, axes))


@pytest.mark.parametrize("interleaved", [False, True])
def test_many_tokens(attn, interleaved):
    """More than one sequence per block of tokens, and batches past one wave's lanes."""
    q_len = [1 + i % 130 for i in range(140)]
    c = make(3, "f32", "f16", q_len=q_len, kv_len=[n + 3 for n in q_len], heads=(2, 1), dim=64,
                      interleaved=interleaved)
    assert sum(q_len) >= 4096
    out, kc, vc = call(attn, c)
    (q, qs), (k, ks), (v, vs) = expected(c)
    near(out, q, qs, "f32", label="q")
    at = R.places(q_len, c["kv_len"])
    p = torch.tensor([int(c["table"][b, n // 16]) for b, n in at])
    off = torch.tensor([n % 16 for _, n in at])
    near(kc.cpu()[p, :, off], k, ks, "f16", label="k")
    near(vc.cpu()[p, :, off], v, vs, "f16", label="v")


@pytest.mark.parametrize("axes", [1, 3])
def test_far_positions(attn, axes):
    """Angles of positions up to 2^30 keep their accuracy."""
    check(attn, make(9, q_len=(40,), kv_len=(40,), axes=axes, far=1 << 30), "far")


def test_negative_positions(attn):
    c = make(10, q_len=(33,), kv_len=(33,), far=64)
    c["positions"] = c["positions"] - 1000000
    check(attn, c, "negative")


def test_pages_that_are_not_in_the_cache(attn):
    """Bad table entries, lengths past the table and more new tokens than kv_len: those are not written."""
    c = make(11, "f16", "f16", q_len=(20, 20, 20), kv_len=(40, 20, 20), heads=(2, 2), dim=64)
    c["table"][0, 1] = -1
    c["table"][1, 0] = c["pages"]
    c["table"][1, 1] = 2 ** 31 - 1
    c["kv_len"][2] = 60                          # the table has 48 places
    check(attn, c, "bad pages")
    c["kv_len"] = [7, -3, 0]
    check(attn, c, "short")


def test_rows_without_a_sequence(attn):
    """Rows before cu_q[0] and past its end keep what q_out holds; offsets past the last row are cut."""
    c = make(12, "f32", "f16", q_len=(3, 4), kv_len=(10, 20), heads=(2, 1), dim=64, norm=False)
    q, k, v = split(c, c["qkv"].cuda())
    for cu, owned in (([2, 3, 5], range(2, 5)), ([0, 3, 90], range(0, 7)), ([-5, 3, 3], range(0, 3))):
        out = torch.full(q.shape, 7.0, device="cuda")
        kc, vc = caches(c, "cuda")
        attn.kv_append(k, v, kc, vc, torch.tensor(c["kv_len"], dtype=torch.int32).cuda(), c["table"].cuda(), q=q,
                       q_out=out, cu_q=torch.tensor(cu, dtype=torch.int32).cuda())
        for t in range(7):
            assert torch.equal(out[t], q[t] if t in owned else torch.full_like(q[t], 7.0)), (cu, t)


def test_in_place_and_without_q(attn):
    c = make(13, "bf16", "bf16", q_len=(5, 3), kv_len=(50, 3))
    whole, kc, vc = call(attn, c)
    qkv = c["qkv"].cuda()
    same, kc2, vc2 = call(attn, c, q_out=split(c, qkv)[0], qkv=qkv)
    none, kc3, vc3 = call(attn, c, with_q=False)
    assert none is None and torch.equal(same, whole)
    for a, b in ((kc, kc2), (vc, vc2), (kc, kc3), (vc, vc3)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.equal(split(c, qkv)[1], split(c, c["qkv"].cuda())[1])


def test_values_that_are_not_finite(attn):
    """They stay in their row and head; 8-bit values clamp at 448, NaN stays NaN."""
    c = make(14, "f32", "e4m3", q_len=(2,), kv_len=(2,), norm=False, rot=0)
    q, k, v = split(c, c["qkv"])
    v[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e30])
    k[1, 1, 0] = float("nan")
    out, kc, vc = call(attn, c)
    p = int(c["table"][0, 0])
    got = vc[p, 0, 0].float().cpu()
    assert got[0] == 448 and got[1] == -448 and got[2].isnan() and got[3] == 448 and got[4:].isfinite().all()
    kk = kc[p].float().cpu()
    assert kk[1, 1, 0].isnan() and kk[1, 1, 1:].isfinite().all() and kk[0].isfinite().all()
    assert torch.equal(out.cpu(), q)


def test_empty(attn):
    c = make(15, q_len=(0, 0), kv_len=(4, 0))
    out, kc, _ = call(attn, c)
    assert out.shape == (0, 4, 128) and bool((kc == 3.0).all())


def test_stream_and_graph(attn):
    c = make(16, "f16", "e4m3", q_len=(3, 30), kv_len=(70, 30))
    want, kc, vc = call(attn, c)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        other, kc2, vc2 = call(attn, c)
    stream.synchronize()
    assert torch.equal(other, want) and torch.equal(kc2.view(torch.uint8), kc.view(torch.uint8))
    q, k, v = split(c, c["qkv"].cuda())
    kc3, vc3 = caches(c, "cuda")
    blank = kc3.clone()
    out = torch.empty_like(want)
    fixed = dict(kv_len=torch.tensor(c["kv_len"], dtype=torch.int32).cuda(), table=c["table"].cuda(),
                 cu_q=R.offsets(c["q_len"]).cuda(), freqs=c["freqs"].cuda(), q_norm=c["q_norm"].cuda(),
                 k_norm=c["k_norm"].cuda(), k_scale=c["k_scale"].cuda(), v_scale=c["v_scale"].cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.kv_append(k, v, kc3, vc3, q=q, q_out=out, **fixed)
    for replay in range(3):
        kc3.view(torch.uint8).copy_(blank.view(torch.uint8))
        vc3.view(torch.uint8).copy_(blank.view(torch.uint8))
        out.fill_(float("nan"))
        call(attn, c)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), replay
        assert torch.equal(kc3.view(torch.uint8), kc.view(torch.uint8)), replay
        assert torch.equal(vc3.view(torch.uint8), vc.view(torch.uint8)), replay
