"""kv_append with q turned in place: k and v may be other columns of q's array, but not q's own elements, which some
blocks would read turned and others not."""

import random

import pytest

torch = pytest.importorskip("torch")
from gemv_tq2_g128_amd import tq2  # noqa: E402
from tests.test_attn_cpu import A, F16, G, append  # noqa: E402

Q = A + 4 * G


def in_place(**over):
    return append(**{**dict(q=Q, q_out=Q, q_ts=1024, o_ts=1024, k_ts=1024, v_ts=1024, k_new=Q + 2048, v_new=Q + 2048 + 1024),
                     **over})


@pytest.mark.parametrize("over", [
    dict(k_new=Q), dict(v_new=Q), dict(k_new=Q + 512), dict(v_new=Q + 2032), dict(k_new=Q + 4096), dict(k_new=Q - 512),
    dict(k_new=Q + 1024, k_hs=512), dict(k_ts=512), dict(v_ts=2048), dict(q_hs=256, o_hs=256, k_new=Q + 512, k_hs=512),
    dict(tokens=1, batch=1, k_new=Q + 512), dict(tokens=1, batch=1, v_new=Q - 512)])
def test_refused(over):
    assert in_place(**over) == tq2.TQ2_ERR_ALIAS


def test_taken():
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible; this check is for GPU-less hosts")
    for over in (dict(), dict(k_new=A + 5 * G), dict(k_new=Q - 1024, v_new=Q - 2048),
                 # heads of q, k and v in turn: a row of q between rows of k
                 dict(q_heads=2, q_hs=384, o_hs=384, k_hs=384, v_hs=384, k_new=Q + 512, v_new=Q + 1024),
                 dict(tokens=1, batch=1, k_ts=256, v_ts=16), dict(q_out=A + 7 * G, k_new=Q, v_new=Q)):
        assert in_place(**over) == tq2.TQ2_ERR_DEVICE, over


def test_against_counting():
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible; this check is for GPU-less hosts")
    rng = random.Random(6)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        tokens, kv_heads, group = rng.randrange(1, 4), rng.randrange(1, 4), rng.randrange(1, 3)
        heads, ts = kv_heads * group, 64 * rng.randrange(6, 24)
        qhs, khs = 64 * rng.randrange(1, 4), 64 * rng.randrange(0, 4)
        at = 64 * rng.randrange(-24, 24)                           # elements of two bytes
        rows = {t * ts + h * qhs for t in range(tokens) for h in range(heads)}
        own = len(rows) < tokens * heads                           # q_out's own rows overlap
        # Every multiple of the token stride counts, as if the array went on.
        meet = any(t * ts + at + h * khs in rows for t in range(-8, 9) for h in range(kv_heads)) if tokens > 1 else \
            any(at + h * khs in rows for h in range(kv_heads))
        got = append(act_type=F16, head_dim=64, rot=64, s0=32, tokens=tokens, batch=tokens, kv_heads=kv_heads,
                     q_heads=heads, q=Q, q_out=Q, q_ts=ts, q_hs=qhs, o_ts=ts, o_hs=qhs, k_new=Q + 2 * at, k_ts=ts,
                     k_hs=khs, v_new=A + 6 * G, k_page_stride=8192, v_page_stride=8192)
        extents = at * 2 < 2 * ((tokens - 1) * ts + (heads - 1) * qhs + 64) and \
            -at * 2 < 2 * ((tokens - 1) * ts + (kv_heads - 1) * khs + 64)
        bad = own or (extents and meet)
        seen[bad] += 1
        assert got == (tq2.TQ2_ERR_ALIAS if bad else tq2.TQ2_ERR_DEVICE), (tokens, heads, kv_heads, ts, qhs, khs, at)
    assert min(seen.values()) > 500
