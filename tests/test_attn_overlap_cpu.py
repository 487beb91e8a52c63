"""Outputs whose own elements overlap (an expanded tensor, windows over one) are refused: blocks would race on them."""

import itertools
import random

import pytest

torch = pytest.importorskip("torch")
from gemv_tq2_g128_amd import tq2  # noqa: E402
from tests.test_attn_cpu import A, G, append, attention  # noqa: E402


@pytest.mark.parametrize("over", [
    dict(o_ts=0), dict(o_hs=0), dict(o_ts=0, o_hs=0), dict(o_ts=64), dict(o_ts=128), dict(o_ts=384), dict(o_hs=64),
    dict(o_ts=128, o_hs=192), dict(q=A + 4 * G, q_out=A + 4 * G, q_ts=0, o_ts=0),
    dict(k_page_stride=0), dict(v_page_stride=64), dict(k_head_stride=0), dict(v_head_stride=64),
    dict(k_token_stride=0), dict(v_token_stride=64)])
def test_append_refuses(over):
    assert append(**over) == tq2.TQ2_ERR_ALIAS


@pytest.mark.parametrize("over", [dict(o_ts=0), dict(o_hs=0), dict(o_ts=128), dict(o_ts=384), dict(o_hs=64),
                                  dict(q=A + 7 * G, q_ts=0, o_ts=0)])
def test_attention_refuses(over):
    assert attention(**over) == tq2.TQ2_ERR_ALIAS


def test_what_is_still_taken():
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible; this check is for GPU-less hosts")
    for over in (dict(o_ts=128, o_hs=384), dict(o_ts=1024, o_hs=256), dict(o_ts=0, tokens=1, batch=1),
                 dict(o_hs=0, q_heads=1, kv_heads=1), dict(o_ts=256, o_hs=768, q_heads=2), dict(q_ts=0), dict(q_hs=0)):
        assert attention(**over) == tq2.TQ2_ERR_DEVICE, over
        assert append(**over) == tq2.TQ2_ERR_DEVICE, over
    for over in (dict(k_page_stride=0, pages=1), dict(k_ts=0, v_hs=0), dict(k_head_stride=0, kv_heads=1)):
        assert append(**over) == tq2.TQ2_ERR_DEVICE, over
    # Attention only reads the cache.
    assert attention(k_page_stride=0, v_head_stride=0, k_token_stride=0) == tq2.TQ2_ERR_DEVICE


def test_against_counting():
    """Every layout of a few rows and heads is refused exactly if two elements share a place."""
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible; this check is for GPU-less hosts")
    rng = random.Random(4)
    for _ in range(3000):
        tokens, heads = rng.randrange(1, 8), rng.randrange(1, 8)
        ts, hs = 16 * rng.randrange(0, 40), 16 * rng.randrange(0, 40)
        starts = sorted(t * ts + h * hs for t, h in itertools.product(range(tokens), range(heads)))
        meet = any(b - a < 64 for a, b in zip(starts, starts[1:]))
        got = attention(tokens=tokens, batch=tokens, kv_heads=1, q_heads=heads, head_dim=64, o_ts=ts, o_hs=hs, q_ts=1024,
                        q_hs=64)
        assert got == (tq2.TQ2_ERR_ALIAS if meet else tq2.TQ2_ERR_DEVICE), (tokens, heads, ts, hs)
