"""GPU parity of tq2_paged_attention over many short sequences, with max_q left to its default (all rows of q).

Tolerances are those of test_paged_attention_gpu.py.
"""

import pytest

torch = pytest.importorskip("torch")
from tests.test_paged_attention_gpu import attn, check, make  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def test_many_short_prompts(attn):  # noqa: F811
    """1,024 prompts of 32 tokens: by the longest that max_q allows, 2^24 blocks."""
    c = make(41, "f16", "f16", q_len=[32] * 1024, kv_len=[32 + b % 9 for b in range(1024)], heads=(64, 8), dim=64)
    check(attn, c, "short prompts", max_q=None)


def test_one_long_prompt_among_single_tokens(attn):  # noqa: F811
    """Steps that the grid has no room for are walked over by its blocks."""
    q_len = [1] * 511 + [2000]
    c = make(42, "bf16", "bf16", q_len=q_len, kv_len=[n + 3 for n in q_len], heads=(64, 16), dim=64)
    check(attn, c, "one long", max_q=None)


def test_decode_batch_with_offsets(attn):  # noqa: F811
    c = make(43, "f32", "e4m3", q_len=[1] * 300 + [0], kv_len=[1 + (b * 7) % 90 for b in range(301)], heads=(8, 2), dim=96)
    check(attn, c, "decode", max_q=None)


@pytest.mark.parametrize("tokens,dim,max_kv", [((1 << 18) + 5, 256, 700), ((1 << 16) + 5, 64, 100000)])
def test_parts_of_many_rows(attn, tokens, dim, max_kv):  # noqa: F811
    """More blocks of the join than one axis of its grid takes: a block for four rows (few parts), a block for each.
    The launch is shaped for single tokens, so that the one sequence's keys are cut into parts."""
    gen = torch.Generator(device="cuda").manual_seed(44)
    q = torch.randn(tokens, 16, dim, generator=gen, device="cuda", dtype=torch.float16)
    k, v = (torch.randn(10, 1, 64, dim, generator=gen, device="cuda", dtype=torch.float16) for _ in "kv")
    table = torch.arange(10, dtype=torch.int32, device="cuda").reshape(1, 10)       # 640 keys for all rows
    lens, cu = torch.tensor([tokens]).int().cuda(), torch.tensor([0, tokens]).int().cuda()
    want = attn.paged_attention(q, k, v, lens, table, cu_q=cu, max_kv=0)            # whole
    print("whole done", flush=True)
    got = attn.paged_attention(q, k, v, lens, table, cu_q=cu, max_q=1, max_kv=max_kv)
    err = float((got.float() - want.float()).abs().max())
    # Each side: half a step of f16 for the probabilities and for the result, f32 sums, all within |v|.
    tol = 2 * (2 * 2.0 ** -11 + 1e-5) * float(v.abs().max())
    print("parts of %d rows: worst err / tol %.3f" % (tokens * 16, err / tol), flush=True)
    assert err <= tol
