"""GPU tests of tq2_sample with four vectors a thread for 16-bit logits: chunks of 32,768 tokens, which rows of more than 16
chunks of half that, or more than 2,048 of those in all, are cut into.  Rules and tolerances of tests/test_sample_gpu.py."""

import pytest

torch = pytest.importorskip("torch")
from tests.test_sample_gpu import TYPES, check, logits_of, sampling  # noqa: E402, F401

pytestmark = pytest.mark.gpu
KINDS = ["f16", "bf16"]


def spread(logits, rows, offset, dtype):
    """Rows in turn of the few, at places from which vectors start differently."""
    few, vocab = logits.shape
    wide = torch.full((rows * (vocab + 3) + 8,), float("inf"), dtype=dtype, device="cuda")
    view = wide.as_strided((rows, vocab), (vocab + 3, 1), offset)
    view.copy_(logits.cuda()[torch.arange(rows, device="cuda") % few])
    return view


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vocab", [(1 << 20) - 5, 9 * 32768, 9 * 32768 + 3, 9 * 32768 + 9])
@pytest.mark.parametrize("offset", [0, 3, 7])
def test_long_rows(sampling, kind, vocab, offset):  # noqa: F811
    # Some rows are drawn among the last tokens, and some among the first.
    logits, u = logits_of(21, 3, vocab, kind, spread=1.0, sure=3.0)
    logits[1, -3:] = 9.0
    logits[2, :2] = 9.0
    view = spread(logits, 3, offset, TYPES[kind])
    for settings in (dict(), dict(top_k=50, top_p=0.9), dict(top_k=vocab // 2), dict(top_p=0.8), dict(min_p=0.05)):
        want = check(sampling, logits, u, **settings)
        assert torch.equal(sampling.sample(view, u.cuda(), **settings), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,vocab", [(256, 151936), (300, 131072 + 5), (1100, 32768 + 5)])
@pytest.mark.parametrize("offset", [0, 5])
def test_many_rows(sampling, kind, rows, vocab, offset):  # noqa: F811
    few = 3
    logits, u = logits_of(22, few, vocab, kind, spread=1.0, sure=3.0)
    logits[1, -3:] = 7.0
    view, us = spread(logits, rows, offset, TYPES[kind]), u.repeat(rows // few + 1)[:rows].cuda()
    for settings in (dict(), dict(top_k=300), dict(top_p=0.8, top_k=vocab // 2), dict(min_p=0.02)):
        want = check(sampling, logits, u, **settings)
        got = sampling.sample(view, us, **settings)
        assert torch.equal(got, want.repeat(rows // few + 1)[:rows])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vocab", [1 << 20, 9 * 32768 + 9])
@pytest.mark.parametrize("offset", [0, 1])
def test_a_bin_that_holds_a_whole_chunk(sampling, kind, vocab, offset):  # noqa: F811
    # All logits equal, and two values in turn: 32,768 and more tokens of a chunk in one bin.
    u = torch.tensor([0.03, 0.52, 0.97])
    logits = torch.full((3, vocab), 1.5).to(TYPES[kind])
    two = logits.clone()
    two[:, 1::2] = 0.5
    two[:, vocab // 3] = -float("inf")
    for rows in (logits, two):
        view = spread(rows, 3, offset, TYPES[kind])
        for settings in (dict(), dict(top_k=vocab // 3), dict(top_p=0.51), dict(top_k=7)):
            want = check(sampling, rows, u, **settings)
            assert torch.equal(sampling.sample(view, u.cuda(), **settings), want)
