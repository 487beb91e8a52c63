"""GPU tests of tq2_sample where one bin holds many tokens: draws and truncations at every place of the order.

At an infinite temperature e is 1 for every finite logit, so that the draw by u is the token of rank floor(u n), exactly for
u of 13 bits and n of 17, and a draw by u = 1 the last one that top_k keeps."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests.test_sample_gpu import TYPES, check, sampling  # noqa: E402, F401

pytestmark = pytest.mark.gpu
INF = float("inf")


def crowd(seed, vocab, kind, spread=25.0):
    return (torch.randn(vocab, generator=torch.Generator().manual_seed(seed)) * spread).to(TYPES[kind])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("vocab", [129, 700, 4099, 32434, 100003])
@pytest.mark.parametrize("top_k", [0, 0.65])
def test_a_draw_at_every_place(sampling, kind, vocab, top_k):  # noqa: F811
    logits = crowd(31, vocab, kind)
    order = torch.sort(logits.double(), descending=True, stable=True).indices
    u = (torch.arange(4096) + 0.5) / 4096
    k = int(top_k * vocab) if top_k else 0
    got = sampling.sample(logits.cuda().expand(4096, vocab), u.cuda(), temperature=INF, top_k=k).cpu()
    rank = (u.double() * (k or vocab)).long()
    assert torch.equal(got.long(), order[rank])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("vocab", [129, 700, 4099, 32434])
def test_every_top_k(sampling, kind, vocab):  # noqa: F811
    logits = crowd(32, vocab, kind)
    order = torch.sort(logits.double(), descending=True, stable=True).indices
    k = (torch.arange(4096) * (vocab - 1) // 4095 + 1).to(torch.int32)
    got = sampling.sample(logits.cuda().expand(4096, vocab), torch.ones(4096, device="cuda"), temperature=INF,
                          top_k=k.cuda()).cpu()
    assert torch.equal(got.long(), order[k.long() - 1])


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("vocab", [700, 5003, 40009])
def test_draws_from_a_crowd_of_unequal_tokens(sampling, kind, vocab):  # noqa: F811
    # A bin is a factor of 1.065 in e: the crowd shares one, and its tokens weigh differently.
    logits = crowd(33, vocab, kind, 0.004)
    e = np.exp(np.sort(logits.double().numpy())[::-1] - float(logits.double().max()))
    upto = np.cumsum(e)
    order = np.argsort(-logits.double().numpy(), kind="stable")
    u = (torch.arange(4096) + 0.5) / 4096
    for top_k in (0, vocab // 3):
        n = top_k or vocab
        want = u.double().numpy() * upto[n - 1]
        at = np.searchsorted(upto[:n], want, side="right")
        near = np.abs(upto[np.stack([np.maximum(at - 1, 0), at])] - want).min(0) > 1.5 * vocab * 2.0 ** -43
        got = sampling.sample(logits.cuda().expand(4096, vocab), u.cuda(), top_k=top_k).cpu().numpy()
        assert near.mean() > 0.99 and np.array_equal(got[near], order[at[near]])
    check(sampling, logits.expand(3, vocab).contiguous(), torch.tensor([0.2, 0.5, 0.8]), top_p=0.6)
