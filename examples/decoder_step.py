"""A decode step on the library's operators: attention, a mixture of experts, the vocabulary and the next token.

    x -> x + attention(x)            examples/attention_layer.py
    x -> experts and their weights   moe.route
    x + sum of the experts           moe.experts, 4-bit or ternary
    x -> logits                      q4.gemv, 4-bit vocabulary
    logits -> tokens                 sampling.sample, by random numbers drawn outside

``python examples/decoder_step.py`` decodes a few tokens for a few sequences from an embedding of random weights, the
whole step captured in a graph: tokens, lengths and random numbers live on the device, so a replay serves every step.
"""

import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
for at in (HERE, os.path.dirname(HERE)):
    if at not in sys.path:
        sys.path.insert(0, at)
import attention_layer as A  # noqa: E402
from gemv_tq2_g128_amd import moe, q4, sampling, tq2  # noqa: E402


class Experts:
    """``router`` [experts, hidden]; ``gate_up`` and ``down`` as moe.experts takes them."""

    def __init__(self, router, gate_up, down, top_k):
        self.router, self.gate_up, self.down, self.top_k = router, gate_up, down, top_k

    def __call__(self, x):
        """x + the experts' sum, for at most moe.MAX_TOKENS rows at a time."""
        out = torch.empty_like(x)
        weights, ids = moe.route(x, self.router, self.top_k)
        for lo in range(0, x.shape[0], moe.MAX_TOKENS):
            part = slice(lo, lo + moe.MAX_TOKENS)
            moe.experts(x[part], self.gate_up, self.down, ids[part], weights[part], experts=self.router.shape[0],
                        residual=x[part], out=out[part])
        return out


class Decoder:
    """One layer, an embedding [vocab, hidden] and a 4-bit vocabulary projection (codes, scales)."""

    def __init__(self, attention, experts, embedding, vocabulary):
        self.attention, self.experts = attention, experts
        self.embedding, self.vocabulary = embedding, vocabulary

    def logits(self, tokens, cache):
        x = self.attention(self.embedding[tokens.long()], cache)
        x = self.experts(x)
        return torch.cat([q4.gemv(*self.vocabulary, x[lo:lo + q4.MAX_M]) for lo in range(0, x.shape[0], q4.MAX_M)])

    def __call__(self, tokens, cache, u, **settings):
        """The token after ``tokens`` of each sequence; cache.kv_len counts these already."""
        return sampling.sample(self.logits(tokens, cache), u, **settings)


def random_decoder(seed, hidden=512, experts=16, inter=256, top_k=4, vocab=4000, ternary=True, group=64, device="cuda"):
    """A decoder of random weights, and the raw tensors it was made from."""
    attention, raw = A.random_layer(seed, hidden=hidden, q_heads=4, kv_heads=2, device=device)
    gen = torch.Generator().manual_seed(seed + 1)

    def four_bit(*shape):
        n, k = shape[-2:]
        return (torch.randint(0, 256, (*shape[:-1], k // 2), generator=gen, dtype=torch.uint8),
                ((torch.rand(*shape[:-1], k // group, generator=gen) + 0.5) * (0.2 / k ** 0.5)).half())

    def blocks(*shape):
        count = shape[0] * shape[1] * shape[2] // 128
        fields = torch.randint(0, 3, (count, 32, 4), generator=gen, dtype=torch.uint8)
        codes = fields[..., 0] | fields[..., 1] << 2 | fields[..., 2] << 4 | fields[..., 3] << 6
        scale = ((torch.rand(count, 1, generator=gen) + 0.5) * (1.2 / shape[2] ** 0.5)).half()
        return torch.cat((codes, scale.view(torch.uint8)), 1).flatten()

    shapes = (experts, 2 * inter, hidden), (experts, hidden, inter)
    raw["gate_up"], raw["down"] = (blocks(*s) if ternary else four_bit(*s) for s in shapes)
    raw["router"] = torch.randn(experts, hidden, generator=gen) / hidden ** 0.5
    raw["embedding"] = torch.randn(vocab, hidden, generator=gen)
    raw["vocabulary"] = four_bit(vocab, hidden)

    def on(w):
        return tuple(t.to(device) for t in w) if isinstance(w, tuple) else w.to(device)

    gate_up, down = (tq2.reformat_aos_to_soa(on(raw[n]), s[0] * s[1], s[2]) if ternary else on(raw[n])
                     for n, s in zip(("gate_up", "down"), shapes))
    layer = Experts(on(raw["router"]), gate_up, down, top_k)
    return Decoder(attention, layer, on(raw["embedding"]), on(raw["vocabulary"])), raw


def main():
    decoder, _ = random_decoder(1)
    batch, steps = 3, 6
    cache = A.Cache(batch, decoder.attention.kv_heads, decoder.attention.head_dim, 16, steps + 2)
    tokens = torch.tensor([5, 17, 230], dtype=torch.int32, device="cuda")
    u = torch.rand(batch, device="cuda")
    settings = dict(temperature=0.8, top_k=50, top_p=0.95)
    cache.kv_len += 1
    decoder(tokens, cache, u, **settings)        # outside the graph once: kernels load on their first call
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens.copy_(decoder(tokens, cache, u, **settings))
    text = []
    for _ in range(steps):
        u.uniform_()
        graph.replay()
        text.append(tokens.tolist())
        cache.kv_len += 1
    print("%d steps of %d sequences: %s" % (steps, batch, list(map(list, zip(*text)))))


if __name__ == "__main__":
    main()
