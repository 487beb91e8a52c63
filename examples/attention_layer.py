"""The attention half of a decoder layer on the library's operators, over a paged cache.

    x -> q, k, v      4-bit projections               q4.gemv (16 tokens a call)
    q, k, v -> cache  norms, rotation, storing        attn.kv_append
    q -> o            attention over the cache        attn.paged_attention
    x + W_o o         ternary projection, residual    tq2.gemm

``python examples/attention_layer.py`` takes in two prompts of random activations and decodes a few steps, the decode
step captured in a graph: lengths and block table live on the device, so a replay serves every step.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gemv_tq2_g128_amd import attn, q4, tq2  # noqa: E402


class AttentionLayer:
    """Weights as a checkpoint holds them: ``qkv`` a pair (codes, scales) of 4-bit rows for q, k and v, ``out`` the
    ternary blocks of W_o [hidden, q_heads * head_dim], both on the device."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, qkv, out, q_norm, k_norm, base=10000.0):
        self.hidden, self.q_heads, self.kv_heads, self.head_dim = hidden, q_heads, kv_heads, head_dim
        self.codes, self.scales = qkv
        self.out = tq2.reformat_aos_to_soa(out, hidden, q_heads * head_dim)
        self.q_norm, self.k_norm = q_norm, k_norm
        half = head_dim // 2
        self.freqs = base ** (-torch.arange(half, dtype=torch.float64, device=self.codes.device) / half)

    def __call__(self, x, cache, cu_q=None, max_q=1):
        """x f32 [tokens, hidden], the new tokens of all sequences; cache.kv_len counts them already."""
        hq, hkv, d = self.q_heads, self.kv_heads, self.head_dim
        qkv = torch.empty(x.shape[0], (hq + 2 * hkv) * d, device=x.device)
        for lo in range(0, x.shape[0], q4.MAX_M):
            q4.gemv(self.codes, self.scales, x[lo:lo + q4.MAX_M], out=qkv[lo:lo + q4.MAX_M])
        q, k, v = (part.unflatten(1, (-1, d)) for part in qkv.split((hq * d, hkv * d, hkv * d), 1))
        q = attn.kv_append(k, v, cache.k, cache.v, cache.kv_len, cache.table, q=q, cu_q=cu_q, freqs=self.freqs,
                           q_norm=self.q_norm, k_norm=self.k_norm)
        o = attn.paged_attention(q, cache.k, cache.v, cache.kv_len, cache.table, cu_q=cu_q, max_q=max_q,
                                 max_kv=cache.most)
        return tq2.gemm(self.out, o.flatten(1), self.hidden, hq * d, residual=x)


class Cache:
    """A paged binary16 cache whose pages are handed out in the order they are asked for."""

    def __init__(self, batch, kv_heads, head_dim, page, most, device="cuda"):
        columns = (most + page - 1) // page
        shape = (batch * columns, kv_heads, page, head_dim)
        self.k = torch.empty(shape, dtype=torch.float16, device=device)
        self.v = torch.empty_like(self.k)
        self.table = torch.arange(batch * columns, dtype=torch.int32, device=device).reshape(columns, batch).t().contiguous()
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device=device)
        self.most = most


def random_layer(seed, hidden=1024, q_heads=8, kv_heads=2, head_dim=128, group=64, device="cuda"):
    """A layer of random weights, and the raw tensors it was made from."""
    gen = torch.Generator().manual_seed(seed)
    rows, wide = (q_heads + 2 * kv_heads) * head_dim, q_heads * head_dim
    raw = {
        "codes": torch.randint(0, 256, (rows, hidden // 2), generator=gen, dtype=torch.uint8),
        "scales": ((torch.rand(rows, hidden // group, generator=gen) + 0.5) * 0.008).half(),
        "q_norm": torch.rand(head_dim, generator=gen) + 0.5, "k_norm": torch.rand(head_dim, generator=gen) + 0.5}
    # Blocks of 32 bytes of codes 0, 1, 2 (four to a byte) and a binary16 scale.
    fields = torch.randint(0, 3, (hidden * wide // 128, 32, 4), generator=gen, dtype=torch.uint8)
    codes = fields[..., 0] | fields[..., 1] << 2 | fields[..., 2] << 4 | fields[..., 3] << 6
    scale = ((torch.rand(hidden * wide // 128, 1, generator=gen) + 0.5) * 0.02).half()
    raw["out"] = torch.cat((codes, scale.view(torch.uint8)), 1).flatten()
    dev = {n: t.to(device) for n, t in raw.items()}
    layer = AttentionLayer(hidden, q_heads, kv_heads, head_dim, (dev["codes"], dev["scales"]), dev["out"],
                           dev["q_norm"], dev["k_norm"])
    return layer, raw


def main():
    layer, _ = random_layer(1)
    prompts, steps = (37, 200), 8
    cache = Cache(len(prompts), layer.kv_heads, layer.head_dim, 16, max(prompts) + steps)
    x = torch.randn(sum(prompts), layer.hidden, device="cuda")
    cache.kv_len += torch.tensor(prompts, dtype=torch.int32, device="cuda")
    cu_q = torch.tensor((0, prompts[0], sum(prompts)), dtype=torch.int32, device="cuda")
    y = layer(x, cache, cu_q, max(prompts))
    print("prompts of %s tokens: output norm %.3f" % (prompts, float(y.norm())))

    token = y[cu_q[1:].long() - 1].contiguous()
    cache.kv_len += 1
    layer(token, cache)                          # outside the graph once: kernels load on their first call
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(token, cache)
    for step in range(steps):
        graph.replay()
        token.copy_(y / y.norm(dim=1, keepdim=True) * layer.hidden ** 0.5)
        cache.kv_len += 1
    print("%d tokens decoded: lengths %s, output norm %.3f" % (steps, (cache.kv_len - 1).tolist(), float(y.norm())))


if __name__ == "__main__":
    main()
