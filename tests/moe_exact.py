"""Experts whose outputs are f32 numbers without any rounding, for as long as every bit of x and of the rows between the
projections counts.

A row of gate or up has two weights, +m and -m, on columns whose x are large and nearly equal whole numbers, so that the
product is a small one; a third column, 2^23, has no weight and sets the power of two of its 128 columns.  silu is its
argument from 20 on, and half of it near zero.  A row of down has four weights on numbers below 2^19 and none on one of
24 bits in each 128 columns.  All sums have at most 24 bits in any order.  scale: of x's two blocks of 128 columns, for
gate and for up."""

import numpy as np


class Exact:
    def __init__(self, seed, tokens, top_k, experts, inter, fmt, group, scale=(1.0, 1.0)):
        rng = np.random.default_rng(seed)
        hidden, m = 256, 7 if fmt == "q4" else 1
        self.fmt, self.group, self.experts, self.hidden, self.inter = fmt, group, experts, hidden, inter
        # Columns 128 b + 2 i and the next: v and v - d.  Products are m d: 20 to 700, and 4095 for pair 62.
        x = np.zeros((tokens, hidden), dtype=np.float64)
        for b in (0, 1):
            v = rng.integers(2 ** 19, 2 ** 21, (tokens, 64)) | 1
            d = rng.integers(20, 700 // m, (tokens, 64))
            d[:, 62] = 4095 // m
            x[:, 128 * b:128 * b + 128:2] = v
            x[:, 128 * b + 1:128 * b + 128:2] = v - d
            x[:, 128 * b + 126] = 2.0 ** 23
            x[:, 128 * b + 127] = 0
            x[:, 128 * b:128 * b + 128] *= scale[b]
        self.x = x
        up = np.zeros((experts, 2 * inter, hidden), dtype=np.int64)
        for e in range(experts):
            for n in range(inter):
                i, j, s = rng.integers(0, 62), rng.integers(0, 62), rng.choice([-1, 1])
                if n % 128 == 5:
                    i, j = 62, 62
                up[e, n, 2 * i], up[e, n, 2 * i + 1] = m, -m
                up[e, inter + n, 128 + 2 * j], up[e, inter + n, 129 + 2 * j] = s * m, -s * m
        down = np.zeros((experts, hidden, inter), dtype=np.int64)
        for e in range(experts):
            for n in range(hidden):
                at = [a for a in rng.permutation(inter)[:8] if a % 128 != 5][:4]
                down[e, n, at] = rng.choice([-1, 1], 4)
        self.up, self.down = up, down
        self.ids = np.stack([rng.permutation(experts)[:top_k] for _ in range(tokens)]).astype(np.int32)
        self.share = rng.choice([0.5, 1.0], (tokens, top_k)).astype(np.float32)

    def packed(self, w, unit=1.0):
        """The framework's codes and scales, all of them `unit`: (codes, scales), or 34-byte blocks."""
        if self.fmt == "q4":
            c = (w + 8).astype(np.uint8)
            return c[..., 0::2] | c[..., 1::2] << 4, np.full(w.shape[:2] + (w.shape[2] // self.group,), unit, dtype=np.float16)
        f = (w + 1).astype(np.uint8).reshape(-1, 32, 4)
        blocks = np.empty((len(f), 34), dtype=np.uint8)
        blocks[:, :32] = f[..., 0] | f[..., 1] << 2 | f[..., 2] << 4 | f[..., 3] << 6
        blocks[:, 32:] = np.full((len(f), 1), unit, dtype=np.float16).view(np.uint8)
        return blocks.reshape(-1)

    def out(self, keep=lambda row: row):
        """The definition in f64; keep: what becomes of a row before each projection."""
        out = np.zeros((len(self.x), self.hidden))
        for t, row in enumerate(self.x):
            for j, e in enumerate(self.ids[t]):
                both = self.up[e] @ keep(row)
                a, b = both[:self.inter], both[self.inter:]
                h = np.where(a >= 20, a, a / 2) * b
                assert np.array_equal(h, h.astype(np.float32)) or keep(row) is not row
                out[t] += self.share[t, j] * (self.down[e] @ keep(h))
        return out


def bits(n):
    """A row in whole numbers of n bits under a power of two for each 128 columns, as the kernels hold it in 30."""
    def keep(row):
        top = np.abs(row).reshape(-1, 128).max(1)
        unit = np.repeat(2.0 ** (np.floor(np.log2(np.where(top > 0, top, 1.0))) + 1 - n), 128)
        return np.rint(row / unit) * unit
    return keep
