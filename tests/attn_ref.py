"""Paged-cache inputs and the operators' definitions in float64 on the CPU (test infrastructure)."""

import math

import torch

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
# Half a step of each type, relative, and half its smallest step.
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10}


def block_table(kv_len, page, gen, spare=0):
    """Shuffled page ids [batch, columns] and the number of pages."""
    cols = max(1, max((n + page - 1) // page for n in kv_len)) + spare
    pages = len(kv_len) * cols
    return torch.randperm(pages, generator=gen).to(torch.int32).reshape(len(kv_len), cols), pages


def offsets(q_len):
    cu = torch.zeros(len(q_len) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(q_len), 0)
    return cu


def places(q_len, kv_len):
    """(sequence, place) of each new token."""
    return [(b, kv_len[b] - q_len[b] + i) for b in range(len(q_len)) for i in range(q_len[b])]


def page_id(table, pages, page, b, n):
    """The page of place n, or None: outside the table, or no page of the cache."""
    if n < 0 or n // page >= table.shape[1]:
        return None
    p = int(table[b, n // page])
    return p if 0 <= p < pages else None


def rotate(x, angle, half, interleaved):
    """x f64 [tokens, heads, dim], angle f64 [tokens, half]; also the bound's |a| + |b| of each component."""
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    y, size = x.clone(), x.abs()
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    size[..., first] = size[..., second] = a.abs() + b.abs()
    return y, size


def normed(x, weight, eps):
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()


def attend(q, k_cache, v_cache, q_len, kv_len, table, window=0, scale=None, k_scale=None, v_scale=None):
    """Attention of the new tokens in float64, and sum_j p_j |v_j| of each output component."""
    tokens, hq, d = q.shape
    pages, hkv, page, _ = k_cache.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(tokens, hq, d, dtype=torch.float64)
    size = torch.zeros_like(out)
    row = 0
    for b in range(len(q_len)):
        keep = [(n, page_id(table, pages, page, b, n)) for n in range(kv_len[b])]
        keep = [(n, p) for n, p in keep if p is not None]
        here = torch.arange(row, row + q_len[b])
        row += q_len[b]
        if not keep or q_len[b] == 0:
            continue
        n = torch.tensor([a for a, _ in keep])
        p = torch.tensor([c for _, c in keep])
        k = k_cache[p, :, n % page].double()                     # [keys, hkv, d]
        v = v_cache[p, :, n % page].double()
        if k_scale is not None:
            k, v = k * k_scale.double()[None, :, None], v * v_scale.double()[None, :, None]
        k = k.repeat_interleave(hq // hkv, 1)
        v = v.repeat_interleave(hq // hkv, 1)
        place = kv_len[b] - q_len[b] + torch.arange(q_len[b])
        seen = n[None] <= place[:, None]
        if window:
            seen &= n[None] > place[:, None] - window
        s = torch.einsum("qhd,khd->hqk", q[here].double(), k) * scale
        s = s.masked_fill(~seen[None], -math.inf)
        w = torch.softmax(s, -1)
        w = torch.where(seen.any(-1)[None, :, None], w, torch.zeros_like(w))
        w = torch.where(seen[None], w, torch.zeros_like(w))
        # Places that are not seen take no part, whatever they hold.
        v0 = torch.where(seen.any(0)[:, None, None], v, torch.zeros_like(v))
        out[here] = torch.einsum("hqk,khd->qhd", w, v0)
        size[here] = torch.einsum("hqk,khd->qhd", w, v0.abs())
    return out, size
