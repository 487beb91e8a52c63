"""The mixture-of-experts operators in float64, from their definitions, and inputs for their tests."""

import numpy as np

import oracle

torch = __import__("torch")


def q4_weight(rng, experts, n, k, group, spread=0.02):
    return (rng.integers(0, 256, (experts, n, k // 2), dtype=np.uint8),
            rng.uniform(-spread, spread, (experts, n, k // group)).astype(np.float16))


def q4_values(weight):
    codes, scales = weight
    w = np.empty(codes.shape[:2] + (2 * codes.shape[2],))
    w[..., 0::2] = (codes & 15).astype(np.float64) - 8
    w[..., 1::2] = (codes >> 4).astype(np.float64) - 8
    return w * np.repeat(scales.astype(np.float64), w.shape[2] // scales.shape[2], axis=2)


def ternary_weight(rng, experts, n, k, spread=0.05):
    """Blocks of 34 bytes, [experts * n * k / 128, 34] flat."""
    count = experts * n * k // 128
    blocks = np.empty((count, 34), dtype=np.uint8)
    fields = rng.integers(0, 3, (count, 32, 4), dtype=np.uint8)
    blocks[:, :32] = fields[..., 0] | fields[..., 1] << 2 | fields[..., 2] << 4 | fields[..., 3] << 6
    blocks[:, 32:] = rng.uniform(-spread, spread, (count, 1)).astype(np.float16).view(np.uint8)
    return blocks.reshape(-1)


def ternary_values(blocks, experts, n, k):
    return oracle.dequantize(blocks, experts * n, k).astype(np.float64).reshape(experts, n, k)


def units(row):
    """2^-30 of the largest of each 128 columns, for each column."""
    return np.repeat(np.abs(row).reshape(-1, 128).max(1), 128) * 2.0 ** -30


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1 + np.exp(-v))


def experts(x, gate_up, down, ids, weights, residual, tol):
    """out, and how far a kernel may be from it whose projections keep tol * sum |x w|.

    gate_up f64 [experts, 2 inter, hidden], down f64 [experts, hidden, inter].  A projection keeps tol * sum |x w| and half
    a unit of its 31-bit integers, 2^-30 of the largest of the row's 128 columns.  silu's slope is below 1.1; its f32
    exponential, quotient and product add 4 roundings, the weighted sum one for each place and two more."""
    x = x.astype(np.float64)
    out = np.zeros(x.shape) if residual is None else residual.astype(np.float64).copy()
    bound, size = np.zeros(x.shape), np.abs(out)
    inter, step = down.shape[2], 2.0 ** -24
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < gate_up.shape[0]:
                continue
            both, s = gate_up[e] @ x[t], np.abs(gate_up[e]) @ (np.abs(x[t]) + units(x[t]) / tol)
            g, u, dg, du = both[:inter], both[inter:], tol * s[:inter], tol * s[inter:]
            h = silu(g) * u
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + 4 * step * np.abs(h)
            w = float(weights[t, j])
            out[t] += w * (down[e] @ h)
            reach = abs(w) * (np.abs(down[e]) @ np.abs(h))
            bound[t] += abs(w) * (np.abs(down[e]) @ (dh + units(h))) * (1 + tol) + tol * reach
            size[t] += reach
    return out, bound + (len(ids[0]) + 2) * step * size if len(ids) else bound


def route(x, weight, top_k, bias, scoring, renormalize, scale):
    """(weights, ids) by the definition; x and weight are float arrays that f64 holds exactly."""
    s = x.astype(np.float64) @ weight.astype(np.float64).T
    if scoring == "softmax":
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    else:
        p = 1 / (1 + np.exp(-s))
    by = s if bias is None else p + bias.astype(np.float64)
    ids = np.argsort(-by, axis=1, kind="stable")[:, :top_k]
    w = np.take_along_axis(p, ids, 1)
    if renormalize:
        w = w / w.sum(1, keepdims=True)
    return w * scale, ids
