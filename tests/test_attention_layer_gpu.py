"""The example layer (examples/attention_layer.py) against float64 on the CPU: prompts, then single tokens.

Tolerance.  The projection's 1e-5 of sum |x w|, binary16 keys and values (2^-11 each) and a binary16 o for more than 16
tokens (2^-11 of sum |o w|) reach the output through sums of random signs; 2e-3 of the attention part's largest value
bounds four such roundings with a factor of one for the softmax's own slope.
"""

import importlib.util
import os

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
from tests import attn_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", at)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Plain:
    """The layer in float64, one sequence at a time, with all keys and values kept."""

    def __init__(self, layer, raw):
        self.l = layer
        w = torch.stack((raw["codes"] & 15, raw["codes"] >> 4), -1).flatten(1).double() - 8
        self.qkv = w * raw["scales"].double().repeat_interleave(w.shape[1] // raw["scales"].shape[1], 1)
        self.norms = raw["q_norm"], raw["k_norm"]
        self.out = torch.from_numpy(oracle.dequantize(raw["out"].numpy(), layer.hidden, layer.q_heads * layer.head_dim))
        self.k, self.v = [], []

    def __call__(self, x):
        hq, hkv, d = self.l.q_heads, self.l.kv_heads, self.l.head_dim
        y = x.double() @ self.qkv.T
        q, k, v = (p.unflatten(1, (-1, d)) for p in y.split((hq * d, hkv * d, hkv * d), 1))
        place = torch.arange(len(self.k), len(self.k) + len(x), dtype=torch.float64)
        angle = place[:, None] * self.l.freqs.cpu()
        q, _ = R.rotate(R.normed(q, self.norms[0], 1e-6), angle, d // 2, False)
        k, _ = R.rotate(R.normed(k, self.norms[1], 1e-6), angle, d // 2, False)
        self.k += list(k)
        self.v += list(v)
        keys = torch.stack(self.k).repeat_interleave(hq // hkv, 1)
        values = torch.stack(self.v).repeat_interleave(hq // hkv, 1)
        s = torch.einsum("qhd,khd->hqk", q, keys) / d ** 0.5
        s = s.masked_fill(torch.arange(len(self.k))[None, None] > place[None, :, None], -float("inf"))
        o = torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), values)
        return o.flatten(1) @ self.out.T


def test_prompts_and_single_tokens(example):
    layer, raw = example.random_layer(3)
    prompts = (5, 40)
    cache = example.Cache(2, layer.kv_heads, layer.head_dim, 16, 50)
    plain = [Plain(layer, raw) for _ in prompts]
    gen = torch.Generator().manual_seed(4)
    for new in (prompts, (1, 1), (1, 1), (2, 3)):
        x = torch.randn(sum(new), layer.hidden, generator=gen)
        cache.kv_len += torch.tensor(new, dtype=torch.int32, device="cuda")
        cu = None if new == (1, 1) else R.offsets(list(new)).cuda()
        y = layer(x.cuda(), cache, cu, max(new)).double().cpu()
        want = torch.cat([p(part) for p, part in zip(plain, x.split(new))])
        err = float((y - x.double() - want).abs().max()) / float(want.abs().max())
        print(new, "worst error of the largest value %.2g" % err, flush=True)
        assert err <= 2e-3, new


def test_the_example_runs(example, capsys):
    example.main()
    assert "8 tokens decoded: lengths [45, 208]" in capsys.readouterr().out
