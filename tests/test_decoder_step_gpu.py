"""The example decode step (examples/decoder_step.py) against float64 on the CPU: attention, experts, vocabulary, token.

Tolerance of the logits.  Attention: 2e-3 of its largest value, as in test_attention_layer_gpu.  The layer behind it has
slopes of a few: random weights of unit gain in each of three products, so that 2e-3 of the stream's error reaches the
logits within a factor of 4 of the largest logit.
The sampled token: the definition on the kernel's own logits, which tests/sample_ref.py gives exactly.
"""

import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import moe_ref as M  # noqa: E402
from tests import sample_ref as S  # noqa: E402
from tests.test_attention_layer_gpu import Plain  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_step.py")
    spec = importlib.util.spec_from_file_location("decoder_step", at)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("ternary", [True, False])
def test_steps(example, ternary):
    decoder, raw = example.random_decoder(7, ternary=ternary)
    batch, hidden, experts, inter, top_k = 3, 512, 16, 256, 4
    cache = example.A.Cache(batch, decoder.attention.kv_heads, decoder.attention.head_dim, 16, 20)
    plain = [Plain(decoder.attention, raw) for _ in range(batch)]
    if ternary:
        up = M.ternary_values(raw["gate_up"].numpy(), experts, 2 * inter, hidden)
        down = M.ternary_values(raw["down"].numpy(), experts, hidden, inter)
    else:
        up, down = (M.q4_values(tuple(t.numpy() for t in raw[n])) for n in ("gate_up", "down"))
    vocabulary = M.q4_values(tuple(t.numpy()[None] for t in raw["vocabulary"]))[0]
    tokens = torch.tensor([3, 99, 3999], dtype=torch.int32)
    gen = torch.Generator().manual_seed(2)
    for step in range(4):
        cache.kv_len += 1
        on = tokens.cuda()
        logits = decoder.logits(on, cache).double().cpu().numpy()
        x = raw["embedding"][tokens.long()].double()
        x = (x + torch.cat([p(row[None]) for p, row in zip(plain, x)])).numpy()
        weights, ids = M.route(x, raw["router"].numpy(), top_k, None, "softmax", True, 1.0)
        y, _ = M.experts(x, up, down, ids, weights, x, 1e-5)
        want = y @ vocabulary.T
        err = np.abs(logits - want).max() / np.abs(want).max()
        print("step %d: worst error of the largest logit %.2g" % (step, err), flush=True)
        assert err <= 8e-3
        u = torch.rand(batch, generator=gen)
        settings = dict(temperature=0.8, top_k=50, top_p=0.95)
        # The same call again: the cache's last place is written with what it holds already.
        got = decoder(on, cache, u.cuda(), **settings).cpu()
        for r in range(batch):
            token, _, margin = S.sample(logits[r], float(u[r]), **settings)
            assert margin > 1.5 * 4000 * 2.0 ** -43 and int(got[r]) == token
        tokens = got


def test_the_example_runs(example, capsys):
    example.main()
    assert "6 steps of 3 sequences" in capsys.readouterr().out
