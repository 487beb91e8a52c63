"""GPU parity of tq2_paged_attention where the scores' scale is zero, tiny, negative or large: every form of the kernel
(single tokens, chunks, prompts) has to give softmax attention with that scale.

Tolerances are those of test_paged_attention_gpu.py; a scale of zero makes every score exactly zero.
"""

import pytest

torch = pytest.importorskip("torch")
from tests.test_paged_attention_gpu import attn, check, make  # noqa: E402, F401

pytestmark = pytest.mark.gpu

LENGTHS = [((1, 1, 1), (5, 33, 200)), ((5, 3), (40, 300)), ((70, 1, 90), (70, 50, 400))]


@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("q_len,kv_len", LENGTHS)
@pytest.mark.parametrize("window", [0, 37])
def test_key_scales_of_any_sign(attn, act, q_len, kv_len, window):  # noqa: F811
    """A head of zeros (scale 0: the mean of the values that are seen), a negative scale and an ordinary one."""
    c = make(31, act, "e4m3", q_len=q_len, kv_len=kv_len, heads=(6, 3), dim=64)
    c["k_scale"] = torch.tensor([0.0, -0.13, 0.11])
    c["v_scale"] = torch.tensor([0.1, 0.0, -0.2])
    out = check(attn, c, "%s %s" % (act, q_len), window=window)
    assert bool((out[:, 2:4] == 0).all())
    c["k_scale"] = torch.tensor([-3.0, -0.002, 0.0])              # one far past the others' weight, and nearly none
    check(attn, c, "%s %s far" % (act, q_len), window=window)


@pytest.mark.parametrize("act,cache", [("f32", "f16"), ("f32", "e4m3"), ("f16", "f16"), ("f16", "e4m3"),
                                       ("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("q_len,kv_len", LENGTHS)
@pytest.mark.parametrize("scale", [1e-300, 1e-60, 1e-44, 1e-30])
def test_tiny_scales(attn, act, cache, q_len, kv_len, scale):  # noqa: F811
    """Below the least f32 number, among the subnormal ones and above them: the mean of what is seen."""
    c = make(32, act, cache, q_len=q_len, kv_len=kv_len, heads=(4, 2), dim=96)
    check(attn, c, "%s %s %g" % (act, cache, scale), scale=scale)


@pytest.mark.parametrize("q_len,kv_len", LENGTHS)
def test_large_scale_of_tiny_scores(attn, q_len, kv_len):  # noqa: F811
    """The largest scale, with q so small that the scores are ordinary."""
    c = make(33, "f32", "f16", q_len=q_len, kv_len=kv_len, heads=(4, 2), dim=64)
    c["q"] *= 2.0 ** -120
    check(attn, c, "large", scale=2.0 ** 117)
