"""GPU tests of tq2_sample at temperatures and logits that bring the bins' arithmetic to its ends, against the definition in
float64 by the rules of tests/test_sample_gpu.py: tokens equal, inputs checked to lie off every border."""

import pytest

torch = pytest.importorskip("torch")
from tests.test_sample_gpu import TYPES, check, sampling  # noqa: E402, F401

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("temperature", [1e10, 1e20, 1e30, 3e38, INF])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-1e-9, -1e-20, -1e-37])
def test_negative_logits_that_share_the_bin_of_zero(sampling, temperature, kind, low):  # noqa: F811
    # l / T times the bins of a factor of two lies below the least f32: all are in one bin, far below the least number there.
    for vocab in (70, 5003):
        logits = torch.full((4, vocab), low)
        logits[1] = low * (1 + torch.arange(vocab).float() / vocab)
        logits[2, vocab // 2] = 0.0
        logits[3, ::3] = -INF
        logits, u = logits.to(TYPES[kind]), (torch.arange(4) * 2 + 1).float() / 9
        for settings in (dict(), dict(top_k=1), dict(top_k=40), dict(top_p=0.7), dict(min_p=0.9), dict(temperature=0.0)):
            check(sampling, logits, u, **{"temperature": temperature, **settings})
