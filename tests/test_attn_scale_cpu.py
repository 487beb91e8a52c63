"""The score scale of tq2_paged_attention has to be above zero and, times log2 e, a finite f32 number."""

import pytest

torch = pytest.importorskip("torch")
from gemv_tq2_g128_amd import tq2  # noqa: E402
from tests.test_attn_cpu import attention  # noqa: E402


@pytest.mark.parametrize("scale", [2.4e38, 3e38, 1e39, float("inf"), 0.0, -1e-300, float("nan")])
def test_scales_out_of_range(scale):
    assert attention(scale=scale) == tq2.TQ2_ERR_INVALID


@pytest.mark.parametrize("scale", [1e-300, 1e-44, 1.0, 2.0 ** 127, 2.3e38])
def test_scales_in_range(scale):
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible; this check is for GPU-less hosts")
    assert attention(scale=scale) == tq2.TQ2_ERR_DEVICE
