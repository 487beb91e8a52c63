"""A block table without columns is an array like others: its address (NULL) is not asked for."""

import pytest

torch = pytest.importorskip("torch")
from gemv_tq2_g128_amd import tq2  # noqa: E402
from tests.test_attn_cpu import append, attention  # noqa: E402


def test_table_without_columns():
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible; this check is for GPU-less hosts")
    for call in (append, attention):
        assert call(table=0, table_cols=0) == tq2.TQ2_ERR_DEVICE
        assert call(table=0, table_cols=0, pages=0, k=0, v=0) == tq2.TQ2_ERR_DEVICE
        assert call(table=0, table_cols=1) == tq2.TQ2_ERR_INVALID
