"""An empty cache: a block table without columns, no pages."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [0, 3])
@pytest.mark.parametrize("q_len", [1, 40])
def test_empty_table(pages, q_len):
    """Nothing is stored, rows see nothing, and q is turned all the same."""
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    from gemv_tq2_g128_amd import attn
    gen = torch.Generator().manual_seed(61)
    q, k = (torch.randn(2 * q_len, h, 64, generator=gen).cuda() for h in (4, 2))
    kc, vc = (torch.full((pages, 2, 16, 64), 7.0, dtype=torch.float16, device="cuda") for _ in "kv")
    lens = torch.tensor([0, q_len]).int().cuda()
    table = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    cu = None if q_len == 1 else torch.tensor([0, q_len, 2 * q_len]).int().cuda()
    out = attn.kv_append(k, k, kc, vc, lens, table, q=q, cu_q=cu)
    assert torch.equal(out, q)
    y = attn.paged_attention(q, kc, vc, lens, table, cu_q=cu)
    torch.cuda.synchronize()
    assert bool((y == 0).all()) and bool((kc == 7).all()) and bool((vc == 7).all())
