"""GPU parity of tq2_kv_append for more tokens than one axis of a grid of single blocks takes."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_very_many_tokens():
    """2^26 + 5 tokens of one sequence, of which the table holds the last 2^20 + 5: each is stored at its place, turned
    by its own angle.  All tokens have one key, so that the angle tells them apart."""
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    from gemv_tq2_g128_amd import attn
    tokens, page, d = (1 << 26) + 5, 1 << 20, 64
    gen = torch.Generator().manual_seed(51)
    row = torch.randn(1, 2, d, generator=gen).half()
    k, v = (row[:, i:i + 1].cuda().expand(tokens, 1, d) for i in range(2))
    kc, vc = (torch.full((2, 1, page, d), float("nan"), dtype=torch.float16, device="cuda") for _ in "kv")
    table = torch.full((1, 65), -1, dtype=torch.int32)
    table[0, 63], table[0, 64] = 1, 0
    freqs = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
    lens, cu = torch.tensor([tokens]).int().cuda(), torch.tensor([0, tokens]).int().cuda()
    attn.kv_append(k, v, kc, vc, lens, table.cuda(), cu_q=cu, freqs=freqs)
    torch.cuda.synchronize()
    print("appended", flush=True)
    half = d // 2
    a, b = row[0, 0, :half].double().cuda(), row[0, 0, half:].double().cuda()
    for at, first, count in ((1, 63 * page, page), (0, 64 * page, 5)):
        angle = torch.arange(first, first + count, device="cuda", dtype=torch.float64)[:, None] * freqs
        cos, sin = torch.cos(angle), torch.sin(angle)
        want = torch.cat((a * cos - b * sin, b * cos + a * sin), 1)
        # The rounding to f16, f32 products and sums of |a| + |b|, and angles to 2^-53 of 7e7.
        tol = 2.0 ** -11 * want.abs() + 2.0 ** -25 + (2.0 ** -22 + 1e-7) * (a.abs() + b.abs()).repeat(2)
        err = (kc[at, 0, :count].double() - want).abs()
        print("page %d worst err / tol %.3f" % (at, float((err / tol).max())), flush=True)
        assert bool((err <= tol).all())
        assert torch.equal(vc[at, 0, :count], row[:, 1].cuda().expand(count, d))
    assert bool(kc[0, 0, 5:].isnan().all()) and bool(vc[0, 0, 5:].isnan().all())
