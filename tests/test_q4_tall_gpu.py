"""GPU parity of tq2_q4_gemv for four rows of x or fewer on both sides of where rows are split over the waves.

The tolerance is that of test_q4_gpu.py; the reference is taken on the GPU, in float64.
"""

import pytest

torch = pytest.importorskip("torch")
from tests.test_q4_gpu import TOL, q4  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [65536, 262143, 262144, 262157])
@pytest.mark.parametrize("m,k,group", [(1, 128, 128), (1, 4224, 32), (2, 1152, 64), (4, 384, 128), (5, 256, 32)])
def test_few_rows_of_x(q4, n, m, k, group):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(n + m + k)
    codes = torch.randint(0, 256, (n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(n, k // group, generator=gen, device="cuda") * 0.04 - 0.02).half()
    x = torch.randn(m, k, generator=gen, device="cuda")
    res = torch.randn(m, n, generator=gen, device="cuda") if m != 2 else None
    y = q4.gemv(codes, scales, x, residual=res).double()
    xt, at = x.double().t().contiguous(), x.double().abs().t().contiguous()
    for lo in range(0, n, 65536):
        part = slice(lo, lo + 65536)
        w = (torch.stack((codes[part] & 15, codes[part] >> 4), -1).flatten(1).double() - 8) * \
            scales[part].double().repeat_interleave(group, 1)
        ref, s = torch.mm(w, xt).t(), torch.mm(w.abs(), at).t()
        if res is not None:
            ref, s = ref + res[:, part], s + res[:, part].abs()
        assert bool(((y[:, part] - ref).abs() <= TOL * s).all()), lo
