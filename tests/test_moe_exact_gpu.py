"""GPU tests of tq2_moe_experts that hold its accuracy closer than tests/test_moe_experts_gpu.py does.

Outputs that have no rounding at all (tests/moe_exact.py) are equal.  On random inputs each projection keeps a count of its
f32 roundings: three for the sums over a scale's columns (joined, scaled), one for each of these added to a wave's sum, and
one for each of the at most 16 waves' sums: K / group + 19 steps of 2^-24 of sum |x w|, beside the 31-bit integers."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import moe_ref as M  # noqa: E402
from tests.moe_exact import Exact  # noqa: E402
from tests.test_moe_experts_gpu import FORMATS, Case, moe  # noqa: E402, F401

pytestmark = pytest.mark.gpu
SCALES = {"ones": (1.0, 1.0), "tiny": (2.0 ** -70, 2.0 ** -70), "tiny up": (1.0, 2.0 ** -133), "large": (2.0 ** 40, 2.0 ** 20)}


def on_gpu(c, unit=1.0):
    from gemv_tq2_g128_amd import tq2
    if c.fmt == "q4":
        return [tuple(torch.from_numpy(a).cuda() for a in c.packed(w, unit)) for w in (c.up, c.down)]
    return [tq2.reformat_aos_to_soa(torch.from_numpy(c.packed(w, unit)).cuda(), w.shape[0] * w.shape[1], w.shape[2])
            for w in (c.up, c.down)]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("tokens,top_k,experts,inter", [(1, 2, 6, 256), (5, 2, 3, 384), (20, 2, 4, 256), (40, 2, 5, 256)])
@pytest.mark.parametrize("scale", list(SCALES))
def test_outputs_without_rounding(moe, fmt, group, tokens, top_k, experts, inter, scale):  # noqa: F811
    # One launch for down and the sum, a block row for each expert or pair, and pairs sorted by expert.
    c = Exact(2, tokens, top_k, experts, inter, fmt, group, SCALES[scale])
    y = moe.experts(torch.from_numpy(c.x.astype(np.float32)).cuda(), *on_gpu(c), torch.from_numpy(c.ids).cuda(),
                    torch.from_numpy(c.share).cuda(), experts=experts)
    want = c.out()
    assert np.array_equal(want, want.astype(np.float32))
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("unit", [2.0 ** -24, 2.0 ** -20, 2.0 ** 15])
@pytest.mark.parametrize("tokens", [1, 40])
def test_scales_at_the_ends_of_binary16(moe, fmt, group, tokens, unit):  # noqa: F811
    c = Exact(3, tokens, 2, 4, 256, fmt, group)
    y = moe.experts(torch.from_numpy((c.x / unit).astype(np.float32)).cuda(), *on_gpu(c, unit), torch.from_numpy(c.ids).cuda(),
                    torch.from_numpy(c.share).cuda(), experts=4)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), c.out() * unit)


def check(c, y, least=0.0):
    """least: what the steps of the smallest f32 numbers add."""
    tol = (max(c.up.shape[2], c.down.shape[2]) / c.group + 19) * 2.0 ** -24
    want, bound = M.experts(c.x.float().numpy(), c.up, c.down, c.ids.numpy(), c.share.numpy(), None, tol)
    assert bound.max() < 1e-2 * np.abs(want).max()
    err = np.abs(y.double().cpu().numpy() - want)
    print("worst error of its bound %.3f" % (err / (bound + least)).max(), flush=True)
    assert (err <= bound + least).all()


def case(fmt, group, *sizes, power=0):
    c = Case(*sizes, fmt, group)
    c.group = group
    c.x = c.x * 2.0 ** power
    return c


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("tokens,top_k,experts,hidden,inter", [(1, 4, 8, 512, 256), (5, 3, 8, 384, 256), (33, 2, 5, 256, 640),
                                                               (50, 4, 11, 384, 256), (3, 1, 2, 2176, 1408)])
def test_roundings(moe, fmt, group, tokens, top_k, experts, hidden, inter):  # noqa: F811
    c = case(fmt, group, 21, tokens, top_k, experts, hidden, inter)
    check(c, c.run(moe))


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("tokens", [2, 40])
@pytest.mark.parametrize("power", [-62, -60, -50, -20])
def test_small_rows(moe, fmt, group, tokens, power):  # noqa: F811
    # Rows between the projections go with the square of x: 2^-120 and below, where f32 ends at 2^-149.  Half a step of
    # these, 2^-150, for each group's sum and a place's: of weights below 0.2 in down less than 2^-140 for all columns.
    c = case(fmt, group, 22, tokens, 3, 6, 512, 256, power=power)
    check(c, c.run(moe), 2.0 ** -140)
