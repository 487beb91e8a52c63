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


def neighbours(top, steps):
    """f32 numbers so many steps below top > 0."""
    return (torch.tensor(top).view(torch.int32) - torch.as_tensor(steps, dtype=torch.int32)).view(torch.float32)


@pytest.mark.parametrize("top,temperature", [(31.972586, 3.76e-6), (25.823309, 3e-6), (25.823309, 1e-5), (11.3, 1e-6),
                                             (57.0, 1e-6), (3.1, 1e-7), (25.823309, 1e-7), (1e5, 0.01), (1e6, 0.05),
                                             (3e38, 1e31), (20.0, 1e-30)])
def test_min_p_among_neighbours_at_low_temperatures(sampling, top, temperature):  # noqa: F811
    # Every number of steps below the top, min_p on both sides of each e.
    vocab = 4500
    near = neighbours(top, list(range(12)))
    logits = torch.full((2, vocab), -5.0)
    logits[0, 40:52] = near
    logits[1, 4400:4412] = near.flip(0)              # another chunk's
    u = torch.tensor([0.95, 0.5])
    e = torch.exp((near.double() - near[0].double()) / temperature)
    for least in {float(x) * s for x in e[1:] if x > 1e-6 for s in (0.98, 1.02)} | {0.5}:
        check(sampling, logits, u, temperature=temperature, min_p=least)
        check(sampling, logits, u, temperature=temperature, min_p=least, top_k=3)


@pytest.mark.parametrize("top", [25.823309, 31.9, 17.1, 1000.1])
def test_a_crowd_far_below_one_at_low_temperatures(sampling, top):  # noqa: F811
    # Neighbours whose e is 9e-8: 3,000 of them hold 3e-4 of the row.
    two = neighbours(top, [0, 1])
    temperature = float(two[0] - two[1]) / 16.2
    logits = two[1].repeat(3, 3003)
    logits[:, 77] = two[0]
    u = torch.tensor([0.5, 0.9998, 0.9999])
    ids = check(sampling, logits, u, temperature=temperature)
    assert int(ids[0]) == 77 and 77 not in ids[1:].tolist()
    check(sampling, logits, u, temperature=temperature, top_p=0.99993)
    check(sampling, logits, u, temperature=temperature, top_k=2500)


def test_a_row_whose_chunks_lie_on_both_sides_of_the_border(sampling):  # noqa: F811
    # l / T times 11 / ln 2 around 2^22, where places change from f32 to f64; each chunk's largest on its own side.
    g = torch.Generator().manual_seed(4)
    border = 2.0 ** 22 * 0.6931471805599453 / 11
    logits = (border + 12 * torch.rand(4, 40000, generator=g) - 6 + torch.linspace(8, -8, 40000))
    logits[2:] = -logits[2:]
    u = torch.rand(4, generator=g)
    for settings in (dict(), dict(top_k=300), dict(top_p=0.7), dict(min_p=0.01), dict(temperature=2.0), dict(temperature=0.5)):
        check(sampling, logits, u, **settings)
        check(sampling, logits.flip(1), u, **settings)


@pytest.mark.parametrize("temperature", [1e40, 1e300, INF])
@pytest.mark.parametrize("least", [1.0, 0.9, 0.5])
def test_min_p_at_temperatures_past_f32(sampling, temperature, least):  # noqa: F811
    # e is 1 wherever the logits lie (at 1e40 within 1.7e-2 of it), over several bins.
    g = torch.Generator().manual_seed(5)
    logits = (torch.rand(3, 9000, generator=g) * 2 - 1) * 3.3e38
    logits[1, 8000] = 3.4e38
    logits[2, 3::7] = -INF
    u = torch.tensor([0.31, 0.62, 0.93])
    check(sampling, logits, u, temperature=temperature, min_p=least)
    check(sampling, logits, u, temperature=temperature, min_p=least, top_k=4000)
