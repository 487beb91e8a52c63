"""CPU checks of the token choice's bins (csrc/tq2_sample_bins.h, compiled for the host)."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HARNESS = r"""
#include "tq2_sample_bins.h"
extern "C" void bins(double temperature, float top, const float* l, int n, int32_t* out) {
  tq2::Bins b;
  b.set_rate(1.4426950408889634 / temperature);
  b.set_top(top);
  for (int i = 0; i < n; ++i) out[i] = b.bin(l[i]);
}
extern "C" float sieve(double temperature, float top, int cut) {
  tq2::Bins b;
  b.set_rate(1.4426950408889634 / temperature);
  b.set_top(top);
  return b.sieve(cut);
}
extern "C" int last_bin(double temperature, double min_p) {
  tq2::Bins b;
  b.set_rate(1.4426950408889634 / temperature);
  return b.last_bin(min_p);
}
"""
INF = float("inf")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("bins")
    (at / "bins.cc").write_text(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-ffp-contract=off",
                    "-fsanitize=undefined", "-fno-sanitize-recover", "-I",
                    os.path.join(ROOT, "gemv_tq2_g128_amd", "csrc"), str(at / "bins.cc"), "-o", str(at / "bins.so")],
                   check=True)
    lib = ctypes.CDLL(str(at / "bins.so"))
    lib.sieve.restype = ctypes.c_float
    return lib


def bins(host, temperature, top, logits):
    l = np.ascontiguousarray(logits, dtype=np.float32)
    out = np.empty(len(l), dtype=np.int32)
    host.bins(ctypes.c_double(temperature), ctypes.c_float(top), l.ctypes.data_as(ctypes.c_void_p), len(l),
              out.ctypes.data_as(ctypes.c_void_p))
    return out


def below(top, rng):
    """f32 values from top down: its neighbours, and some at every distance."""
    top = np.float32(top)
    order = np.int64(np.abs(top).view(np.int32)) * (1 if top >= 0 else -1)          # f32 in order, as whole numbers
    least = -0x7F7FFFFF
    span = max(order - least, 1)
    steps = np.unique(np.concatenate([np.arange(200), (2.0 ** rng.uniform(0, np.log2(span), 4000)).astype(np.int64)]))
    at = order - steps[steps <= span]
    bits = np.abs(at).astype(np.int32)
    return np.where(at < 0, -bits.view(np.float32), bits.view(np.float32)).astype(np.float32)


TEMPERATURES = [1e-36, 1e-30, 1e-20, 1e-10, 1e-7, 1e-6, 3e-6, 1e-5, 1e-3, 0.05, 0.7, 1.0, 2.0, 100.0, 1e10, 1e20, 1e30,
                1e36, 3e38, 1e39, 1e300, INF]
TOPS = [0.0, -0.0, 1e-45, -1e-45, -1e-38, 1e-20, -1e-20, -1e-12, -1e-9, -1e-3, 0.3, -1.0, 25.823309, 31.972586, -77.0, 1e4,
        6e5, -6e5, 1e10, -1e10, 3e38, -3e38, 3.4028235e38, -3.4028235e38]


@pytest.mark.parametrize("temperature", TEMPERATURES)
def test_the_sieve_passes_all_of_its_bins(host, temperature):
    rng = np.random.default_rng(1)
    for top in TOPS:
        logits = below(top, rng)
        at = bins(host, temperature, top, logits)
        assert at[0] == 0 and (np.diff(at) >= 0).all()
        for cut in (0, 1, 2, 3, 13, 100, 510, 511):
            bound = host.sieve(ctypes.c_double(temperature), ctypes.c_float(top), cut)
            lost = logits[(at <= cut) & ~(logits >= np.float32(bound))]
            assert len(lost) == 0, (top, cut, bound, lost[:3])


def test_what_lies_above_the_top_or_is_no_number(host):
    for temperature in TEMPERATURES:
        for top in (INF, 3.0, -1e-20, -3e38):
            assert bins(host, temperature, top, [np.nan, top]).tolist() == [512, 0]
    assert bins(host, 1.0, INF, [3e38, 0.0]).tolist() == [512, 512]


@pytest.mark.parametrize("temperature", [t for t in TEMPERATURES if t < 1e38])
def test_bins_are_as_far_as_the_logits(host, temperature):
    """11 bins for each factor of two in e: the distance, rounded down at both ends to whole bins and, near, to eighths.  The
    grid is rounded twice to 24 bits, less than 2^-12 over 512 bins."""
    rng = np.random.default_rng(2)
    for top in TOPS:
        logits = below(top, rng)
        at = bins(host, temperature, top, logits)
        far = (np.float64(np.float32(top)) - logits.astype(np.float64)) * 11 * 1.4426950408889634 / temperature
        off = np.abs(at - far)[far < 510]
        assert off.max() < 1.25 + 2.0 ** -12, (top, off.max())
        assert (at[far < 510] < 512).all() and (at[far > 514] == 512).all()


@pytest.mark.parametrize("temperature", TEMPERATURES)
def test_chunks_agree_on_their_bins(host, temperature):
    """A logit's bin below a row's top is its chunk's top's and its own below that, on whichever side of the border between
    f32 and f64 each top lies."""
    rng = np.random.default_rng(3)
    border = 2.0 ** 22 * temperature / (11 * 1.4426950408889634)
    tops = TOPS + [s * border * (1 + d) for s in (1, -1) for d in (-1025 / 2 ** 22, -1023 / 2 ** 22, -1e-5, -1e-7, 1e-7, 1e-4)
                   if border < 3e38]
    for top in tops:
        logits = below(top, rng)
        row = bins(host, temperature, top, logits)
        logits, row = logits[row < 512], row[row < 512]
        for i in rng.integers(0, len(logits), 12):
            mine = logits <= logits[i]
            chunk = bins(host, temperature, logits[i], logits[mine])
            assert (row[i] + chunk == row[mine]).all(), (top, logits[i])


@pytest.mark.parametrize("temperature", TEMPERATURES)
def test_min_p_keeps_its_bins(host, temperature):
    rng = np.random.default_rng(4)
    for top in TOPS:
        logits = below(top, rng)
        logits = logits[np.isfinite(logits)]
        at = bins(host, temperature, top, logits)
        e = np.exp2((logits.astype(np.float64) - np.float64(logits[0])) * (1.4426950408889634 / temperature))
        for least in (1.0, 0.999, 0.9, 0.5, 0.02, 1e-6, 1e-12, 1e-14):
            last = host.last_bin(ctypes.c_double(temperature), ctypes.c_double(least))
            lost = logits[(e >= least) & (at > last)]
            assert len(lost) == 0 or (least < 1e-13 and (at[(e >= least) & (at > last)] == 512).all()), (top, least, lost[:3])
    assert host.last_bin(ctypes.c_double(temperature), ctypes.c_double(0.0)) == 511
    assert host.last_bin(ctypes.c_double(0.7), ctypes.c_double(0.5)) in (2 + 11, 2 + 12)
