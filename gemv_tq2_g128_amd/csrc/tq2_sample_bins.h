// Bins of a row's logits: plain arithmetic, shared by the kernels of the token choice and
// (compiled for the host) their CPU test.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __HIP__
#define TQ2_HD __host__ __device__ __forceinline__
#else
#define TQ2_HD inline
#endif

namespace tq2 {

constexpr int kBins = 512;
constexpr float kGrid = 11.f;              // bins of a factor of two: 2^46.5 over all, more than a weight's 43 bits

// Places on the grid below this are f32, which has quarters there; larger ones are f64, where l * grid is exact (f64 for
// all: 256 rows of 151,936 f32 logits 115 us where this takes 110, with min-p 75 and 71).
constexpr float kNear = 0x1p22f;

// A logit's place is floor(l * grid), its bin how far that lies below the top's place; the grid is absolute, so that chunks
// of a row agree on it.  Logits around a top far from zero, or at low temperatures, have large places: f32 would move a
// bin by the step of its numbers, and so past what min_p keeps or past the last bin.
struct Bins {
  float grid;                              // bins of the logits' unit
  bool far;                                // from the top's place on logits of the bins may lie past kNear
  float base;                              // the top's place
  double far_base;

  // rate: log2(e) / T.
  TQ2_HD void set_rate(double rate) { grid = fmaxf(kGrid * float(rate), 0x1p-126f); }       // at an infinite T too
  // Rises with l: f32 rounds no product to a whole number that the other side of kNear passes.
  TQ2_HD double place(float l) const {
    const float p = l * grid;
    return fabsf(p) < kNear ? double(floorf(p)) : floor(double(l) * double(grid));
  }
  TQ2_HD void set_top(float l) {
    base = floorf(l * grid);
    far = !(fabsf(base) < kNear - 2 * kBins);
    far_base = place(l);
  }
  // Bins from the top's; NaN and what is too far give kBins.
  TQ2_HD int near_bin(float l) const {
    const float d = base - floorf(l * grid);
    return d < float(kBins) ? int(d) : kBins;
  }
  TQ2_HD int far_bin(float l) const {
    const double p = place(l), d = p == far_base ? 0.0 : far_base - p;      // +infinity is one place
    return d < double(kBins) ? int(d) : kBins;
  }
  TQ2_HD int bin(float l) const { return far ? far_bin(l) : near_bin(l); }
  // A bound that no logit of bins 0 .. cut lies below.  edge is off by a few 2^-24 of itself.  l * grid rounds to whole
  // least subnormals as well, half of which are 2^-150 / grid in l: negative logits that far below 0 still share its bin.
  // At temperatures past 1e13, where this is no small number, everything passes.
  TQ2_HD float sieve(int cut) const {
    const float edge = far ? float((far_base - cut) / double(grid)) : (base - float(cut)) / grid;
    return grid >= 0x1p-40f && fabsf(edge) < 3e38f ? edge - fabsf(edge) * 0x1p-20f - 0x1p-100f : -INFINITY;
  }
  // The last bin that min_p leaves anything of, for a largest logit that is the row's or below it, with one to spare; all
  // where the grid is at its least, which is finer than 11 bins for a factor of two.
  TQ2_HD int last_bin(double min_p) const {
    if (!(min_p > 0.0) || grid == 0x1p-126f) return kBins - 1;
    const int last = 2 - int(floor(log2(fmin(min_p, 1.0)) * double(kGrid)));
    return last < kBins - 1 ? last : kBins - 1;
  }
};

}  // namespace tq2
