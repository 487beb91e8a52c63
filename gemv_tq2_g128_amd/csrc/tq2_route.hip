// Router of a mixture of experts: scores x W^T in 64 bits, and the choice of top_k of them.
//
// Why 64 bits.  The choice is a whole number: two experts whose scores differ by less than the rounding of a 32-bit sum
// (1e-7 of sum |x w|) would change places from one kernel to the next, some token in every few thousand.  Products of
// 32- and 16-bit operands are exact in f64.
//
// Scores, two forms.  dot_kernel: a wave for one expert and up to kDots tokens, on the vector ALUs; the weight is read
// once, which is all there is to a few tokens.  tile_kernel: v_mfma_f64_16x16x4_f64 over 16 tokens by 16 or 32 experts, a
// block's waves and further blocks sharing the hidden axis; its bound is the f64 rate of the matrix cores (4099 tokens by 60
// experts, K = 4096: 55 us, 37 TFLOP/s), no faster than the vector ALUs' but with no operand conversion in its way.
// The order of a sum over the hidden axis is fixed by the sizes alone.
//
// Choice.  A wave for each token: f64 scores as unsigned keys of the same order, one maximum over the wave (DPP moves)
// for each chosen expert, the lowest index by a ballot over equal keys.
//
// Measured (us): one token, hidden 2048, 8 of 128 experts: 3.3 for the scores, 4.0 for the choice, each a chain of trips to
// memory and maxima.  64 tokens, 7168, 8 of 256: 10.9 and 7.6.  4099 tokens, 4096, 4 of 60: 55 and 5.5 (58 among other calls).
#include "tq2_device.h"
#include "tq2_moe_internal.h"
#include "tq2_types.h"

namespace tq2 {
namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));

// Eight consecutive values as f32 (exact for all types).
template <class T>
__device__ __forceinline__ void load8(const typename T::elem* p, float (&v)[8]) {
  const f32x4_t a = load4(T(), p), b = load4(T(), p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}

__device__ __forceinline__ double shuffle_xor(double v, int mask) {
  return __shfl_xor(v, mask);
}

constexpr int kDots = 4;             // tokens of a wave of dot_kernel
constexpr int kDotWaves = 4;

// scores f64 [tokens, experts].
template <class X, class W>
__global__ __launch_bounds__(64 * kDotWaves) void dot_kernel(const typename X::elem* __restrict__ x,
                                                             const typename W::elem* __restrict__ w, int tokens,
                                                             int experts, int hidden, double* __restrict__ scores) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * kDotWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (e >= experts) return;
  const int t0 = blockIdx.y * kDots, n = min(kDots, tokens - t0);
  double sum[kDots] = {};
  const typename W::elem* row = w + size_t(e) * hidden;
#pragma unroll 4
  for (int h = lane * 8; h < hidden; h += 512) {
    float b[8];
    load8<W>(row + h, b);
#pragma unroll
    for (int i = 0; i < kDots; ++i) {
      if (i >= n) break;
      float a[8];
      load8<X>(x + size_t(t0 + i) * hidden + h, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[i] = __builtin_fma(double(a[j]), double(b[j]), sum[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kDots; ++i) {
    if (i >= n) break;
#pragma unroll
    for (int m = 32; m; m >>= 1) sum[i] += shuffle_xor(sum[i], m);
    if (lane == 0) scores[size_t(t0 + i) * experts + e] = sum[i];
  }
}

constexpr int kTileWaves = 8;
constexpr int kMaxParts = 8;

// scores f64 [parts, tokens, experts] of 16 tokens by 16 TILES experts; part blockIdx.z takes `span` of the hidden axis (a
// multiple of 32), its waves a 32-wide step each in turn.  A lane holds eight neighbouring values of one row: lane group
// g's j-th is column 8 g + j of the step, in both operands.  Several tiles share the conversion of x to f64.
template <class X, class W, int TILES>
__global__ __launch_bounds__(64 * kTileWaves) void tile_kernel(const typename X::elem* __restrict__ x,
                                                               const typename W::elem* __restrict__ w, int tokens,
                                                               int experts, int hidden, int span,
                                                               double* __restrict__ scores) {
  __shared__ double join[kTileWaves][TILES * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const int t0 = blockIdx.x * 16, e0 = blockIdx.y * 16 * TILES;
  // Rows past the end repeat the last one; their products are not stored.
  const typename X::elem* xr = x + size_t(min(t0 + r16, tokens - 1)) * hidden;
  const typename W::elem* wr[TILES];
#pragma unroll
  for (int i = 0; i < TILES; ++i) wr[i] = w + size_t(min(e0 + i * 16 + r16, experts - 1)) * hidden;
  const int from = blockIdx.z * span, end = min(hidden, from + span);
  f64x4_t acc[TILES] = {};
  float a[8] = {}, b[TILES][8] = {};
  const auto load = [&](int h) {
    if (h < end) {
      load8<X>(xr + h, a);
#pragma unroll
      for (int i = 0; i < TILES; ++i) load8<W>(wr[i] + h, b[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = 0.f;
#pragma unroll
        for (int i = 0; i < TILES; ++i) b[i][j] = 0.f;
      }
    }
  };
  load(from + wave * 32 + g4 * 8);
  for (int h0 = from + wave * 32; h0 < end; h0 += 32 * kTileWaves) {
    float c[8], d[TILES][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = a[j];
#pragma unroll
      for (int i = 0; i < TILES; ++i) d[i][j] = b[i][j];
    }
    load(h0 + 32 * kTileWaves + g4 * 8);                // the next step's, under this one's products
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double v = double(c[j]);
#pragma unroll
      for (int i = 0; i < TILES; ++i) acc[i] = __builtin_amdgcn_mfma_f64_16x16x4f64(v, double(d[i][j]), acc[i], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) join[wave][(i * 4 + r) * 64 + lane] = acc[i][r];
  __syncthreads();
  double* out = scores + size_t(blockIdx.z) * tokens * experts;
  for (int at = threadIdx.x; at < TILES * 256; at += 64 * kTileWaves) {
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < kTileWaves; ++i) v += join[i][at];
    // Lane group g holds rows g, 4 + g, 8 + g, 12 + g.
    const int t = t0 + (at >> 6 & 3) * 4 + (at >> 4 & 3), e = e0 + (at >> 8) * 16 + (at & 15);
    if (t < tokens && e < experts) out[size_t(t) * experts + e] = v;
  }
}

// f64 as unsigned keys of the same order; NaN below all numbers, 0 is no key.
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v == 0.0 ? 0.0 : v);     // -0 and 0 are equal
  const uint64_t k = u >> 63 ? ~u : u | uint64_t(1) << 63;
  return v == v ? k : 1;
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROW_MASK, 0xF, false)));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0xB1, 0xF>(v);
  v = dpp_max<0x4E, 0xF>(v);
  v = dpp_max<0x141, 0xF>(v);
  v = dpp_max<0x140, 0xF>(v);
  v = dpp_max<0x142, 0xA>(v);
  v = dpp_max<0x143, 0xC>(v);
  return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

constexpr int kChoiceWaves = 4;

// NE: scores of a lane, experts lane + 64 i.
template <int NE>
__global__ __launch_bounds__(64 * kChoiceWaves) void choice_kernel(const double* __restrict__ scores, int parts,
                                                                   const float* __restrict__ bias, int tokens,
                                                                   int experts, int top_k, bool sigmoid,
                                                                   bool renormalize, double scale,
                                                                   float* __restrict__ weights,
                                                                   int32_t* __restrict__ ids) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kChoiceWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= tokens) return;
  const double low = -__builtin_inf();
  double p[NE];
  uint64_t key[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    p[i] = low;
    if (e < experts) {
      // All parts are loaded at once; those that are not there count as zeros.
      double part[kMaxParts];
#pragma unroll
      for (int s = 0; s < kMaxParts; ++s)
        part[s] = s < parts ? scores[(size_t(s) * tokens + t) * experts + e] : 0.0;
      p[i] = part[0];
#pragma unroll
      for (int s = 1; s < kMaxParts; ++s) p[i] += part[s];
    }
    key[i] = e < experts ? key_of(p[i]) : 0;
  }
  double sum = 0.0;                                       // of the softmax, over all experts
  bool nan = false;
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] = 1.0 / (1.0 + exp(-p[i]));
  } else {
    double top = low;
#pragma unroll
    for (int i = 0; i < NE; ++i) top = fmax(top, p[i]);
#pragma unroll
    for (int m = 32; m; m >>= 1) top = fmax(top, shuffle_xor(top, m));
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      p[i] = lane + 64 * i < experts ? exp(p[i] - top) : 0.0;
      sum += p[i];
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) sum += shuffle_xor(sum, m);
    nan = sum != sum;
    if (nan && bias) {
      // The choice goes on without the NaN scores: equals of an infinite top share the softmax.
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        if (p[i] != p[i] && key[i] > 1) p[i] = 1.0;       // infinity less itself
        if (p[i] == p[i]) sum += p[i];
      }
#pragma unroll
      for (int m = 32; m; m >>= 1) sum += shuffle_xor(sum, m);
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] /= sum;
  }
  if (bias) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      if (e < experts) key[i] = key_of(p[i] + double(bias[e]));
    }
  }
  double mine = 0.0, total = 0.0;                         // lane j keeps the j-th choice
  int id = 0;
  for (int j = 0; j < top_k; ++j) {
    // The largest key, by its upper and then its lower half.
    uint32_t upper = 0, lower = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) upper = max(upper, uint32_t(key[i] >> 32));
    upper = wave_max(upper);
#pragma unroll
    for (int i = 0; i < NE; ++i) lower = max(lower, uint32_t(key[i] >> 32) == upper ? uint32_t(key[i]) : 0);
    lower = wave_max(lower);
    const uint64_t best = uint64_t(upper) << 32 | lower;
    double chosen = 0.0;
    int at = -1;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const uint64_t same = __ballot(key[i] == best);
      if (at < 0 && same) {
        const int from = __builtin_ctzll(same);
        at = 64 * i + from;
        const uint64_t bits = __builtin_bit_cast(uint64_t, p[i]);
        const uint32_t lo = __builtin_amdgcn_readlane(int(bits), from), hi = __builtin_amdgcn_readlane(int(bits >> 32), from);
        chosen = __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
        if (lane == from) key[i] = 0;
      }
    }
    total += chosen;
    if (lane == j) mine = chosen, id = at;
  }
  if (renormalize && total < 0x1p-800) {
    // Probabilities near or past f64's least number, of which the sum knows too little or nothing: their ratios are those
    // of exp(score), for the sigmoid too, whose 1 + exp(score) is 1 here.
    double score = low;
    if (lane < top_k) {
      score = 0.0;
      for (int s = 0; s < parts; ++s) score += scores[(size_t(s) * tokens + t) * experts + id];
    }
    double most = score;
#pragma unroll
    for (int m = 32; m; m >>= 1) most = fmax(most, shuffle_xor(most, m));
    mine = lane >= top_k ? 0.0 : score == most ? 1.0 : exp(score - most);
    total = mine;
#pragma unroll
    for (int m = 32; m; m >>= 1) total += shuffle_xor(total, m);
  }
  if (lane < top_k) {
    if (renormalize) mine /= total;
    if (nan) mine = __builtin_nan("");
    weights[size_t(t) * top_k + lane] = float(mine * scale);
    ids[size_t(t) * top_k + lane] = id;
  }
}

// Few tokens by the vector ALUs, from 9 on by tiles of 16.
constexpr int64_t kDotTokens = 8;

// Expert tiles of a block, and parts of the hidden axis.  Two tiles share x's conversion where that leaves a block for
// each of the 256 CUs.  Parts: fewest rounds of blocks over the CUs, 3 hundredths of a round for each part's sums (4099
// tokens by 60 experts, K = 4096, two tiles: 71 us in one part, 58 in four to six; 64 by 256, K = 7168, one tile: 32 in one,
// 15 in four; 1024 by 128, K = 2048: 18 in one, 22 in six).
struct Split {
  int tiles, parts;
};
Split split_of(int64_t tokens, int64_t experts, int64_t hidden) {
  const int64_t rows = (tokens + 15) / 16, two = rows * ((experts + 31) / 32), one = rows * ((experts + 15) / 16);
  Split s = {two >= 256 ? 2 : 1, 1};
  const int64_t blocks = s.tiles == 2 ? two : one;
  const int64_t most = hidden / (32 * kTileWaves);       // at least a step for each wave
  int64_t least = INT64_MAX;
  for (int parts = 1; parts <= kMaxParts && (parts == 1 || parts <= most); ++parts) {
    const int64_t cost = (blocks * parts + 255) / 256 * 100 / parts + 3 * parts;
    if (cost < least) least = cost, s.parts = parts;
  }
  return s;
}

}  // namespace

int route_parts(int64_t tokens, int64_t experts, int64_t hidden) {
  return tokens <= kDotTokens ? 1 : split_of(tokens, experts, hidden).parts;
}

namespace {

template <class X, class W, int TILES>
hipError_t launch_tiles(const tq2_moe_route_args& a, int parts, hipStream_t stream) {
  const int tokens = int(a.tokens), experts = int(a.experts), hidden = int(a.hidden);
  const int span = ((hidden + parts - 1) / parts + 31) & ~31;
  const dim3 grid((tokens + 15) / 16, (experts + 16 * TILES - 1) / (16 * TILES), parts);
  hipLaunchKernelGGL((tile_kernel<X, W, TILES>), grid, dim3(64 * kTileWaves), 0, stream,
                     static_cast<const typename X::elem*>(a.x), static_cast<const typename W::elem*>(a.weight), tokens,
                     experts, hidden, span, static_cast<double*>(a.workspace));
  return hipGetLastError();
}

template <class X, class W>
hipError_t launch_scores(const tq2_moe_route_args& a, int parts, hipStream_t stream) {
  const auto* x = static_cast<const typename X::elem*>(a.x);
  const auto* w = static_cast<const typename W::elem*>(a.weight);
  const int tokens = int(a.tokens), experts = int(a.experts), hidden = int(a.hidden);
  double* scores = static_cast<double*>(a.workspace);
  if (tokens <= kDotTokens) {
    const dim3 grid((experts + kDotWaves - 1) / kDotWaves, (tokens + kDots - 1) / kDots);
    hipLaunchKernelGGL((dot_kernel<X, W>), grid, dim3(64 * kDotWaves), 0, stream, x, w, tokens, experts, hidden, scores);
  } else {
    return split_of(tokens, experts, hidden).tiles == 1 ? launch_tiles<X, W, 1>(a, parts, stream)
                                                        : launch_tiles<X, W, 2>(a, parts, stream);
  }
  return hipGetLastError();
}

template <class X>
hipError_t launch_scores(const tq2_moe_route_args& a, int parts, hipStream_t stream) {
  if (a.weight_type == TQ2_TYPE_F32) return launch_scores<X, F32>(a, parts, stream);
  if (a.weight_type == TQ2_TYPE_F16) return launch_scores<X, F16>(a, parts, stream);
  return launch_scores<X, BF16>(a, parts, stream);
}

}  // namespace

hipError_t launch_moe_route(const tq2_moe_route_args& a, hipStream_t stream) {
  const int parts = route_parts(a.tokens, a.experts, a.hidden);
  const hipError_t err = a.act_type == TQ2_TYPE_F32   ? launch_scores<F32>(a, parts, stream)
                         : a.act_type == TQ2_TYPE_F16 ? launch_scores<F16>(a, parts, stream)
                                                      : launch_scores<BF16>(a, parts, stream);
  if (err != hipSuccess) return err;
  const int ne = int(a.experts + 63) / 64;
  auto fn = ne <= 1 ? choice_kernel<1> : ne <= 2 ? choice_kernel<2> : ne <= 4 ? choice_kernel<4>
            : ne <= 8 ? choice_kernel<8> : choice_kernel<16>;
  hipLaunchKernelGGL(fn, dim3((a.tokens + kChoiceWaves - 1) / kChoiceWaves), dim3(64 * kChoiceWaves), 0, stream,
                     static_cast<const double*>(a.workspace), parts, a.bias, int(a.tokens), int(a.experts),
                     int(a.top_k), a.scoring == TQ2_MOE_SIGMOID, a.renormalize != 0, a.scale, a.weights, a.ids);
  return hipGetLastError();
}

}  // namespace tq2
