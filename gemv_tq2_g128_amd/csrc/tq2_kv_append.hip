// New tokens into a paged cache: normalise, rotate, store.
//     x' = x / sqrt(mean x^2 + eps) * w,   (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//
// Bound.  q, k and v are read once, q_out and the cache entries written once:
// HBM for prompts, launch latency for single tokens.
//
// Work split.  A head is held by head_dim / 8 lanes (a group of 8, 16 or 32),
// each with the two runs of four components that its four rotation pairs
// need: (i .. i + 3) and (i + rot / 2 ..), or eight neighbours for interleaved
// pairs, so the rotation needs no exchange between lanes and the norm one sum
// over the group.  All heads of a token share its angles: a block computes
// them once for its tokens (angle, quarter turns and polynomial in f64: the
// position times a frequency needs all of them at far positions) and keeps
// sines and cosines in LDS.
//
// Measured: 5,500 ragged prompt tokens with three axes, f32 to f16: 50.5 us, 4.5 TB/s;
// one token: 3.0 us on the GPU; 256 tokens into e4m3: 4.9 us.
#include "tq2_attn_internal.h"
#include "tq2_device.h"
#include "tq2_types.h"

namespace tq2 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = TQ2_ATTN_MAX_HEAD_DIM / 2;
constexpr int64_t kNowhere = -1;                 // a token without a place in the cache
constexpr int64_t kUnowned = -2;                 // a row that belongs to no sequence

// Sine and cosine of a in f64: quarter turns off with a two-part pi / 2, then
// the Taylor series on |r| <= pi / 4, whose first term left out is below 3e-14.
__device__ __forceinline__ float2 sine_cosine(double a) {
  const double turns = __builtin_rint(a * 0.63661977236758134308);
  double r = __builtin_fma(-turns, 1.57079632679489655800, a);
  r = __builtin_fma(-turns, 6.12323399573676603587e-17, r);
  const double r2 = r * r;
  double s = 1.0 / 6227020800.0;
  s = __builtin_fma(s, r2, -1.0 / 39916800.0);
  s = __builtin_fma(s, r2, 1.0 / 362880.0);
  s = __builtin_fma(s, r2, -1.0 / 5040.0);
  s = __builtin_fma(s, r2, 1.0 / 120.0);
  s = __builtin_fma(s, r2, -1.0 / 6.0);
  s = __builtin_fma(s * r2, r, r);
  double c = -1.0 / 87178291200.0;
  c = __builtin_fma(c, r2, 1.0 / 479001600.0);
  c = __builtin_fma(c, r2, -1.0 / 3628800.0);
  c = __builtin_fma(c, r2, 1.0 / 40320.0);
  c = __builtin_fma(c, r2, -1.0 / 720.0);
  c = __builtin_fma(c, r2, 1.0 / 24.0);
  c = __builtin_fma(c, r2, -0.5);
  c = __builtin_fma(c, r2, 1.0);
  const int q = int(turns - 4.0 * __builtin_rint(turns * 0.25));     // -2 .. 2
  const float fs = float(s), fc = float(c);
  const float sn = (q & 1) ? fc : fs, cs = (q & 1) ? fs : fc;
  return float2{(q & 2) ? -sn : sn, ((q + 1) & 2) ? -cs : cs};
}

// Sum over the lane's group of G lanes.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  v += dpp_move<0xB1, 0xF>(v);
  v += dpp_move<0x4E, 0xF>(v);
  v += dpp_move<0x141, 0xF>(v);
  if constexpr (G >= 16) v += dpp_move<0x140, 0xF>(v);
  if constexpr (G >= 32) v += __shfl_xor(v, 16);
  return v;
}

// T tokens of a block; blockIdx.y shares a token's heads out.
template <class Act, class Cache, int G, int T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendArgs a) {
  __shared__ float2 turn[T * kMaxHalf];          // sine, cosine
  __shared__ int64_t at_k[T], at_v[T];           // offset of the token in the caches, kNowhere or kUnowned
  const Pages& p = a.pages;
  const int wave = threadIdx.x >> 6;
  const int t0 = ((blockIdx.z << kRowShift) + blockIdx.x) * T;
  // One wave finds a token's sequence, its place and its angles.
  for (int i = wave; i < T; i += kThreads / 64) {
    const int t = t0 + i;
    int64_t to_k = kUnowned, to_v = kUnowned;
    int place = 0;
    const int b = t < p.tokens ? owner(p, t) : p.batch;
    if (b < p.batch) {
      const Seq s = sequence(p, b);
      if (t >= s.q0 && t < s.q0 + s.q_len) {
        place = s.first + (t - s.q0);
        const int id = page_of(p, b, place);
        const int in = place & ((1 << p.page_shift) - 1);
        to_k = to_v = kNowhere;
        if (id >= 0) {
          to_k = id * p.k_page + in * p.k_token;
          to_v = id * p.v_page + in * p.v_token;
        }
      }
    }
    if ((threadIdx.x & 63) == 0) {
      at_k[i] = to_k;
      at_v[i] = to_v;
    }
    if (t < p.tokens) {
      for (int j = threadIdx.x & 63; j < a.half; j += 64) {
        int pos = place;
        if (a.positions) {
          const int axis = (j >= a.cut[0]) + (j >= a.cut[1]);
          pos = a.positions[int64_t(axis) * p.tokens + t];
        }
        turn[i * kMaxHalf + j] = sine_cosine(double(pos) * a.freqs[j]);
      }
    }
  }
  __syncthreads();

  constexpr int kGroups = kThreads / G;
  const int lane = threadIdx.x & (G - 1), group = threadIdx.x / G;
  const int dim = p.head_dim;
  const bool live = lane * 8 < dim;              // head_dim 96 and 192 leave lanes over
  // The lane's two runs of four components and its first pair.
  const int pair = lane * 4;
  int at_a = lane * 8, at_b = lane * 8 + 4;
  const bool turned = a.interleaved ? lane * 8 < 2 * a.half : pair < a.half;
  if (turned && !a.interleaved) {
    at_a = pair;
    at_b = pair + a.half;
  }
  const int heads_q = a.q ? p.q_heads : 0;
  const int heads = heads_q + 2 * p.kv_heads;
  typedef typename Act::elem act_t;
  typedef typename Cache::elem cache_t;
  for (int i = 0; i < T; ++i) {
    const int t = t0 + i;
    if (at_k[i] == kUnowned) continue;           // rows past the last one as well
    float2 sc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sc[j] = turned ? turn[i * kMaxHalf + pair + j] : float2{0.f, 1.f};
    for (int h = blockIdx.y * kGroups + group; h < heads; h += gridDim.y * kGroups) {
      const int kind = h < heads_q ? 0 : (h < heads_q + p.kv_heads ? 1 : 2);
      const int hh = kind == 0 ? h : (kind == 1 ? h - heads_q : h - heads_q - p.kv_heads);
      const act_t* src = kind == 0   ? static_cast<const act_t*>(a.q) + t * a.q_token + hh * a.q_head
                         : kind == 1 ? static_cast<const act_t*>(a.k) + t * a.k_token + hh * a.k_head
                                     : static_cast<const act_t*>(a.v) + t * a.v_token + hh * a.v_head;
      const int64_t to = kind == 1 ? at_k[i] : (kind == 2 ? at_v[i] : 0);
      f32x4_t x = {0.f, 0.f, 0.f, 0.f}, y = x;
      if (live) {
        x = load4(Act(), src + at_a);
        y = load4(Act(), src + at_b);
      }
      const float* norm = kind == 0 ? a.q_norm : (kind == 1 ? a.k_norm : nullptr);
      if (norm) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = __builtin_fmaf(x[j], x[j], __builtin_fmaf(y[j], y[j], sum));
        const float r = rsqrtf(group_sum<G>(sum) / float(dim) + a.eps);
        if (live) {
          x = x * r * load4(F32(), norm + at_a);
          y = y * r * load4(F32(), norm + at_b);
        }
      }
      if (kind != 2 && turned) {
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float u = x[2 * j], v = x[2 * j + 1], m = y[2 * j], n = y[2 * j + 1];
            x[2 * j] = u * sc[j].y - v * sc[j].x;
            x[2 * j + 1] = v * sc[j].y + u * sc[j].x;
            y[2 * j] = m * sc[2 + j].y - n * sc[2 + j].x;
            y[2 * j + 1] = n * sc[2 + j].y + m * sc[2 + j].x;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float u = x[j], v = y[j];
            x[j] = u * sc[j].y - v * sc[j].x;
            y[j] = v * sc[j].y + u * sc[j].x;
          }
        }
      }
      if (!live) continue;
      if (kind == 0) {
        act_t* dst = static_cast<act_t*>(a.q_out) + t * a.o_token + hh * a.o_head;
        store4(Act(), dst + at_a, x);
        store4(Act(), dst + at_b, y);
      } else if (to >= 0) {
        const float* scale = kind == 1 ? a.k_scale : a.v_scale;
        if (scale) {
          const float s = scale[hh];
          x = x / s;
          y = y / s;
        }
        cache_t* dst = (kind == 1 ? static_cast<cache_t*>(a.k_cache) + hh * p.k_head
                                  : static_cast<cache_t*>(a.v_cache) + hh * p.v_head) + to;
        store4(Cache(), dst + at_a, x);
        store4(Cache(), dst + at_b, y);
      }
    }
  }
}

template <class Act, class Cache, int G, int T>
hipError_t launch(const AppendArgs& a, hipStream_t stream) {
  const int heads = (a.q ? a.pages.q_heads : 0) + 2 * a.pages.kv_heads;
  const int rounds = (heads * G + kThreads - 1) / kThreads;
  const Grid grid = append_grid(a.pages.tokens, T, rounds);
  hipLaunchKernelGGL((kv_append_kernel<Act, Cache, G, T>), dim3(grid.x, grid.y, grid.z), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <class Act, class Cache, int G>
hipError_t launch_tokens(const AppendArgs& a, hipStream_t stream) {
  // Four tokens share a block, so that all four waves compute angles, once there are
  // blocks for every CU many times over (6,000 tokens: 36.2 us, 39.0 by one; 1,500
  // tokens: 13.0 us, 10.6 by one).
  if (a.pages.tokens >= 4096) return launch<Act, Cache, G, 4>(a, stream);
  return launch<Act, Cache, G, 1>(a, stream);
}

template <class Act, class Cache>
hipError_t launch_dim(const AppendArgs& a, hipStream_t stream) {
  if (a.pages.head_dim <= 64) return launch_tokens<Act, Cache, 8>(a, stream);
  if (a.pages.head_dim <= 128) return launch_tokens<Act, Cache, 16>(a, stream);
  return launch_tokens<Act, Cache, 32>(a, stream);
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, int act, int cache, hipStream_t stream) {
  const bool narrow = cache == TQ2_TYPE_E4M3;
  if (act == TQ2_TYPE_F32)
    return narrow ? launch_dim<F32, E4M3>(a, stream) : launch_dim<F32, F16>(a, stream);
  if (act == TQ2_TYPE_F16)
    return narrow ? launch_dim<F16, E4M3>(a, stream) : launch_dim<F16, F16>(a, stream);
  return narrow ? launch_dim<BF16, E4M3>(a, stream) : launch_dim<BF16, BF16>(a, stream);
}

}  // namespace tq2
