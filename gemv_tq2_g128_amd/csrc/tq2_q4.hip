// 4-bit matrix-vector products with group scales, 1 <= M <= 16 rows of x:
//     out[m, n] = residual[m, n] + sum_g d[n, g] sum_{k in g} x[m, k] (c[n, k] - 8).
//
// Bound.  Every weight is read once: N K / 2 bytes of codes and 2 N K / group
// of scales against HBM.  On the vector ALUs a weight would cost two
// instructions (half a mask, half a packed subtract, one mixed FMA) per row of
// x, which is already 80 % of the issue slots at 8 TB/s for one row; on the
// matrix cores it costs one instruction for any M up to 16.
//
// Matrix form.  One v_mfma_f32_16x16x32_f16 takes 16 weight rows as its
// columns and up to 16 rows of x halves as its rows: x = hi + lo in binary16
// under a power of two (exact weights, so the products carry x's 22 leading
// bits); rows 0..7 hold hi and 8..15 lo for M <= 8, else two MFMAs.
// Accumulation is f32: the codes of one group are summed by the matrix core,
// then scaled by d (one lane holds one weight row) and by the power of two.
//
// Work split.  A block of 8 waves owns all of K for a step of RT * 16 weight
// rows; each wave takes an eighth of the 128-wide blocks of K, and the eight
// partial sums meet in LDS.  x is converted once per block into LDS in
// operand order, so a wave's inner loop is: one 16-byte load per lane (a row
// segment of 64 bytes per row and 128-wide block, next to the one the same wave
// reads for the following block), four LDS operand reads shared by RT row
// tiles, decode, MFMA.  Blocks walk over row steps, with the next step's
// codes in flight before the present step is computed.
//
// Groups.  A lane's 16 bytes are 32 consecutive weights.  For group 128 any
// order of k inside the 128-wide block will do, so word s of lane group g
// serves MFMA step s.  For groups of 32 and 64 a step must stay inside one
// group: the four lane groups transpose their words (two swaps of 32-lane
// halves, two of 16-lane rows), after which step s covers group s of 32.
#include "tq2_internal.h"
#include "tq2_device.h"
#include "tq2_q4_internal.h"

namespace tq2 {
namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxKb = 4;                       // 128-wide blocks of K per wave and pass

// The 8 weights of one word as exact binary16 values code - 8, in the order
// 0, 4, 1, 5, 2, 6, 3, 7: masks leave a pair of nibbles 16 bits apart in the
// low mantissa bits of 1024 + c or of 1024 + 16 c.
__device__ __forceinline__ half8_t decode8(uint32_t w) {
  const uint32_t magic = 0x64006400u;
  const half2_t one16 = {_Float16(0.0625f), _Float16(0.0625f)};
  const half2_t off16 = {_Float16(-72.0f), _Float16(-72.0f)};
  const half2_t off1 = {_Float16(-1032.0f), _Float16(-1032.0f)};
  const uint32_t v = w >> 8;
  const half2_t a = __builtin_bit_cast(half2_t, and_or(w, 0x000F000Fu, magic)) + off1;
  const half2_t b = __builtin_bit_cast(half2_t, and_or(w, 0x00F000F0u, magic)) * one16 + off16;
  const half2_t c = __builtin_bit_cast(half2_t, and_or(v, 0x000F000Fu, magic)) + off1;
  const half2_t d = __builtin_bit_cast(half2_t, and_or(v, 0x00F000F0u, magic)) * one16 + off16;
  return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Transpose the 4 words of the four 16-lane groups: afterwards lane group g
// holds in word s what lane group s held in word g.
__device__ __forceinline__ void transpose4(u32x4_t& w) {
  auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w = u32x4_t{c[0], c[1], d[0], d[1]};
}

// Largest |x| over aligned groups of 16 lanes, in every lane.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_move<0xB1, 0xF>(v));
  v = fmaxf(v, dpp_move<0x4E, 0xF>(v));
  v = fmaxf(v, dpp_move<0x141, 0xF>(v));
  v = fmaxf(v, dpp_move<0x140, 0xF>(v));
  return v;
}

// MT: rows of the matrix operand x fills (8: hi and lo in one operand, 16:
// one operand each).  LDS: x operand words [kb][step][lane group][column],
// the powers of two [kb][16], and two buffers of partial sums.
template <int MT>
struct Shape {
  __host__ __device__ static int columns(int m) { return MT == 8 ? 2 * m : 32; }
  __host__ __device__ static size_t x_bytes(int kb, int m) { return size_t(kb) * 256 * columns(m); }
  __host__ __device__ static size_t bytes(int kb, int m, int rt) {
    return x_bytes(kb, m) + size_t(kb) * 64 + size_t(2) * kWaves * rt * MT * 64;
  }
};

// Convert rows 0..m-1 of x, columns [k0, k0 + 128 kbs), into LDS.  Sixteen
// consecutive threads hold one row's 128 columns, so the power of two of that
// stretch is a DPP maximum: 2^13 <= |x| 2^e < 2^14 keeps hi normal and
// leaves lo 2^-25 absolute, 2^-39 of the largest value.
template <int G, int MT>
__device__ __forceinline__ void stage_x(const float* __restrict__ x, int m, int64_t k, int64_t k0,
                                        int kbs, half8_t* __restrict__ xf, float* __restrict__ xs) {
  const int cols = Shape<MT>::columns(m);
  const int hi_lo = MT == 8 ? m : 16;
  for (int i = threadIdx.x; i < m * kbs * 16; i += kThreads) {
    const int u = i & 15, kb = (i >> 4) % kbs, row = (i >> 4) / kbs;
    const float4* src = reinterpret_cast<const float4*>(x + row * k + k0 + kb * 128 + u * 8);
    const float4 p = src[0], q = src[1];
    const float v[8] = {p.x, q.x, p.y, q.y, p.z, q.z, p.w, q.w};   // decode8's order
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
    top = row16_max(top);
    const int e = int((__builtin_bit_cast(uint32_t, top) >> 23) & 255) - 127;
    const int up = top > 0.f ? min(13 - e, 126) : 0;
    const float s = __builtin_ldexpf(1.0f, up);
    half8_t hi, lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = v[j] * s;
      hi[j] = _Float16(t);
      lo[j] = _Float16(t - float(hi[j]));
    }
    const int step = G == 128 ? (u & 3) : (u >> 2), grp = G == 128 ? (u >> 2) : (u & 3);
    half8_t* dst = xf + (size_t(kb * 4 + step) * 4 + grp) * cols + row;
    dst[0] = hi;
    dst[hi_lo] = lo;
    if (u == 0) {
      const float back = __builtin_ldexpf(1.0f, -up);
      xs[kb * 16 + row] = back;
      if (MT == 8) xs[kb * 16 + 8 + row] = back;
    }
  }
}

template <int G>
struct Codes {
  u32x4_t w;
  uint32_t d[G == 32 ? 2 : 1];                  // binary16 scales of the lane's row, 128 / G of them
};

template <int G>
__device__ __forceinline__ void load_codes(const uint8_t* __restrict__ codes,
                                           const uint16_t* __restrict__ scales, uint32_t code_off,
                                           uint32_t scale_off, Codes<G>& c) {
  c.w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(codes + code_off));
  if constexpr (G == 128) {
    c.d[0] = scales[scale_off];
  } else if constexpr (G == 64) {
    c.d[0] = *reinterpret_cast<const uint32_t*>(scales + scale_off);
  } else {
    const uint2 d = *reinterpret_cast<const uint2*>(scales + scale_off);
    c.d[0] = d.x;
    c.d[1] = d.y;
  }
}

template <int G>
__device__ __forceinline__ float scale_of(const Codes<G>& c, int s) {
  if constexpr (G == 128) return float(__builtin_bit_cast(_Float16, uint16_t(c.d[0])));
  const int i = G == 64 ? s >> 1 : s;           // group of 32-wide step s
  return float(__builtin_bit_cast(_Float16, uint16_t(c.d[i >> 1] >> (16 * (i & 1)))));
}

template <int G, int MT, int RT>
__global__ __launch_bounds__(kThreads, 2) void q4_kernel(
    const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
    const float* __restrict__ x, const float* __restrict__ residual, float* __restrict__ out,
    int m, int n, int64_t k, int pass_kb) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g4 = lane >> 4;
  const int cols = Shape<MT>::columns(m);
  half8_t* xf = reinterpret_cast<half8_t*>(smem);
  const int all_kb = int(k >> 7);
  const int first = min(all_kb, pass_kb);
  float* xs = reinterpret_cast<float*>(smem + Shape<MT>::x_bytes(first, m));
  float* red = xs + first * 16;
  const int col = MT == 8 ? ((r16 & 7) < m ? (r16 >> 3) * m + (r16 & 7) : 0) : (r16 < m ? r16 : 0);
  const int steps = (n + RT * 16 - 1) / (RT * 16);
  const int64_t row_bytes = k >> 1, row_scales = k / G;

  for (int pass = 0; pass < all_kb; pass += pass_kb) {
    const int kbs = min(pass_kb, all_kb - pass);
    const int nk = (kbs + kWaves - 1) / kWaves;           // <= kMaxKb
    const int kb0 = wave * nk;
    const int mine = max(0, min(nk, kbs - kb0));
    Codes<G> c[2][kMaxKb][RT];
    auto load = [&](int step, Codes<G> (&into)[kMaxKb][RT]) {
      const int64_t row0 = int64_t(step) * (RT * 16);
      const uint8_t* cb = codes + row0 * row_bytes;
      const uint16_t* sb = scales + row0 * row_scales;
#pragma unroll
      for (int j = 0; j < kMaxKb; ++j) {
        if (j >= mine) continue;
        const uint32_t kb = uint32_t(pass + kb0 + j);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          // Rows past the end read the last row; their sums are not stored.
          const uint32_t r = uint32_t(min(int64_t(t * 16 + r16), n - 1 - row0));
          load_codes<G>(cb, sb, r * uint32_t(row_bytes) + kb * 64 + g4 * 16,
                        r * uint32_t(row_scales) + kb * (128 / G), into[j][t]);
        }
      }
    };
    int parity = 0;
    auto compute = [&](int step, Codes<G> (&from)[kMaxKb][RT]) {
      float acc[RT][4];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = 0.f;
#pragma unroll
      for (int j = 0; j < kMaxKb; ++j) {
        if (j >= mine) continue;
        const int kb = kb0 + j;
        const float4_t back = *reinterpret_cast<const float4_t*>(xs + kb * 16 + g4 * 4);
        if constexpr (G != 128) {
#pragma unroll
          for (int t = 0; t < RT; ++t) transpose4(from[j][t].w);
        }
        float4_t sum[RT];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const half8_t* a = xf + (size_t(kb * 4 + s) * 4 + g4) * cols + col;
          const half8_t a0 = a[0];
          half8_t a1;
          if constexpr (MT == 16) a1 = a[16];
          const bool fresh = s % (G / 32) == 0;           // a group's first step
          const bool whole = (s + 1) % (G / 32) == 0;     // and its last
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const half8_t b = decode8(from[j][t].w[s]);
            sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                a0, b, fresh ? float4_t{0.f, 0.f, 0.f, 0.f} : sum[t], 0, 0, 0);
            if constexpr (MT == 16)
              sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, b, sum[t], 0, 0, 0);
            if (whole) {
              const float d = scale_of<G>(from[j][t], s);
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[t][r] = __builtin_fmaf(d * back[r], sum[t][r], acc[t][r]);
            }
          }
        }
      }
      // Partial sums [wave][tile][row of x][weight row] of this step; lane
      // groups 0 and 1 (MT == 8) or all four hold rows 4 g4 .. 4 g4 + 3.
      float* buf = red + parity * (kWaves * RT * MT * 16);
      parity ^= 1;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float v = acc[t][r];
          if constexpr (MT == 8) v += __shfl_xor(v, 32);  // hi + lo
          if (MT == 16 || g4 < 2) buf[((wave * RT + t) * MT + g4 * 4 + r) * 16 + r16] = v;
        }
      }
      __syncthreads();
      // A buffer is written again two steps on, behind the next step's barrier.
      const int o = threadIdx.x, on = o & 15, om = (o >> 4) % MT, ot = (o >> 4) / MT;
      const int64_t row = int64_t(step) * (RT * 16) + ot * 16 + on;
      if (ot < RT && om < m && row < n) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += buf[((w * RT + ot) * MT + om) * 16 + on];
        const size_t at = size_t(om) * size_t(n) + size_t(row);
        if (pass > 0) v += out[at];
        else if (residual) v += residual[at];
        out[at] = v;
      }
    };

    // The first step's codes are in flight while x is converted (the grid has no
    // more blocks than steps).  Every wave
    // takes part in each step's barrier: the walk is uniform over the block.
    int step = blockIdx.x;
    load(step, c[0]);
    if (pass > 0) __syncthreads();                        // the last step has read x and red
    stage_x<G, MT>(x, m, k, int64_t(pass) * 128, kbs, xf, xs);
    __syncthreads();
    const int hop = gridDim.x;
    while (step < steps) {
      if (step + hop < steps) load(step + hop, c[1]);
      compute(step, c[0]);
      step += hop;
      if (step >= steps) break;
      if (step + hop < steps) load(step + hop, c[0]);
      compute(step, c[1]);
      step += hop;
    }
  }
}

template <int G, int MT, int RT>
hipError_t launch(const Q4Args& a, hipStream_t stream) {
  const int all_kb = int(a.k >> 7);
  const int pass_kb = MT == 8 ? kWaves * kMaxKb : kWaves * kMaxKb / 2;
  const size_t lds = Shape<MT>::bytes(all_kb < pass_kb ? all_kb : pass_kb, int(a.m), RT);
  const int steps = int((a.n + RT * 16 - 1) / (RT * 16));
  const int per_cu = lds <= 80 * 1024 ? 2 : 1;
  const int grid = steps < 256 * per_cu ? steps : 256 * per_cu;
  auto fn = q4_kernel<G, MT, RT>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3(grid), dim3(kThreads), lds, stream, a.codes, a.scales, a.x,
                     a.residual, a.out, int(a.m), int(a.n), a.k, pass_kb);
  return hipGetLastError();
}

template <int G>
hipError_t launch_group(const Q4Args& a, hipStream_t stream) {
  if (a.m > 8) return launch<G, 16, 1>(a, stream);
  // Two row tiles per step share the operand reads of x once every CU has
  // work for them; below that one tile per step fills more CUs.
  if (a.n >= 32 * 512) return launch<G, 8, 2>(a, stream);
  return launch<G, 8, 1>(a, stream);
}

}  // namespace

hipError_t launch_q4_gemv(const Q4Args& a, int group, hipStream_t stream) {
  if (group == 32) return launch_group<32>(a, stream);
  if (group == 64) return launch_group<64>(a, stream);
  return launch_group<128>(a, stream);
}

}  // namespace tq2
