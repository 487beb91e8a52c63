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
// Work split.  x is converted once per block into LDS in operand order; a wave's
// inner loop is one 16-byte load per lane (a row segment of 64 bytes for each of 16
// rows and 128-wide block of K), four LDS operand reads, decode, MFMA.  q4_kernel
// splits K: a block of 8 waves walks over steps of 16 weight rows, each wave takes
// an eighth of the 128-wide blocks, and the eight partial sums meet in LDS.
// q4_tall_kernel, for many rows, gives each wave tiles of 16 rows and all of K, with
// no barrier.  Both have the next step's codes in flight before the present one is
// computed.  131072 x 4096, eight rows of x: 63 us (4.5 TB/s, 48 us without the
// arithmetic and the scales); 4096 x 4096, one row: 5.2 us, most of it the launch
// and one trip to memory after another.
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
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
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
  // Operand words from one lane group's columns to the next's: one more than the columns,
  // so that the 16 lanes that write a stretch of x write to different banks (eight rows by
  // 4096 x 4096: 10.5 -> 9.8 us), but for four rows or fewer, where it would cost the
  // second block of a CU.
  __host__ __device__ static int columns(int m) { return MT == 16 ? 33 : (m > 4 ? 2 * m + 1 : 2 * m); }
  __host__ __device__ static size_t x_bytes(int kb, int m) { return size_t(kb) * 256 * columns(m); }
  __host__ __device__ static size_t bytes(int kb, int m, bool sums) {
    return x_bytes(kb, m) + size_t(kb) * 64 + (sums ? size_t(2) * kWaves * MT * 64 : 0);
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

// N consecutive 128-wide blocks of K of the lane's row: its 16 bytes of each, and the
// scales of all, which lie side by side.  (One load of up to 16 bytes for several
// blocks' scales: a load of its own for each cost 19 of 66 us at 131072 x 4096.)
template <int G, int N>
struct Codes {
  u32x4_t w[N];
  uint32_t d[N * (64 / G) + (G == 128 ? N / 2 + 1 : 0)];  // words of scales; G == 128: from bit `down` on
  uint32_t down;
};

// Past the range of either resource: zeros.
constexpr uint32_t kNowhere = 0x80000000u;

// codes and scales of 16 rows or, at the end, fewer.  The word that holds the last scale
// is in range as a whole.
struct Rows {
  rsrc_t codes, scales;
};
__device__ __forceinline__ Rows rows_at(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                                        int64_t row0, uint32_t live, int64_t row_bytes, int64_t row_scales) {
  return Rows{make_rsrc(codes + row0 * row_bytes, live * uint32_t(row_bytes)),
              make_rsrc(scales + row0 * row_scales, (live * uint32_t(row_scales) * 2 + 3) & ~3u)};
}

// Every load is issued, whether the row or the block of K exists or not (those give
// zeros): behind a branch the count of loads in flight would be unknown, and each wait
// would take in the loads of the next step too.  kb: the first block, of which the lane
// takes the bytes at code_off + 64 kb; `count` of them exist.
template <int G, int N>
__device__ __forceinline__ void load_codes(const Rows& rows, uint32_t code_off, uint32_t scale_off, uint32_t kb,
                                           int count, Codes<G, N>& c) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    c.w[j] = __builtin_amdgcn_raw_buffer_load_b128(rows.codes, j < count ? code_off + (kb + j) * 64 : kNowhere, 0,
                                                   kStreamOnce);
  const uint32_t at = count > 0 ? scale_off + kb * (256 / G) : kNowhere;
  if constexpr (G == 128) {
    // Two-byte scales may start in the middle of a word, where buffer loads do not: the
    // words around them, moved down by half a word there.
    uint32_t w[N / 2 + 1];
    if constexpr (N == 4) {
      const u32x2_t d = __builtin_amdgcn_raw_buffer_load_b64(rows.scales, at & ~3u, 0, 0);
      w[0] = d[0];
      w[1] = d[1];
    } else {
      const u32x4_t d = __builtin_amdgcn_raw_buffer_load_b128(rows.scales, at & ~3u, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = d[i];
    }
    w[N / 2] = __builtin_amdgcn_raw_buffer_load_b32(rows.scales, (at & ~3u) + N * 2, 0, 0);
    c.down = (at & 2) * 8;
#pragma unroll
    for (int i = 0; i <= N / 2; ++i) c.d[i] = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < N * (256 / G) / 16; ++i) {
      const u32x4_t d = __builtin_amdgcn_raw_buffer_load_b128(rows.scales, at + i * 16, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) c.d[4 * i + e] = d[e];
    }
  }
}

// The scale of 32-wide step s of block j.
template <int G, int N>
__device__ __forceinline__ float scale_of(const Codes<G, N>& c, int j, int s) {
  const int i = j * (128 / G) + s / (G / 32);
  uint32_t w = c.d[i >> 1];
  if constexpr (G == 128) w = __builtin_amdgcn_alignbit(c.d[(i >> 1) + 1], w, c.down);
  return float(__builtin_bit_cast(_Float16, uint16_t(w >> (16 * (i & 1)))));
}

// One 128-wide block of K (block j of c): the codes' four matrix steps against x, scaled
// into acc (rows 4 g4 + r of x, weight row r16).  The weight scale meets the sum before the
// power of two does: their product alone would leave the normal numbers for x below 2^-113.
template <int G, int MT, int N>
__device__ __forceinline__ void multiply(Codes<G, N>& c, int j, const half8_t* __restrict__ a, const float4_t& back,
                                         int cols, float (&acc)[4]) {
  if constexpr (G != 128) transpose4(c.w[j]);
  float4_t sum;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const half8_t a0 = a[size_t(s) * 4 * cols];
    const half8_t b = decode8(c.w[j][s]);
    const bool fresh = s % (G / 32) == 0;                 // a group's first step
    const bool whole = (s + 1) % (G / 32) == 0;           // and its last
    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, b, fresh ? float4_t{0.f, 0.f, 0.f, 0.f} : sum, 0, 0, 0);
    if constexpr (MT == 16)
      sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[size_t(s) * 4 * cols + 16], b, sum, 0, 0, 0);
    if (whole) {
      const float d = scale_of<G, N>(c, j, s);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(d * sum[r], back[r], acc[r]);
    }
  }
}

// The column of the matrix operand x that the lane's row reads.
template <int MT>
__device__ __forceinline__ int operand_column(int r16, int m) {
  if (MT == 8) return (r16 & 7) < m ? (r16 >> 3) * m + (r16 & 7) : 0;
  return r16 < m ? r16 : 0;
}

// K split over the waves: one step of 16 weight rows at a time.
template <int G, int MT>
__global__ __launch_bounds__(kThreads, 2) void q4_kernel(
    const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
    const float* __restrict__ x, const float* __restrict__ residual, float* __restrict__ out,
    int m, int n, int64_t k, int pass_kb) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const int cols = Shape<MT>::columns(m);
  half8_t* xf = reinterpret_cast<half8_t*>(smem);
  const int all_kb = int(k >> 7);
  const int first = min(all_kb, pass_kb);
  float* xs = reinterpret_cast<float*>(smem + Shape<MT>::x_bytes(first, m));
  float* red = xs + first * 16;
  const int col = operand_column<MT>(r16, m);
  const int steps = (n + 15) / 16;
  const int64_t row_bytes = k >> 1, row_scales = k / G;

  for (int pass = 0; pass < all_kb; pass += pass_kb) {
    const int kbs = min(pass_kb, all_kb - pass);
    const int nk = (kbs + kWaves - 1) / kWaves;           // <= kMaxKb
    const int kb0 = wave * nk;
    const int mine = max(0, min(nk, kbs - kb0));
    Codes<G, kMaxKb> c[2];
    auto load = [&](int step, Codes<G, kMaxKb>& into) {
      const int64_t row0 = int64_t(step < steps ? step : 0) * 16;
      const uint32_t live = step < steps ? uint32_t(min(int64_t(16), n - row0)) : 0;
      load_codes<G, kMaxKb>(rows_at(codes, scales, row0, live, row_bytes, row_scales),
                            r16 * uint32_t(row_bytes) + g4 * 16, r16 * uint32_t(row_scales) * 2,
                            uint32_t(pass + kb0), mine, into);
    };
    // The thread's output of a step, and what is added to it; loaded in front of the
    // next step's codes, so that its wait does not take them in.
    const int on = threadIdx.x & 15, om = threadIdx.x >> 4;
    const float* add = pass > 0 ? out : residual;
    auto load_add = [&](int step) {
      const int64_t row = int64_t(step) * 16 + on;
      return add && om < m && row < n ? add[size_t(om) * size_t(n) + size_t(row)] : 0.f;
    };
    int parity = 0;
    auto compute = [&](int step, Codes<G, kMaxKb>& from, float added) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kMaxKb; ++j) {
        if (j >= mine) continue;
        const int kb = kb0 + j;
        multiply<G, MT, kMaxKb>(from, j, xf + (size_t(kb) * 16 + g4) * cols + col,
                                *reinterpret_cast<const float4_t*>(xs + kb * 16 + g4 * 4), cols, acc);
      }
      // Partial sums [wave][row of x][weight row] of this step; lane groups 0 and 1
      // (MT == 8) or all four hold rows 4 g4 .. 4 g4 + 3.
      float* buf = red + parity * (kWaves * MT * 16);
      parity ^= 1;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = acc[r];
        if constexpr (MT == 8) v += __shfl_xor(v, 32);    // hi + lo
        if (MT == 16 || g4 < 2) buf[(wave * MT + g4 * 4 + r) * 16 + r16] = v;
      }
      __syncthreads();
      // A buffer is written again two steps on, behind the next step's barrier.
      const int64_t row = int64_t(step) * 16 + on;
      if (om < m && row < n) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += buf[(w * MT + om) * 16 + on];
        out[size_t(om) * size_t(n) + size_t(row)] = v + added;
      }
    };

    // The first step's codes are in flight while x is converted (the grid has no
    // more blocks than steps).  Every wave takes part in each step's barrier: the
    // walk is uniform over the block.
    int step = blockIdx.x;
    load(step, c[0]);
    if (pass > 0) __syncthreads();                        // the last step has read x and red
    stage_x<G, MT>(x, m, k, int64_t(pass) * 128, kbs, xf, xs);
    __syncthreads();
    const int hop = gridDim.x;
    while (step < steps) {
      float added = load_add(step);
      load(step + hop, c[1]);
      compute(step, c[0], added);
      step += hop;
      if (step >= steps) break;
      added = load_add(step);
      load(step + hop, c[0]);
      compute(step, c[1], added);
      step += hop;
    }
  }
}

// Rows split over the waves: each walks over tiles of 16 weight rows and all of K by
// itself, kFlight blocks of K ahead of its matrix steps, with no barrier.
constexpr int kFlight = 8;

template <int G, int MT>
__global__ __launch_bounds__(kThreads, 2) void q4_tall_kernel(
    const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
    const float* __restrict__ x, const float* __restrict__ residual, float* __restrict__ out,
    int m, int n, int64_t k, int pass_kb) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const int cols = Shape<MT>::columns(m);
  half8_t* xf = reinterpret_cast<half8_t*>(smem);
  const int all_kb = int(k >> 7);
  float* xs = reinterpret_cast<float*>(smem + Shape<MT>::x_bytes(min(all_kb, pass_kb), m));
  const int col = operand_column<MT>(r16, m);
  const int tiles = (n + 15) / 16, hop = gridDim.x * kWaves;
  const int64_t row_bytes = k >> 1, row_scales = k / G;
  const uint32_t row_code = r16 * uint32_t(row_bytes) + g4 * 16, row_scale = r16 * uint32_t(row_scales) * 2;

  for (int pass = 0; pass < all_kb; pass += pass_kb) {
    const int kbs = min(pass_kb, all_kb - pass);
    const int rounds = (kbs + kFlight - 1) / kFlight;     // of a tile
    const float* add = pass > 0 ? out : residual;
    Codes<G, kFlight> c[2];
    auto load = [&](int tile, int round, Codes<G, kFlight>& into) {
      const int64_t row0 = int64_t(tile < tiles ? tile : 0) * 16;
      const uint32_t live = tile < tiles ? uint32_t(min(int64_t(16), n - row0)) : 0;
      load_codes<G, kFlight>(rows_at(codes, scales, row0, live, row_bytes, row_scales), row_code, row_scale,
                             uint32_t(pass + round * kFlight), kbs - round * kFlight, into);
    };
    float acc[4], added[4];
    auto compute = [&](int round, Codes<G, kFlight>& from) {
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const int kb = round * kFlight + j;
        if (kb >= kbs) continue;
        multiply<G, MT, kFlight>(from, j, xf + (size_t(kb) * 16 + g4) * cols + col,
                                 *reinterpret_cast<const float4_t*>(xs + kb * 16 + g4 * 4), cols, acc);
      }
    };
    // Lane groups 0 and 1 (MT == 8) or all four hold rows 4 g4 + r of x.
    auto begin = [&](int tile) {
      const int64_t row = int64_t(tile) * 16 + r16;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        acc[r] = 0.f;
        added[r] = add && g4 * 4 + r < m && row < n ? add[size_t(g4 * 4 + r) * size_t(n) + size_t(row)] : 0.f;
      }
    };
    auto end = [&](int tile) {
      const int64_t row = int64_t(tile) * 16 + r16;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v = acc[r];
        if constexpr (MT == 8) v += __shfl_xor(v, 32);    // hi + lo
        if (g4 * 4 + r < m && row < n) out[size_t(g4 * 4 + r) * size_t(n) + size_t(row)] = v + added[r];
      }
    };

    int tile = blockIdx.x * kWaves + wave, round = 0;
    load(tile, 0, c[0]);
    if (pass > 0) __syncthreads();                        // every wave has read x
    stage_x<G, MT>(x, m, k, int64_t(pass) * 128, kbs, xf, xs);
    __syncthreads();
    auto walk = [&](Codes<G, kFlight>& now, Codes<G, kFlight>& then) {
      const bool last = round + 1 == rounds;
      const int next = last ? tile + hop : tile, next_round = last ? 0 : round + 1;
      if (round == 0) begin(tile);
      load(next, next_round, then);
      compute(round, now);
      if (last) end(tile);
      tile = next;
      round = next_round;
    };
    while (tile < tiles) {
      walk(c[0], c[1]);
      if (tile >= tiles) break;
      walk(c[1], c[0]);
    }
  }
}

template <int G, int MT>
hipError_t launch(const Q4Args& a, hipStream_t stream) {
  const int all_kb = int(a.k >> 7);
  const int pass_kb = MT == 8 ? kWaves * kMaxKb : kWaves * kMaxKb / 2;
  // Rows over the waves once there are two tiles for each of 2048 waves; for four rows of x
  // or fewer, where two blocks on a CU hide each other's joins, once there are eight.  K split
  // and rows over the waves, K = 4096 in groups of 128 (us): 65536 rows, one of x 31.5 and 34.1,
  // eight 39.3 and 35.8; 131072, one 58.7 and 58.1, four 63.9 both ways, eight 71.0 and 64.2; 200000,
  // one 91.0 and 91.5, four 97.5 and 100.5; 262144, one 119.3 and 108.9, four 124.0 and 119.7.
  // 49152 rows, eight of x: 31.5 and 34.3.
  const bool tall = a.n >= (a.m > 4 ? 65536 : 262144);
  const size_t lds = Shape<MT>::bytes(all_kb < pass_kb ? all_kb : pass_kb, int(a.m), !tall);
  const int64_t tiles = (a.n + 15) / 16, steps = tall ? (tiles + kWaves - 1) / kWaves : tiles;
  const int per_cu = lds <= 80 * 1024 ? 2 : 1;
  const int grid = steps < 256 * per_cu ? int(steps) : 256 * per_cu;
  auto fn = tall ? q4_tall_kernel<G, MT> : q4_kernel<G, MT>;
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
  return a.m > 8 ? launch<G, 16>(a, stream) : launch<G, 8>(a, stream);
}

}  // namespace

hipError_t launch_q4_gemv(const Q4Args& a, int group, hipStream_t stream) {
  if (group == 32) return launch_group<32>(a, stream);
  if (group == 64) return launch_group<64>(a, stream);
  return launch_group<128>(a, stream);
}

}  // namespace tq2
