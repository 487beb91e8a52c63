// The chosen experts' feed-forward for a few tokens, on 4-bit or ternary weights:
//     h[p] = silu(x G_e^T) * (x U_e^T),  y[p] = w[p] h[p] D_e^T,  out[t] = residual[t] + sum of t's y
// for each pair p = (token t, place j) with e = ids[t, j].
//
// Bound.  Every touched expert's weights are read once against HBM (3 H I weights of 4.125 to 4.5 or 2.125 bits); a few
// tokens meet each of them, so that everything else is kept off that stream.
//
// Matrix form, as in the 4-bit products: one v_mfma_f32_16x16x32_f16 takes 16 weight rows as its columns and up to
// eight rows of x as hi and lo binary16 halves under a power of two per row and 128 columns; codes are decoded to exact
// binary16 integers, a group's sum meets its scale in f32, then the power of two.
//
// Work split.  Three launches: rows_kernel for gate and up (SwiGLU in its epilogue), rows_kernel for down, and the sum
// of each token's weighted rows.  A block of rows_kernel has an expert and walks over column tiles of 16; its eight
// waves are `wk` parts of K by 8 / wk tiles (gate and up tiles of the same columns side by side), whose partial sums meet
// in LDS once a step.  The expert's rows of x lie in LDS, eight at a time; the next step's codes are in flight before the
// present one is computed.
//
// Who has which expert is found by each block from ids itself (at most 2048 of them): with fewer pairs than experts a
// block row stands for a pair and works if no earlier pair has its expert, otherwise it stands for an expert.
#include "tq2_device.h"
#include "tq2_internal.h"
#include "tq2_moe_internal.h"
#include "tq2_types.h"

namespace tq2 {
namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 8;                        // rows of x in one matrix operand, beside their low halves
constexpr int kUnits = 4;                       // 64-byte pieces of a weight row that a wave has in flight
constexpr int kLds = 160 * 1024;

// A weight format: G, the columns of a scale; kBlocks, the 128-wide blocks of a row's 64 bytes.
struct Q4G32 {
  static constexpr int kGroup = 32, kBlocks = 1;
};
struct Q4G64 {
  static constexpr int kGroup = 64, kBlocks = 1;
};
struct Q4G128 {
  static constexpr int kGroup = 128, kBlocks = 1;
};
struct Ternary {
  static constexpr int kGroup = 128, kBlocks = 2;
};

// The 8 weights of one 4-bit word as exact binary16 values code - 8, in the order 0, 4, 1, 5, 2, 6, 3, 7: masks leave a
// pair of nibbles 16 bits apart in the low mantissa bits of 1024 + c or of 1024 + 16 c.
__device__ __forceinline__ half8_t decode_q4(uint32_t w) {
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

// The lower 8 codes of each half-word of a ternary word (columns 0 .. 7 of its 16; of the word moved down by a byte,
// columns 8 .. 15) as exact binary16 values code - 1.
__device__ __forceinline__ half8_t decode_ternary(uint32_t w) {
  const uint32_t magic = 0x64006400u;
  const half2_t m1 = {_Float16(0.25f), _Float16(0.25f)};
  const half2_t m2 = {_Float16(0.0625f), _Float16(0.0625f)};
  const half2_t m3 = {_Float16(0.015625f), _Float16(0.015625f)};
  const half2_t o0 = {_Float16(-1025.0f), _Float16(-1025.0f)};
  const half2_t o1 = {_Float16(-257.0f), _Float16(-257.0f)};
  const half2_t o2 = {_Float16(-65.0f), _Float16(-65.0f)};
  const half2_t o3 = {_Float16(-17.0f), _Float16(-17.0f)};
  const half2_t a = __builtin_bit_cast(half2_t, and_or(w, 0x00030003u, magic)) + o0;
  const half2_t b = __builtin_bit_cast(half2_t, and_or(w, 0x000C000Cu, magic)) * m1 + o1;
  const half2_t c = __builtin_bit_cast(half2_t, and_or(w, 0x00300030u, magic)) * m2 + o2;
  const half2_t d = __builtin_bit_cast(half2_t, and_or(w, 0x00C000C0u, magic)) * m3 + o3;
  return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Where the eight columns 8 u .. 8 u + 7 of a 128-wide block stand in the matrix steps: step and lane group, which
// follow from where a lane's 16 bytes of codes lie.
//   groups of 128: a lane's word s is step s (columns 32 g + 8 s);
//   groups of 32 and 64: after the transposition of words step s is columns 32 s + 8 g;
//   ternary: after the swap of halves lane group g has words 4 (g & 1) + 2 (g >> 1) and the next one, two steps each.
template <class F>
__device__ __forceinline__ void place_of(int u, int* step, int* grp) {
  if (F::kBlocks == 2) {
    *step = u & 3;
    *grp = u >> 3 | (u >> 1 & 2);
  } else if (F::kGroup == 128) {
    *step = u & 3;
    *grp = u >> 2;
  } else {
    *step = u >> 2;
    *grp = u & 3;
  }
}

// A lane's pieces of kUnits consecutive 64-byte units of its row, and the scales of their blocks.
template <class F>
struct Codes {
  static constexpr int kBlocks = kUnits * F::kBlocks;
  static constexpr int kScales = kBlocks * (128 / F::kGroup);      // binary16
  static constexpr int kWords = F::kGroup == 128 ? kScales / 2 + 1 : kScales / 2;
  u32x4_t w[kUnits];
  uint32_t d[kWords];                                               // kGroup == 128: from bit `down` on
  uint32_t down;
};

// Past the range of either resource: zeros.
constexpr uint32_t kNowhere = 0x80000000u;

struct Rows {
  rsrc_t codes, scales;
};

struct Weight {
  const uint8_t* codes;
  const uint16_t* scales;
  uint32_t row_bytes, row_scales;              // of one row
};

// Sixteen rows from row0 on, which all exist.
__device__ __forceinline__ Rows rows_at(const Weight& w, int64_t row0) {
  return Rows{make_rsrc(w.codes + row0 * w.row_bytes, 16 * w.row_bytes),
              make_rsrc(w.scales + row0 * w.row_scales, (16 * w.row_scales * 2 + 3) & ~3u)};
}

// Units unit .. unit + kUnits - 1 of the lane's row; `count` of them are wanted.  Every load is issued, wanted or not
// (those give zeros): behind a branch the count of loads in flight would be unknown to the waits.
template <class F>
__device__ __forceinline__ void load_codes(const Rows& rows, uint32_t row_bytes, uint32_t code_off, uint32_t scale_off,
                                           uint32_t unit, int count, uint32_t in_row, Codes<F>& c) {
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t at = (unit + j) * 64 + in_row;
    // The last half unit of a ternary row is the next row's.
    const bool ok = j < count && (F::kBlocks == 1 || at < row_bytes);
    c.w[j] = __builtin_amdgcn_raw_buffer_load_b128(rows.codes, ok ? code_off + (unit + j) * 64 : kNowhere, 0,
                                                   kStreamOnce);
  }
  const uint32_t at = count > 0 ? scale_off + unit * (F::kBlocks * 256 / F::kGroup) : kNowhere;
  if constexpr (F::kGroup == 128) {
    // Two-byte scales may start in the middle of a word, where buffer loads do not: the words around them.
    if constexpr (F::kBlocks == 1) {
      const u32x2_t d = __builtin_amdgcn_raw_buffer_load_b64(rows.scales, at & ~3u, 0, 0);
      c.d[0] = d[0];
      c.d[1] = d[1];
    } else {
      const u32x4_t d = __builtin_amdgcn_raw_buffer_load_b128(rows.scales, at & ~3u, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) c.d[i] = d[i];
    }
    c.d[Codes<F>::kWords - 1] =
        __builtin_amdgcn_raw_buffer_load_b32(rows.scales, (at & ~3u) + (Codes<F>::kWords - 1) * 4, 0, 0);
    c.down = (at & 2) * 8;
  } else {
#pragma unroll
    for (int i = 0; i < Codes<F>::kWords / 4; ++i) {
      const u32x4_t d = __builtin_amdgcn_raw_buffer_load_b128(rows.scales, at + i * 16, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) c.d[4 * i + e] = d[e];
    }
  }
}

// The scale of 32-wide step s of block b.
template <class F>
__device__ __forceinline__ float scale_of(const Codes<F>& c, int b, int s) {
  const int i = b * (128 / F::kGroup) + s / (F::kGroup / 32);
  uint32_t w = c.d[i >> 1];
  if constexpr (F::kGroup == 128) w = __builtin_amdgcn_alignbit(c.d[(i >> 1) + 1], w, c.down);
  return float(__builtin_bit_cast(_Float16, uint16_t(w >> (16 * (i & 1)))));
}

// Lane groups exchange words so that each step stays inside one scale's columns.
template <class F>
__device__ __forceinline__ void arrange(u32x4_t& w) {
  if constexpr (F::kBlocks == 2) {
    // Afterwards words 0 and 1 are of the unit's first block in all lanes, 2 and 3 of its second.
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    w = u32x4_t{a[0], b[0], a[1], b[1]};
  } else if constexpr (F::kGroup != 128) {
    // Lane group g holds in word s what lane group s held in word g.
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = u32x4_t{c[0], c[1], d[0], d[1]};
  }
}

// Block b of unit j (b < F::kBlocks): four matrix steps against x, scaled into acc (rows 4 g4 + r of x, weight row r16).
template <class F>
__device__ __forceinline__ void multiply(const Codes<F>& c, int j, int b, const half8_t* __restrict__ a,
                                         const float4_t& back, int cols, float (&acc)[4]) {
  float4_t sum;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const half8_t a0 = a[size_t(s) * 4 * cols];
    half8_t w;
    if constexpr (F::kBlocks == 2) {
      const uint32_t word = c.w[j][2 * b + (s >> 1)];
      w = decode_ternary(s & 1 ? word >> 8 : word);
    } else {
      w = decode_q4(c.w[j][s]);
    }
    const bool fresh = s % (F::kGroup / 32) == 0;
    const bool whole = (s + 1) % (F::kGroup / 32) == 0;
    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, w, fresh ? float4_t{0.f, 0.f, 0.f, 0.f} : sum, 0, 0, 0);
    if (whole) {
      const float d = scale_of<F>(c, j * F::kBlocks + b, s);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(d * sum[r], back[r], acc[r]);
    }
  }
}

// Largest |x| over aligned groups of 16 lanes, in every lane.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_move<0xB1, 0xF>(v));
  v = fmaxf(v, dpp_move<0x4E, 0xF>(v));
  v = fmaxf(v, dpp_move<0x141, 0xF>(v));
  v = fmaxf(v, dpp_move<0x140, 0xF>(v));
  return v;
}

// Operand words from one lane group's columns to the next's; an odd number keeps the lanes that write a stretch of x
// off each other's banks.
__host__ __device__ inline int columns_of(int m) { return m > 4 ? 2 * m + 1 : 2 * m; }
// Bytes of LDS for m rows of `blocks` 128-wide blocks: operands and powers of two.
__host__ __device__ inline int x_bytes(int blocks, int m) { return blocks * (256 * columns_of(m) + 4 * 2 * kRows); }
constexpr int kRedBytes = 2 * kWaves * kRows * 16 * 4;

// Convert m rows of x (row i at x + row_of(i) * stride) into LDS.  Sixteen consecutive threads hold one row's 128
// columns, so the power of two of that stretch is a DPP maximum: 2^13 <= |x| 2^e < 2^14.
template <class F, class X, class RowOf>
__device__ __forceinline__ void stage_x(const typename X::elem* __restrict__ x, int64_t stride, RowOf row_of, int m,
                                        int blocks, half8_t* __restrict__ xf, float* __restrict__ xs) {
  const int cols = columns_of(m);
  for (int i = threadIdx.x; i < m * blocks * 16; i += kThreads) {
    const int u = i & 15, kb = (i >> 4) % blocks, row = (i >> 4) / blocks;
    const typename X::elem* src = x + row_of(row) * stride + kb * 128 + u * 8;
    const f32x4_t p = load4(X(), src), q = load4(X(), src + 4);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[F::kBlocks == 2 ? j : 2 * j] = p[j];                     // the order of the decoded codes
      v[F::kBlocks == 2 ? j + 4 : 2 * j + 1] = q[j];
    }
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
    int step, grp;
    place_of<F>(u, &step, &grp);
    half8_t* dst = xf + (size_t(kb * 4 + step) * 4 + grp) * cols + row;
    dst[0] = hi;
    dst[m] = lo;
    if (u == 0) {
      const float back = __builtin_ldexpf(1.0f, -up);
      xs[kb * 16 + row] = back;
      xs[kb * 16 + kRows + row] = back;
    }
  }
}

struct Shape {
  int pairs, top_k, experts;
  int rows;                  // of x in LDS at a time
  int blocks;                // 128-wide blocks of K
  int tiles;                 // column tiles of an expert (of gate, and as many of up)
  int wk;                    // parts of K
  bool by_pair;
};

// GATE: x are the tokens' rows, out the rows between the projections, f32 [pairs, 16 tiles].  Otherwise x are those
// and out the weighted rows, f32 [pairs, 16 tiles].
template <class F, class X, bool GATE>
__global__ __launch_bounds__(kThreads, 2) void rows_kernel(Weight weight, const typename X::elem* __restrict__ x,
                                                           const int32_t* __restrict__ ids,
                                                           const float* __restrict__ share, float* __restrict__ out,
                                                           Shape sh) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ uint16_t list[TQ2_MOE_MAX_TOKENS * TQ2_MOE_MAX_TOP_K];
  __shared__ int counts[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const int e = __builtin_amdgcn_readfirstlane(sh.by_pair ? ids[blockIdx.y] : int(blockIdx.y));
  if (uint32_t(e) >= uint32_t(sh.experts)) return;

  // The wave's part: a tile of each step, and units of K.
  const int units = (sh.blocks + F::kBlocks - 1) / F::kBlocks;
  const int wn = kWaves / sh.wk, slot = wave / sh.wk, part = wave % sh.wk;
  const int part_units = (units + sh.wk - 1) / sh.wk;
  const int unit0 = part * part_units, mine = max(0, min(part_units, units - unit0));
  const int rounds = (part_units + kUnits - 1) / kUnits, per = (part_units + rounds - 1) / rounds;
  const int per_step = GATE ? wn / 2 : wn;
  const int steps = sh.tiles / per_step;
  const int64_t width = int64_t(sh.tiles) * 16;
  const int64_t expert_row = int64_t(e) * width * (GATE ? 2 : 1);
  const uint32_t code_off = r16 * weight.row_bytes + g4 * 16, scale_off = r16 * weight.row_scales * 2;

  Codes<F> c[2];
  auto load = [&](int step, int round, Codes<F>& into) {
    const bool there = step < steps;
    const int64_t tile = int64_t(there ? step : 0) * per_step + (GATE ? slot >> 1 : slot);
    const int64_t row0 = expert_row + (GATE && (slot & 1) ? width : 0) + tile * 16;
    load_codes<F>(rows_at(weight, row0), weight.row_bytes, code_off, scale_off, uint32_t(unit0 + round * per),
                  there ? min(per, mine - round * per) : 0, g4 * 16, into);
  };
  int step = blockIdx.x, round = 0;
  load(step, 0, c[0]);                                   // in flight while the rows are found and converted

  // The pairs of this expert, in order.
  int found = 0;
  for (int p0 = 0; p0 < sh.pairs; p0 += kThreads) {
    const int p = p0 + threadIdx.x;
    const bool here = p < sh.pairs && ids[p] == e;
    const uint64_t all = __ballot(here);
    if (lane == 0) counts[wave] = __popcll(all);
    __syncthreads();
    int at = found;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) at += counts[w];
      found += counts[w];
    }
    if (here) list[at + __popcll(all & ((uint64_t(1) << lane) - 1))] = uint16_t(p);
    __syncthreads();
  }
  if (found == 0 || (sh.by_pair && list[0] != blockIdx.y)) return;

  half8_t* xf = reinterpret_cast<half8_t*>(smem);
  float* xs = reinterpret_cast<float*>(smem + sh.blocks * 256 * columns_of(sh.rows));
  float* red = reinterpret_cast<float*>(smem + x_bytes(sh.blocks, sh.rows));

  for (int first = 0; first < found; first += sh.rows) {
    const int m = min(sh.rows, found - first), cols = columns_of(m);
    if (first > 0) {
      step = blockIdx.x;
      round = 0;
      load(step, 0, c[0]);
      __syncthreads();                                   // the last step has read x and red
    }
    stage_x<F, X>(x, GATE ? int64_t(sh.blocks) * 128 : int64_t(sh.blocks) * 128,
                  [&](int i) { return int64_t(GATE ? list[first + i] / sh.top_k : list[first + i]); }, m, sh.blocks, xf,
                  xs);
    __syncthreads();
    const int col = (r16 & 7) < m ? (r16 >> 3) * m + (r16 & 7) : 0;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int parity = 0;
    auto compute = [&](Codes<F>& from) {
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        const int unit = unit0 + round * per + j;
        if (j >= per || round * per + j >= mine) continue;
        arrange<F>(from.w[j]);
#pragma unroll
        for (int b = 0; b < F::kBlocks; ++b) {
          const int kb = unit * F::kBlocks + b;
          if (F::kBlocks > 1 && kb >= sh.blocks) continue;
          multiply<F>(from, j, b, xf + (size_t(kb) * 16 + g4) * cols + col,
                      *reinterpret_cast<const float4_t*>(xs + kb * 16 + g4 * 4), cols, acc);
        }
      }
    };
    // Partial sums [wave][row of x][weight row] of a step meet; a buffer is written again two steps on, behind the
    // next step's barrier.
    auto finish = [&]() {
      float* buf = red + parity * (kWaves * kRows * 16);
      parity ^= 1;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = acc[r] + __shfl_xor(acc[r], 32);              // hi + lo
        acc[r] = 0.f;
        if (g4 < 2) buf[(wave * kRows + g4 * 4 + r) * 16 + r16] = v;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < per_step * kRows * 16; i += kThreads) {
        const int n = i & 15, row = i >> 4 & (kRows - 1), tile = i >> 7;
        if (row >= m) continue;
        const int p = list[first + row];
        const float* at = buf + row * 16 + n;
        float a = 0.f, b = 0.f;
        for (int w = 0; w < sh.wk; ++w) {
          a += at[((GATE ? 2 * tile : tile) * sh.wk + w) * (kRows * 16)];
          if (GATE) b += at[((2 * tile + 1) * sh.wk + w) * (kRows * 16)];
        }
        const float v = GATE ? a / (1.f + expf(-a)) * b : a * share[p];
        out[p * width + (int64_t(step) * per_step + tile) * 16 + n] = v;
      }
    };
    auto walk = [&](Codes<F>& now, Codes<F>& then) {
      const bool last = round + 1 == rounds;
      const int next = last ? step + int(gridDim.x) : step, next_round = last ? 0 : round + 1;
      load(next, next_round, then);
      compute(now);
      if (last) finish();
      step = next;
      round = next_round;
    };
    while (step < steps) {
      walk(c[0], c[1]);
      if (step >= steps) break;
      walk(c[1], c[0]);
    }
  }
}

// out[t] = residual[t] + the token's weighted rows in the order of their places; four columns a thread.
template <class X>
__global__ __launch_bounds__(256) void sum_kernel(const float* __restrict__ y, const int32_t* __restrict__ ids,
                                                  const typename X::elem* residual, typename X::elem* out, int top_k,
                                                  int experts, int hidden) {
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
  if (n >= hidden) return;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < top_k; ++j) {
    const int p = t * top_k + j;
    if (uint32_t(ids[p]) < uint32_t(experts)) sum += load4(F32(), y + size_t(p) * hidden + n);
  }
  if (residual) sum += load4(X(), residual + size_t(t) * hidden + n);
  store4(X(), out + size_t(t) * hidden + n, sum);
}

// Parts of K: as many as keep a wave's share at kUnits units, or all waves (half of them where gate and up share the
// block).
template <class F>
int parts_of(int blocks, int most) {
  const int units = (blocks + F::kBlocks - 1) / F::kBlocks;
  int wk = 1;
  while (wk < most && wk * kUnits < units) wk *= 2;
  return wk;
}

template <class F, class X, bool GATE>
hipError_t launch_rows(const tq2_moe_experts_args& a, const Weight& w, const void* x, float* out, int64_t n, int64_t k,
                       hipStream_t stream) {
  Shape s;
  s.pairs = int(a.tokens * a.top_k);
  s.top_k = int(a.top_k);
  s.experts = int(a.experts);
  s.blocks = int(k / 128);
  s.tiles = int(n / 16);
  s.wk = parts_of<F>(s.blocks, GATE ? kWaves / 2 : kWaves);
  s.by_pair = s.pairs < s.experts;
  // Rows of x at a time: no more than an expert can have, as many as LDS holds beside the list and the sums.
  s.rows = s.pairs < kRows ? s.pairs : kRows;
  const int room = kLds - kRedBytes - TQ2_MOE_MAX_TOKENS * TQ2_MOE_MAX_TOP_K * 2 - 64;
  while (x_bytes(s.blocks, s.rows) > room) --s.rows;
  const int lds = x_bytes(s.blocks, s.rows) + kRedBytes;
  const int per_step = (kWaves / s.wk) / (GATE ? 2 : 1), steps = s.tiles / per_step;
  const int experts = s.by_pair ? s.pairs : s.experts;
  int across = (1024 + experts - 1) / experts;
  if (across > steps) across = steps;
  auto fn = rows_kernel<F, X, GATE>;
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3(across, experts), dim3(kThreads), lds, stream, w,
                     static_cast<const typename X::elem*>(x), a.ids, a.weights, out, s);
  return hipGetLastError();
}

template <class F>
Weight weight_of(const void* codes, const void* scales, int64_t rows, int64_t k) {
  Weight w;
  w.codes = static_cast<const uint8_t*>(codes);
  w.row_bytes = uint32_t(F::kBlocks == 2 ? k / 4 : k / 2);
  w.row_scales = uint32_t(k / F::kGroup);
  w.scales = reinterpret_cast<const uint16_t*>(F::kBlocks == 2 ? w.codes + scales_offset(rows, k)
                                                               : static_cast<const uint8_t*>(scales));
  return w;
}

template <class F, class X>
hipError_t launch(const tq2_moe_experts_args& a, const MoePlan& plan, hipStream_t stream) {
  float* h = static_cast<float*>(a.workspace);
  float* y = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + plan.y_offset);
  hipError_t e = launch_rows<F, X, true>(a, weight_of<F>(a.gate_up, a.gate_up_scales, 2 * a.experts * a.inter, a.hidden),
                                         a.x, h, a.inter, a.hidden, stream);
  if (e != hipSuccess) return e;
  e = launch_rows<F, F32, false>(a, weight_of<F>(a.down, a.down_scales, a.experts * a.hidden, a.inter), h, y, a.hidden,
                                 a.inter, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sum_kernel<X>, dim3((a.hidden + 1023) / 1024, a.tokens), dim3(256), 0, stream, y, a.ids,
                     static_cast<const typename X::elem*>(a.residual), static_cast<typename X::elem*>(a.out),
                     int(a.top_k), int(a.experts), int(a.hidden));
  return hipGetLastError();
}

template <class F>
hipError_t launch(const tq2_moe_experts_args& a, const MoePlan& plan, hipStream_t stream) {
  if (a.act_type == TQ2_TYPE_F32) return launch<F, F32>(a, plan, stream);
  if (a.act_type == TQ2_TYPE_F16) return launch<F, F16>(a, plan, stream);
  return launch<F, BF16>(a, plan, stream);
}

}  // namespace

MoePlan plan_moe(const tq2_moe_experts_args& a) {
  MoePlan p;
  p.y_offset = align256(size_t(a.tokens) * size_t(a.top_k) * size_t(a.inter) * 4);
  p.workspace = p.y_offset + size_t(a.tokens) * size_t(a.top_k) * size_t(a.hidden) * 4;
  return p;
}

hipError_t launch_moe_experts(const tq2_moe_experts_args& a, const MoePlan& plan, hipStream_t stream) {
  if (a.format == TQ2_MOE_TERNARY) return launch<Ternary>(a, plan, stream);
  if (a.group == 32) return launch<Q4G32>(a, plan, stream);
  if (a.group == 64) return launch<Q4G64>(a, plan, stream);
  return launch<Q4G128>(a, plan, stream);
}

}  // namespace tq2
