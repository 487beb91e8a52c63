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

// The masked bits of a word in binary16 mantissas.  Not in inline asm: the compiler keeps instructions that it knows, but
// not asm, off the result registers of a matrix instruction in flight whose values nobody reads.
__device__ __forceinline__ half2_t mantissas(uint32_t w, uint32_t mask) {
  return __builtin_bit_cast(half2_t, (w & mask) | 0x64006400u);
}

// The 8 weights of one 4-bit word as exact binary16 values code - 8, in the order 0, 4, 1, 5, 2, 6, 3, 7: masks leave a
// pair of nibbles 16 bits apart in the low mantissa bits of 1024 + c or of 1024 + 16 c.
__device__ __forceinline__ half8_t decode_q4(uint32_t w) {
  const half2_t one16 = {_Float16(0.0625f), _Float16(0.0625f)};
  const half2_t off16 = {_Float16(-72.0f), _Float16(-72.0f)};
  const half2_t off1 = {_Float16(-1032.0f), _Float16(-1032.0f)};
  const uint32_t v = w >> 8;
  const half2_t a = mantissas(w, 0x000F000Fu) + off1;
  const half2_t b = mantissas(w, 0x00F000F0u) * one16 + off16;
  const half2_t c = mantissas(v, 0x000F000Fu) + off1;
  const half2_t d = mantissas(v, 0x00F000F0u) * one16 + off16;
  return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The lower 8 codes of each half-word of a ternary word (columns 0 .. 7 of its 16; of the word moved down by a byte,
// columns 8 .. 15) as exact binary16 values code - 1.
__device__ __forceinline__ half8_t decode_ternary(uint32_t w) {
  const half2_t m1 = {_Float16(0.25f), _Float16(0.25f)};
  const half2_t m2 = {_Float16(0.0625f), _Float16(0.0625f)};
  const half2_t m3 = {_Float16(0.015625f), _Float16(0.015625f)};
  const half2_t o0 = {_Float16(-1025.0f), _Float16(-1025.0f)};
  const half2_t o1 = {_Float16(-257.0f), _Float16(-257.0f)};
  const half2_t o2 = {_Float16(-65.0f), _Float16(-65.0f)};
  const half2_t o3 = {_Float16(-17.0f), _Float16(-17.0f)};
  const half2_t a = mantissas(w, 0x00030003u) + o0;
  const half2_t b = mantissas(w, 0x000C000Cu) * m1 + o1;
  const half2_t c = mantissas(w, 0x00300030u) * m2 + o2;
  const half2_t d = mantissas(w, 0x00C000C0u) * m3 + o3;
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

// How rows of x fill the matrix operands.
enum Mode {
  kPacked,                                      // 8 rows as hi, and their lo as 8 more
  kHigh,                                        // 16 rows as hi: 16-bit values need no lo
  kBoth                                         // 16 rows as hi, and lo as an operand of its own
};
template <Mode M>
constexpr int kRowsOf = M == kPacked ? 8 : 16;

// Operand words from one lane group's columns to the next's; an odd number keeps the lanes that write a stretch of x
// off each other's banks.
template <Mode M>
__host__ __device__ inline int columns_of(int m) {
  const int n = M == kHigh ? m : 2 * m;
  return m > 4 ? n | 1 : n;
}
// Bytes of LDS for m rows of `blocks` 128-wide blocks (operands and powers of two), and for partial sums.
template <Mode M>
__host__ __device__ inline int x_bytes(int blocks, int m) { return blocks * (256 * columns_of<M>(m) + 64); }
template <Mode M>
constexpr int kRedBytes = 2 * kWaves * kRowsOf<M> * 16 * 4;

// The column of the matrix operand x that the lane's row reads.
template <Mode M>
__device__ __forceinline__ int operand_column(int r16, int m) {
  if (M == kPacked) return (r16 & 7) < m ? (r16 >> 3) * m + (r16 & 7) : 0;
  return r16 < m ? r16 : 0;
}

// Block b of unit j (b < F::kBlocks): four matrix steps against x, scaled into acc (rows 4 g4 + r of x, weight row r16).
template <class F, Mode M>
__device__ __forceinline__ void multiply(const Codes<F>& c, int j, int b, const half8_t* __restrict__ a,
                                         const float4_t& back, int cols, int m, float (&acc)[4]) {
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
    if constexpr (M == kBoth)
      sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[size_t(s) * 4 * cols + m], w, sum, 0, 0, 0);
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

// Convert eight columns (the u-th eight of 128-wide block kb) of row `row` of m into LDS.  The sixteen lanes of a block
// call together: their power of two is a DPP maximum, 2^13 <= |x| 2^e < 2^14.  `share` multiplies the row.
template <class F, Mode M, class X>
__device__ __forceinline__ void stage8(const typename X::elem* __restrict__ src, int u, int kb, int row, int m, int cols,
                                       float share, half8_t* __restrict__ xf, float* __restrict__ xs) {
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
  if (M != kHigh) dst[m] = lo;
  if (u == 0) {
    const float back = __builtin_ldexpf(1.0f, -up) * share;
    xs[kb * 16 + row] = back;
    if (M == kPacked) xs[kb * 16 + 8 + row] = back;
  }
}

// One launch of rows_kernel; all of it follows from the sizes.
struct Shape {
  int pairs, top_k, experts;
  uint32_t top_k_inverse;    // pair * top_k_inverse >> 16 is its token
  int rows;                  // of x in LDS at a time
  int blocks;                // 128-wide blocks of K
  uint32_t blocks_inverse;   // i * blocks_inverse >> 20 is i / blocks
  int units;                 // 64-byte pieces of a weight row
  int tiles;                 // column tiles of an expert (of gate, and as many of up)
  int wk_shift;              // log2 of the parts of K
  int part_units, rounds, per;         // units of a part, its rounds, units of a round
  int steps;                 // of column tiles that the block's waves take together
  bool by_pair;
};

// GATE: x are the tokens' rows, out the rows between the projections, f32 [pairs, 16 tiles].  Otherwise x are those
// and out the weighted rows, f32 [pairs, 16 tiles].
template <class F, class X, bool GATE, Mode M>
__global__ __launch_bounds__(kThreads, 2) void rows_kernel(Weight weight, const typename X::elem* __restrict__ x,
                                                           const int32_t* __restrict__ ids,
                                                           const float* __restrict__ share, float* __restrict__ out,
                                                           Shape sh) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int kRows = kRowsOf<M>;
  half8_t* xf = reinterpret_cast<half8_t*>(smem);
  float* xs = reinterpret_cast<float*>(smem + sh.blocks * 256 * columns_of<M>(sh.rows));
  float* red = reinterpret_cast<float*>(smem + x_bytes<M>(sh.blocks, sh.rows));
  int* counts = reinterpret_cast<int*>(smem + x_bytes<M>(sh.blocks, sh.rows) + kRedBytes<M>);
  uint16_t* list = reinterpret_cast<uint16_t*>(counts + kWaves);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const bool few = sh.pairs <= 64;                       // ids of all pairs in one load
  const int id = few && lane < sh.pairs ? ids[lane] : -1;
  const int e = !sh.by_pair ? int(blockIdx.y)
                : few       ? __builtin_amdgcn_readlane(id, blockIdx.y)
                            : __builtin_amdgcn_readfirstlane(ids[blockIdx.y]);
  if (uint32_t(e) >= uint32_t(sh.experts)) return;
  const uint64_t mask = __ballot(id == e);
  if (few && (mask == 0 || (sh.by_pair && __builtin_ctzll(mask) != int(blockIdx.y)))) return;

  // The wave's part: a tile of each step, and units of K.
  const int slot = wave >> sh.wk_shift, part = wave & ((1 << sh.wk_shift) - 1);
  const int unit0 = part * sh.part_units, mine = min(sh.part_units, sh.units - unit0);
  const int per_step = (kWaves >> sh.wk_shift) >> (GATE ? 1 : 0);
  const int64_t width = int64_t(sh.tiles) * 16;
  const int64_t expert_row = int64_t(e) * width * (GATE ? 2 : 1);
  const uint32_t code_off = r16 * weight.row_bytes + g4 * 16, scale_off = r16 * weight.row_scales * 2;

  Codes<F> c[2];
  auto load = [&](int step, int round, Codes<F>& into) {
    const bool there = step < sh.steps;
    const int64_t tile = int64_t(there ? step : 0) * per_step + (GATE ? slot >> 1 : slot);
    const int64_t row0 = expert_row + (GATE && (slot & 1) ? width : 0) + tile * 16;
    load_codes<F>(rows_at(weight, row0), weight.row_bytes, code_off, scale_off, uint32_t(unit0 + round * sh.per),
                  there ? min(sh.per, mine - round * sh.per) : 0, g4 * 16, into);
  };
  int step = blockIdx.x, round = 0;
  load(step, 0, c[0]);                                   // in flight while the rows are found and converted

  // The pairs of this expert, in order.
  int found = 0;
  if (few) {
    found = __popcll(mask);
    if (id == e) list[__popcll(mask & ((uint64_t(1) << lane) - 1))] = uint16_t(lane);    // by every wave, for itself
    __builtin_amdgcn_wave_barrier();
  } else {
    for (int p0 = 0; p0 < sh.pairs; p0 += kThreads) {
      const int p = p0 + threadIdx.x;
      const bool here = p < sh.pairs && ids[p] == e;
      const uint64_t all = __ballot(here);
      if (lane == 0) counts[wave] = __popcll(all);
      __syncthreads();
      int at = found;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        at += w < wave ? counts[w] : 0;
        found += counts[w];
      }
      if (here) list[at + __popcll(all & ((uint64_t(1) << lane) - 1))] = uint16_t(p);
      __syncthreads();
    }
    if (found == 0 || (sh.by_pair && list[0] != blockIdx.y)) return;
  }

  for (int first = 0; first < found; first += sh.rows) {
    const int m = min(sh.rows, found - first), cols = columns_of<M>(m);
    if (first > 0) {
      step = blockIdx.x;
      round = 0;
      load(step, 0, c[0]);
      __syncthreads();                                   // the last step has read x and red
    }
    for (int i = threadIdx.x; i < m * sh.blocks * 16; i += kThreads) {
      const int row = int((uint32_t(i >> 4) * sh.blocks_inverse) >> 20), kb = (i >> 4) - row * sh.blocks;
      const uint32_t pair = list[first + row], from = GATE ? pair * sh.top_k_inverse >> 16 : pair;
      stage8<F, M, X>(x + (int64_t(from) * sh.blocks + kb) * 128 + (i & 15) * 8, i & 15, kb, row, m, cols, 1.f, xf, xs);
    }
    __syncthreads();
    const int col = operand_column<M>(r16, m);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int parity = 0;
    auto compute = [&](Codes<F>& from) {
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        const int unit = unit0 + round * sh.per + j;
        if (j >= sh.per || round * sh.per + j >= mine) continue;
        arrange<F>(from.w[j]);
#pragma unroll
        for (int b = 0; b < F::kBlocks; ++b) {
          const int kb = unit * F::kBlocks + b;
          if (F::kBlocks > 1 && kb >= sh.blocks) continue;
          multiply<F, M>(from, j, b, xf + (size_t(kb) * 16 + g4) * cols + col,
                         *reinterpret_cast<const float4_t*>(xs + kb * 16 + g4 * 4), cols, m, acc);
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
        float v = acc[r];
        if (M == kPacked) v += __shfl_xor(v, 32);                     // hi + lo
        acc[r] = 0.f;
        if (M != kPacked || g4 < 2) buf[(wave * kRows + g4 * 4 + r) * 16 + r16] = v;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < per_step * kRows * 16; i += kThreads) {
        const int n = i & 15, row = i >> 4 & (kRows - 1), tile = i / (16 * kRows);
        if (row >= m) continue;
        const int p = list[first + row];
        const float* at = buf + row * 16 + n;
        float a = 0.f, b = 0.f;
        for (int w = 0; w < 1 << sh.wk_shift; ++w) {
          a += at[(((GATE ? 2 * tile : tile) << sh.wk_shift) + w) * (kRows * 16)];
          if (GATE) b += at[(((2 * tile + 1) << sh.wk_shift) + w) * (kRows * 16)];
        }
        const float v = GATE ? a / (1.f + expf(-a)) * b : a * share[p];
        out[p * width + (int64_t(step) * per_step + tile) * 16 + n] = v;
      }
    };
    auto walk = [&](Codes<F>& now, Codes<F>& then) {
      const bool last = round + 1 == sh.rounds;
      const int next = last ? step + int(gridDim.x) : step, next_round = last ? 0 : round + 1;
      load(next, next_round, then);
      compute(now);
      if (last) finish();
      step = next;
      round = next_round;
    };
    while (step < sh.steps) {
      walk(c[0], c[1]);
      if (step >= sh.steps) break;
      walk(c[1], c[0]);
    }
  }
}

// Down and the sum over a token's experts at once, for few tokens: a block has a token and a tile of 16 columns, its
// waves take rounds of units over all of the token's places in turn, and their sums meet in LDS.  An expert that several
// tokens chose is read for each of them.
template <class F, class X>
__global__ __launch_bounds__(kThreads, 2) void token_kernel(Weight weight, const float* __restrict__ h,
                                                            const int32_t* __restrict__ ids,
                                                            const float* __restrict__ share,
                                                            const typename X::elem* residual, typename X::elem* out,
                                                            Shape sh) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ float red[kWaves][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4, t = blockIdx.y;
  constexpr int kCols = 2;
  const int all_blocks = sh.top_k * sh.blocks;
  half8_t* xf = reinterpret_cast<half8_t*>(smem);
  float* xs = reinterpret_cast<float*>(smem + all_blocks * 256 * kCols);
  const int id = lane < sh.top_k ? ids[t * sh.top_k + lane] : -1;
  const float part = lane < sh.top_k ? share[t * sh.top_k + lane] : 0.f;
  const uint32_t code_off = r16 * weight.row_bytes + g4 * 16, scale_off = r16 * weight.row_scales * 2;
  const int64_t hidden = int64_t(sh.tiles) * 16;

  // Round r is part r % rounds of place r / rounds; the wave has rounds wave, wave + kWaves, ...
  const int all_rounds = sh.top_k * sh.rounds;
  Codes<F> c[2];
  int place = 0, round = wave;                           // of the round that is loaded next
  auto settle = [&]() {
    while (round >= sh.rounds && place < sh.top_k) round -= sh.rounds, ++place;
  };
  struct At {
    int place, unit, count;
  };
  auto load = [&](Codes<F>& into) {
    settle();
    const bool there = place < sh.top_k;
    const int e = __builtin_amdgcn_readlane(id, there ? place : 0);
    const bool real = there && uint32_t(e) < uint32_t(sh.experts);
    const At at = {place, round * sh.per, real ? min(sh.per, sh.units - round * sh.per) : 0};
    load_codes<F>(rows_at(weight, (real ? int64_t(e) * hidden : 0) + int64_t(blockIdx.x) * 16), weight.row_bytes,
                  code_off, scale_off, uint32_t(at.unit), at.count, g4 * 16, into);
    round += kWaves;
    return at;
  };
  At now = load(c[0]);
  for (int i = threadIdx.x; i < all_blocks * 16; i += kThreads) {
    const int kb = i >> 4, j = int((uint32_t(kb) * sh.blocks_inverse) >> 20);
    stage8<F, kPacked, F32>(h + (int64_t(t) * all_blocks + kb) * 128 + (i & 15) * 8, i & 15, kb, 0, 1, kCols,
                            __shfl(part, j), xf, xs);
  }
  __syncthreads();
  const int col = operand_column<kPacked>(r16, 1);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  auto compute = [&](Codes<F>& from, const At& at) {
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      if (j >= at.count) continue;
      arrange<F>(from.w[j]);
#pragma unroll
      for (int b = 0; b < F::kBlocks; ++b) {
        const int k = (at.unit + j) * F::kBlocks + b, kb = at.place * sh.blocks + k;
        if (F::kBlocks > 1 && k >= sh.blocks) continue;
        multiply<F, kPacked>(from, j, b, xf + (size_t(kb) * 16 + g4) * kCols + col,
                             *reinterpret_cast<const float4_t*>(xs + kb * 16 + g4 * 4), kCols, 1, acc);
      }
    }
  };
  for (int done = wave; done < all_rounds;) {
    const At then = load(c[1]);
    compute(c[0], now);
    done += kWaves;
    if (done >= all_rounds) break;
    now = load(c[0]);
    compute(c[1], then);
    done += kWaves;
  }
  const float v = acc[0] + __shfl_xor(acc[0], 32);       // row 0: hi of lane group 0, lo of lane group 2
  if (g4 == 0) red[wave][r16] = v;
  __syncthreads();
  if (threadIdx.x < 16) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += red[w][threadIdx.x];
    const int64_t at = int64_t(t) * hidden + int64_t(blockIdx.x) * 16 + threadIdx.x;
    if (residual) sum += float(residual[at]);
    out[at] = typename X::elem(sum);
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

// The launch for n columns and k of K over `most` parts of it.
template <class F>
Shape shape_of(const tq2_moe_experts_args& a, int64_t n, int64_t k, int most, bool gate) {
  Shape s;
  s.pairs = int(a.tokens * a.top_k);
  s.top_k = int(a.top_k);
  s.experts = int(a.experts);
  s.top_k_inverse = uint32_t((65536 + a.top_k - 1) / a.top_k);
  s.blocks = int(k / 128);
  s.blocks_inverse = uint32_t(((1 << 20) + s.blocks - 1) / s.blocks);
  s.units = (s.blocks + F::kBlocks - 1) / F::kBlocks;
  s.tiles = int(n / 16);
  // Parts of K: as many as keep a wave's share at kUnits units.
  s.wk_shift = 0;
  while ((1 << s.wk_shift) < most && (kUnits << s.wk_shift) < s.units) ++s.wk_shift;
  s.part_units = (s.units + (1 << s.wk_shift) - 1) >> s.wk_shift;
  s.rounds = (s.part_units + kUnits - 1) / kUnits;
  s.per = (s.part_units + s.rounds - 1) / s.rounds;
  s.steps = s.tiles / ((kWaves >> s.wk_shift) >> (gate ? 1 : 0));
  s.by_pair = s.pairs < s.experts;
  return s;
}

hipError_t allow_lds(const void* fn, int lds) {
  return lds <= 48 * 1024 ? hipSuccess
                          : hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

// LDS of rows_kernel beside x: partial sums, the list of pairs and its counts.
template <Mode M>
int rest_bytes(int pairs) { return kRedBytes<M> + (kWaves * 4 + pairs * 2 + 15) / 16 * 16; }

// Rows of x at a time: no more than an expert can have, as many as LDS holds.
template <Mode M>
int rows_at_once(int pairs, int blocks) {
  int rows = pairs < kRowsOf<M> ? pairs : kRowsOf<M>;
  while (x_bytes<M>(blocks, rows) + rest_bytes<M>(pairs) > kLds) --rows;
  return rows;
}

template <class F, class X, bool GATE, Mode M>
hipError_t launch_rows(const tq2_moe_experts_args& a, const Weight& w, const void* x, float* out, int64_t n, int64_t k,
                       hipStream_t stream) {
  Shape s = shape_of<F>(a, n, k, GATE ? kWaves / 2 : kWaves, GATE);
  s.rows = rows_at_once<M>(s.pairs, s.blocks);
  const int lds = x_bytes<M>(s.blocks, s.rows) + rest_bytes<M>(s.pairs);
  const int experts = s.by_pair ? s.pairs : s.experts;
  int across = (1024 + experts - 1) / experts;
  if (across > s.steps) across = s.steps;
  const auto fn = rows_kernel<F, X, GATE, M>;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(across, experts), dim3(kThreads), lds, stream, w,
                     static_cast<const typename X::elem*>(x), a.ids, a.weights, out, s);
  return hipGetLastError();
}

// Up to 16 rows of f32 at a time where experts have more than 8 and LDS holds more.
bool many_rows(const tq2_moe_experts_args& a, int64_t k) {
  return a.tokens * a.top_k > 6 * a.experts && rows_at_once<kBoth>(int(a.tokens * a.top_k), int(k / 128)) > 8;
}

// LDS of token_kernel, whose blocks hold all of a token's rows.
int token_lds(const tq2_moe_experts_args& a) { return x_bytes<kPacked>(int(a.top_k * (a.inter / 128)), 1); }

bool by_token(const tq2_moe_experts_args& a) {
  return a.tokens * a.top_k <= 32 && token_lds(a) + kWaves * 64 <= kLds;
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
  const Weight up = weight_of<F>(a.gate_up, a.gate_up_scales, 2 * a.experts * a.inter, a.hidden);
  const Weight down = weight_of<F>(a.down, a.down_scales, a.experts * a.hidden, a.inter);
  hipError_t e;
  if constexpr (sizeof(typename X::elem) == 2) {
    e = launch_rows<F, X, true, kHigh>(a, up, a.x, h, a.inter, a.hidden, stream);
  } else {
    e = many_rows(a, a.hidden) ? launch_rows<F, X, true, kBoth>(a, up, a.x, h, a.inter, a.hidden, stream)
                               : launch_rows<F, X, true, kPacked>(a, up, a.x, h, a.inter, a.hidden, stream);
  }
  if (e != hipSuccess) return e;
  const auto* residual = static_cast<const typename X::elem*>(a.residual);
  auto* out = static_cast<typename X::elem*>(a.out);
  if (by_token(a)) {
    const Shape s = shape_of<F>(a, a.hidden, a.inter, 1, false);
    const auto fn = token_kernel<F, X>;
    e = allow_lds(reinterpret_cast<const void*>(fn), token_lds(a));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fn, dim3(s.tiles, uint32_t(a.tokens)), dim3(kThreads), token_lds(a), stream, down, h, a.ids,
                       a.weights, residual, out, s);
    return hipGetLastError();
  }
  e = many_rows(a, a.inter) ? launch_rows<F, F32, false, kBoth>(a, down, h, y, a.hidden, a.inter, stream)
                            : launch_rows<F, F32, false, kPacked>(a, down, h, y, a.hidden, a.inter, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sum_kernel<X>, dim3((a.hidden + 1023) / 1024, a.tokens), dim3(256), 0, stream, y, a.ids, residual,
                     out, int(a.top_k), int(a.experts), int(a.hidden));
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
