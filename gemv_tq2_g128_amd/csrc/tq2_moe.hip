// The chosen experts' feed-forward for a few tokens, on 4-bit or ternary weights:
//     h[p] = silu(x G_e^T) * (x U_e^T),  y[p] = w[p] h[p] D_e^T,  out[t] = residual[t] + sum of t's y
// for each pair p = (token t, place j) with e = ids[t, j].
//
// Bound.  Every touched expert's weights are read once against HBM (3 H I weights of 4.125 to 4.5 or 2.125 bits); a few
// tokens meet each of them, so that everything else is kept off that stream.
//
// Whole numbers.  A row of x becomes 31-bit integers under a power of two per 128 columns, as four signed bytes each; the
// codes are small integers as they lie in memory (a mask, or a shift and a mask, for four of them: a fifth of what their
// binary16 values cost).  One v_mfma_i32_16x16x64_i8 takes 16 weight rows as its columns and four tokens' bytes as its
// 16 rows; its sums are exact, start at minus the codes' middle times the sum of x, and a lane has one token's four bytes
// of one weight row.  They become f32 once for each scale: bytes joined, times the scale, times the power of two.
//
// Work split.  rows_kernel for gate and up (SwiGLU in its epilogue), rows_kernel for down, and the sum of each token's
// weighted rows; for few tokens down and the sum are one launch, token_kernel.  A block of rows_kernel has an expert, up to
// eight of its tokens in LDS, and walks over column tiles of 16; its waves are parts of K by tiles (gate and up tiles of
// the same columns side by side), whose partial sums meet in LDS once a step.  The next step's codes are in flight before
// the present one is computed.
//
// Who has which expert: up to 64 pairs are one load and a ballot in each wave; more are sorted by items_kernel into items
// of an expert and up to eight of its pairs, so that experts of many tokens take more blocks instead of longer ones.
//
// Measured (us a call; share of the bytes that it cannot do without at a copy's 4.97 TB/s).  Hidden 2048, inter 768, 8 of
// 128 experts, groups of 128, one token: 7.7 for gate and up, 6.1 for down and sum (0.30: two chains of id, weights, join).
// 4096, 11008, 2 of 8, ternary, one token: 15.4 and 11.1 (0.57).  2048, 768, 8 of 128, groups of 64, 64 tokens: 5 for the
// items, 55, 28 to 38, 5 for the sum (83 to 96 among other calls, whose ends overlap: 0.66 to 0.77).  4096, 1408, 6 of 64,
// ternary, 128 tokens: 5, 96 to 109, 57 to 64, 5 (0.38: the same loads without the products take 107 in all, as an expert's
// 12 tokens are two items that each read its weights; the products hide behind them in part).
#include "tq2_device.h"
#include "tq2_internal.h"
#include "tq2_moe_internal.h"
#include "tq2_types.h"

namespace tq2 {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kTokenWaves = 16;                 // of a block of token_kernel
constexpr int kMaxRows = 8;                     // rows of x that a block has at a time, four to a matrix operand
constexpr int kUnits = 2;                       // 64-byte pieces that a wave of rows_kernel takes of each row at a time
constexpr int kTokenUnits = 4;                  // and one of token_kernel
constexpr int kLds = 160 * 1024;

// A weight format: kGroup, the columns of a scale; kBlocks, the 128-wide blocks of a row's 64 bytes; kMiddle, the code
// that stands for zero.
struct Q4G32 {
  static constexpr int kGroup = 32, kBlocks = 1, kMiddle = 8;
};
struct Q4G64 {
  static constexpr int kGroup = 64, kBlocks = 1, kMiddle = 8;
};
struct Q4G128 {
  static constexpr int kGroup = 128, kBlocks = 1, kMiddle = 8;
};
struct Ternary {
  static constexpr int kGroup = 128, kBlocks = 2, kMiddle = 1;
};
template <class F>
constexpr int kGroups = 128 / F::kGroup;        // scales of a block
template <class F>
constexpr int kSteps = F::kGroup == 32 ? 4 : 2; // matrix steps of a block, of 32 or 64 columns

// Where eight columns of a 128-wide block stand in the matrix steps, which follows from where a lane's 16 bytes of codes
// lie: step, lane group and half of the lane group's 16 bytes (steps of 32: all of its 8).  The eight are 8 u .. 8 u + 7,
// for ternary weights 16 (u >> 1) + 4 (u & 1) and the next three, and the four that are eight further.
//   groups of 128: a lane's words 2 s and 2 s + 1 are step s;
//   groups of 64: after the swap of halves step s is group s, of which lane group g has half a lane's words;
//   groups of 32: after the transposition of words step s is columns 32 s + 8 g;
//   ternary: after the swap lane group g has words 4 (g & 1) + 2 (g >> 1) and the next one, a step each.
template <class F>
__device__ __forceinline__ void place_of(int u, int* step, int* grp, int* half) {
  if (F::kBlocks == 2) {
    const int word = u >> 1;
    *step = word & 1;
    *grp = word >> 2 | (word & 2);
    *half = u & 1;
  } else if (F::kGroup == 128) {
    *step = u >> 1 & 1;
    *grp = u >> 2;
    *half = u & 1;
  } else if (F::kGroup == 64) {
    *step = u >> 3;
    *grp = (u >> 2 & 1) | (u & 2);
    *half = u & 1;
  } else {
    *step = u >> 2;
    *grp = u & 3;
    *half = 0;
  }
}

// A lane's pieces of N consecutive 64-byte units of its row, and the scales of their blocks.
template <class F, int N>
struct Codes {
  static constexpr int kBlocks = N * F::kBlocks;
  static constexpr int kScales = kBlocks * (128 / F::kGroup);      // binary16
  static constexpr int kWords = F::kGroup == 128 ? kScales / 2 + 1 : kScales / 2;
  u32x4_t w[N];
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

// Units unit .. unit + N - 1 of the lane's row; `count` of them are wanted.  Every load is issued, wanted or not
// (those give zeros): behind a branch the count of loads in flight would be unknown to the waits.
template <class F, int N>
__device__ __forceinline__ void load_codes(const Rows& rows, uint32_t row_bytes, uint32_t code_off, uint32_t scale_off,
                                           uint32_t unit, int count, uint32_t in_row, Codes<F, N>& c) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t at = (unit + j) * 64 + in_row;
    // The last half unit of a ternary row is the next row's.
    const bool ok = j < count && (F::kBlocks == 1 || at < row_bytes);
    // Without the hint that they are read once (111 us against 118 for 64 tokens, 188 against 211 for 128): a line of 128
    // bytes is two loads, and items of one expert share its weights.
    c.w[j] = __builtin_amdgcn_raw_buffer_load_b128(rows.codes, ok ? code_off + (unit + j) * 64 : kNowhere, 0, 0);
  }
  constexpr int kWords = Codes<F, N>::kWords;
  uint32_t at = count > 0 ? scale_off + unit * (F::kBlocks * 256 / F::kGroup) : kNowhere;
  // Two-byte scales may start in the middle of a word, where buffer loads do not: the words around them.
  c.down = (at & 2) * 8;
  at &= ~3u;
#pragma unroll
  for (int i = 0; i + 4 <= kWords; i += 4) {
    const u32x4_t d = __builtin_amdgcn_raw_buffer_load_b128(rows.scales, at + i * 4, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) c.d[i + e] = d[e];
  }
  if constexpr (kWords & 2) {
    constexpr int i = kWords & ~3;
    const u32x2_t d = __builtin_amdgcn_raw_buffer_load_b64(rows.scales, at + i * 4, 0, 0);
    c.d[i] = d[0];
    c.d[i + 1] = d[1];
  }
  if constexpr (kWords & 1)
    c.d[kWords - 1] = __builtin_amdgcn_raw_buffer_load_b32(rows.scales, at + (kWords - 1) * 4, 0, 0);
}

// The power of two that undoes a row's is split, so that both parts and what they meet stay normal numbers of f32 for all
// rows: 2^-kInScale goes with the scales (in the step that converts them, at no cost), the rest with the row.
constexpr int kInScale = 24;
constexpr int kMostUp = 126 + kInScale;

// The scale of 32-wide step s of block b, times 2^-kInScale.
template <class F, int N>
__device__ __forceinline__ float scale_of(const Codes<F, N>& c, int b, int s) {
  const int i = b * (128 / F::kGroup) + s / (F::kGroup / 32);
  uint32_t w = c.d[i >> 1];
  if constexpr (F::kGroup == 128) w = __builtin_amdgcn_alignbit(c.d[(i >> 1) + 1], w, c.down);
  return __builtin_fmaf(float(__builtin_bit_cast(_Float16, uint16_t(w >> (16 * (i & 1))))), 0x1p-24f, 0.f);
}

// Lane groups exchange words so that each step stays inside one scale's columns.
template <class F>
__device__ __forceinline__ void arrange(u32x4_t& w) {
  if constexpr (F::kBlocks == 2 || F::kGroup == 64) {
    // Afterwards words 0 and 1 are of the first half of the lanes' columns, 2 and 3 of the second, in all lanes.
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    w = u32x4_t{a[0], b[0], a[1], b[1]};
  } else if constexpr (F::kGroup == 32) {
    // Lane group g holds in word s what lane group s held in word g.
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = u32x4_t{c[0], c[1], d[0], d[1]};
  }
}

// x of up to kMaxRows rows in LDS:
//   operands  [block][step][lane group][columns_of(m)] of 16 bytes (steps of 32: 8), column 4 row + byte
//   starts    [block][group][row] of 4 integers: minus kMiddle times the sums of the row's bytes
//   backs     [block][row]: the power of two that undoes the row's, but for what the scales have of it
// An odd number of columns keeps the lanes that write a stretch of x off each other's banks.
__host__ __device__ inline int columns_of(int m) { return m > 1 ? 4 * m + 1 : 4; }
template <class F>
__host__ __device__ inline int operand_bytes(int blocks, int m) { return (blocks * 128 * columns_of(m) + 15) & ~15; }
template <class F>
__host__ __device__ inline int start_bytes(int blocks, int m) { return blocks * kGroups<F> * m * 16; }
template <class F>
__host__ __device__ inline int x_bytes(int blocks, int m) {
  return operand_bytes<F>(blocks, m) + start_bytes<F>(blocks, m) + (blocks * m * 4 + 15) / 16 * 16;
}
struct Rows31 {
  char* operands;
  i32x4_t* starts;
  float* backs;
};
template <class F>
__device__ __forceinline__ Rows31 rows_in(unsigned char* smem, int blocks, int m) {
  Rows31 r;
  r.operands = reinterpret_cast<char*>(smem);
  r.starts = reinterpret_cast<i32x4_t*>(smem + operand_bytes<F>(blocks, m));
  r.backs = reinterpret_cast<float*>(smem + operand_bytes<F>(blocks, m) + start_bytes<F>(blocks, m));
  return r;
}

// One DPP lane move of an integer.
template <int CTRL>
__device__ __forceinline__ int move(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false); }

// Four words of bytes 0 .. 3 to four words of one byte each.
__device__ __forceinline__ u32x4_t by_byte(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t ab01 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab23 = __builtin_amdgcn_perm(b, a, 0x07030602u);
  const uint32_t cd01 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd23 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  return u32x4_t{__builtin_amdgcn_perm(cd01, ab01, 0x05040100u), __builtin_amdgcn_perm(cd01, ab01, 0x07060302u),
                 __builtin_amdgcn_perm(cd23, ab23, 0x05040100u), __builtin_amdgcn_perm(cd23, ab23, 0x07060302u)};
}

// Convert eight columns (the u-th eight, as place_of says) of 128-wide block kb of row `row` of m into LDS.  The sixteen
// lanes of a block call together: their power of two is a DPP maximum, 2^29 <= |x| 2^e < 2^30, at most kMostUp, by which
// every f32 number is whole.  `share` multiplies the row.
template <class F, class X>
__device__ __forceinline__ void stage8(const typename X::elem* __restrict__ block, int u, int kb, int row, int m,
                                       int cols, float share, const Rows31& r) {
  const typename X::elem* src = block + (F::kBlocks == 2 ? (u >> 1) * 16 + (u & 1) * 4 : u * 8);
  const f32x4_t p = load4(X(), src), q = load4(X(), src + (F::kBlocks == 2 ? 8 : 4));
  const float v[8] = {p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
  int top = 0;                                           // bits of the largest |x|: NaN above infinity
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __builtin_bit_cast(int, v[j]) & 0x7FFFFFFF);
  top = max(top, move<0xB1>(top));
  top = max(top, move<0x4E>(top));
  top = max(top, move<0x141>(top));
  top = max(top, move<0x140>(top));
  const int up = top > 0 ? min(29 + 127 - (top >> 23), kMostUp) : 0;
  uint32_t b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    b[j] = (uint32_t(int(__builtin_rintf(__builtin_ldexpf(v[j], up)))) + 0x00808080u) ^ 0x00808080u;   // signed bytes
  // The order of the codes' bytes: nibbles of a word, or 2-bit fields of bytes.
  const u32x4_t first = F::kBlocks == 2 ? by_byte(b[0], b[4], b[1], b[5]) : by_byte(b[0], b[2], b[4], b[6]);
  const u32x4_t second = F::kBlocks == 2 ? by_byte(b[2], b[6], b[3], b[7]) : by_byte(b[1], b[3], b[5], b[7]);
  int step, grp, half;
  place_of<F>(u, &step, &grp, &half);
  constexpr int kWide = F::kGroup == 32 ? 8 : 16;
  char* dst = r.operands + (size_t(kb * kSteps<F> + step) * 4 + grp) * cols * kWide + half * 8;
  i32x4_t sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    *reinterpret_cast<u32x2_t*>(dst + (row * 4 + i) * kWide) = u32x2_t{first[i], second[i]};
    int n = __builtin_amdgcn_sdot4(int(first[i]), 0x01010101, 0, false);
    n = __builtin_amdgcn_sdot4(int(second[i]), 0x01010101, n, false);
    n += move<0xB1>(n);
    n += move<0x4E>(n);                                  // four lanes: 32 columns
    if (F::kGroup >= 64) n += move<0x141>(n);            // eight
    if (F::kGroup == 128) n += move<0x140>(n);
    sum[i] = -F::kMiddle * n;
  }
  constexpr int kLanes = F::kGroup / 8;
  if (u % kLanes == 0) r.starts[(kb * kGroups<F> + u / kLanes) * m + row] = sum;
  if (u == 0)
    r.backs[kb * m + row] = top >= 0x7F800000 ? __builtin_nanf("") : __builtin_ldexpf(1.0f, kInScale - up) * share;
}

// Bytes from a step's operands to lane group g4's of a column.
template <class F>
__device__ __forceinline__ int operand_at(int g4, int cols, int column) {
  return (g4 * cols + column) * (F::kGroup == 32 ? 8 : 16);
}

// Block b of unit j (b < F::kBlocks) of TILES times 16 weight rows against SETS times four rows of x: lane group g4 adds
// row 4 set + g4's product with weight row r16 to acc[tile][set].  at: the bytes from a step's operands to the lane's; row:
// its group's rows.  All other terms of the addresses are the wave's own.
template <class F, int N, int TILES, int SETS>
__device__ __forceinline__ void multiply(const Codes<F, N> (&c)[TILES], int j, int b, int kb, const Rows31& x, int cols,
                                         const int (&at)[SETS], const int (&row)[SETS], int m,
                                         float (&acc)[TILES][SETS]) {
  constexpr int kWide = F::kGroup == 32 ? 8 : 16;
  float back[SETS];
#pragma unroll
  for (int q = 0; q < SETS; ++q) back[q] = (x.backs + kb * m)[row[q]];
#pragma unroll
  for (int g = 0; g < kGroups<F>; ++g) {
    i32x4_t sum[TILES][SETS];
#pragma unroll
    for (int q = 0; q < SETS; ++q) {
      sum[0][q] = (x.starts + (kb * kGroups<F> + g) * m)[row[q]];
#pragma unroll
      for (int t = 1; t < TILES; ++t) sum[t][q] = sum[0][q];
    }
#pragma unroll
    for (int s = g * kSteps<F> / kGroups<F>; s < (g + 1) * kSteps<F> / kGroups<F>; ++s) {
      const char* operand = x.operands + (kb * kSteps<F> + s) * 4 * cols * kWide;
      if constexpr (F::kGroup == 32) {
        long a[SETS];
#pragma unroll
        for (int q = 0; q < SETS; ++q) a[q] = *reinterpret_cast<const long*>(operand + at[q]);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          const uint32_t w = c[t].w[j][s];
          const u32x2_t codes = {w & 0x0F0F0F0Fu, w >> 4 & 0x0F0F0F0Fu};
#pragma unroll
          for (int q = 0; q < SETS; ++q)
            sum[t][q] = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[q], __builtin_bit_cast(long, codes), sum[t][q], 0, 0, 0);
        }
      } else {
        i32x4_t a[SETS];
#pragma unroll
        for (int q = 0; q < SETS; ++q) a[q] = *reinterpret_cast<const i32x4_t*>(operand + at[q]);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          u32x4_t codes;
          if constexpr (F::kBlocks == 2) {
            const uint32_t w = c[t].w[j][2 * b + s];
            codes = u32x4_t{w & 0x03030303u, w >> 2 & 0x03030303u, w >> 4 & 0x03030303u, w >> 6 & 0x03030303u};
          } else {
            const uint32_t w = c[t].w[j][2 * s], v = c[t].w[j][2 * s + 1];
            codes = u32x4_t{w & 0x0F0F0F0Fu, w >> 4 & 0x0F0F0F0Fu, v & 0x0F0F0F0Fu, v >> 4 & 0x0F0F0F0Fu};
          }
#pragma unroll
          for (int q = 0; q < SETS; ++q)
            sum[t][q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[q], __builtin_bit_cast(i32x4_t, codes), sum[t][q], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const float d = scale_of<F, N>(c[t], j * F::kBlocks + b, g * (F::kGroup / 32));
#pragma unroll
      for (int q = 0; q < SETS; ++q) {
        // Two bytes joined are whole numbers below 2^27; f32 rounds them and the four.
        const i32x4_t v = sum[t][q];
        const float four = __builtin_fmaf(float((v[3] << 8) + v[2]), 65536.f, float((v[1] << 8) + v[0]));
        acc[t][q] = __builtin_fmaf(d * four, back[q], acc[t][q]);
      }
    }
  }
}

// An expert and up to kMaxRows of its pairs, order[first .. first + count).
struct Item {
  int expert, first, count;
};
// What items_kernel leaves in the workspace.
struct Items {
  int* count;
  Item* item;
  uint16_t* order;
};

// One launch of rows_kernel; all of it follows from the sizes.
struct Shape {
  int pairs, top_k, experts;
  uint32_t top_k_inverse;    // pair * top_k_inverse >> 16 is its token
  int rows;                  // of x in LDS at a time
  int row_blocks;            // 128-wide blocks of K
  int pieces, blocks;        // K in pieces of `blocks`, whose rows fit LDS; each piece's sums are rows of their own
  uint32_t blocks_inverse;   // i * blocks_inverse >> 20 is i / blocks
  int units;                 // 64-byte units of a weight row in a piece
  int tiles;                 // column tiles of an expert (of gate, and as many of up): a multiple of 8
  int wk_shift;              // log2 of the parts of K
  int part_units, rounds, per;         // units of a part, its rounds, units of a round
  int steps;                 // of column tiles that the block's waves take together
  bool few, by_pair;         // no items: a block row for each pair, or for each expert
};

// Pairs sorted by their expert, and experts cut into items of `rows` pairs.  The order of an expert's pairs is left to the
// atomics: a pair's row is computed from itself alone, in whichever item it is.
constexpr int kItemThreads = 1024;
__global__ __launch_bounds__(kItemThreads) void items_kernel(const int32_t* __restrict__ ids, int pairs, int experts,
                                                             int rows, Items out) {
  __shared__ uint32_t next[TQ2_MOE_MAX_EXPERTS];
  __shared__ uint32_t part[2][kItemThreads / 64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  constexpr int kMine = TQ2_MOE_MAX_TOKENS * TQ2_MOE_MAX_TOP_K / kItemThreads;
  int id[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) id[i] = t + i * kItemThreads < pairs ? ids[t + i * kItemThreads] : -1;
  next[t] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (uint32_t(id[i]) < uint32_t(experts)) atomicAdd(&next[id[i]], 1u);
  __syncthreads();
  // Thread t's expert: where its pairs and its items start.
  const uint32_t n = next[t], cut = (n + rows - 1) / rows;
  uint32_t pair = n, item = cut;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t a = __shfl_up(pair, d), b = __shfl_up(item, d);
    if (lane >= d) pair += a, item += b;
  }
  if (lane == 63) part[0][wave] = pair, part[1][wave] = item;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kItemThreads / 64; ++w)
    if (w < wave) pair += part[0][w], item += part[1][w];
  next[t] = pair - n;
  if (t == kItemThreads - 1) *out.count = int(item);
  for (uint32_t i = 0; i < cut; ++i)
    out.item[item - cut + i] = Item{t, int(pair - n + i * rows), int(min(n - i * rows, uint32_t(rows)))};
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (uint32_t(id[i]) < uint32_t(experts)) out.order[atomicAdd(&next[id[i]], 1u)] = uint16_t(t + i * kItemThreads);
}

// GATE: x are the tokens' rows, out the rows between the projections, f32 [pairs, 16 tiles].  Otherwise x are those
// and out the weighted rows, f32 [pieces, pairs, 16 tiles].
template <class F, class X, bool GATE, int WAVES, int SETS>
__global__ __launch_bounds__(64 * WAVES, 4) void rows_kernel(Weight weight, const typename X::elem* __restrict__ x,
                                                             const int32_t* __restrict__ ids, Items items,
                                                             const float* __restrict__ share, float* __restrict__ out,
                                                             Shape sh) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int kThreads = 64 * WAVES, kRows = 4 * SETS;
  float* red = reinterpret_cast<float*>(smem + x_bytes<F>(sh.blocks, sh.rows));
  uint16_t* list = reinterpret_cast<uint16_t*>(red + 2 * WAVES * kRows * 16);    // after [wave][tile][row][column]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  // Few pairs: the block has the steps blockIdx.x, blockIdx.x + gridDim.x, ... of its expert.  Otherwise a share of the
  // steps of all items, one after another, which may begin and end inside one.
  int e = 0, found = 0, step = 0, hop, end = 0, piece = sh.few ? blockIdx.z : 0;
  int64_t now_at = 0, stop_at = 0;                       // of all items' steps
  if (sh.few) {
    // The ids of all pairs, at most 64, are one load; every wave lists the expert's pairs for itself.
    const int id = lane < sh.pairs ? ids[lane] : -1;
    e = sh.by_pair ? __builtin_amdgcn_readlane(id, blockIdx.y) : int(blockIdx.y);
    if (uint32_t(e) >= uint32_t(sh.experts)) return;
    const uint64_t mask = __ballot(id == e);
    if (mask == 0 || (sh.by_pair && __builtin_ctzll(mask) != int(blockIdx.y))) return;
    found = __popcll(mask);
    if (id == e) list[__popcll(mask & ((uint64_t(1) << lane) - 1))] = uint16_t(lane);
    step = blockIdx.x;
    hop = gridDim.x;
    end = sh.steps;
  } else {
    const int64_t all = int64_t(*items.count) * sh.pieces * sh.steps;
    // Blocks go round the dies by number: neighbouring shares are one die's, whose L2 then has an expert's weights for
    // its second item too (128 tokens, ternary: 165 us with shares in the blocks' order, 159 so).
    const int per_die = gridDim.x / 8, block = (blockIdx.x & 7) * per_die + (blockIdx.x >> 3);
    now_at = all * block / gridDim.x;
    stop_at = all * (block + 1) / gridDim.x;
    if (now_at >= stop_at) return;
    hop = 1;
  }
  // The wave's part: two tiles of each step (gate and up, or neighbours), which share what is read of x, and units of K.
  const int slot = wave >> sh.wk_shift, part = wave & ((1 << sh.wk_shift) - 1);
  const int unit0 = part * sh.part_units;
  int blocks = 0, mine = 0;                              // of the piece, and the wave's units of it
  auto take = [&]() {
    blocks = min(sh.blocks, sh.row_blocks - piece * sh.blocks);
    mine = min(sh.part_units, (blocks + F::kBlocks - 1) / F::kBlocks - unit0);
  };
  const int per_step = WAVES >> sh.wk_shift, twos = GATE ? sh.tiles : sh.tiles / 2;
  const int64_t width = int64_t(sh.tiles) * 16;
  const uint32_t code_off = r16 * weight.row_bytes + g4 * 16, scale_off = r16 * weight.row_scales * 2;

  Codes<F, kUnits> c[2][2];
  auto load = [&](int step, int round, Codes<F, kUnits> (&into)[2]) {
    const int two = step * per_step + slot;
    const bool there = step < end && two < twos;
    const int64_t row0 = int64_t(e) * width * (GATE ? 2 : 1) + (there ? two * (GATE ? 16 : 32) : 0);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      load_codes<F, kUnits>(rows_at(weight, row0 + (GATE ? i * width : i * 16)), weight.row_bytes, code_off, scale_off,
                            uint32_t(piece * sh.units + unit0 + round * sh.per),
                            there ? min(sh.per, mine - round * sh.per) : 0, g4 * 16, into[i]);
  };
  int round = 0, begin = 0;
  for (bool more = true; more;) {
    if (!sh.few) {
      const int at = int(now_at / sh.steps);
      const Item item = items.item[GATE ? at : at / sh.pieces];
      piece = GATE ? 0 : at % sh.pieces;
      e = __builtin_amdgcn_readfirstlane(item.expert);
      found = __builtin_amdgcn_readfirstlane(item.count);
      begin = int(now_at - int64_t(at) * sh.steps);
      end = int(min(int64_t(sh.steps), begin + stop_at - now_at));
      now_at += end - begin;
      more = now_at < stop_at;
      step = begin;
      round = 0;
      take();
      load(step, 0, c[0]);                               // in flight while x is converted
      __syncthreads();                                   // the last item's rows, sums and list have been read
      if (lane < found) list[lane] = items.order[item.first + lane];
    } else {
      begin = blockIdx.x;
      take();
      load(step, 0, c[0]);
      more = false;
    }
    __builtin_amdgcn_wave_barrier();

    for (int first = 0; first < found; first += sh.rows) {
      const int m = min(sh.rows, found - first), cols = columns_of(m);
      const Rows31 rows = rows_in<F>(smem, sh.blocks, m);
      if (first > 0) {
        step = begin;
        round = 0;
        load(step, 0, c[0]);
        __syncthreads();                                   // the last step has read x and red
      }
      for (int i = threadIdx.x; i < m * sh.blocks * 16; i += kThreads) {
        const int row = int((uint32_t(i >> 4) * sh.blocks_inverse) >> 20), kb = (i >> 4) - row * sh.blocks;
        const uint32_t pair = list[first + row], from = GATE ? pair * sh.top_k_inverse >> 16 : pair;
        if (kb < blocks)
          stage8<F, X>(x + (int64_t(from) * sh.row_blocks + piece * sh.blocks + kb) * 128, i & 15, kb, row, m, cols, 1.f,
                       rows);
      }
      __syncthreads();
      // The lane's operand columns and its group's rows; past the last row they repeat the first one's.
      int at[SETS], own[SETS];
#pragma unroll
      for (int q = 0; q < SETS; ++q) {
        at[q] = operand_at<F>(g4, cols, q * 4 + (r16 >> 2) < m ? q * 16 + r16 : r16 & 3);
        own[q] = q * 4 + g4 < m ? q * 4 + g4 : 0;
      }
      float acc[2][SETS] = {};
      auto compute = [&](Codes<F, kUnits> (&from)[2]) {
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
          const int unit = unit0 + round * sh.per + j;
          if (j >= sh.per || round * sh.per + j >= mine) continue;
          arrange<F>(from[0].w[j]);
          arrange<F>(from[1].w[j]);
#pragma unroll
          for (int b = 0; b < F::kBlocks; ++b) {
            const int kb = unit * F::kBlocks + b;
            if (F::kBlocks > 1 && kb >= blocks) continue;
            multiply<F, kUnits, 2, SETS>(from, j, b, kb, rows, cols, at, own, m, acc);
          }
        }
      };
      // Partial sums [wave][tile][row of x][weight row] of a step meet.
      auto finish = [&]() {
        __syncthreads();                                   // the last step's have been read
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = 0; q < SETS; ++q) {
            red[((wave * 2 + i) * kRows + q * 4 + g4) * 16 + r16] = acc[i][q];
            acc[i][q] = 0.f;
          }
        __syncthreads();
        // GATE: a gate and an up tile give one of the output; otherwise each tile its own.
        constexpr int kOut = GATE ? 1 : 2;
        for (int i = threadIdx.x; i < per_step * kOut * kRows * 16; i += kThreads) {
          const int n = i & 15, row = i >> 4 & (kRows - 1), tile = i / (16 * kRows);
          const int two = step * per_step + tile / kOut;
          if (row >= m || two >= twos) continue;
          const int p = list[first + row];
          const float* from = red + ((((tile / kOut) << sh.wk_shift) * 2 + tile % kOut) * kRows + row) * 16 + n;
          float a = 0.f, b = 0.f;
          for (int w = 0; w < 1 << sh.wk_shift; ++w) {
            a += from[w * (2 * kRows * 16)];
            if (GATE) b += from[w * (2 * kRows * 16) + kRows * 16];
          }
          const float v = GATE ? a / (1.f + expf(-a)) * b : a * share[p];
          out[(int64_t(piece) * sh.pairs + p) * width + int64_t(two) * (16 * kOut) + tile % kOut * 16 + n] = v;
        }
      };
      auto walk = [&](Codes<F, kUnits> (&now)[2], Codes<F, kUnits> (&then)[2]) {
        const bool last = round + 1 == sh.rounds;
        const int next = last ? step + hop : step, next_round = last ? 0 : round + 1;
        load(next, next_round, then);
        compute(now);
        if (last) finish();
        step = next;
        round = next_round;
      };
      while (step < end) {
        walk(c[0], c[1]);
        if (step >= end) break;
        walk(c[1], c[0]);
      }
    }
  }
}

// Down and the sum over a token's experts at once, for few tokens: a block has a token and a tile of 16 columns, its
// waves take rounds of units over all of the token's places in turn, and their sums meet in LDS.  An expert that several
// tokens chose is read for each of them.
template <class F, class X>
__global__ __launch_bounds__(64 * kTokenWaves) void token_kernel(Weight weight, const float* __restrict__ h,
                                                                    const int32_t* __restrict__ ids,
                                                                    const float* __restrict__ share,
                                                                    const typename X::elem* residual,
                                                                    typename X::elem* out, Shape sh) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ float red[kTokenWaves][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4, t = blockIdx.y;
  const int all_blocks = sh.top_k * sh.blocks, cols = columns_of(1);
  const Rows31 rows = rows_in<F>(smem, all_blocks, 1);
  const int id = lane < sh.top_k ? ids[t * sh.top_k + lane] : -1;
  const float part = lane < sh.top_k ? share[t * sh.top_k + lane] : 0.f;
  const uint32_t code_off = r16 * weight.row_bytes + g4 * 16, scale_off = r16 * weight.row_scales * 2;
  const int64_t hidden = int64_t(sh.tiles) * 16;

  // Round r is part r % rounds of place r / rounds; the wave has rounds wave, wave + kTokenWaves, ...
  const int all_rounds = sh.top_k * sh.rounds;
  Codes<F, kTokenUnits> c[2][1];
  int place = 0, round = wave;                           // of the round that is loaded next
  struct At {
    int place, unit, count;
  };
  auto load = [&](Codes<F, kTokenUnits> (&into)[1]) {
    while (round >= sh.rounds && place < sh.top_k) round -= sh.rounds, ++place;
    const bool there = place < sh.top_k;
    const int e = __builtin_amdgcn_readlane(id, there ? place : 0);
    const bool real = there && uint32_t(e) < uint32_t(sh.experts);
    const At at = {place, round * sh.per, real ? min(sh.per, sh.units - round * sh.per) : 0};
    load_codes<F, kTokenUnits>(rows_at(weight, (real ? int64_t(e) * hidden : 0) + int64_t(blockIdx.x) * 16),
                               weight.row_bytes, code_off, scale_off, uint32_t(at.unit), at.count, g4 * 16, into[0]);
    round += kTokenWaves;
    return at;
  };
  At now = load(c[0]);
  for (int i = threadIdx.x; i < all_blocks * 16; i += 64 * kTokenWaves) {
    const int kb = i >> 4, j = int((uint32_t(kb) * sh.blocks_inverse) >> 20);
    // The first lanes are among those that are here: the lanes end in front of one that is not.
    stage8<F, F32>(h + (int64_t(t) * all_blocks + kb) * 128, i & 15, kb, 0, 1, cols, __shfl(part, j), rows);
  }
  __syncthreads();
  const int at[1] = {operand_at<F>(g4, cols, r16 & 3)}, own[1] = {0};
  float acc[1][1] = {};
  auto compute = [&](Codes<F, kTokenUnits> (&from)[1], const At& a) {
#pragma unroll
    for (int j = 0; j < kTokenUnits; ++j) {
      if (j >= a.count) continue;
      arrange<F>(from[0].w[j]);
#pragma unroll
      for (int b = 0; b < F::kBlocks; ++b) {
        const int k = (a.unit + j) * F::kBlocks + b;
        if (F::kBlocks > 1 && k >= sh.blocks) continue;
        multiply<F, kTokenUnits, 1, 1>(from, j, b, a.place * sh.blocks + k, rows, cols, at, own, 1, acc);
      }
    }
  };
  for (int done = wave; done < all_rounds;) {
    const At then = load(c[1]);
    compute(c[0], now);
    done += kTokenWaves;
    if (done >= all_rounds) break;
    now = load(c[0]);
    compute(c[1], then);
    done += kTokenWaves;
  }
  if (g4 == 0) red[wave][r16] = acc[0][0];
  __syncthreads();
  if (threadIdx.x < 16) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kTokenWaves; ++w) sum += red[w][threadIdx.x];
    const int64_t to = int64_t(t) * hidden + int64_t(blockIdx.x) * 16 + threadIdx.x;
    if (residual) sum += float(residual[to]);
    out[to] = typename X::elem(sum);
  }
}

// out[t] = residual[t] + the token's weighted rows in the order of their places and pieces; four columns a thread.
template <class X>
__global__ __launch_bounds__(256) void sum_kernel(const float* __restrict__ y, const int32_t* __restrict__ ids,
                                                  const typename X::elem* residual, typename X::elem* out, int pieces,
                                                  int pairs, int top_k, int experts, int hidden) {
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
  if (n >= hidden) return;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < top_k; ++j) {
    const int p = t * top_k + j;
    if (uint32_t(ids[p]) >= uint32_t(experts)) continue;
    for (int i = 0; i < pieces; ++i) sum += load4(F32(), y + (size_t(i) * pairs + p) * hidden + n);
  }
  if (residual) sum += load4(X(), residual + size_t(t) * hidden + n);
  store4(X(), out + size_t(t) * hidden + n, sum);
}

// Blocks of each of `pieces` of a row, whole units.
template <class F>
int piece_blocks(int blocks, int pieces) {
  const int units = (blocks + F::kBlocks - 1) / F::kBlocks, each = (units + pieces - 1) / pieces * F::kBlocks;
  return each < blocks ? each : blocks;
}

// LDS of rows_kernel.
template <class F>
int lds_bytes(int blocks, int rows, int waves) {
  return x_bytes<F>(blocks, rows) + 2 * waves * (rows > 4 ? 8 : 4) * 64 + 128;          // sums of two tiles, the list
}

// Rows of x at a time: as many as LDS holds of the hidden axis.  A token hardly names an expert twice.  Four rows are one
// matrix operand, enough for most experts of a batch that has up to two pairs for each.
template <class F>
int rows_at_once(const tq2_moe_experts_args& a) {
  int rows = a.tokens < kMaxRows ? int(a.tokens) : kMaxRows;
  if (rows > 4 && a.tokens * a.top_k <= 2 * a.experts) rows = 4;
  while (lds_bytes<F>(int(a.hidden / 128), rows, 16) > kLds) --rows;
  return rows;
}

// Pieces of K for down, so that LDS holds as many rows of each as gate and up have: two or three rows at a time would read
// an expert's weights again for every few tokens.
template <class F>
int pieces_of(const tq2_moe_experts_args& a) {
  const int rows = rows_at_once<F>(a), blocks = int(a.inter / 128);
  int pieces = 1;
  while (lds_bytes<F>(piece_blocks<F>(blocks, pieces), rows, 16) > kLds) ++pieces;
  const int each = piece_blocks<F>(blocks, pieces);
  return (blocks + each - 1) / each;                     // no empty ones
}

// The launch for n columns and k of K: `waves` of a block share it, `units` of a row at a time.
template <class F>
Shape shape_of(const tq2_moe_experts_args& a, int64_t n, int64_t k, int waves, int units, int twos, int pieces) {
  Shape s;
  s.pairs = int(a.tokens * a.top_k);
  s.top_k = int(a.top_k);
  s.experts = int(a.experts);
  s.top_k_inverse = uint32_t((65536 + a.top_k - 1) / a.top_k);
  s.rows = rows_at_once<F>(a);
  s.row_blocks = int(k / 128);
  s.blocks = piece_blocks<F>(s.row_blocks, pieces);
  s.pieces = (s.row_blocks + s.blocks - 1) / s.blocks;
  s.blocks_inverse = uint32_t(((1 << 20) + s.blocks - 1) / s.blocks);
  s.units = (s.blocks + F::kBlocks - 1) / F::kBlocks;
  s.tiles = int(n / 16);
  s.few = s.pairs <= 64;
  s.by_pair = s.pairs < s.experts;
  // Parts of K that take the fewest rounds of all waves; among equals the most parts, whose steps are shared out most
  // evenly.  Where blocks walk over many steps, one of a single round pays an eighth more for meeting in LDS (64 tokens on
  // 128 experts of 768: 102 us with single rounds, 99 with two; on 64 of 1408: 110 and 107).
  int64_t best = INT64_MAX;
  for (int shift = 0; (1 << shift) <= waves; ++shift) {
    const int part = (s.units + (1 << shift) - 1) >> shift, rounds = (part + units - 1) / units;
    const int per_step = waves >> shift, steps = (twos + per_step - 1) / per_step;
    const int64_t cost = int64_t(steps) * (rounds == 1 && !s.few ? 9 : 8 * rounds);
    if (cost > best) continue;
    best = cost;
    s.wk_shift = shift;
    s.part_units = part;
    s.rounds = rounds;
    s.per = (part + rounds - 1) / rounds;
    s.steps = steps;
  }
  return s;
}

hipError_t allow_lds(const void* fn, int lds) {
  return lds <= 48 * 1024 ? hipSuccess
                          : hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

template <class F, class X, bool GATE, int WAVES, int SETS>
hipError_t launch_rows(const tq2_moe_experts_args& a, const Weight& w, const void* x, const Items& items, float* out,
                       int64_t n, int64_t k, int pieces, hipStream_t stream) {
  const Shape s = shape_of<F>(a, n, k, WAVES, kUnits, int(n / (GATE ? 16 : 32)), pieces);
  const int lds = lds_bytes<F>(s.blocks, s.rows, WAVES);
  // As many blocks as the card holds at a time, two of 8 waves or one of 16 for each CU: the prologue (who, which rows,
  // their conversion) is paid once, and steps are shared out evenly.
  dim3 grid(256 * (16 / WAVES));
  if (s.few) {
    grid.y = s.by_pair ? s.pairs : s.experts;
    grid.z = s.pieces;
    grid.x = (512 + grid.y - 1) / grid.y;
    if (grid.x > uint32_t(s.steps)) grid.x = s.steps;
  }
  const auto fn = rows_kernel<F, X, GATE, WAVES, SETS>;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, grid, dim3(64 * WAVES), lds, stream, w,
                     static_cast<const typename X::elem*>(x), a.ids, items, a.weights, out, s);
  return hipGetLastError();
}

// Blocks of 8 waves where two of them share a CU's LDS, otherwise one of 16.
template <class F, class X, bool GATE>
hipError_t launch_rows(const tq2_moe_experts_args& a, const Weight& w, const void* x, const Items& items, float* out,
                       int64_t n, int64_t k, int pieces, hipStream_t stream) {
  const int rows = rows_at_once<F>(a);
  const bool two = 2 * lds_bytes<F>(piece_blocks<F>(int(k / 128), pieces), rows, 8) <= kLds;
  if (rows <= 4) return two ? launch_rows<F, X, GATE, 8, 1>(a, w, x, items, out, n, k, pieces, stream)
                            : launch_rows<F, X, GATE, 16, 1>(a, w, x, items, out, n, k, pieces, stream);
  return two ? launch_rows<F, X, GATE, 8, 2>(a, w, x, items, out, n, k, pieces, stream)
             : launch_rows<F, X, GATE, 16, 2>(a, w, x, items, out, n, k, pieces, stream);
}

// LDS of token_kernel, whose blocks hold all of a token's rows.
template <class F>
int token_lds(const tq2_moe_experts_args& a) { return x_bytes<F>(int(a.top_k * (a.inter / 128)), 1); }

template <class F>
bool by_token(const tq2_moe_experts_args& a) {
  // Against a second launch of 4 us: weights that several tokens share come from the caches again, up to 32 MB of them
  // (8 tokens on two of 8 experts of 12 MB each: 141 us by tokens, 133 by experts; 4 on all of 8 of 0.8 MB: 16 and 20).
  const int64_t pairs = a.tokens * a.top_k, twice = pairs > a.experts ? pairs - a.experts : 0;
  return pairs <= 32 && twice * a.hidden * a.inter * (F::kBlocks == 2 ? 17 : 34) / 64 <= int64_t(32) << 20 &&
         token_lds<F>(a) + kTokenWaves * 64 <= kLds;
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
  char* ws = static_cast<char*>(a.workspace);
  float* h = reinterpret_cast<float*>(ws);
  float* y = reinterpret_cast<float*>(ws + plan.y_offset);
  Items items;
  items.count = reinterpret_cast<int*>(ws + plan.items_offset);
  items.item = reinterpret_cast<Item*>(items.count + 4);
  items.order = reinterpret_cast<uint16_t*>(items.item + a.tokens * a.top_k);
  const Weight up = weight_of<F>(a.gate_up, a.gate_up_scales, 2 * a.experts * a.inter, a.hidden);
  const Weight down = weight_of<F>(a.down, a.down_scales, a.experts * a.hidden, a.inter);
  hipError_t e;
  if (a.tokens * a.top_k > 64) {
    hipLaunchKernelGGL(items_kernel, dim3(1), dim3(kItemThreads), 0, stream, a.ids, int(a.tokens * a.top_k),
                       int(a.experts), rows_at_once<F>(a), items);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  e = launch_rows<F, X, true>(a, up, a.x, items, h, a.inter, a.hidden, 1, stream);
  if (e != hipSuccess) return e;
  const auto* residual = static_cast<const typename X::elem*>(a.residual);
  auto* out = static_cast<typename X::elem*>(a.out);
  if (by_token<F>(a)) {
    const Shape s = shape_of<F>(a, a.hidden, a.inter, 1, kTokenUnits, 1, 1);
    const auto fn = token_kernel<F, X>;
    e = allow_lds(reinterpret_cast<const void*>(fn), token_lds<F>(a));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fn, dim3(s.tiles, uint32_t(a.tokens)), dim3(64 * kTokenWaves), token_lds<F>(a), stream, down, h,
                       a.ids, a.weights, residual, out, s);
    return hipGetLastError();
  }
  e = launch_rows<F, F32, false>(a, down, h, items, y, a.hidden, a.inter, pieces_of<F>(a), stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sum_kernel<X>, dim3((a.hidden + 1023) / 1024, a.tokens), dim3(256), 0, stream, y, a.ids, residual,
                     out, pieces_of<F>(a), int(a.tokens * a.top_k), int(a.top_k), int(a.experts), int(a.hidden));
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
  const int pieces = a.format == TQ2_MOE_TERNARY ? pieces_of<Ternary>(a)
                     : a.group == 32             ? pieces_of<Q4G32>(a)
                     : a.group == 64             ? pieces_of<Q4G64>(a)
                                                 : pieces_of<Q4G128>(a);
  const size_t pairs = size_t(a.tokens) * size_t(a.top_k);
  MoePlan p;
  p.y_offset = align256(pairs * size_t(a.inter) * 4);
  p.items_offset = p.y_offset + align256(pairs * size_t(pieces) * size_t(a.hidden) * 4);
  p.workspace = p.items_offset + 16 + pairs * (sizeof(Item) + 2);
  return p;
}

hipError_t launch_moe_experts(const tq2_moe_experts_args& a, const MoePlan& plan, hipStream_t stream) {
  if (a.format == TQ2_MOE_TERNARY) return launch<Ternary>(a, plan, stream);
  if (a.group == 32) return launch<Q4G32>(a, plan, stream);
  if (a.group == 64) return launch<Q4G64>(a, plan, stream);
  return launch<Q4G128>(a, plan, stream);
}

}  // namespace tq2
