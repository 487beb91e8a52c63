// Attention of new tokens over a paged cache, streaming form.
//     o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q.k_j - m),   c = scale log2 e
// with the running maximum m of a row: one pass over the keys, f32 sums.
//
// Bound.  A decode step reads every visible key and value once and does a
// few operations with each: HBM.  So keys and values go straight from memory
// to the operand registers of the matrix cores, with no LDS in between and no
// barrier in the loop; each wave walks over its own tiles of 32 keys with its
// own m, sum and output, and the waves of a block meet once at the end.
//
// Matrix form (v_mfma_f32_16x16x32, 16 rows: the new tokens times the query
// heads that share a key head).
//   S^T = K Q^T: a lane reads 16 bytes of one key, and holds four keys' scores
//     of one row for each 16 keys.
//   O^T = V^T P^T: the eight probabilities of a lane (two tiles of 16 keys) are
//     its operand words as they are, with the keys of a matrix step in the order
//     4 g + j, 16 + 4 g + j of lane group g.  For V^T a lane reads the same 8
//     components of those eight keys (rows of 256 bytes by 16 lanes), and byte
//     permutes turn its 8 x 8 block: word i of the eight keys is the operand of
//     matrix step i, whose row c is component 8 c + i.
// Softmax statistics are per lane (a row) and its 16-lane group's keys; the
// maximum is joined across the four groups each tile, the sum once at the end.
//
// 32-bit q is split into two binary16 parts under a power of two per row, and
// so are the probabilities (scaled by 2^14): two matrix steps each.  16-bit q enters
// as it is.  e4m3 codes become binary16 (keys: q's type) exactly.  With 16-bit q the
// probabilities are rounded once to the products' type: half a step each, of random
// sign, which makes the error 1.1 to 1.4 times that of the output's own
// rounding; a second part would double the matrix steps of the second product.
//
// Masks.  A 16-key run lies in one page; its buffer resource ends at the last
// key that counts, so that everything past it (or in a page that is not there)
// loads as zero.  Tiles that every row sees whole skip the comparisons.  Where
// rows differ in what they see, a value that is not finite is kept from rows
// that do not see it (zero times infinity would reach them).
//
// Parts.  Long sequences are cut into parts of keys, one block each, whose states
// join_kernel puts together.  Measured: 64 sequences of up to 8,192 tokens, bf16:
// 188 us, 5.9 TB/s; 4 of up to 131,071, e4m3: 130 us, 5.6 TB/s; one token over 1,001
// keys: 9.6 us in 8 parts, a chain of trips to memory (length, page, keys, parts).
#include "tq2_attn_device.h"

namespace tq2 {
namespace {

// Maximum and sum over the lanes 16, 32 and 48 on (a row's four lane groups).
__device__ __forceinline__ float over_groups_max(float v) {
  float2 a = halves32(v);
  a = halves16(fmaxf(a.x, a.y));
  return fmaxf(a.x, a.y);
}
__device__ __forceinline__ float over_groups_sum(float v) {
  float2 a = halves32(v);
  a = halves16(a.x + a.y);
  return a.x + a.y;
}

__device__ __forceinline__ float row16_top(float v) {
  v = fmaxf(v, dpp_move<0xB1, 0xF>(v));
  v = fmaxf(v, dpp_move<0x4E, 0xF>(v));
  v = fmaxf(v, dpp_move<0x141, 0xF>(v));
  return fmaxf(v, dpp_move<0x140, 0xF>(v));
}

// Components per lane of the value chunks that make up a head: 128, 64 or 32 wide.
template <int D>
struct Chunks {
  static constexpr int count = D == 96 || D == 192 || D == 256 ? 2 : 1;
  __host__ __device__ static constexpr int per_lane(int c) {
    return D == 64 ? 4 : D == 96 ? (c == 0 ? 4 : 2) : D == 192 ? (c == 0 ? 8 : 4) : 8;
  }
  __host__ __device__ static constexpr int start(int c) { return c == 0 ? 0 : (D == 96 ? 64 : 128); }
  __host__ __device__ static constexpr int tile(int c) { return c == 0 ? 0 : per_lane(0); }
};

// A 16-key run: where its keys and values start, and how many count.
struct Run {
  rsrc_t k, v;
  int count;
};

// Waves per SIMD that the register budget aims at.
template <int D, int MT>
constexpr int kMinWaves = D * MT <= 128 ? 2 : 1;

// LDS of a block: q in operand order during the loop, then every wave's output,
// maximum and sum of each row (rows are four floats apart, so that 16 rows' words lie
// in 16 bank groups).
template <class Act, int D, int MT, int W>
struct StreamLds {
  static constexpr size_t q = size_t(__is_same(Act, F32) ? 2 : 1) * MT * (D / 32) * 1024;
  static constexpr int row = D + 4;
  static constexpr size_t states = size_t(W) * MT * 16 * row * 4;
  static constexpr size_t bytes = q > states ? q : states;
};

template <class Act, class Cache, int D, int MT, int W>
__global__ __launch_bounds__(64 * W, (kMinWaves<D, MT>)) void stream_kernel(AttnArgs a) {
  typedef typename Kinds<Act, Cache>::QK QK;
  typedef typename Kinds<Act, Cache>::PV PV;
  typedef typename Act::elem act_t;
  typedef typename Cache::elem cache_t;
  constexpr bool kSplit = __is_same(Act, F32);                   // q and probabilities in two parts
  constexpr float kLift = __is_same(PV, F16) ? 14.f : 0.f;       // log2: keeps small probabilities normal
  constexpr int kSize = int(sizeof(cache_t));
  constexpr int kSteps = D / 32;
  constexpr int kTiles = D / 16;
  constexpr int kState = StreamLds<Act, D, MT, W>::row;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  u32x4_t* qf = reinterpret_cast<u32x4_t*>(smem);                // [part][MT][step][64]
  float* states = reinterpret_cast<float*>(smem);                // [wave][row]: output; maximum, sum
  __shared__ float back[MT * 16];                                // power of two of each row of q

  const Pages& p = a.pages;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const uint32_t group = a.group;
  const int head = blockIdx.x % p.kv_heads;
  const int split = blockIdx.z;
  const int b = blockIdx.y;
  if (b >= p.batch) return;
  const Seq s = sequence(p, b);
  const uint32_t rows = uint32_t(s.q_len) * group;               // below 2^31
  const Parts parts = parts_of(s, a.window, a.splits, a.split_keys);
  if (split >= parts.count) return;
  const int start = parts.base + split * parts.per;
  const int part_end = s.keys - start < parts.per ? s.keys : start + parts.per;

  for (uint32_t row0 = blockIdx.x / p.kv_heads * (MT * 16); row0 < rows; row0 += gridDim.x / p.kv_heads * (MT * 16)) {
    // Keys of this part that any of the rows sees.
    const uint32_t live_rows = rows - row0 < MT * 16 ? rows - row0 : MT * 16;
    const int place_lo = s.first + int(row0 / group), place_hi = s.first + int((row0 + live_rows - 1) / group);
    const int hi = place_hi + 1 < part_end ? place_hi + 1 : part_end;
    int lo = start;
    if (a.window) {
      const int64_t edge = int64_t(place_lo) - a.window + 1;
      if (edge > lo) lo = edge < part_end ? int(edge) & ~31 : part_end;
    }

    // q: 16 lanes for each row, 8 components each.
    constexpr int kUnits = (D / 8 + 15) / 16, kPasses = (MT * 4 + W - 1) / W;
    f32x4_t qx[kPasses][kUnits][2];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t r = (i * W + wave) * 4 + g4;
      const bool live = r < live_rows;
      const uint32_t row = row0 + r, token = row / group;
      const act_t* src = static_cast<const act_t*>(a.q) +
                         (live ? int64_t(s.q0 + token) * a.q_token + (head * group + row - token * group) * a.q_head : 0);
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        const int u = r16 + 16 * j;
        qx[i][j][0] = qx[i][j][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (live && u < D / 8) {
          qx[i][j][0] = load4(Act(), src + u * 8);
          qx[i][j][1] = load4(Act(), src + u * 8 + 4);
        }
      }
    }

    float scale[MT], m[MT], sum[MT];
    f32x4_t o[MT][kTiles];
    int place[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint32_t row = row0 + mt * 16 + r16;
      place[mt] = row < rows ? s.first + int(row / group) : -1;
    }
    const int all = hi > lo ? (hi - lo + 31) >> 5 : 0;           // tiles of 32 keys
    const int mine = wave < all ? (all - wave + W - 1) / W : 0;
    const cache_t* kbase = static_cast<const cache_t*>(a.k_cache) + head * p.k_head;
    const cache_t* vbase = static_cast<const cache_t*>(a.v_cache) + head * p.v_head;
    const uint32_t ktok = uint32_t(p.k_token) * kSize, vtok = uint32_t(p.v_token) * kSize;
    int ids = -1;                                                // page of run `lane` of the next 64

    auto runs = [&](int j, Run (&run)[2]) {
      const int key0 = lo + (j * W + wave) * 32;
      if ((j & 31) == 0) {
        const int64_t key = lo + (int64_t(j + (lane >> 1)) * W + wave) * 32 + (lane & 1) * 16;
        ids = key < hi ? page_of(p, b, int(key)) : -1;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int id = __builtin_amdgcn_readlane(ids, (j & 31) * 2 + h);
        const int key = key0 + h * 16;
        const int count = id < 0 ? 0 : (hi - key < 16 ? hi - key : 16);
        const int in = key & ((1 << p.page_shift) - 1);
        const int64_t page = id < 0 ? 0 : id;
        run[h].count = count;
        run[h].k = uniform_rsrc(kbase + page * p.k_page + in * p.k_token, count ? (count - 1) * ktok + D * kSize : 0);
        run[h].v = uniform_rsrc(vbase + page * p.v_page + in * p.v_token, count ? (count - 1) * vtok + D * kSize : 0);
      }
    };
    u32x4_t kf[2][kSteps];                                       // operand words of two 16-key runs
    auto load_k = [&](const Run (&run)[2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t row = r16 * ktok;
        if constexpr (kSize == 2) {
#pragma unroll
          for (int t = 0; t < kSteps; ++t)
            kf[h][t] = __builtin_amdgcn_raw_buffer_load_b128(run[h].k, row + t * 64 + g4 * 16, 0, kStreamOnce);
        } else {
          // Raw codes; two steps' worth in the first one's words.
#pragma unroll
          for (int t = 0; t + 1 < kSteps; t += 2)
            kf[h][t] = __builtin_amdgcn_raw_buffer_load_b128(run[h].k, row + t * 32 + g4 * 16, 0, kStreamOnce);
          if constexpr (kSteps & 1) {
            const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(run[h].k, row + (D - 32) + g4 * 8, 0, kStreamOnce);
            kf[h][kSteps - 1] = u32x4_t{w[0], w[1], 0, 0};
          }
        }
      }
    };
    auto key_words = [&](int h, int t) -> u32x4_t {
      if constexpr (kSize == 2) return kf[h][t];
      const u32x4_t w = kf[h][t & ~1];
      const uint32_t x = (t & 1) ? w[2] : w[0], y = (t & 1) ? w[3] : w[1];
      return u32x4_t{widen2<false>(QK(), x), widen2<true>(QK(), x), widen2<false>(QK(), y), widen2<true>(QK(), y)};
    };
    // Eight keys' words of each value chunk: per_lane components of a key.
    u32x4_t vf[Chunks<D>::count][8];
    auto load_v = [&](const Run (&run)[2]) {
#pragma unroll
      for (int c = 0; c < Chunks<D>::count; ++c) {
        constexpr int kMost = 8;
        const int n = Chunks<D>::per_lane(c);
#pragma unroll
        for (int j = 0; j < kMost; ++j) {
          const rsrc_t r = run[j >> 2].v;
          const uint32_t off = (g4 * 4 + (j & 3)) * vtok + (Chunks<D>::start(c) + r16 * n) * kSize;
          const int bytes = n * kSize;
          if (bytes == 16) {
            vf[c][j] = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kStreamOnce);
          } else if (bytes == 8) {
            const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, kStreamOnce);
            vf[c][j] = u32x4_t{w[0], w[1], 0, 0};
          } else if (bytes == 4) {
            vf[c][j] = u32x4_t{__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, kStreamOnce), 0, 0, 0};
          } else {
            vf[c][j] = u32x4_t{__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, kStreamOnce), 0, 0, 0};
          }
        }
      }
    };
    // Word e of key j of chunk c as two 16-bit values.
    auto value_word = [&](int c, int j, int e) -> uint32_t {
      if constexpr (kSize == 2) return vf[c][j][e];
      const uint32_t w = vf[c][j][e >> 1];
      return (e & 1) ? widen2<true>(PV(), w) : widen2<false>(PV(), w);
    };

    auto sees = [&](int at, int key) {
      return key <= at && (a.window == 0 || int64_t(key) > int64_t(at) - a.window);
    };
    auto is_clean = [&](int key0, const Run (&run)[2]) {         // every row sees every key
      return run[0].count == 16 && run[1].count == 16 && key0 + 31 <= place_lo &&
             (a.window == 0 || int64_t(key0) > int64_t(place_hi) - a.window);
    };
    // Zeros for the values that are not finite; whether the wave has any.  Adding one
    // to an exponent of all ones reaches the sign bit, and no other does.
    constexpr uint32_t kTop = kSize == 1 ? 0x7F7F7F7Fu : (__is_same(Cache, F16) ? 0x7C007C00u : 0x7F807F80u);
    constexpr uint32_t kOne = kSize == 1 ? 0x01010101u : (__is_same(Cache, F16) ? 0x04000400u : 0x00800080u);
    constexpr uint32_t kSign = kSize == 1 ? 0x80808080u : 0x80008000u;
    auto tame_values = [&]() {
      uint32_t any = 0;
#pragma unroll
      for (int c = 0; c < Chunks<D>::count; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < (Chunks<D>::per_lane(c) * kSize + 3) / 4; ++e) any |= (vf[c][k][e] & kTop) + kOne;
      if (__builtin_expect(__ballot((any & kSign) != 0) == 0, 1)) return false;
#pragma unroll
      for (int c = 0; c < Chunks<D>::count; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < (Chunks<D>::per_lane(c) * kSize + 3) / 4; ++e) {
            const uint32_t odd = ((vf[c][k][e] & kTop) + kOne) & kSign;        // top bit of each such value
            vf[c][k][e] &= ~(odd | (odd - (odd >> (kSize == 1 ? 7 : 15))));
          }
      return true;
    };
    // What tame_values left out, added where a row sees it.
    auto add_wild = [&](int key0, const Run& run) {
#pragma unroll 1
      for (int k = 0; k < run.count; ++k)
#pragma unroll
        for (int c = 0; c < Chunks<D>::count; ++c)
#pragma unroll
          for (int i = 0; i < Chunks<D>::per_lane(c); ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int comp = Chunks<D>::start(c) + (4 * g4 + r) * Chunks<D>::per_lane(c) + i;
              const uint32_t off = uint32_t(k) * vtok + comp * kSize;
              float x;
              asm volatile("" ::: "memory");                     // one load at a time: registers are short
              if constexpr (kSize == 1) {
                x = __builtin_amdgcn_cvt_f32_fp8(__builtin_amdgcn_raw_buffer_load_b8(run.v, off, 0, 0), 0);
              } else {
                const uint16_t w = __builtin_amdgcn_raw_buffer_load_b16(run.v, off, 0, 0);
                x = float(__builtin_bit_cast(cache_t, w));
              }
              if (fabsf(x) < __builtin_inff()) continue;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                if (sees(place[mt], key0 + k)) o[mt][Chunks<D>::tile(c) + i][r] += x;
            }
    };

    Run run[2], next[2];
    if (mine > 0) {
      runs(0, run);
      load_k(run);
      load_v(run);
    }
    __syncthreads();                                             // the last rows are done with LDS
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t r = (i * W + wave) * 4 + g4;
      float lift = 1.f;
      if constexpr (kSplit) {
        // 2^13 <= |q| 2^up < 2^14: high parts normal, low parts down to 2^-39 of the largest.
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < kUnits; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(qx[i][j][0][k]), fabsf(qx[i][j][1][k])));
        top = row16_top(top);
        const int e = int((word(top) >> 23) & 255) - 127;
        const int up = top > 0.f ? min(13 - e, 126) : 0;
        lift = __builtin_ldexpf(1.f, up);
        if (r16 == 0 && r < MT * 16) back[r] = __builtin_ldexpf(1.f, -up);
      }
      const int mt = r >> 4, rr = r & 15;
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        const int u = r16 + 16 * j;
        if (u >= D / 8 || r >= MT * 16) continue;
        const bool pairs = kSize == 1 && u < 8 * (D / 64);
        const int t = pairs ? 2 * (u / 8) + (u & 1) : u / 4;
        const int g = pairs ? (u % 8) / 2 : u % 4;
        const f32x4_t y = qx[i][j][0] * lift, z = qx[i][j][1] * lift;
        qf[(mt * kSteps + t) * 64 + g * 16 + rr] =
            u32x4_t{pack2(QK(), y[0], y[1]), pack2(QK(), y[2], y[3]), pack2(QK(), z[0], z[1]), pack2(QK(), z[2], z[3])};
        if constexpr (kSplit)
          qf[((MT + mt) * kSteps + t) * 64 + g * 16 + rr] =
              u32x4_t{pack2_rest(QK(), y[0], y[1]), pack2_rest(QK(), y[2], y[3]),
                      pack2_rest(QK(), z[0], z[1]), pack2_rest(QK(), z[2], z[3])};
      }
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      scale[mt] = a.scale;
      if constexpr (kSplit) scale[mt] *= back[mt * 16 + r16];
      if constexpr (kSize == 1) scale[mt] *= a.k_scale[head];
      m[mt] = kNone;
      sum[mt] = 0.f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) o[mt][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    bool wild = false;
    for (int j = 0; j < mine; ++j) {
      const int key0 = lo + (j * W + wave) * 32;
      f32x4_t sc[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) sc[mt][0] = sc[mt][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < kSteps; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4_t k = key_words(h, t);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            sc[mt][h] = mfma(QK(), k, qf[(mt * kSteps + t) * 64 + lane], sc[mt][h]);
            if constexpr (kSplit)
              sc[mt][h] = mfma(QK(), k, qf[((MT + mt) * kSteps + t) * 64 + lane], sc[mt][h]);
          }
        }
      const bool more = j + 1 < mine;
      if (more) {
        runs(j + 1, next);
        load_k(next);
      }
      const bool clean = is_clean(key0, run);
      u32x4_t pf[MT], pl[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = sc[mt][i >> 2][i & 3] * scale[mt];
        if (!clean) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int in = g4 * 4 + (i & 3);
            if (in >= run[i >> 2].count || !sees(place[mt], key0 + (i >> 2) * 16 + in)) x[i] = kNone;
          }
        }
        float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        top = fmaxf(m[mt], over_groups_max(top));
        const float base = top == kNone ? 0.f : top;             // no key yet: every p is 2^-inf
        const float shrink = __builtin_amdgcn_exp2f(m[mt] - base);
        m[mt] = top;
        float total = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = __builtin_amdgcn_exp2f(x[i] - base + kLift);
          total += x[i];
        }
        sum[mt] = sum[mt] * shrink + total;
        pf[mt] = u32x4_t{pack2(PV(), x[0], x[1]), pack2(PV(), x[2], x[3]), pack2(PV(), x[4], x[5]), pack2(PV(), x[6], x[7])};
        if constexpr (kSplit)
          pl[mt] = u32x4_t{pack2_rest(PV(), x[0], x[1]), pack2_rest(PV(), x[2], x[3]),
                           pack2_rest(PV(), x[4], x[5]), pack2_rest(PV(), x[6], x[7])};
#pragma unroll
        for (int i = 0; i < kTiles; ++i) o[mt][i] = o[mt][i] * shrink;
      }
      // Values that are not finite must not meet the zeros of rows that do not see them.
      if (!clean) wild |= tame_values();
#pragma unroll
      for (int c = 0; c < Chunks<D>::count; ++c)
#pragma unroll
        for (int e = 0; e < Chunks<D>::per_lane(c) / 2; ++e) {
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = value_word(c, k, e);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t pick = half ? 0x07060302u : 0x05040100u;
            u32x4_t v;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __builtin_amdgcn_perm(w[2 * k + 1], w[2 * k], pick);
            const int tile = Chunks<D>::tile(c) + 2 * e + half;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[mt][tile] = mfma(PV(), v, pf[mt], o[mt][tile]);
              if constexpr (kSplit) o[mt][tile] = mfma(PV(), v, pl[mt], o[mt][tile]);
            }
          }
        }
      if (more) {
        load_v(next);
        run[0] = next[0];
        run[1] = next[1];
      }
    }

    // Rare: once more over the tiles whose rows differ in what they see.
    if (__builtin_expect(wild, 0)) {
      for (int j = 0; j < mine; ++j) {
        runs(j, run);
        const int key0 = lo + (j * W + wave) * 32;
        if (is_clean(key0, run)) continue;
        add_wild(key0, run[0]);
        add_wild(key0 + 16, run[1]);
      }
    }

    // Join the waves.  Lane (r16, g4) holds row r16 and, of chunk c, components
    // start + (4 g4 + r) n + 0 .. n - 1.
    __syncthreads();                                             // q is done with
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      sum[mt] = over_groups_sum(sum[mt]);
      if (uint32_t(mt * 16 + r16) >= live_rows) continue;
      float* to = states + (wave * (MT * 16) + mt * 16 + r16) * kState;
#pragma unroll
      for (int c = 0; c < Chunks<D>::count; ++c) {
        constexpr int kLeast = 2;
        const int n = Chunks<D>::per_lane(c);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int i = 0; i < n; i += n < 4 ? kLeast : 4) {
            const int t = Chunks<D>::tile(c) + i, at = Chunks<D>::start(c) + (4 * g4 + r) * n + i;
            if (n >= 4)
              *reinterpret_cast<f32x4_t*>(to + at) =
                  f32x4_t{o[mt][t][r], o[mt][t + 1][r], o[mt][t + (n < 4 ? 0 : 2)][r], o[mt][t + (n < 4 ? 0 : 3)][r]};
            else
              *reinterpret_cast<float2*>(to + at) = float2{o[mt][t][r], o[mt][t + 1][r]};
          }
      }
      if (g4 == 0) {
        to[D] = m[mt];
        to[D + 1] = sum[mt];
      }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < live_rows * (D / 4); i += 64 * W) {
      const uint32_t r = i / (D / 4), c = i % (D / 4) * 4;
      const float* from = states + r * kState;
      float top = kNone, all = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, from[w * (MT * 16) * kState + D]);
      const float base = top == kNone ? 0.f : top;
      f32x4_t y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float* at = from + w * (MT * 16) * kState;
        const float f = __builtin_amdgcn_exp2f(at[D] - base);    // 0 where the wave had no key for the row
        all += at[D + 1] * f;
        y += *reinterpret_cast<const f32x4_t*>(at + c) * f;
      }
      const uint32_t row = row0 + r, token = row / group;
      const int qh = head * group + (row - token * group);
      const int64_t at = s.q0 + token;
      if (a.splits > 1) {
        float* part = a.part + ((at * p.q_heads + qh) * a.splits + split) * (D + 4);
        store4(F32(), part + 4 + c, y);
        if (c == 0) {
          part[0] = top;
          part[1] = all;
        }
      } else {
        const float vs = kSize == 1 ? a.v_scale[head] : 1.f;
        const float f = all > 0.f || all != all ? vs / all : 0.f;
        store4(Act(), static_cast<act_t*>(a.out) + at * a.o_token + qh * a.o_head + c, y * f);
      }
    }
  }
}

// Join the parts of a row (a new token and head).  G groups of L lanes, four components
// to a lane, take every G-th part; then their states meet in LDS.
template <class Act, int D, int G>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a) {
  constexpr int L = D <= 64 ? 16 : (D <= 128 ? 32 : 64);
  constexpr int kRows = 256 / (L * G);
  __shared__ float states[G > 1 ? G : 1][D + 4];
  const Pages& p = a.pages;
  const int lane = threadIdx.x % L, g = threadIdx.x / L % G;
  const uint32_t row = ((blockIdx.y << kRowShift) + blockIdx.x) * kRows + threadIdx.x / (L * G);
  const uint32_t tokens = uint32_t(p.tokens), token = row / uint32_t(p.q_heads);  // rows past the last one: no token
  const int qh = int(row % uint32_t(p.q_heads));
  const float* part = a.part + int64_t(row) * a.splits * (D + 4);
  const int c = lane * 4;
  // Parts are read kBatch at a time, the first ones before it is known how many the row
  // has (the workspace holds a.splits of them).
  constexpr int kBatch = 8;
  float pm[kBatch], ps[kBatch];
  f32x4_t py[kBatch];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * G;
      pm[j] = kNone;
      ps[j] = 0.f;
      py[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (i < a.splits && token < tokens && c < D) {
        const float* at = part + i * (D + 4);
        pm[j] = at[0];
        ps[j] = at[1];
        py[j] = load4(F32(), at + 4 + c);
      }
    }
  };
  fetch(g);
  int b = 0, parts = 0;
  constexpr int kPerWave = G == 1 ? 64 / L : 1;                  // rows of a wave
#pragma unroll
  for (int i = 0; i < kPerWave; ++i) {
    const uint32_t t = __builtin_amdgcn_readlane(token, i * L);
    const int of = t < tokens ? owner(p, int(t)) : p.batch;
    if (kPerWave == 1 || int(threadIdx.x & 63) / L == i) b = of;
  }
  bool live = token < tokens && b < p.batch;
  if (live) {
    const Seq s = sequence(p, b);
    live = int(token) >= s.q0 && int(token) < s.q0 + s.q_len;
    parts = live ? parts_of(s, a.window, a.splits, a.split_keys).count : 0;
  }
  float m = kNone, base = 0.f, sum = 0.f;
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = g; i0 < parts; i0 += kBatch * G) {
    if (i0 > g) fetch(i0);
    float top = m;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (i0 + j * G < parts) top = fmaxf(top, pm[j]);
    base = top == kNone ? 0.f : top;
    const float shrink = __builtin_amdgcn_exp2f(m - base);
    m = top;
    sum *= shrink;
    y *= shrink;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (i0 + j * G >= parts) continue;
      const float f = __builtin_amdgcn_exp2f(pm[j] - base);      // 0 for a part with no key for the row
      sum += ps[j] * f;
      y += py[j] * f;
    }
  }
  if constexpr (G > 1) {
    if (c < D) *reinterpret_cast<f32x4_t*>(&states[g][c]) = y;
    if (lane == 0) {
      states[g][D] = m;
      states[g][D + 1] = sum;
    }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 0; i < G; ++i) m = fmaxf(m, states[i][D]);
    base = m == kNone ? 0.f : m;
    sum = 0.f;
    y = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float f = __builtin_amdgcn_exp2f(states[i][D] - base);
      sum += states[i][D + 1] * f;
      if (c < D) y += *reinterpret_cast<const f32x4_t*>(&states[i][c]) * f;
    }
  }
  if (!live || c >= D) return;
  const float vs = a.v_scale ? a.v_scale[qh / int(a.group)] : 1.f;
  const float f = sum > 0.f || sum != sum ? vs / sum : 0.f;
  typedef typename Act::elem act_t;
  store4(Act(), static_cast<act_t*>(a.out) + int64_t(token) * a.o_token + qh * a.o_head + c, y * f);
}

template <class Act, class Cache, int D, int MT, int W>
hipError_t launch_stream(const AttnArgs& a, const AttnPlan& plan, hipStream_t stream) {
  constexpr size_t lds = StreamLds<Act, D, MT, W>::bytes;
  auto fn = stream_kernel<Act, Cache, D, MT, W>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  const Grid grid = stream_grid(plan, a.pages.kv_heads, a.pages.batch);
  hipLaunchKernelGGL(fn, dim3(grid.x, grid.y, grid.z), dim3(64 * W), lds, stream, a);
  return hipGetLastError();
}

template <class Act, class Cache, int D>
hipError_t launch_rows(const AttnArgs& a, const AttnPlan& plan, hipStream_t stream) {
  if constexpr (D <= 128) {
    if (plan.row_tiles == 2) return launch_stream<Act, Cache, D, 2, 4>(a, plan, stream);
  }
  return launch_stream<Act, Cache, D, 1, 4>(a, plan, stream);
}

template <class Act, class Cache>
hipError_t launch_dim(const AttnArgs& a, const AttnPlan& plan, hipStream_t stream) {
  switch (a.pages.head_dim) {
    case 64: return launch_rows<Act, Cache, 64>(a, plan, stream);
    case 96: return launch_rows<Act, Cache, 96>(a, plan, stream);
    case 128: return launch_rows<Act, Cache, 128>(a, plan, stream);
    case 192: return launch_rows<Act, Cache, 192>(a, plan, stream);
    default: return launch_rows<Act, Cache, 256>(a, plan, stream);
  }
}

hipError_t launch_streaming(const AttnArgs& a, const AttnPlan& plan, int act, int cache, hipStream_t stream) {
  const bool narrow = cache == TQ2_TYPE_E4M3;
  if (act == TQ2_TYPE_F32)
    return narrow ? launch_dim<F32, E4M3>(a, plan, stream) : launch_dim<F32, F16>(a, plan, stream);
  if (act == TQ2_TYPE_F16)
    return narrow ? launch_dim<F16, E4M3>(a, plan, stream) : launch_dim<F16, F16>(a, plan, stream);
  return narrow ? launch_dim<BF16, E4M3>(a, plan, stream) : launch_dim<BF16, BF16>(a, plan, stream);
}

template <class Act, int D>
hipError_t launch_join(const AttnArgs& a, hipStream_t stream) {
  constexpr int L = D <= 64 ? 16 : (D <= 128 ? 32 : 64);
  const int64_t rows = int64_t(a.pages.tokens) * a.pages.q_heads;
  // A whole block for each row once there are parts for all of it.
  const Grid grid = row_grid(a.splits > 8 ? rows : pieces(rows, 256 / L));
  if (a.splits > 8)
    hipLaunchKernelGGL((join_kernel<Act, D, 256 / L>), dim3(grid.x, grid.y), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((join_kernel<Act, D, 1>), dim3(grid.x, grid.y), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <class Act>
hipError_t launch_join_dim(const AttnArgs& a, hipStream_t stream) {
  switch (a.pages.head_dim) {
    case 64: return launch_join<Act, 64>(a, stream);
    case 96: return launch_join<Act, 96>(a, stream);
    case 128: return launch_join<Act, 128>(a, stream);
    case 192: return launch_join<Act, 192>(a, stream);
    default: return launch_join<Act, 256>(a, stream);
  }
}

}  // namespace

hipError_t launch_paged_attention(const AttnArgs& a, const AttnPlan& plan, int act, int cache,
                                  hipStream_t stream) {
  const hipError_t e = plan.tiled ? launch_attention_tiles(a, plan, act, cache, stream)
                                  : launch_streaming(a, plan, act, cache, stream);
  if (e != hipSuccess || plan.splits == 1) return e;
  if (act == TQ2_TYPE_F32) return launch_join_dim<F32>(a, stream);
  if (act == TQ2_TYPE_F16) return launch_join_dim<F16>(a, stream);
  return launch_join_dim<BF16>(a, stream);
}

}  // namespace tq2
