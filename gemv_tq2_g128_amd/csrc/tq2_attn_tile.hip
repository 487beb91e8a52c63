// Attention of new tokens over a paged cache, tiled form for many rows.
//
// Bound.  A block of 128 rows (new tokens times the query heads that share a key
// head) does 256 operations with every key and value component it reads: the
// matrix cores, with the exponentials close behind (one for each 4 * head_dim
// operations).
//
// Work split.  Four waves of 32 rows share tiles of 64 keys in LDS, filled two
// tiles deep by loads that go to LDS directly; two blocks fit on a CU, so that
// one's softmax runs under the other's products.  Query, running maximum, sum and
// output stay in registers.
//
// Matrix form (v_mfma_f32_32x32x16).  S^T = K Q^T: a lane holds 16 of 32 keys'
// scores of one row.  O^T = V^T P^T: packed in pairs these are the operand words
// of two matrix steps as they are, with the keys of a step in the order
// 4 h + j, 8 + 4 h + j of lane half h; the LDS transpose read gives V^T's words in
// that order: four keys of one component at a time.
//
// Running maximum.  The output is rescaled only when a row's maximum has grown by
// more than 2^8 since the last time; until then probabilities run up to 2^8, which
// f32 sums and (with the lift of 2^7) binary16 words hold as exactly.
//
// LDS.  Rows of keys lie 16-byte chunk by chunk, rows of values by 64 bytes, under an
// exclusive or with the row number that keeps the rows read together in different banks.
// The loads apply it on the address they read from.
//
// f32 q, e4m3 caches, masks and the rounding of probabilities as in the streaming form.
//
// Measured: 512 new tokens over 16,895 keys, 32 heads of 128 on 8 key heads, f16: 161 us
// with joining (867 TFLOP/s); two prompts of up to 4,096, bf16: 260 us (873).  Matrix
// cores are busy 43 % of the cycles, the vector ALU 41 %: what runs of one under the
// other is what two waves a SIMD happen to overlap.
#include "tq2_attn_device.h"

namespace tq2 {
namespace {

constexpr int kWaves = 4;
static_assert(kTileRows == 32 * kWaves, "32 rows a wave");
constexpr int kKeys = 64;                        // keys of a tile: one 16-key run per wave
constexpr float kSlack = 8.f;                    // log2 of the growth that is left unscaled

constexpr int kAhead = 4;                        // reads of keys in front of their matrix steps

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t* lds_s16x4_t;
typedef __attribute__((address_space(3))) const u32x4_t* lds_u32x4_t;
typedef __attribute__((address_space(3))) unsigned char* lds_byte_t;

// Where 16-byte chunk c of row r of a tile lies within its row.  LDS has 256 bytes of
// banks: 16 rows' chunks c of keys, and the two neighbouring 32-byte pieces of four rows
// of values that half a wave's transpose read takes, have to lie in different ones.
template <int D>
struct Place {
  static constexpr int chunks = D / 8;
  static constexpr int key_turn = D == 96 ? 4 : (D == 64 || D == 192 ? 8 : 16);  // chunks a turn moves among
  __device__ __forceinline__ static int key(int r, int c) {
    return c ^ (D == 96 ? (r >> 2) & 3 : (D == 64 || D == 192 ? (r >> 1) & 7 : r & 15));
  }
  // Values by 64 bytes: a 32-component tile of the output.
  static constexpr int value_turn = D == 96 ? 1 : (D == 64 || D == 192 ? 2 : 4);
  __device__ __forceinline__ static int value_tile(int r, int dt) {
    return dt ^ (D == 96 ? 0 : (D == 64 || D == 192 ? (r >> 1) & 1 : r & 3));
  }
  __device__ __forceinline__ static int value(int r, int c) { return value_tile(r, c >> 2) * 4 + (c & 3); }
};

// 16 bytes a lane from base + off to LDS at + 16 * lane; past the range: zeros.  The
// compiler does not see the load: the five wait states that it would put between a
// vector instruction's write of a resource word (a lane read) and the load are here.  m0 is
// named as written: the compiler keeps no value there (hence its warning), but must not
// move this between a write of its own and the use.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(rsrc_t r, uint32_t off, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               ::"s"(at), "v"(off), "s"(r) : "memory", "m0");
}
#pragma clang diagnostic pop
// The larger of two; NaN if one is (fmaxf would first quiet its operands).
__device__ __forceinline__ float largest(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Every load to LDS of this wave is in, then every wave's.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16 bytes of a key at + off; four values of a component at + off and as many at
// + off + far.
__device__ __forceinline__ u32x4_t lds_keys(uint32_t at, int off) {
  return *reinterpret_cast<lds_u32x4_t>(reinterpret_cast<lds_byte_t>(at) + off);
}
__device__ __forceinline__ u32x4_t lds_values(uint32_t at, int off, int far) {
  const lds_byte_t from = reinterpret_cast<lds_byte_t>(at) + off;
  const s16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4_t>(from));
  const s16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4_t>(from + far));
  const u32x2_t u = __builtin_bit_cast(u32x2_t, x), v = __builtin_bit_cast(u32x2_t, y);
  return u32x4_t{u[0], u[1], v[0], v[1]};
}

// Waves per SIMD that the register budget aims at.
template <class Act, int D>
constexpr int kMinWaves = D <= 64 || (D <= 128 && !__is_same(Act, F32)) ? 2 : 1;

template <class Act, class Cache, int D>
__global__ __launch_bounds__(64 * kWaves, (kMinWaves<Act, D>)) void tile_kernel(AttnArgs a, int steps) {
  typedef typename Kinds<Act, Cache>::QK QK;
  typedef typename Kinds<Act, Cache>::PV PV;
  typedef typename Act::elem act_t;
  typedef typename Cache::elem cache_t;
  constexpr bool kSplit = __is_same(Act, F32);                   // q and probabilities in two parts
  constexpr float kLift = __is_same(PV, F16) ? 7.f : 0.f;
  constexpr int kSize = int(sizeof(cache_t));
  constexpr int kSteps = D / 16;                                 // matrix steps of a score
  constexpr int kTiles = D / 32;                                 // 32-component tiles of the output
  constexpr int kRows = kTileRows;
  constexpr int kRowBytes = 2 * D;
  constexpr int kTileBytes = kKeys * kRowBytes;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];  // K, K, V, V, flag
  int* flag = reinterpret_cast<int*>(smem + 4 * kTileBytes);     // a tile had values that are not finite

  const Pages& p = a.pages;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  const uint32_t group = a.group;
  // Key heads vary fastest: with 8 of them each XCD's cache holds one head.
  // Later tokens, which see more keys, come first.
  uint32_t id = blockIdx.x;
  const int head = id % p.kv_heads;
  id /= p.kv_heads;
  const int split = id % a.splits;
  id /= a.splits;
  const int step = steps - 1 - int(id);
  const int b = blockIdx.y;
  const Seq s = sequence(p, b);
  const uint32_t rows = uint32_t(s.q_len) * group;               // below 2^31
  const Parts parts = parts_of(s, a.window, a.splits, a.split_keys);
  if (split >= parts.count) return;

  const uint32_t lds = uint32_t(uintptr_t((__attribute__((address_space(3))) unsigned char*)(smem)));
  const cache_t* kbase = static_cast<const cache_t*>(a.k_cache) + head * p.k_head;
  const cache_t* vbase = static_cast<const cache_t*>(a.v_cache) + head * p.v_head;
  const uint32_t ktok = uint32_t(p.k_token) * kSize, vtok = uint32_t(p.v_token) * kSize;

  for (uint32_t row0 = uint32_t(step) * kRows; row0 < rows; row0 += uint32_t(steps) * kRows) {
    const int last = int(row0 + kRows < rows ? kRows : rows - row0) - 1;
    const int block_hi = s.first + int((row0 + last) / group), block_lo = s.first + int(row0 / group);
    const int start = parts.base + split * parts.per;
    const int part_end = s.keys - start < parts.per ? s.keys : start + parts.per;
    const int hi = block_hi + 1 < part_end ? block_hi + 1 : part_end;
    int lo = start;
    if (a.window) {
      const int64_t edge = int64_t(block_lo) - a.window + 1;
      if (edge > lo) lo = edge < part_end ? int(edge) & ~31 : part_end;
    }
    const int tiles = hi > lo ? (hi - lo + kKeys - 1) / kKeys : 0;

    // The wave's rows, and q in operand order: components 16 t + 8 h + 0 .. 7 of row r32.
    const uint32_t wave_row = row0 + wave * 32;
    const uint32_t wave_end = wave_row + 32 <= rows ? wave_row + 31 : rows - 1;
    const int place_lo = s.first + int(wave_row / group);
    const int place_hi = wave_row < rows ? s.first + int(wave_end / group) : -1;
    const uint32_t row = wave_row + r32;
    const bool live = row < rows;
    const int place = live ? s.first + int(row / group) : -1;
    const int64_t token = s.q0 + row / group;
    const int qh = head * group + row % group;
    const int64_t out_of = a.window ? int64_t(place) - a.window : -1;
    const int below = out_of < -1 ? -1 : int(out_of);            // keys up to here are out of the window
    float scale = a.scale;
    if constexpr (kSize == 1) scale *= a.k_scale[head];
    // Scores meet the mask and the maximum before they meet the scale, which therefore has to
    // be positive: a negative one turns q's sign, and zero becomes the least number, which
    // leaves every score at 0 and a masked one at -infinity.
    const bool turned = kSize == 1 && scale < 0.f;
    u32x4_t q[kSteps], q2[kSplit ? kSteps : 1];
    const act_t* src = static_cast<const act_t*>(a.q) + (live ? token * a.q_token + qh * a.q_head : 0) + 8 * h;
    float lift = 1.f;
    f32x4_t x[kSplit ? kSteps : 1][2];
    if constexpr (kSplit) {
      float top = 0.f;
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        x[t][0] = x[t][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (live) {
          x[t][0] = load4(Act(), src + t * 16);
          x[t][1] = load4(Act(), src + t * 16 + 4);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(x[t][0][j]), fabsf(x[t][1][j])));
      }
      const float2 both = halves32(top);
      top = fmaxf(both.x, both.y);
      const int e = int((word(top) >> 23) & 255) - 127;
      const int up = top > 0.f ? min(13 - e, 126) : 0;
      lift = turned ? -__builtin_ldexpf(1.f, up) : __builtin_ldexpf(1.f, up);
      scale *= __builtin_ldexpf(1.f, -up);
    }
    scale = scale == 0.f ? 0x1p-149f : fabsf(scale);
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      if constexpr (kSplit) {
        const f32x4_t y = x[t][0] * lift, z = x[t][1] * lift;
        q[t] = u32x4_t{pack2(QK(), y[0], y[1]), pack2(QK(), y[2], y[3]), pack2(QK(), z[0], z[1]), pack2(QK(), z[2], z[3])};
        q2[t] = u32x4_t{pack2_rest(QK(), y[0], y[1]), pack2_rest(QK(), y[2], y[3]),
                        pack2_rest(QK(), z[0], z[1]), pack2_rest(QK(), z[2], z[3])};
      } else {
        q[t] = live ? *reinterpret_cast<const u32x4_t*>(src + t * 16) : u32x4_t{0, 0, 0, 0};
        if constexpr (kSize == 1) q[t] ^= turned ? 0x80008000u : 0u;
      }
    }
    float m = kNone, sum = 0.f;
    f32x16_t o[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] = 0.f;

    // Loads of a tile: wave w fills the 16 rows of run w.
    int ids = -1;                                                // page of run `lane` of the next 16 tiles
    uint64_t missing = 0;                                        // runs of them that have none
    rsrc_t run_k, run_v;
    auto find = [&](int j) {
      if ((j & 15) == 0) {
        const int64_t key = lo + (int64_t(j) * 4 + lane) * 16;
        ids = key < hi ? page_of(p, b, int(key)) : -1;
        missing = __ballot(ids < 0);
      }
      const int key = lo + j * kKeys + wave * 16;
      const int page = __builtin_amdgcn_readlane(ids, (j & 15) * 4 + wave);
      const int count = page < 0 ? 0 : (hi - key < 16 ? hi - key : 16);
      const int in = key & ((1 << p.page_shift) - 1);
      const int64_t at = page < 0 ? 0 : page;
      run_k = uniform_rsrc(kbase + at * p.k_page + in * p.k_token, count ? (count - 1) * ktok + D * kSize : 0);
      run_v = uniform_rsrc(vbase + at * p.v_page + in * p.v_token, count ? (count - 1) * vtok + D * kSize : 0);
    };
    constexpr int kCodes = (D + 63) / 64;                        // 16-byte loads of e4m3 codes per lane
    u32x4_t codes_k[kSize == 1 ? kCodes : 1], codes_v[kSize == 1 ? kCodes : 1];
    auto load = [&](int buf) {
      if constexpr (kSize == 2) {
        const uint32_t to_k = lds + buf * kTileBytes + wave * (16 * kRowBytes), to_v = to_k + 2 * kTileBytes;
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
          const int i = n * 64 + lane, r = i / Place<D>::chunks, c = i % Place<D>::chunks;
          load_to_lds(run_k, r * ktok + Place<D>::key(r, c) * 16, to_k + n * 1024);
          load_to_lds(run_v, r * vtok + Place<D>::value(r, c) * 16, to_v + n * 1024);
        }
      } else {
#pragma unroll
        for (int n = 0; n < kCodes; ++n) {
          const int i = n * 64 + lane, r = i / (D / 16), c = i % (D / 16);
          codes_k[n] = __builtin_amdgcn_raw_buffer_load_b128(run_k, r * ktok + c * 16, 0, 0);
          codes_v[n] = __builtin_amdgcn_raw_buffer_load_b128(run_v, r * vtok + c * 16, 0, 0);
        }
      }
    };
    auto store = [&](int buf) {                                  // e4m3: widened into the tile
      if constexpr (kSize == 1) {
        unsigned char* to_k = smem + buf * kTileBytes + wave * (16 * kRowBytes);
        unsigned char* to_v = to_k + 2 * kTileBytes;
#pragma unroll
        for (int n = 0; n < kCodes; ++n) {
          const int i = n * 64 + lane, r = i / (D / 16), c = i % (D / 16);
          if (D % 64 && i >= D) continue;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t k0 = codes_k[n][2 * e], k1 = codes_k[n][2 * e + 1];
            const uint32_t v0 = codes_v[n][2 * e], v1 = codes_v[n][2 * e + 1];
            *reinterpret_cast<u32x4_t*>(to_k + r * kRowBytes + Place<D>::key(r, 2 * c + e) * 16) =
                u32x4_t{widen2<false>(QK(), k0), widen2<true>(QK(), k0), widen2<false>(QK(), k1), widen2<true>(QK(), k1)};
            *reinterpret_cast<u32x4_t*>(to_v + r * kRowBytes + Place<D>::value(r, 2 * c + e) * 16) =
                u32x4_t{widen2<false>(PV(), v0), widen2<true>(PV(), v0), widen2<false>(PV(), v1), widen2<true>(PV(), v1)};
          }
        }
      }
    };
    // Operand addresses in a tile.  Keys: chunk 2 t + h of row r32, whose low bits the
    // exclusive or turns; the others, and the second 32 rows, are constant offsets.
    // Values: lane l16 of a 16-lane group reads 8 bytes of row 4 h + l16 / 4, and so on.
    constexpr int kTurn = Place<D>::key_turn, kValueTurn = Place<D>::value_turn;
    const int l16 = lane & 15;
    uint32_t key_at[kTurn / 2], value_at[kValueTurn];
#pragma unroll
    for (int t = 0; t < kTurn / 2; ++t) key_at[t] = lds + r32 * kRowBytes + Place<D>::key(r32, 2 * t + h) * 16;
#pragma unroll
    for (int dt = 0; dt < kValueTurn; ++dt)
      value_at[dt] = lds + 2 * kTileBytes + (4 * h + (l16 >> 2)) * kRowBytes + (l16 & 3) * 8 +
                     Place<D>::value_tile(l16 >> 2, dt) * 64 + ((lane >> 4) & 1) * 32;
    // The wave's 16 rows of values: zeros for what is not finite, and the flag.
    auto tame = [&](int buf) {
      constexpr uint32_t kTop = __is_same(PV, F16) ? 0x7C00u : 0x7F80u;
      u32x4_t* at = reinterpret_cast<u32x4_t*>(smem + (2 + buf) * kTileBytes + wave * (16 * kRowBytes)) + lane;
#pragma unroll 1
      for (int n = 0; n < D / 32; ++n, at += 64) {
        u32x4_t v = *at;
        uint32_t any = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w = v[e];
          if ((w & kTop) == kTop) w &= 0xFFFF0000u;
          if ((w >> 16 & kTop) == kTop) w &= 0xFFFFu;
          any |= w ^ v[e];
          v[e] = w;
        }
        if (any) {
          *at = v;
          *flag = 1;
        }
      }
    };

    bool wild = false;
    uint32_t gone = 0;                                           // runs of the tile without a page
    __syncthreads();                                             // the last rows' tiles are done with
    if (threadIdx.x == 0) *flag = 0;
    if (tiles > 0) {
      find(0);
      gone = uint32_t(missing) & 15;
      load(0);
      store(0);
    }
    tile_barrier();
    for (int j = 0; j < tiles; ++j) {
      const int buf = j & 1;
      const bool more = j + 1 < tiles;
      const int key0 = lo + j * kKeys;
      // Where rows of the block differ in what they see, the values that are not finite
      // become zeros: they must not meet the zeros of rows that do not see them.
      if (gone != 0 || key0 + kKeys - 1 > block_lo || key0 + kKeys > hi ||
          (a.window != 0 && int64_t(key0) <= int64_t(block_hi) - a.window)) {
        tame(buf);
        tile_barrier();
        wild = *flag != 0;
      }
      uint32_t next_gone = 0;
      if (more) {
        find(j + 1);
        next_gone = uint32_t(missing >> (((j + 1) & 15) * 4)) & 15;
        load(buf ^ 1);
      }
      const bool some = key0 <= place_hi &&
                        (a.window == 0 || int64_t(key0) + kKeys - 1 > int64_t(place_lo) - a.window);
      const bool clean = gone == 0 && key0 + kKeys - 1 <= place_lo && key0 + kKeys <= hi &&
                         (a.window == 0 || int64_t(key0) > int64_t(place_hi) - a.window);
      if (some) {
        // Scores.  Reads of keys run kAhead in front of the matrix steps that take them.
        f32x16_t x[2];
#pragma unroll
        for (int r = 0; r < 16; ++r) x[0][r] = x[1][r] = 0.f;
        u32x4_t kf[2 * kSteps];
        auto read_key = [&](int i) {                             // step i / 2 of the 32 keys i % 2
          kf[i] = lds_keys(key_at[i / 2 % (kTurn / 2)] + buf * kTileBytes,
                           (i & 1) * 32 * kRowBytes + i / 2 / (kTurn / 2) * kTurn * 16);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) read_key(i);
#pragma unroll
        for (int i = 0; i < 2 * kSteps; ++i) {
          if (i + kAhead < 2 * kSteps) read_key(i + kAhead);
          __builtin_amdgcn_sched_barrier(0);
          x[i & 1] = mfma(QK(), kf[i], q[i / 2], x[i & 1]);
          if constexpr (kSplit) x[i & 1] = mfma(QK(), kf[i], q2[i / 2], x[i & 1]);
          __builtin_amdgcn_sched_barrier(0);
        }
        u32x4_t vf[2][kTiles];
        auto read_value = [&](int t, int dt) {
          vf[t & 1][dt] = lds_values(value_at[dt % kValueTurn] + buf * kTileBytes,
                                     16 * t * kRowBytes + dt / kValueTurn * kValueTurn * 64, 8 * kRowBytes);
        };
#pragma unroll
        for (int dt = 0; dt < kTiles; ++dt) read_value(0, dt);
        if (!clean) {
          const int upto = (place < hi ? place : hi - 1) - key0 - 4 * h, over = below - key0 - 4 * h;
#pragma unroll
          for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int key = kt * 32 + 8 * (r >> 2) + (r & 3);  // and 4 h
              if (key > upto || key <= over || (gone >> (kt * 2 + (r >> 3)) & 1)) x[kt][r] = kNone;
            }
        }
        float top = kNone;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int r = 0; r < 16; r += 2) top = largest(largest(x[kt][r], x[kt][r + 1]), top);
        const float2 both = halves32(top);
        top = largest(both.x, both.y) * scale;
        if (__ballot(top > m + kSlack) != 0) {
          const float grown = fmaxf(m, top);
          const float shrink = grown == kNone ? 1.f : __builtin_amdgcn_exp2f(m - grown);
          m = grown;
          sum *= shrink;
#pragma unroll
          for (int i = 0; i < kTiles; ++i) o[i] = o[i] * shrink;
        }
        const float base = m == kNone ? 0.f : m - kLift;
        // Probabilities, two at a time: those of the second 32 keys, and the reads of the
        // next step's values, lie between the matrix steps of the first 32.
        u32x4_t pf[4], pl[kSplit ? 4 : 1];
        auto probabilities = [&](int kt, int i) {
          const float u = __builtin_amdgcn_exp2f(__builtin_fmaf(x[kt][2 * i], scale, -base));
          const float v = __builtin_amdgcn_exp2f(__builtin_fmaf(x[kt][2 * i + 1], scale, -base));
          sum += u + v;
          pf[kt * 2 + (i >> 2)][i & 3] = pack2(PV(), u, v);
          if constexpr (kSplit) pl[kt * 2 + (i >> 2)][i & 3] = pack2_rest(PV(), u, v);
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) probabilities(0, i);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int dt = 0; dt < kTiles; ++dt) {
            const int slot = t * kTiles + dt;
            if (t < 3) read_value(t + 1, dt);
            __builtin_amdgcn_sched_barrier(0);
            o[dt] = mfma(PV(), vf[t & 1][dt], pf[t], o[dt]);
            if constexpr (kSplit) o[dt] = mfma(PV(), vf[t & 1][dt], pl[t], o[dt]);
            if (t < 2) {
#pragma unroll
              for (int i = slot * 8 / (2 * kTiles); i < (slot + 1) * 8 / (2 * kTiles); ++i) probabilities(1, i);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
      }
      gone = next_gone;
      if (more) store(buf ^ 1);
      tile_barrier();
    }
    // Rare: what was left out, added where a row sees it.
    if (wild) {
#pragma unroll 1
      for (int key = lo; key < hi; ++key) {
        const int page = page_of(p, b, key);
        if (page < 0) continue;
        const int in = key & ((1 << p.page_shift) - 1);
        const cache_t* v = vbase + page * p.v_page + in * p.v_token + 4 * h;
#pragma unroll
        for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            asm volatile("" ::: "memory");                       // one load at a time: registers are short
            const cache_t w = v[dt * 32 + 8 * (r >> 2) + (r & 3)];
            float x;
            if constexpr (kSize == 1) x = __builtin_amdgcn_cvt_f32_fp8(w, 0);
            else x = float(w);
            if (fabsf(x) < __builtin_inff()) continue;
            if (key <= place && key > below) o[dt][r] += x;
          }
      }
    }
    // Lane (r32, h) holds components 32 dt + 8 i + 4 h + 0 .. 3 of row r32.
    const float2 both = halves32(sum);
    const float all = both.x + both.y;
    if (!live) continue;
    const float vs = kSize == 1 ? a.v_scale[head] : 1.f;
    const float f = a.splits > 1 ? 1.f : (all > 0.f || all != all ? vs / all : 0.f);
    float* part = a.part + ((token * p.q_heads + qh) * a.splits + split) * (D + 4);
    act_t* dst = static_cast<act_t*>(a.out) + token * a.o_token + qh * a.o_head;
#pragma unroll
    for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4_t y = f32x4_t{o[dt][4 * i], o[dt][4 * i + 1], o[dt][4 * i + 2], o[dt][4 * i + 3]} * f;
        const int at = 32 * dt + 8 * i + 4 * h;
        if (a.splits > 1) store4(F32(), part + 4 + at, y);
        else store4(Act(), dst + at, y);
      }
    if (a.splits > 1 && h == 0) {
      part[0] = m;
      part[1] = all;
    }
  }
}

template <class Act, class Cache, int D>
hipError_t launch(const AttnArgs& a, const AttnPlan& plan, hipStream_t stream) {
  constexpr size_t lds = size_t(4) * kKeys * 2 * D + 16;
  auto fn = tile_kernel<Act, Cache, D>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  const Grid grid = tile_grid(plan, a.pages.kv_heads, a.pages.batch);
  hipLaunchKernelGGL(fn, dim3(grid.x, grid.y, grid.z), dim3(64 * kWaves), lds, stream, a, plan.steps);
  return hipGetLastError();
}

template <class Act, class Cache>
hipError_t launch_dim(const AttnArgs& a, const AttnPlan& plan, hipStream_t stream) {
  switch (a.pages.head_dim) {
    case 64: return launch<Act, Cache, 64>(a, plan, stream);
    case 96: return launch<Act, Cache, 96>(a, plan, stream);
    case 128: return launch<Act, Cache, 128>(a, plan, stream);
    case 192: return launch<Act, Cache, 192>(a, plan, stream);
    default: return launch<Act, Cache, 256>(a, plan, stream);
  }
}

}  // namespace

hipError_t launch_attention_tiles(const AttnArgs& a, const AttnPlan& plan, int act, int cache, hipStream_t stream) {
  const bool narrow = cache == TQ2_TYPE_E4M3;
  if (act == TQ2_TYPE_F32)
    return narrow ? launch_dim<F32, E4M3>(a, plan, stream) : launch_dim<F32, F16>(a, plan, stream);
  if (act == TQ2_TYPE_F16)
    return narrow ? launch_dim<F16, E4M3>(a, plan, stream) : launch_dim<F16, F16>(a, plan, stream);
  return narrow ? launch_dim<BF16, E4M3>(a, plan, stream) : launch_dim<BF16, BF16>(a, plan, stream);
}

}  // namespace tq2
