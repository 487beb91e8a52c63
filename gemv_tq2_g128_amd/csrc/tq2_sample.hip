// The next token of each row of logits: temperature, top-k, min-p, top-p, and a draw by a given random number.
//
// Order.  All truncations keep a run from the top of the order (logit falling, index rising), and so does the draw: the
// token is where the running sum of e = exp((l - max) / T), from the top, passes u times the kept sum.  So nothing is
// sorted: a histogram over the logits, of counts and of sums, says in which bin the k-th token, the end of top-p's run
// or the drawn one lies, and only that bin's tokens are put in order.
//
// Whole numbers.  e is computed in f64 and rounded to a multiple of 2^-43 of the largest of its chunk; sums are then
// u64, exact in any order, which is what makes LDS atomics allowed here and the result one that repeats.  (32-bit
// exponentials would give another token than the definition once in a few dozen draws over 10^5 tokens: that many
// borders lie within 1e-7 of u.)
//
// Two launches.  bins_kernel: blocks for chunks of each row, held in registers: their largest logit, then counts and sums
// in bins of a fixed grid (11 to a factor of two in e, so that chunks agree on them), and the tokens' places ordered by
// bin.  What min_p or top_k drop of a chunk alone is dropped at once.  choice_kernel: a block for each row, which joins the
// chunks' bins at the row's largest logit and reads the tokens of the bins it needs.  Bound: logits are read from HBM
// once, two bytes are written for each that is not dropped.
//
// Measured (us): one row of 32,000 f32 logits with top-k and top-p 5.8 and 12.1, one of 131,072 with top-p 8 and 14 to 26 (more for others),
// by how many tokens share the run's last bin: chains of dependent steps, not bytes.  64 rows of 128,255 in bf16 of mixed
// settings 20 and 34.  256 rows of 151,936 f32 logits with min-p 50 (3.1 TB/s) and 21.
#include "tq2_device.h"
#include "tq2_sample_bins.h"
#include "tq2_sample_internal.h"
#include "tq2_types.h"

#pragma clang fp contract(off)

namespace tq2 {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kMaxChunks = 64;
constexpr int kThreads = 1024;             // of bins_kernel
constexpr int kRowThreads = kBins;         // of the choice: a thread for each bin
constexpr int kRowWaves = kRowThreads / 64;
constexpr uint32_t kList = 4096;           // tokens of a bin that are held in LDS
constexpr uint32_t kFew = kRowThreads / 4; // tokens that are put in order at once: four threads for each
constexpr int kUnit = 43;                  // a token of the largest logit weighs 2^43
constexpr double kCoolest = 1e-36;         // temperatures below act as this one

struct Args {
  const void* logits;
  const float* u;
  int32_t* ids;
  float* logprob;
  const float* temperatures;
  const int32_t* top_ks;
  const float* top_ps;
  const float* min_ps;
  int32_t top_k, vocab, chunks;
  int32_t chunk_shift;                     // log2 of a chunk's vectors
  int64_t row_stride;
  double temperature, top_p, min_p;
  uint64_t* sums;                          // [rows, chunks, kBins]
  uint32_t* counts;                        // the same: where the bin's tokens start in `order`, in the upper half, and their number
  float* tops;                             // [rows, chunks]: largest logit
  uint16_t* order;                         // [rows, chunks, chunk_tokens]: places in the chunk, by bins
  int32_t chunk_tokens;
};

// Element types by their bits, f32 by f32.  kNone, a NaN, fills places past the row: it has no bin at any temperature,
// where -infinity times a large enough grid shares one with finite logits.
template <class T>
struct Bits;
template <>
struct Bits<F32> {
  static constexpr int kVec = 4;
  static constexpr uint32_t kNone = 0x7FC00000u;
  static __device__ float get(u32x4_t v, int i) { return __builtin_bit_cast(float, uint32_t(v[i])); }
  static __device__ float one(const void* p, int i) { return static_cast<const float*>(p)[i]; }
};
template <>
struct Bits<F16> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNone = 0x7E007E00u;
  static __device__ float get(u32x4_t v, int i) {
    const uint32_t w = v[i >> 1];
    return float(__builtin_bit_cast(_Float16, uint16_t(i & 1 ? w >> 16 : w)));
  }
  static __device__ float one(const void* p, int i) { return float(static_cast<const _Float16*>(p)[i]); }
};
template <>
struct Bits<BF16> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNone = 0x7FC07FC0u;
  static __device__ float get(u32x4_t v, int i) {
    const uint32_t w = v[i >> 1];
    return __builtin_bit_cast(float, i & 1 ? w & 0xFFFF0000u : w << 16);
  }
  static __device__ float one(const void* p, int i) {
    return __builtin_bit_cast(float, uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
  }
};

// A row's logits: `head` elements up to the first 16-byte boundary, `vecs` vectors of 16 bytes, and the rest.  Chunk 0
// has the head too, the last chunk the rest.
template <class T>
struct Row {
  static constexpr int kVec = Bits<T>::kVec;
  const typename T::elem* p;
  const u32x4_t* body;
  int vocab, head, vecs;

  __device__ Row(const Args& a, int row) {
    p = static_cast<const typename T::elem*>(a.logits) + row * a.row_stride;
    vocab = a.vocab;
    const int past = int(reinterpret_cast<uintptr_t>(p) & 15) / int(sizeof(typename T::elem));
    head = min(vocab, past ? kVec - past : 0);
    vecs = (vocab - head) / kVec;
    body = reinterpret_cast<const u32x4_t*>(p + head);
  }
  // The index of the thread's element among the head (a first chunk's) and the rest (a last one's), or -1.
  __device__ int loose(bool first, bool last) const {
    const int t = threadIdx.x, rest = head + vecs * kVec;
    if (first && t < head) return t;
    if (last && t >= 64 && t - 64 < vocab - rest) return rest + t - 64;
    return -1;
  }
};

// A row's settings, and what becomes of a logit; `top` is the largest logit that weights are counted from.
struct Rule : Bins {
  double rate;                             // log2(e) / T
  float top;
  bool greedy;

  __device__ Rule(const Args& a, int row) {
    const double heat = a.temperatures ? double(a.temperatures[row]) : a.temperature;
    greedy = !(heat > 0.0);                // the first of the order, at any temperature
    rate = 1.4426950408889634 / (greedy ? 1.0 : fmax(heat, kCoolest));
    set_rate(rate);
  }
  __device__ void set_top(float l) {
    top = l;
    Bins::set_top(l);
  }
  __device__ double power(float l) const { return l == top ? 0.0 : (double(l) - double(top)) * rate; }
  // 2^y, y <= 0: f = y - n, |f| <= 1/2, by the Taylor polynomial of degree 11, which leaves 6.3e-15 of it.
  static __device__ double exp2_of(double y) {
    const double n = __builtin_rint(y), f = y - n;
    double s = 4.44553827187081e-10;                    // ln(2)^k / k!, k = 11 .. 0
    s = __builtin_fma(s, f, 7.054911620801121e-09);
    s = __builtin_fma(s, f, 1.0178086009239696e-07);
    s = __builtin_fma(s, f, 1.3215486790144305e-06);
    s = __builtin_fma(s, f, 1.5252733804059838e-05);
    s = __builtin_fma(s, f, 0.00015403530393381606);
    s = __builtin_fma(s, f, 0.0013333558146428441);
    s = __builtin_fma(s, f, 0.009618129107628477);
    s = __builtin_fma(s, f, 0.055504108664821576);
    s = __builtin_fma(s, f, 0.2402265069591007);
    s = __builtin_fma(s, f, 0.6931471805599453);
    s = __builtin_fma(s, f, 1.0);
    return __builtin_ldexp(s, int(n));
  }
  __device__ double e(float l) const {
    const double y = power(l);
    return y > -1000.0 ? exp2_of(y) : 0.0;
  }
  // e in units of 2^-kUnit, rounded to a whole number by adding 2^52.  Free of branches, and right for a logit whose bin
  // is below kBins; any number for others.
  __device__ uint64_t near_weight(float l) const {
    const double y = fmax(power(l), -64.0);             // fmax passes NaN by
    const double whole = __builtin_fma(exp2_of(y), double(uint64_t(1) << kUnit), 4503599627370496.0);
    return __builtin_bit_cast(uint64_t, whole) & ((uint64_t(1) << 52) - 1);
  }
};

// Logits as unsigned numbers of the same order, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float l) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l == 0.f ? 0.f : l);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t o) {
  return __builtin_bit_cast(float, o >> 31 ? o & 0x7FFFFFFFu : ~o);
}
// Largest first: the logit, then the index, lowest first.
__device__ __forceinline__ uint64_t key_of(float l, int index) {
  return uint64_t(order_of(l)) << 32 | uint32_t(~index);
}

// One lane move of the maximum over a wave; lanes outside ROW_MASK keep theirs.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float max_move(float v) {
  const int x = __builtin_bit_cast(int, v);
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(x, x, CTRL, ROW_MASK, 0xF, false)));
}
__device__ __forceinline__ float wave_max(float v) {
  v = max_move<0xB1, 0xF>(v);
  v = max_move<0x4E, 0xF>(v);
  v = max_move<0x141, 0xF>(v);
  v = max_move<0x140, 0xF>(v);
  v = max_move<0x142, 0xA>(v);
  v = max_move<0x143, 0xC>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Inclusive sums over the bins, one for each of the first kBins threads; part: two values for each of their waves.
template <class A>
__device__ __forceinline__ void scan(A& sum, uint32_t& count, A* part_sum, uint32_t* part_count) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave < kBins / 64) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const A o = __shfl_up(sum, d);
      const uint32_t c = __shfl_up(count, d);
      if (lane >= d) sum += o, count += c;
    }
    if (lane == 63) part_sum[wave] = sum, part_count[wave] = count;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBins / 64; ++w)
    if (w < wave) sum += part_sum[w], count += part_count[w];
}

// Tokens of a chunk: those of its vectors, and for the first and the last one the row's loose ones.
template <class T, int VECS>
constexpr int kChunkTokens = kThreads * VECS * Bits<T>::kVec + 16;

template <class T, int VECS>
__global__ __launch_bounds__(kThreads) void bins_kernel(Args a) {
  constexpr int kVec = Bits<T>::kVec;
  __shared__ unsigned long long sums[kBins];
  __shared__ uint32_t counts[kBins], starts[kBins], part_a[kBins / 64], part_b[kBins / 64];
  __shared__ __attribute__((aligned(16))) uint16_t order[kChunkTokens<T, VECS>];
  __shared__ float part[kThreads / 64];
  __shared__ int last;
  __shared__ uint32_t all;
  const int chunk = blockIdx.x, row = blockIdx.y, t = threadIdx.x;
  const Row<T> r(a, row);
  u32x4_t x[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int v = chunk * (kThreads * VECS) + i * kThreads + t;
    x[i] = u32x4_t{Bits<T>::kNone, Bits<T>::kNone, Bits<T>::kNone, Bits<T>::kNone};
    if (v < r.vecs) x[i] = r.body[v];
  }
  const int loose = r.loose(chunk == 0, chunk == a.chunks - 1);
  const float single = loose >= 0 ? Bits<T>::one(r.p, loose) : -__builtin_inff();
  for (int i = t; i < kBins; i += kThreads) sums[i] = 0, counts[i] = 0;
  Rule rule(a, row);
  const double min_p = a.min_ps ? double(a.min_ps[row]) : a.min_p;
  const int top_k = rule.greedy ? 1 : a.top_ks ? a.top_ks[row] : a.top_k;
  float top = fmaxf(single, -__builtin_inff());         // fmaxf passes NaN by
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) top = fmaxf(top, Bits<T>::get(x[i], j));
  const float mine = top;
  top = wave_max(top);
  if ((t & 63) == 0) part[t >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) top = fmaxf(top, part[w]);
  const size_t at = size_t(row) * a.chunks + chunk;
  if (t == 0) a.tops[at] = top;
  if (top == -__builtin_inff()) return;                 // its bins are not read
  rule.set_top(top);
  // Each token's bin and its number there.  What min_p drops of a chunk by itself is no part of the row's either.
  constexpr uint32_t kDropped = ~0u;
  int cut = rule.last_bin(min_p);
  if (top_k > 0 && top_k <= kThreads / 2) {
    // Nor is what lies below top_k threads' own largest tokens: a first cut by these, one a thread.
    const int b = rule.bin(mine);
    if (b < kBins && mine > -__builtin_inff()) atomicAdd(&counts[b], 1u);
    if (t == 0) last = cut;
    __syncthreads();
    const uint32_t own = t < kBins ? counts[t] : 0;
    uint32_t upto = own, none = 0;
    scan(upto, none, part_a, part_b);
    if (t < kBins && upto >= uint32_t(top_k) && upto - own < uint32_t(top_k)) last = min(cut, t);
    if (t < kBins) counts[t] = 0;
    __syncthreads();
    cut = last;
  }
  const float from = rule.sieve(cut);                   // one comparison for most tokens
  const auto place = [&](float l, int b) {
    return b <= cut && l > -__builtin_inff() ? uint32_t(b) << 16 | atomicAdd(&counts[b], 1u) : kDropped;
  };
  uint32_t code[VECS][kVec];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      code[i][j] = kDropped;
      any |= Bits<T>::get(x[i], j) >= from;
    }
    if (!__any(any)) continue;
    if (rule.far) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) code[i][j] = place(Bits<T>::get(x[i], j), rule.far_bin(Bits<T>::get(x[i], j)));
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) code[i][j] = place(Bits<T>::get(x[i], j), rule.near_bin(Bits<T>::get(x[i], j)));
    }
  }
  const uint32_t code_single = loose >= 0 ? place(single, rule.bin(single)) : kDropped;
  if (t == 0) last = cut;
  __syncthreads();
  const uint32_t own = t < kBins ? counts[t] : 0;
  uint32_t upto = own, none = 0;
  scan(upto, none, part_a, part_b);
  if (t < kBins) {
    starts[t] = upto - own;
    // Nor is what top_k drops.
    if (top_k > 0 && upto >= uint32_t(top_k) && upto - own < uint32_t(top_k)) last = t;
  }
  __syncthreads();
  cut = last;
  if (t == cut) all = upto;
  __syncthreads();
  // The tokens by their bins, and weights.  Where most were dropped the others are gone through as they are ordered, their
  // logits read again; otherwise from the registers, a vector's exponentials side by side: each is one long chain.
  const bool sparse = all * 4 <= uint32_t(kChunkTokens<T, VECS>);
  const int base = chunk == 0 ? 0 : r.head + chunk * (kThreads * VECS * kVec);
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < kVec; ++j) any |= int(code[i][j] >> 16) <= cut;
    if (!__any(any)) continue;
    const int first = r.head + (chunk * (kThreads * VECS) + i * kThreads + t) * kVec - base;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int b = int(code[i][j] >> 16);
      if (b <= cut) order[starts[b] + (code[i][j] & 0xFFFFu)] = uint16_t(first + j);
    }
    if (sparse) continue;
    uint64_t w[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j] = rule.near_weight(Bits<T>::get(x[i], j));
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int b = int(code[i][j] >> 16);
      if (b <= cut) atomicAdd(&sums[b], static_cast<unsigned long long>(w[j]));
    }
  }
  if (int(code_single >> 16) <= cut) {
    const int b = int(code_single >> 16);
    if (!sparse) atomicAdd(&sums[b], static_cast<unsigned long long>(rule.near_weight(single)));
    order[starts[b] + (code_single & 0xFFFFu)] = uint16_t(loose - base);
  }
  __syncthreads();
  if (sparse) {
    for (uint32_t i = t; i < all; i += kThreads) {
      const float l = Bits<T>::one(r.p, base + order[i]);
      atomicAdd(&sums[rule.bin(l)], static_cast<unsigned long long>(rule.near_weight(l)));
    }
    __syncthreads();
  }
  if (t < kBins) {
    a.sums[at * kBins + t] = sums[t];
    a.counts[at * kBins + t] = t <= cut ? starts[t] << 16 | own : all << 16;
  }
  u32x4_t* out = reinterpret_cast<u32x4_t*>(a.order + at * a.chunk_tokens);
  for (int i = t; i * 8 < int(all); i += kThreads) out[i] = reinterpret_cast<const u32x4_t*>(order)[i];
}

// LDS of the choice.
struct Shared {
  uint64_t list[kList], weights[kList];    // keys of the tokens at hand and their weights
  uint64_t sums[kBins];
  uint64_t part_a[kRowWaves], part_b[kRowWaves];
  uint32_t counts[kBins];
  uint32_t part_c[kRowWaves];
  double factor[kMaxChunks];               // of a chunk's sums
  int32_t shift[kMaxChunks];               // from the row's bins to the chunk's; kBins: no chunk to look at
  uint32_t from[kMaxChunks], past[kMaxChunks];         // of a chunk's tokens at hand: the first in its order, where they end
  uint64_t few_key[kFew], few_sum[kFew];
  uint32_t few, count, upto;
  int bin;
  uint64_t before, inside, key, all;
  uint32_t count_before;
};

// What is looked for in the order: the `count`-th token (count > 0), or the first whose sum from the top reaches `sum`.
struct Goal {
  uint32_t count;
  uint64_t sum;
  // Sums of tokens weighed at the row's top may miss those of the chunks by their last units: no more than is there.
  __device__ void cut(uint64_t all, uint32_t n) {
    if (count) count = min(count, n);
    else if (all == 0) count = 1;
    else sum = sum < all ? sum : all;
  }
  __device__ bool here(uint64_t upto, uint64_t own, uint32_t upto_n, uint32_t n) const {
    return count ? upto_n >= count && upto_n - n < count : upto >= sum && upto - own < sum;
  }
};

// The smallest logit (as order_of gives it) that `holds`, which is false below it and true from it on up to `most`, by
// one wave: first among the 64 around a guess, then by 64 tries at a time.
template <class F>
__device__ __forceinline__ uint32_t first_logit(float guess, uint32_t most, F holds) {
  const int lane = threadIdx.x & 63;
  const uint32_t near = order_of(guess), from = near > 32 ? near - 32 : 0;
  const uint32_t mine = from + lane < most ? from + lane : most;
  uint64_t yes = __ballot(holds(logit_of(mine)));
  if (yes && !(yes & 1)) return __builtin_amdgcn_readlane(int(mine), __builtin_ctzll(yes));
  uint32_t lo = order_of(-__builtin_inff()), hi = most;           // the answer lies in (lo, hi]
  while (hi - lo > 1) {
    const uint32_t step = (hi - lo + 63) / 64;
    const uint64_t at = uint64_t(lo) + uint64_t(step) * (lane + 1);
    const uint32_t probe = at < hi ? uint32_t(at) : hi;
    yes = __ballot(holds(logit_of(probe)));
    const int n = yes ? __builtin_ctzll(yes) : 63;
    hi = __builtin_amdgcn_readlane(int(probe), n);
    if (n > 0) lo = __builtin_amdgcn_readlane(int(probe), n - 1);
  }
  return hi;
}

__device__ __forceinline__ uint64_t wave_sum(uint64_t v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(static_cast<unsigned long long>(v), m);
  return v;
}

template <class T>
struct Choice {
  Shared& s;
  const Args& a;
  const Rule& rule;
  const Row<T>& row;
  int index;                               // of the row
  // Thread t's bin: sum and count, by itself and through it from the top.
  uint64_t own, sum;
  uint32_t mine, count;
  // Bins whose tokens are at hand: listed if they fit, and in order if there are few.
  int low = 0, high = -1;
  bool listed = false, ordered = false;
  uint32_t tokens = 0;
  // Of those in order, a token for four threads: its key and weight, the sum and count from the first through it; what
  // lies above the first.
  uint64_t key = 0, weight = 0, upto = 0, above = 0;
  uint32_t rank = 0, above_n = 0;

  __device__ uint64_t weight_of(uint64_t k) const { return rule.near_weight(logit_of(uint32_t(k >> 32))); }

  // f(place, key) for the tokens at hand, from the chunks' orders: a wave for a chunk at a time.
  template <class F>
  __device__ void read(F f) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int c = wave; c < a.chunks; c += kRowWaves) {
      const uint32_t at = c ? s.past[c - 1] : 0, n = s.past[c] - at, from = s.from[c];
      const uint16_t* order = a.order + (size_t(index) * a.chunks + c) * a.chunk_tokens + from;
      const int base = c == 0 ? 0 : row.head + (c << a.chunk_shift) * Bits<T>::kVec;
      for (uint32_t i = lane; i < n; i += 64) {
        const int token = base + order[i];
        f(at + i, key_of(Bits<T>::one(row.p, token), token));
      }
    }
  }
  // Have the tokens of a bin at hand, and all above them if these are few.
  __device__ void open(int bin) {
    if (bin >= low && bin <= high) return;
    const int t = threadIdx.x;
    __syncthreads();
    if (t == bin) s.upto = count, s.count = mine, s.before = sum - own;
    __syncthreads();
    const bool all = s.upto <= kFew;
    low = all ? 0 : bin, high = bin;
    above = all ? 0 : s.before;
    above_n = all ? 0 : s.upto - s.count;
    tokens = all ? s.upto : s.count;
    if (t < 64) {
      uint32_t n = 0;
      if (t < a.chunks) {
        const int first = max(low - s.shift[t], 0), last = bin - s.shift[t];
        if (last >= 0) {
          const uint32_t* packed = a.counts + (size_t(index) * a.chunks + t) * kBins;
          const uint32_t end = packed[last], begin = first > 0 ? packed[first] >> 16 : 0;
          s.from[t] = begin;
          n = (end >> 16) + (end & 0xFFFFu) - begin;
        }
      }
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(n, d);
        if (t >= d) n += o;
      }
      s.past[t] = n;
    }
    __syncthreads();
    listed = tokens <= kList;
    ordered = tokens <= kFew;
    if (!listed) return;
    read([&](uint32_t i, uint64_t k) {
      s.list[i] = k;
      s.weights[i] = weight_of(k);
    });
    __syncthreads();
    if (ordered) count_order(s.list, s.weights, tokens);
  }
  // Put at most kFew tokens in order by counting: key, weight, upto and rank of the thread's.
  __device__ void count_order(const uint64_t* keys, const uint64_t* weights, uint32_t n) {
    const int t = threadIdx.x;
    const uint32_t i = t >> 2;
    key = i < n ? keys[i] : 0;
    weight = i < n ? weights[i] : 0;
    upto = 0, rank = 0;
    if (i < n) {
#pragma unroll 4
      for (uint32_t j = t & 3; j < n; j += 4)
        if (keys[j] >= key) upto += weights[j], ++rank;
#pragma unroll
      for (int m = 1; m < 4; m *= 2)
        upto += __shfl_xor(static_cast<unsigned long long>(upto), m), rank += __shfl_xor(rank, m);
      if (rank == n) s.all = upto;
    }
    __syncthreads();
  }
  // f(key, weight) for the tokens at hand.
  template <class F>
  __device__ void each(F f) {
    if (listed) {
      for (uint32_t i = threadIdx.x; i < tokens; i += kRowThreads) f(s.list[i], s.weights[i]);
    } else {
      read([&](uint32_t, uint64_t k) { f(k, weight_of(k)); });       // the bin by itself
    }
  }
  // Sums over the block.
  __device__ void total(uint64_t& v, uint32_t& n) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(static_cast<unsigned long long>(v), m), n += __shfl_xor(n, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.part_a[threadIdx.x >> 6] = v, s.part_c[threadIdx.x >> 6] = n;
    __syncthreads();
    v = 0, n = 0;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) v += s.part_a[w], n += s.part_c[w];
  }
  // What is kept by min_p: the tokens whose logit's order is `border` or above, of which `bin` has the last.
  __device__ void cut(uint32_t border, int bin, uint64_t* kept, uint32_t* left) {
    const int t = threadIdx.x;
    open(bin);
    uint64_t part = 0;
    uint32_t n = 0;
    each([&](uint64_t k, uint64_t w) {
      const uint32_t l = uint32_t(k >> 32);
      if (l >= border && (low == high || rule.bin(logit_of(l)) == bin)) part += w, ++n;
    });
    total(part, n);
    if (t == bin) {
      s.before = sum - own + (part < own ? part : own);      // no more than the bins hold
      s.count = count - mine + n;
    }
    __syncthreads();
    *kept = s.before, *left = s.count;
  }
  // The goal's token; *through becomes the sum from the top through it.  Called by all threads alike.
  __device__ uint64_t find(Goal g, uint64_t* through) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    __syncthreads();
    if (g.here(sum, own, count, mine)) {
      s.bin = t;
      s.before = sum - own;
      s.inside = own;
      s.count_before = count - mine;
    }
    __syncthreads();
    const int bin = s.bin;
    const uint64_t before = s.before, end = before + s.inside;
    const uint32_t before_n = s.count_before;
    open(bin);
    // No more is kept than the bins hold, so that what is drawn lies in the kept run.
    if (ordered) {
      if (g.count) g.count -= above_n;
      else g.sum -= above;
      g.cut(s.all, tokens);
      __syncthreads();
      if (uint32_t(t >> 2) < tokens && g.here(upto, weight, rank, 1)) s.key = key, s.before = upto;
      __syncthreads();
      const uint64_t got = above + s.before;
      *through = got < end ? got : end;
      return s.key;
    }
    // More than kFew: the bin by itself is at hand.
    if (g.count) g.count -= before_n;
    else g.sum -= before;
    uint64_t lo = 0, hi = ~uint64_t(0), passed = 0;
    uint32_t n = tokens;
    while (n > kFew) {
      // The keys' range, then bins over it.
      uint64_t least = ~uint64_t(0), most = 0;
      each([&](uint64_t k, uint64_t) {
        if (k < lo || k > hi) return;
        least = k < least ? k : least;
        most = k > most ? k : most;
      });
#pragma unroll
      for (int m = 32; m; m >>= 1) {
        const uint64_t x = __shfl_xor(static_cast<unsigned long long>(least), m);
        const uint64_t y = __shfl_xor(static_cast<unsigned long long>(most), m);
        least = x < least ? x : least;
        most = y > most ? y : most;
      }
      __syncthreads();
      if (lane == 0) s.part_a[wave] = least, s.part_b[wave] = most;
      s.sums[t] = 0;
      s.counts[t] = 0;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kRowWaves; ++w) {
        least = s.part_a[w] < least ? s.part_a[w] : least;
        most = s.part_b[w] > most ? s.part_b[w] : most;
      }
      const int width = 64 - __builtin_clzll((most - least) | 1), shift = width > 9 ? width - 9 : 0;
      each([&](uint64_t k, uint64_t w) {
        if (k < lo || k > hi) return;
        const int b = int((most - k) >> shift);
        atomicAdd(reinterpret_cast<unsigned long long*>(&s.sums[b]), static_cast<unsigned long long>(w));
        atomicAdd(&s.counts[b], 1u);
      });
      __syncthreads();
      const uint64_t part = s.sums[t];
      const uint32_t part_n = s.counts[t];
      uint64_t upto_b = part;
      uint32_t upto_n = part_n;
      scan(upto_b, upto_n, s.part_a, s.part_c);
      if (t == kBins - 1) s.all = upto_b;
      __syncthreads();
      g.cut(s.all, n);
      if (g.here(upto_b, part, upto_n, part_n)) {
        s.bin = t;
        s.before = upto_b - part;
        s.count_before = upto_n - part_n;
        s.count = part_n;
      }
      __syncthreads();
      hi = most - (uint64_t(s.bin) << shift);
      // The last bin may reach past the least key: no lower than before, where other tokens follow.
      const uint64_t below = (uint64_t(1) << shift) - 1;
      if (hi - lo > below) lo = hi - below;
      n = s.count;
      passed += s.before;
      if (g.count) g.count -= s.count_before;
      else g.sum -= s.before;
    }
    // Few: put in order by counting.
    __syncthreads();
    if (t == 0) s.few = 0;
    __syncthreads();
    each([&](uint64_t k, uint64_t w) {
      if (k < lo || k > hi) return;
      const uint32_t at = atomicAdd(&s.few, 1u);
      if (at < kFew) s.few_key[at] = k, s.few_sum[at] = w;
    });
    __syncthreads();
    count_order(s.few_key, s.few_sum, n);
    g.cut(s.all, n);
    if (uint32_t(t >> 2) < n && g.here(upto, weight, rank, 1)) s.key = key, s.before = upto;
    __syncthreads();
    const uint64_t got = before + passed + s.before;
    *through = got < end ? got : end;
    return s.key;
  }
};

template <class T>
__global__ __launch_bounds__(kRowThreads) void choice_kernel(Args a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  const int index = blockIdx.x, t = threadIdx.x, lane = t & 63;
  Rule rule(a, index);
  const double min_p = a.min_ps ? double(a.min_ps[index]) : a.min_p;
  const int top_k = a.top_ks ? a.top_ks[index] : a.top_k;
  const double top_p = a.top_ps ? double(a.top_ps[index]) : a.top_p;
  const float u = a.u[index];
  const size_t first_chunk = size_t(index) * a.chunks;
  const float chunk_top = a.tops[first_chunk + min(lane, a.chunks - 1)];
  const float top = wave_max(chunk_top);
  const auto none = [&]() {
    if (t == 0) {
      a.ids[index] = -1;
      if (a.logprob) a.logprob[index] = -__builtin_inff();
    }
  };
  if (top == -__builtin_inff()) {
    none();
    return;
  }
  rule.set_top(top);
  if (t < a.chunks) {                                   // at most kMaxChunks: the first wave
    const bool any = chunk_top > -__builtin_inff();
    s.shift[t] = any ? rule.bin(chunk_top) : kBins;
    s.factor[t] = any ? rule.e(chunk_top) : 0.0;
  }
  __syncthreads();
  // The thread's bin of the row, from all chunks.
  uint64_t own = 0;
  uint32_t mine = 0;
#pragma unroll 4
  for (int c = 0; c < a.chunks; ++c) {
    const int at = t - s.shift[c];
    const size_t from = (first_chunk + c) * kBins + max(at, 0);
    const bool here = at >= 0;
    const uint64_t sum = here ? a.sums[from] : 0;
    mine += here ? a.counts[from] & 0xFFFFu : 0;
    const double f = s.factor[c];
    own += f == 1.0 ? sum : uint64_t(double(sum) * f);
  }
  uint64_t sum = own;
  uint32_t count = mine;
  scan(sum, count, s.part_a, s.part_c);
  if (t == kBins - 1) s.before = sum, s.count = count;
  __syncthreads();
  uint64_t kept = s.before;                             // the sum and the count of what is kept so far
  uint32_t left = s.count;
  // The top weighs 2^kUnit.  Were it missing, no bin would hold what is looked for: a search needs a sum above zero.
  if (kept == 0) {
    none();
    return;
  }
  const Row<T> row(a, index);
  Choice<T> pick{s, a, rule, row, index, own, sum, mine, count};
  if (!rule.greedy && min_p > 0.0) {
    // The least logit with e >= min_p.
    const double least = fmin(min_p, 1.0);
    const float guess = float(double(top) + log2(least) / rule.rate);
    const uint32_t border = first_logit(guess < top ? guess : top, order_of(top), [&](float l) { return rule.e(l) >= least; });
    const int bin = rule.bin(logit_of(border));
    if (bin < kBins) pick.cut(border, bin, &kept, &left);
  }
  uint64_t key = 0;
  for (int stage = 0; stage < 3; ++stage) {
    Goal g{0, 1};
    if (stage == 0) {
      if (rule.greedy || top_k <= 0 || uint32_t(top_k) >= left) continue;
      g = Goal{uint32_t(top_k), 0};
    } else if (stage == 1) {
      if (rule.greedy || !(top_p < 1.0)) continue;
      const uint64_t want = uint64_t(ceil(fmax(top_p, 0.0) * double(kept)));
      g.sum = want < 1 ? 1 : want > kept ? kept : want;
    } else if (!rule.greedy && u > 0.f) {
      const uint64_t past = uint64_t(fmin(double(u), 1.0) * double(kept));
      g.sum = (past < kept ? past : kept - 1) + 1;
    }
    uint64_t through;
    key = pick.find(g, &through);
    if (stage < 2) kept = through > 0 ? through : 1;
  }
  if (t == 0) {
    a.ids[index] = int(~uint32_t(key));
    if (a.logprob) {
      const double y = rule.power(logit_of(uint32_t(key >> 32)));
      a.logprob[index] = rule.greedy ? 0.f
                                     : float(y * 0.6931471805599453 - log(__builtin_ldexp(double(kept), -kUnit)));
    }
  }
}

// Chunks of 1, 2 or 4 vectors a thread: small ones for the number of blocks, but at most 16, which the choice joins
// (131,072 logits, both kernels: 33 us with 32 chunks of one vector, 28 with 16 of two), and large ones once there are blocks enough.
struct Chunks {
  int vecs, count, tokens;                 // vectors of a thread, chunks of a row, places of a chunk's order
};
Chunks chunks_of(int64_t rows, int64_t vocab, int64_t type) {
  const int64_t vec = type == TQ2_TYPE_F32 ? 4 : 8, vecs = vocab / vec;
  Chunks c;
  for (c.vecs = 1; c.vecs < 4; c.vecs *= 2) {
    const int64_t n = (vecs + kThreads * c.vecs - 1) / (kThreads * c.vecs);
    if (n <= 16 && rows * n <= 2048) break;
  }
  c.count = int((vecs + kThreads * c.vecs - 1) / (kThreads * c.vecs));
  if (c.count < 1) c.count = 1;
  c.tokens = int(kThreads * c.vecs * vec + 16);
  return c;
}

template <class T>
hipError_t launch(const Args& a, int vecs, int64_t rows, hipStream_t stream) {
  const dim3 grid(a.chunks, uint32_t(rows));
  const auto bins = vecs == 1 ? bins_kernel<T, 1> : vecs == 2 ? bins_kernel<T, 2> : bins_kernel<T, 4>;
  hipLaunchKernelGGL(bins, grid, dim3(kThreads), 0, stream, a);
  const auto fn = choice_kernel<T>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(Shared)));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(uint32_t(rows)), dim3(kRowThreads), sizeof(Shared), stream, a);
  return hipGetLastError();
}

}  // namespace

size_t sample_workspace(int64_t rows, int64_t vocab, int64_t type) {
  const Chunks c = chunks_of(rows, vocab, type);
  return size_t(rows) * size_t(c.count) * (kBins * 12 + size_t(c.tokens) * 2 + 4);
}

hipError_t launch_sample(const tq2_sample_args& q, hipStream_t stream) {
  const Chunks chunks = chunks_of(q.rows, q.vocab, q.logits_type);
  Args a;
  a.logits = q.logits;
  a.u = q.u;
  a.ids = q.ids;
  a.logprob = q.logprob;
  a.temperatures = q.temperatures;
  a.top_ks = q.top_ks;
  a.top_ps = q.top_ps;
  a.min_ps = q.min_ps;
  a.top_k = int32_t(q.top_k < 0 ? 0 : q.top_k < TQ2_SAMPLE_MAX_VOCAB ? q.top_k : TQ2_SAMPLE_MAX_VOCAB);
  a.vocab = int32_t(q.vocab);
  a.chunks = chunks.count;
  a.chunk_shift = __builtin_ctz(unsigned(kThreads * chunks.vecs));
  a.row_stride = q.row_stride;
  a.temperature = q.temperature;
  a.top_p = q.top_p;
  a.min_p = q.min_p;
  const size_t parts = size_t(q.rows) * size_t(chunks.count);
  a.sums = static_cast<uint64_t*>(q.workspace);
  a.counts = reinterpret_cast<uint32_t*>(a.sums + parts * kBins);
  a.order = reinterpret_cast<uint16_t*>(a.counts + parts * kBins);
  a.chunk_tokens = chunks.tokens;
  a.tops = reinterpret_cast<float*>(a.order + parts * size_t(chunks.tokens));
  if (q.logits_type == TQ2_TYPE_F32) return launch<F32>(a, chunks.vecs, q.rows, stream);
  if (q.logits_type == TQ2_TYPE_F16) return launch<F16>(a, chunks.vecs, q.rows, stream);
  return launch<BF16>(a, chunks.vecs, q.rows, stream);
}

}  // namespace tq2
