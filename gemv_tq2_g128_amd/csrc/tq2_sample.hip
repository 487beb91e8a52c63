// The next token of each row of logits: temperature, top-k, min-p, top-p, and a draw by a given random number.
//
// Order.  All truncations keep a run from the top of the order (logit falling, index rising), and so does the draw: the
// token is where the running sum of e = exp((l - max) / T), from the top, passes u times the kept sum.  So nothing is
// sorted: a histogram over the logits' range, of counts and of sums, says in which bin the k-th token, the end of top-p's
// run or the drawn one lies, and only that bin's few tokens are put in order.
//
// Whole numbers.  e is computed in f64 and rounded to a multiple of 2^-43; sums are then u64, exact in any order, which
// is what makes LDS atomics allowed here and the result one that repeats.  (32-bit exponentials would give another token
// than the definition once in a few dozen draws over 10^5 tokens: that many borders lie within 1e-7 of u.)
//
// Three launches.  max_kernel and bins_kernel: blocks for chunks of each row, so that one row uses many CUs;
// choice_kernel: a block for each row, which joins the chunks' bins and reads only those chunks again that have tokens in
// a bin it needs.  Bound: logits are read from HBM once (the second time from the caches); the f64 exponential costs about
// 17 instructions an element, which is as long as the read.
#include "tq2_device.h"
#include "tq2_sample_internal.h"
#include "tq2_types.h"

#pragma clang fp contract(off)

namespace tq2 {
namespace {

constexpr int kBins = 512;
constexpr int kMaxChunks = 32;
constexpr int kThreads = 256;              // of the chunk kernels
constexpr int kRowThreads = kBins;         // of the choice: a thread for each bin
constexpr int kList = 4096;                // tokens of a bin that are held in LDS
constexpr int kUnit = 43;                  // a token of the largest logit weighs 2^43

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
  int64_t row_stride;
  double temperature, top_p, min_p;
  float2* ends;                            // [rows, chunks]: largest and least logit
  uint64_t* sums;                          // [rows, chunks, kBins]
  uint32_t* counts;
};

// A row's logits: `head` elements up to the first 16-byte boundary, vectors of 16 bytes, and the rest.
template <class T>
struct Row {
  static constexpr int kVec = 16 / sizeof(typename T::elem);
  const typename T::elem* p;
  int vocab, head, vecs, per_chunk;        // per_chunk: vectors of a chunk

  __device__ Row(const Args& a, int row) {
    p = static_cast<const typename T::elem*>(a.logits) + row * a.row_stride;
    vocab = a.vocab;
    const int past = int(reinterpret_cast<uintptr_t>(p) & 15) / int(sizeof(typename T::elem));
    head = min(vocab, past ? kVec - past : 0);
    vecs = (vocab - head) / kVec;
    per_chunk = (vecs + a.chunks - 1) / a.chunks;
  }
  __device__ static float value(const typename T::elem* p) {
    const float v = float(*p);
    return v == v ? v : -__builtin_inff();            // NaN counts as -infinity
  }
  // f(value, index) for the elements of a chunk, shared by `threads` threads.  Chunk 0 has the head, the last one the rest.
  template <class F>
  __device__ void each(int chunk, int chunks, int threads, F f) const {
    const int from = min(vecs, chunk * per_chunk), to = min(vecs, from + per_chunk);
    const typename T::elem* body = p + head;
    constexpr int kAhead = 4;
    for (int v0 = from + threadIdx.x; v0 < to; v0 += kAhead * threads) {
      f32x4_t x[kAhead][kVec / 4];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int v = min(v0 + i * threads, to - 1);
#pragma unroll
        for (int j = 0; j < kVec / 4; ++j) x[i][j] = load4(T(), body + v * kVec + 4 * j);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int v = v0 + i * threads;
        if (v >= to) break;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float y = x[i][j / 4][j % 4];
          f(y == y ? y : -__builtin_inff(), head + v * kVec + j);
        }
      }
    }
    const int t = threadIdx.x;
    if (chunk == 0 && t < head) f(value(p + t), t);
    const int rest = head + vecs * kVec;
    if (chunk == chunks - 1 && t < vocab - rest) f(value(p + rest + t), rest + t);
  }
};

// A row's settings, and the two functions of a logit that all kernels share.
struct Rule {
  float top, slope;                        // bin = (top - l) * slope
  double heat, rate;                       // temperature; log2(e) / T
  double least;                            // min_p
  bool greedy;

  __device__ Rule(const Args& a, int row, float top, float low) : top(top) {
    heat = a.temperatures ? double(a.temperatures[row]) : a.temperature;
    greedy = !(heat > 0.0);
    rate = greedy ? 0.0 : 1.4426950408889634 / heat;
    least = a.min_ps ? double(a.min_ps[row]) : a.min_p;
    least = least > 0.0 ? fmin(least, 1.0) : 0.0;
    // Bins over what lies within 32 temperatures of the top, or over less.
    slope = greedy ? 0.f : float(kBins - 1) / fminf(float(32.0 * heat), top - low);
  }
  __device__ int bin(float l) const {
    return l == top ? 0 : int(fminf((top - l) * slope, float(kBins - 1)));
  }
  // log2 of e.
  __device__ double power(float l) const {
    if (l == top) return 0.0;
    return greedy ? -__builtin_inf() : (double(l) - double(top)) * rate;
  }
  // e in units of 2^-kUnit; 0 below min_p.
  __device__ uint64_t weight(float l) const {
    const double y = power(l);
    if (!(y > -(kUnit + 2))) return 0;                  // NaN as well: -infinity at an infinite temperature
    // 2^f, |f| <= 1/2, by its Taylor polynomial of degree 11, which leaves 6.3e-15 of it.
    const double n = __builtin_rint(y), f = y - n;
    double s = 4.44553827187081e-10;                     // ln(2)^k / k!, k = 11 .. 0
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
    s = __builtin_ldexp(s, int(n));
    if (s < least) return 0;
    // Rounded to a whole number by adding 2^52.
    const double whole = __builtin_fma(s, double(uint64_t(1) << kUnit), 4503599627370496.0);
    return __builtin_bit_cast(uint64_t, whole) & ((uint64_t(1) << 52) - 1);
  }
};

// Largest first: a logit's bits in its order, then the index, lowest first.
__device__ __forceinline__ uint64_t key_of(float l, int index) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l == 0.f ? 0.f : l);
  const uint32_t o = b >> 31 ? ~b : b | 0x80000000u;
  return uint64_t(o) << 32 | uint32_t(~index);
}

__device__ __forceinline__ float2 join(float2 a, float2 b) { return make_float2(fmaxf(a.x, b.x), fminf(a.y, b.y)); }

__device__ __forceinline__ float2 wave_ends(float2 v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = join(v, make_float2(__shfl_xor(v.x, m), __shfl_xor(v.y, m)));
  return v;
}

template <class T>
__global__ __launch_bounds__(kThreads) void max_kernel(Args a) {
  __shared__ float2 part[kThreads / 64];
  const int chunk = blockIdx.x, row = blockIdx.y;
  float2 v = make_float2(-__builtin_inff(), __builtin_inff());
  // -infinity is no least logit: bins are spread over what can be taken.
  Row<T>(a, row).each(chunk, a.chunks, kThreads, [&](float l, int) {
    v.x = fmaxf(v.x, l);
    v.y = fminf(v.y, l > -__builtin_inff() ? l : __builtin_inff());
  });
  v = wave_ends(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 64; ++i) v = join(v, part[i]);
    a.ends[row * a.chunks + chunk] = v;
  }
}

// The row's largest and least logit, in every thread of each wave.
__device__ __forceinline__ float2 row_ends(const Args& a, int row) {
  const int lane = threadIdx.x & 63;
  return wave_ends(a.ends[row * a.chunks + min(lane, a.chunks - 1)]);
}

template <class T>
__global__ __launch_bounds__(kThreads) void bins_kernel(Args a) {
  __shared__ uint64_t sums[kBins];
  __shared__ uint32_t counts[kBins];
  const int chunk = blockIdx.x, row = blockIdx.y;
  for (int i = threadIdx.x; i < kBins; i += kThreads) sums[i] = 0, counts[i] = 0;
  const float2 ends = row_ends(a, row);
  const Rule rule(a, row, ends.x, ends.y);
  __syncthreads();
  Row<T>(a, row).each(chunk, a.chunks, kThreads, [&](float l, int) {
    if (l == -__builtin_inff()) return;
    const uint64_t w = rule.weight(l);
    if (w == 0) return;
    const int b = rule.bin(l);
    atomicAdd(reinterpret_cast<unsigned long long*>(&sums[b]), static_cast<unsigned long long>(w));
    atomicAdd(&counts[b], 1u);
  });
  __syncthreads();
  const size_t at = (size_t(row) * a.chunks + chunk) * kBins;
  for (int i = threadIdx.x; i < kBins; i += kThreads) a.sums[at + i] = sums[i], a.counts[at + i] = counts[i];
}

// LDS of the choice.
struct Shared {
  uint64_t list_key[kList], list_sum[kList];
  uint64_t few_key[64], few_sum[64];
  uint64_t sums[kBins];
  uint32_t counts[kBins];
  uint64_t wave_sum[kRowThreads / 64];
  uint32_t wave_count[kRowThreads / 64];
  uint64_t lo[kRowThreads / 64], hi[kRowThreads / 64];
  uint32_t filled;
  int bin;
  uint64_t before, key;
  uint32_t count_before, count;
};

// Inclusive sums over the block's threads, one bin each.
__device__ __forceinline__ void scan(Shared& s, uint64_t& sum, uint32_t& count) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t o = __shfl_up(static_cast<unsigned long long>(sum), d);
    const uint32_t c = __shfl_up(count, d);
    if (lane >= d) sum += o, count += c;
  }
  if (lane == 63) s.wave_sum[wave] = sum, s.wave_count[wave] = count;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += s.wave_sum[w], count += s.wave_count[w];
  __syncthreads();
}

// What is looked for in the order: the `count`-th token (count > 0), or the first whose sum from the top reaches `sum`.
struct Goal {
  uint32_t count;
  uint64_t sum;
  __device__ bool here(uint64_t upto, uint64_t own, uint32_t upto_n, uint32_t n) const {
    return count ? upto_n >= count && upto_n - n < count : upto >= sum && upto - own < sum;
  }
};

// The bin of the goal, with what lies above it: s.bin, s.before, s.count_before, s.count.  sum and count are the
// thread's inclusive sums, own and n its bin's.
__device__ __forceinline__ void find_bin(Shared& s, const Goal& g, uint64_t sum, uint64_t own, uint32_t count, uint32_t n) {
  if (g.here(sum, own, count, n)) {
    s.bin = threadIdx.x;
    s.before = sum - own;
    s.count_before = count - n;
    s.count = n;
  }
  __syncthreads();
}

template <class T>
struct Choice {
  Shared& s;
  const Args& a;
  const Rule& rule;
  const Row<T>& row;
  int index;                               // of the row
  int listed = -1;                         // the bin that the list holds

  // f(key, weight) for the tokens of a bin, from the chunks that have any.
  template <class F>
  __device__ void tokens(int bin, F f) {
    for (int c = 0; c < a.chunks; ++c) {
      if (a.counts[(size_t(index) * a.chunks + c) * kBins + bin] == 0) continue;
      row.each(c, a.chunks, kRowThreads, [&](float l, int i) {
        if (l == -__builtin_inff() || rule.bin(l) != bin) return;
        const uint64_t w = rule.weight(l);
        if (w) f(key_of(l, i), w);
      });
    }
  }

  // The key of the goal's token among the n of a bin (the goal counted from the bin's start); *upto becomes the sum from
  // the bin's start through it.  Called by all threads alike.
  __device__ uint64_t resolve(int bin, uint32_t n, Goal g, uint64_t* upto) {
    uint64_t lo = 0, hi = ~uint64_t(0), above = 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    bool in_list = listed == bin;
    const auto each = [&](auto f) {
      if (in_list) {
        for (uint32_t i = threadIdx.x; i < s.filled; i += kRowThreads)
          if (s.list_key[i] >= lo && s.list_key[i] <= hi) f(s.list_key[i], s.list_sum[i]);
      } else {
        tokens(bin, [&](uint64_t k, uint64_t w) {
          if (k >= lo && k <= hi) f(k, w);
        });
      }
    };
    if (!in_list && n <= kList) {
      __syncthreads();
      if (threadIdx.x == 0) s.filled = 0;
      __syncthreads();
      tokens(bin, [&](uint64_t k, uint64_t w) {
        const uint32_t at = atomicAdd(&s.filled, 1u);
        s.list_key[at] = k;
        s.list_sum[at] = w;
      });
      __syncthreads();
      listed = bin;
      in_list = true;
    }
    while (n > 64) {
      // The keys' range, then bins over it.
      uint64_t least = ~uint64_t(0), most = 0;
      each([&](uint64_t k, uint64_t) {
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
      if (lane == 0) s.lo[wave] = least, s.hi[wave] = most;
      s.sums[threadIdx.x] = 0;
      s.counts[threadIdx.x] = 0;
      __syncthreads();
      for (int w = 0; w < kRowThreads / 64; ++w) {
        least = s.lo[w] < least ? s.lo[w] : least;
        most = s.hi[w] > most ? s.hi[w] : most;
      }
      const int width = 64 - __builtin_clzll(most - least | 1), shift = width > 9 ? width - 9 : 0;
      each([&](uint64_t k, uint64_t w) {
        const int b = int((most - k) >> shift);
        atomicAdd(reinterpret_cast<unsigned long long*>(&s.sums[b]), static_cast<unsigned long long>(w));
        atomicAdd(&s.counts[b], 1u);
      });
      __syncthreads();
      const uint64_t own = s.sums[threadIdx.x];
      const uint32_t mine = s.counts[threadIdx.x];
      uint64_t sum = own;
      uint32_t count = mine;
      scan(s, sum, count);
      find_bin(s, g, sum, own, count, mine);
      hi = most - (uint64_t(s.bin) << shift);
      lo = hi - ((uint64_t(1) << shift) - 1);
      if (lo > hi) lo = 0;                               // below zero: the last bin may reach past the least key
      n = s.count;
      above += s.before;
      if (g.count) g.count -= s.count_before; else g.sum -= s.before;
      __syncthreads();
    }
    // Few: one wave puts them in order by counting.
    __syncthreads();
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    each([&](uint64_t k, uint64_t w) {
      const uint32_t at = atomicAdd(&s.count, 1u);
      s.few_key[at] = k;
      s.few_sum[at] = w;
    });
    __syncthreads();
    if (wave == 0) {
      const uint64_t k = lane < int(n) ? s.few_key[lane] : 0, w = lane < int(n) ? s.few_sum[lane] : 0;
      uint64_t sum = 0;
      uint32_t count = 0;
      for (uint32_t j = 0; j < n; ++j)
        if (s.few_key[j] >= k) sum += s.few_sum[j], ++count;
      if (lane < int(n) && g.here(sum, w, count, 1)) s.key = k, s.before = sum;
    }
    __syncthreads();
    *upto = above + s.before;
    const uint64_t key = s.key;
    __syncthreads();
    return key;
  }
};

template <class T>
__global__ __launch_bounds__(kRowThreads) void choice_kernel(Args a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  const int index = blockIdx.x, t = threadIdx.x;
  const float2 ends = row_ends(a, index);
  if (ends.x == -__builtin_inff()) {
    if (t == 0) {
      a.ids[index] = -1;
      if (a.logprob) a.logprob[index] = -__builtin_inff();
    }
    return;
  }
  const Rule rule(a, index, ends.x, ends.y);
  const Row<T> row(a, index);
  uint64_t own = 0;
  uint32_t mine = 0;
  for (int c = 0; c < a.chunks; ++c) {
    const size_t at = (size_t(index) * a.chunks + c) * kBins + t;
    own += a.sums[at];
    mine += a.counts[at];
  }
  uint64_t sum = own;
  uint32_t count = mine;
  scan(s, sum, count);
  if (t == kBins - 1) s.before = sum, s.count = count;
  __syncthreads();
  uint64_t kept = s.before;                               // the sum of what is kept so far
  const uint32_t all = s.count;
  __syncthreads();
  Choice<T> pick{s, a, rule, row, index};

  const int top_k = a.top_ks ? a.top_ks[index] : a.top_k;
  if (!rule.greedy && top_k > 0 && uint32_t(top_k) < all) {
    Goal g{uint32_t(top_k), 0};
    find_bin(s, g, sum, own, count, mine);
    const int bin = s.bin;
    const uint32_t n = s.count;
    const uint64_t before = s.before;
    g.count -= s.count_before;
    __syncthreads();
    if (g.count < n) {
      uint64_t upto;
      pick.resolve(bin, n, g, &upto);
      kept = before + upto;
    } else {
      if (t == bin) s.before = sum;                      // the bin as a whole
      __syncthreads();
      kept = s.before;
      __syncthreads();
    }
  }
  const double top_p = a.top_ps ? double(a.top_ps[index]) : a.top_p;
  if (!rule.greedy && top_p < 1.0) {
    const uint64_t want = uint64_t(ceil(fmax(top_p, 0.0) * double(kept)));
    Goal g{0, want < 1 ? 1 : want > kept ? kept : want};
    find_bin(s, g, sum, own, count, mine);
    const int bin = s.bin;
    const uint32_t n = s.count;
    const uint64_t before = s.before;
    g.sum -= before;
    __syncthreads();
    uint64_t upto;
    pick.resolve(bin, n, g, &upto);
    kept = before + upto;
  }
  const float u = a.u[index];
  uint64_t past = rule.greedy || !(u > 0.f) ? 0 : uint64_t(fmin(double(u), 1.0) * double(kept));
  past = past < kept ? past : kept - 1;
  Goal g{0, past + 1};
  find_bin(s, g, sum, own, count, mine);
  const int bin = s.bin;
  const uint32_t n = s.count;
  g.sum -= s.before;
  __syncthreads();
  uint64_t upto;
  const uint64_t key = pick.resolve(bin, n, g, &upto);
  if (t == 0) {
    const int id = int(~uint32_t(key));
    a.ids[index] = id;
    if (a.logprob) {
      const uint32_t o = uint32_t(key >> 32), b = o >> 31 ? o & 0x7FFFFFFFu : ~o;
      const double y = rule.power(__builtin_bit_cast(float, b));
      a.logprob[index] = rule.greedy ? 0.f
                                     : float(y * 0.6931471805599453 - log(__builtin_ldexp(double(kept), -kUnit)));
    }
  }
}

// Chunks of a row: blocks for every CU, of at least 2048 logits each.
int chunks_of(int64_t rows, int64_t vocab) {
  int64_t chunks = 1024 / rows;
  if (chunks > vocab / 2048) chunks = vocab / 2048;
  if (chunks > kMaxChunks) chunks = kMaxChunks;
  return chunks < 1 ? 1 : int(chunks);
}

template <class T>
hipError_t launch(const Args& a, int64_t rows, hipStream_t stream) {
  const dim3 grid(a.chunks, uint32_t(rows));
  hipLaunchKernelGGL(max_kernel<T>, grid, dim3(kThreads), 0, stream, a);
  hipLaunchKernelGGL(bins_kernel<T>, grid, dim3(kThreads), 0, stream, a);
  const auto fn = choice_kernel<T>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(Shared)));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(uint32_t(rows)), dim3(kRowThreads), sizeof(Shared), stream, a);
  return hipGetLastError();
}

}  // namespace

size_t sample_workspace(int64_t rows, int64_t vocab) {
  return size_t(rows) * size_t(chunks_of(rows, vocab)) * (kBins * 12 + sizeof(float2));
}

hipError_t launch_sample(const tq2_sample_args& q, hipStream_t stream) {
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
  a.chunks = chunks_of(q.rows, q.vocab);
  a.row_stride = q.row_stride;
  a.temperature = q.temperature;
  a.top_p = q.top_p;
  a.min_p = q.min_p;
  const size_t parts = size_t(q.rows) * size_t(a.chunks);
  a.sums = static_cast<uint64_t*>(q.workspace);
  a.counts = reinterpret_cast<uint32_t*>(a.sums + parts * kBins);
  a.ends = reinterpret_cast<float2*>(a.counts + parts * kBins);
  if (q.logits_type == TQ2_TYPE_F32) return launch<F32>(a, q.rows, stream);
  if (q.logits_type == TQ2_TYPE_F16) return launch<F16>(a, q.rows, stream);
  return launch<BF16>(a, q.rows, stream);
}

}  // namespace tq2
