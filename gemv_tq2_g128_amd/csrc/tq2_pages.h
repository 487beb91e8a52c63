// Places of a paged cache: plain index arithmetic, shared by the kernels and
// (compiled for the host) their CPU test.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define TQ2_HD __host__ __device__ __forceinline__
#else
#define TQ2_HD inline
#endif

namespace tq2 {

// Places past this are never reached; sums of a place and a tile stay in 32 bits.
constexpr int64_t kMaxKeys = 0x7FFF0000;

// The cache as kernels see it.
struct Pages {
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu_q;                   // nullptr: one new token per sequence
  int32_t batch, tokens, pages, cols;
  int32_t page_shift;
  int32_t kv_heads, q_heads, head_dim;
  int64_t table_stride;
  int64_t k_page, k_head, k_token;       // strides in elements
  int64_t v_page, v_head, v_token;
};

// A sequence's rows of q and its length, cut to what the arrays can hold: the
// rows lie in 0 .. tokens, the length in 0 .. columns * page.  The place of a row
// may be negative (more new tokens than kv_len): it sees no key.
struct Seq {
  int32_t q0, q_len;                     // rows q0 .. q0 + q_len
  int32_t first;                         // place of row q0
  int32_t keys;                          // places 0 .. keys are in the table
};

TQ2_HD Seq sequence(const Pages& p, int32_t b) {
  Seq s;
  const int32_t len = p.kv_len[b];
  int32_t lo = b, hi = b + 1;
  if (p.cu_q) {
    lo = p.cu_q[b];
    hi = p.cu_q[b + 1];
  }
  const int32_t end = hi;
  lo = lo < 0 ? 0 : (lo > p.tokens ? p.tokens : lo);
  hi = hi < lo ? lo : (hi > p.tokens ? p.tokens : hi);
  s.q0 = lo;
  s.q_len = hi - lo;
  const int64_t first = int64_t(len) - (int64_t(end) - lo);  // at most len
  s.first = first < INT32_MIN ? INT32_MIN : int32_t(first);
  int64_t room = int64_t(p.cols) << p.page_shift;
  if (room > kMaxKeys) room = kMaxKeys;
  s.keys = len < 0 ? 0 : (len > room ? int32_t(room) : len);
  return s;
}

// The page of place n, or -1: outside the table, or not a page of the cache.
TQ2_HD int32_t page_of(const Pages& p, int32_t b, int32_t n) {
  if (n < 0) return -1;
  const int32_t col = n >> p.page_shift;
  if (col >= p.cols) return -1;
  const int32_t id = p.table[int64_t(b) * p.table_stride + col];
  return id >= 0 && id < p.pages ? id : -1;
}

// The parts that a sequence's keys are cut into for attention: part i covers
// base + i * per and on, for i < count.  At most `splits` parts of a multiple of
// 32 keys, at least `split_keys`; keys that no row sees through the window
// are left out in front.
struct Parts {
  int32_t base, per, count;
};

TQ2_HD Parts parts_of(const Seq& s, int32_t window, int32_t splits, int32_t split_keys) {
  Parts r;
  const int64_t edge = window ? int64_t(s.first) - window + 1 : 0;
  r.base = edge <= 0 ? 0 : int32_t(edge < s.keys ? edge : s.keys) & ~31;
  const int32_t keys = s.keys - r.base;
  const int64_t even = (int64_t(keys) + splits - 1) / splits;
  const int64_t up = (even + 31) & ~int64_t(31);
  r.per = up > split_keys ? int32_t(up) : split_keys;
  r.count = keys > 0 ? int32_t((int64_t(keys) + r.per - 1) / r.per) : 1;
  return r;
}

#ifdef __HIP__
// Number of sequences that end at or before row t: the one that owns it.  For a
// whole wave.
__device__ __forceinline__ int owner(const Pages& p, int t) {
  if (!p.cu_q) return t;
  int n = 0;
  for (int lo = 0; lo < p.batch; lo += 64) {
    const int b = lo + int(threadIdx.x & 63);
    n += __popcll(__ballot(b < p.batch && p.cu_q[b + 1] <= t));
  }
  return n;
}
#endif

}  // namespace tq2
