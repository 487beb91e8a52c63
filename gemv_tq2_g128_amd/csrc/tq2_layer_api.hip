// C ABI of the operators around the matmuls (tq2_q4.h, tq2_attn.h): argument
// checks, device check, launch.  Same error policy as tq2_api.hip: every failure is a status.
#include "../../include/tq2_attn.h"
#include "../../include/tq2_q4.h"
#include "tq2_attn_internal.h"
#include "tq2_host.h"
#include "tq2_internal.h"
#include "tq2_q4_internal.h"

#include <utility>

namespace {

using tq2::aligned;
using tq2::check_device;
using tq2::launch_status;
using tq2::overlaps;

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxStride = int64_t(1) << 40;

int type_bytes(int64_t t) { return t == TQ2_TYPE_F32 ? 4 : (t == TQ2_TYPE_E4M3 ? 1 : 2); }

bool size_ok(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

// Whether the strides keep rows 16-byte aligned; *bad is set if one is out of range.
bool strides_ok(int64_t bytes, int64_t s0, int64_t s1, int64_t s2, bool* bad) {
  for (int64_t s : {s0, s1, s2})
    if (!size_ok(s, 0, kMaxStride)) *bad = true;
  return !((s0 * bytes) & 15) && !((s1 * bytes) & 15) && !((s2 * bytes) & 15);
}

// Bytes from the first to the last element of a strided [n0, n1, n2, dim] array.
size_t extent(int64_t bytes, int64_t dim, int64_t n0, int64_t s0, int64_t n1, int64_t s1,
              int64_t n2 = 1, int64_t s2 = 0) {
  typedef unsigned __int128 wide;
  const wide most = wide(1) << 62;               // past any array, and no overflow when added to an address
  const wide all = (wide(n0 - 1) * s0 + wide(n1 - 1) * s1 + wide(n2 - 1) * s2 + dim) * bytes;
  return size_t(all < most ? all : most);
}

// Whether no two of the `dim` elements at i * s0 + j * s1, i < n0, j < n1, overlap.
bool apart(int64_t dim, int64_t n0, int64_t s0, int64_t n1, int64_t s1) {
  if (s0 < s1) std::swap(s0, s1), std::swap(n0, n1);
  if ((n0 > 1 && s0 < dim) || (n1 > 1 && s1 < dim)) return false;
  if (n0 <= 1 || n1 <= 1) return true;
  // Rows i apart along s0 lie within the other axis' reach for few i: at most n1.
  const __int128 reach = __int128(n1 - 1) * s1 + dim;
  for (int64_t i = 1; i < n0 && __int128(i) * s0 < reach; ++i) {
    const __int128 off = __int128(i) * s0;
    const int64_t j = int64_t(off / s1), past = int64_t(off % s1);
    if (past < dim || (j + 1 < n1 && s1 - past < dim)) return false;
  }
  return true;
}

// Whether rows of two [tokens, heads, dim] arrays whose extents overlap meet; a and b are
// taken as columns of one array (equal token strides), otherwise as meeting.  All in bytes.
bool rows_meet(int64_t tokens, int64_t wide, const void* a, int64_t a_heads, int64_t a_token, int64_t a_head,
               const void* b, int64_t b_heads, int64_t b_token, int64_t b_head) {
  const int64_t period = tokens > 1 ? a_token : int64_t(1) << 62;
  if (tokens > 1 && (a_token != b_token || a_token <= 0)) return true;
  const int64_t from = int64_t(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const auto place = [&](int64_t off) { return (off % period + period) % period; };
  // Heads of b all past those of a within a token's row.
  const __int128 a_end = __int128(a_heads - 1) * a_head + wide, b_span = __int128(b_heads - 1) * b_head + wide;
  if (place(from) >= a_end && place(from) + b_span <= period) return false;
  for (int64_t i = 0; i < a_heads; ++i)
    for (int64_t j = 0; j < b_heads; ++j) {
      const int64_t off = place(from + j * b_head - i * a_head);
      if (off < wide || period - off < wide) return true;
    }
  return false;
}

// Whether neighbours along each axis of a cache lie apart.
bool cache_apart(const tq2_paged_cache& c) {
  const int64_t d = c.head_dim;
  const auto ok = [&](int64_t page, int64_t head, int64_t token) {
    return (c.pages <= 1 || page >= d) && (c.kv_heads <= 1 || head >= d) && (c.page <= 1 || token >= d);
  };
  return ok(c.k_page_stride, c.k_head_stride, c.k_token_stride) && ok(c.v_page_stride, c.v_head_stride, c.v_token_stride);
}

// Sizes and types of the cache; nothing is dereferenced.
int check_cache_sizes(const tq2_paged_cache& c) {
  if (!size_ok(c.batch, 0, TQ2_ATTN_MAX_BATCH) || !size_ok(c.tokens, 0, kMaxDim) ||
      !size_ok(c.pages, 0, kMaxDim) || !size_ok(c.table_cols, 0, kMaxDim) ||
      !size_ok(c.table_stride, 0, kMaxDim) || !size_ok(c.kv_heads, 1, TQ2_ATTN_MAX_HEADS) ||
      !size_ok(c.q_heads, 1, TQ2_ATTN_MAX_HEADS))
    return TQ2_ERR_INVALID;
  if (c.head_dim != 64 && c.head_dim != 96 && c.head_dim != 128 && c.head_dim != 192 &&
      c.head_dim != 256)
    return TQ2_ERR_INVALID;
  const bool wide = (c.act_type == TQ2_TYPE_F32 && c.cache_type == TQ2_TYPE_F16) ||
                    (c.act_type == TQ2_TYPE_F16 && c.cache_type == TQ2_TYPE_F16) ||
                    (c.act_type == TQ2_TYPE_BF16 && c.cache_type == TQ2_TYPE_BF16);
  const bool narrow = c.cache_type == TQ2_TYPE_E4M3 && size_ok(c.act_type, TQ2_TYPE_F32, TQ2_TYPE_BF16);
  if (!wide && !narrow) return TQ2_ERR_INVALID;
  if (!c.cu_q && c.tokens != c.batch) return TQ2_ERR_INVALID;
  if (!size_ok(c.page, 16, int64_t(1) << 20) || (c.page & (c.page - 1))) return TQ2_ERR_SHAPE;
  if (c.q_heads % c.kv_heads) return TQ2_ERR_SHAPE;
  return TQ2_OK;
}

// Pointers and strides of the cache.
int check_cache_arrays(const tq2_paged_cache& c) {
  // An empty array has no address.
  if ((c.table_cols > 0 && !c.table) || !c.kv_len || (c.pages > 0 && (!c.k || !c.v))) return TQ2_ERR_INVALID;
  const bool narrow = c.cache_type == TQ2_TYPE_E4M3;
  if (narrow != (c.k_scale != nullptr) || narrow != (c.v_scale != nullptr)) return TQ2_ERR_INVALID;
  const int64_t cb = type_bytes(c.cache_type);
  bool bad = false;
  const bool even = strides_ok(cb, c.k_page_stride, c.k_head_stride, c.k_token_stride, &bad) &
                    strides_ok(cb, c.v_page_stride, c.v_head_stride, c.v_token_stride, &bad);
  if (bad) return TQ2_ERR_INVALID;
  if (!even || !aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.table, 4) ||
      !aligned(c.kv_len, 4) || !aligned(c.cu_q, 4) || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4))
    return TQ2_ERR_ALIGN;
  if (c.k && c.k == c.v) return TQ2_ERR_ALIAS;
  return TQ2_OK;
}

size_t k_extent(const tq2_paged_cache& c) {
  return c.pages == 0 ? 0 : extent(type_bytes(c.cache_type), c.head_dim, c.pages, c.k_page_stride, c.kv_heads,
                                   c.k_head_stride, c.page, c.k_token_stride);
}

size_t v_extent(const tq2_paged_cache& c) {
  return c.pages == 0 ? 0 : extent(type_bytes(c.cache_type), c.head_dim, c.pages, c.v_page_stride, c.kv_heads,
                                   c.v_head_stride, c.page, c.v_token_stride);
}

tq2::Pages pages_of(const tq2_paged_cache& c) {
  tq2::Pages p;
  p.table = c.table;
  p.kv_len = c.kv_len;
  p.cu_q = c.cu_q;
  p.batch = int32_t(c.batch);
  p.tokens = int32_t(c.tokens);
  p.pages = int32_t(c.pages);
  p.cols = int32_t(c.table_cols);
  p.page_shift = __builtin_ctzll(uint64_t(c.page));
  p.kv_heads = int32_t(c.kv_heads);
  p.q_heads = int32_t(c.q_heads);
  p.head_dim = int32_t(c.head_dim);
  p.table_stride = c.table_stride;
  p.k_page = c.k_page_stride;
  p.k_head = c.k_head_stride;
  p.k_token = c.k_token_stride;
  p.v_page = c.v_page_stride;
  p.v_head = c.v_head_stride;
  p.v_token = c.v_token_stride;
  return p;
}

// Sizes of an attention call; nothing is dereferenced.
int check_attention_sizes(const tq2_paged_attention_args& a) {
  const int st = check_cache_sizes(a.cache);
  if (st != TQ2_OK) return st;
  if (!size_ok(a.max_q, 0, kMaxDim) || !size_ok(a.max_kv, 0, (int64_t(1) << 31) - 1) ||
      !size_ok(a.window, 0, (int64_t(1) << 31) - 1))
    return TQ2_ERR_INVALID;
  // Rows and heads are counted in 31 bits.
  if (a.cache.tokens * a.cache.q_heads >= (int64_t(1) << 31) - 4096) return TQ2_ERR_INVALID;
  return TQ2_OK;
}

}  // namespace

extern "C" {

int tq2_q4_gemv(const void* codes, const void* scales, const float* x, const float* residual,
                float* out, int64_t m, int64_t n, int64_t k, int group, void* stream) {
  if (m < 0 || n < 0 || k <= 0) return TQ2_ERR_INVALID;
  if (k % 128) return TQ2_ERR_SHAPE;
  if (m > TQ2_Q4_MAX_M || n > kMaxDim || k > tq2::kGemmMaxK) return TQ2_ERR_INVALID;
  if (group != 32 && group != 64 && group != 128) return TQ2_ERR_INVALID;
  if (m == 0 || n == 0) return TQ2_OK;
  if (!codes || !scales || !x || !out) return TQ2_ERR_INVALID;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(x, 16) || !aligned(out, 16) ||
      (residual && !aligned(residual, 16)))
    return TQ2_ERR_ALIGN;
  const size_t ob = size_t(m) * size_t(n) * 4;
  if (overlaps(out, ob, x, size_t(m) * size_t(k) * 4) ||
      overlaps(out, ob, codes, size_t(n) * size_t(k / 2)) ||
      overlaps(out, ob, scales, size_t(n) * size_t(k / group) * 2))
    return TQ2_ERR_ALIAS;
  if (residual && residual != out && overlaps(out, ob, residual, ob)) return TQ2_ERR_ALIAS;
  const int st = check_device();
  if (st != TQ2_OK) return st;
  const tq2::Q4Args a = {static_cast<const uint8_t*>(codes), static_cast<const uint16_t*>(scales),
                         x, residual, out, m, n, k};
  return launch_status(tq2::launch_q4_gemv(a, group, static_cast<hipStream_t>(stream)));
}

int tq2_kv_append(const tq2_kv_append_args* args, void* stream) {
  if (!args) return TQ2_ERR_INVALID;
  const tq2_kv_append_args& a = *args;
  const tq2_paged_cache& c = a.cache;
  int st = check_cache_sizes(c);
  if (st != TQ2_OK) return st;
  if (!size_ok(a.rot, 0, c.head_dim) || !size_ok(a.axes, 1, 3)) return TQ2_ERR_INVALID;
  if (a.rot % 8) return TQ2_ERR_SHAPE;
  if (a.axes > 1 && !a.positions) return TQ2_ERR_INVALID;
  int64_t sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (!size_ok(a.section[i], 0, i < a.axes ? a.rot / 2 : 0)) return TQ2_ERR_INVALID;
    sum += a.section[i];
  }
  if (sum != a.rot / 2) return TQ2_ERR_INVALID;
  if (!(a.eps >= 0.0)) return TQ2_ERR_INVALID;
  if (c.tokens == 0 || c.batch == 0) return TQ2_OK;              // no row has a sequence
  st = check_cache_arrays(c);
  if (st != TQ2_OK) return st;
  if (!a.k || !a.v || (a.q != nullptr) != (a.q_out != nullptr) || (a.rot > 0 && !a.freqs))
    return TQ2_ERR_INVALID;
  const int64_t ab = type_bytes(c.act_type), d = c.head_dim;
  bool bad = false;
  const bool even = strides_ok(ab, a.k_token_stride, a.k_head_stride, 0, &bad) &
                    strides_ok(ab, a.v_token_stride, a.v_head_stride, 0, &bad) &
                    (!a.q || (strides_ok(ab, a.q_token_stride, a.q_head_stride, 0, &bad) &
                              strides_ok(ab, a.q_out_token_stride, a.q_out_head_stride, 0, &bad)));
  if (bad) return TQ2_ERR_INVALID;
  if (!even || !aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.q_out, 16) ||
      !aligned(a.q_norm, 16) || !aligned(a.k_norm, 16) || !aligned(a.freqs, 8) || !aligned(a.positions, 4))
    return TQ2_ERR_ALIGN;
  const size_t kb = extent(ab, d, c.tokens, a.k_token_stride, c.kv_heads, a.k_head_stride);
  const size_t vb = extent(ab, d, c.tokens, a.v_token_stride, c.kv_heads, a.v_head_stride);
  const size_t qb = a.q ? extent(ab, d, c.tokens, a.q_token_stride, c.q_heads, a.q_head_stride) : 0;
  const size_t ob = a.q ? extent(ab, d, c.tokens, a.q_out_token_stride, c.q_heads, a.q_out_head_stride) : 0;
  for (const auto& cache : {std::make_pair(c.k, k_extent(c)), std::make_pair(c.v, v_extent(c))})
    if (overlaps(cache.first, cache.second, a.q, qb) || overlaps(cache.first, cache.second, a.k, kb) ||
        overlaps(cache.first, cache.second, a.v, vb) || overlaps(cache.first, cache.second, a.q_out, ob))
      return TQ2_ERR_ALIAS;
  // In place, q_out's extent is q's own, which k and v may share as other columns of one array.
  const bool in_place = a.q_out == a.q && a.q_out_token_stride == a.q_token_stride &&
                        a.q_out_head_stride == a.q_head_stride;
  if (a.q && !in_place &&
      (overlaps(a.q_out, ob, a.q, qb) || overlaps(a.q_out, ob, a.k, kb) || overlaps(a.q_out, ob, a.v, vb)))
    return TQ2_ERR_ALIAS;
  const auto meets_q = [&](const void* in, size_t bytes, int64_t token, int64_t head) {
    return overlaps(a.q, qb, in, bytes) && rows_meet(c.tokens, d * ab, a.q, c.q_heads, a.q_token_stride * ab,
                                                     a.q_head_stride * ab, in, c.kv_heads, token * ab, head * ab);
  };
  if (a.q && in_place && (meets_q(a.k, kb, a.k_token_stride, a.k_head_stride) ||
                          meets_q(a.v, vb, a.v_token_stride, a.v_head_stride)))
    return TQ2_ERR_ALIAS;
  if (!cache_apart(c) || (a.q && !apart(d, c.tokens, a.q_out_token_stride, c.q_heads, a.q_out_head_stride)))
    return TQ2_ERR_ALIAS;
  st = check_device();
  if (st != TQ2_OK) return st;
  tq2::AppendArgs g;
  g.pages = pages_of(c);
  g.q = a.q;
  g.k = a.k;
  g.v = a.v;
  g.q_out = a.q_out;
  g.k_cache = c.k;
  g.v_cache = c.v;
  g.q_token = a.q_token_stride;
  g.q_head = a.q_head_stride;
  g.k_token = a.k_token_stride;
  g.k_head = a.k_head_stride;
  g.v_token = a.v_token_stride;
  g.v_head = a.v_head_stride;
  g.o_token = a.q_out_token_stride;
  g.o_head = a.q_out_head_stride;
  g.freqs = a.freqs;
  g.positions = a.positions;
  g.q_norm = a.q_norm;
  g.k_norm = a.k_norm;
  g.k_scale = c.k_scale;
  g.v_scale = c.v_scale;
  g.eps = float(a.eps);
  g.half = int32_t(a.rot / 2);
  g.cut[0] = int32_t(a.section[0]);
  g.cut[1] = int32_t(a.section[0] + a.section[1]);
  g.interleaved = a.interleaved != 0;
  return launch_status(
      tq2::launch_kv_append(g, int(c.act_type), int(c.cache_type), static_cast<hipStream_t>(stream)));
}

size_t tq2_paged_attention_workspace_bytes(const tq2_paged_attention_args* args) {
  if (!args || check_attention_sizes(*args) != TQ2_OK || args->cache.tokens == 0 ||
      args->cache.batch == 0)
    return 0;
  return tq2::plan_attention(*args).workspace;
}

int tq2_paged_attention(const tq2_paged_attention_args* args, void* stream) {
  if (!args) return TQ2_ERR_INVALID;
  const tq2_paged_attention_args& a = *args;
  const tq2_paged_cache& c = a.cache;
  int st = check_attention_sizes(a);
  if (st != TQ2_OK) return st;
  const double scale = a.scale * 1.4426950408889634;             // scores as exponents of two
  if (!(a.scale > 0.0) || !(scale <= double(__FLT_MAX__))) return TQ2_ERR_INVALID;
  if (c.tokens == 0 || c.batch == 0) return TQ2_OK;              // no row has a sequence
  st = check_cache_arrays(c);
  if (st != TQ2_OK) return st;
  if (!a.q || !a.out) return TQ2_ERR_INVALID;
  const int64_t ab = type_bytes(c.act_type), cb = type_bytes(c.cache_type), d = c.head_dim;
  bool bad = false;
  const bool even = strides_ok(ab, a.q_token_stride, a.q_head_stride, 0, &bad) &
                    strides_ok(ab, a.out_token_stride, a.out_head_stride, 0, &bad);
  // A buffer resource spans 16 tokens of a page.
  const int64_t most = (int64_t(1) << 31) - 4096;
  if (bad || c.k_token_stride * cb * 16 > most || c.v_token_stride * cb * 16 > most) return TQ2_ERR_INVALID;
  const tq2::AttnPlan plan = tq2::plan_attention(a);
  if (a.workspace_bytes < 0 || (plan.workspace > 0 && (!a.workspace || size_t(a.workspace_bytes) < plan.workspace)))
    return TQ2_ERR_INVALID;
  if (!even || !aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.workspace, 16)) return TQ2_ERR_ALIGN;
  const size_t qb = extent(ab, d, c.tokens, a.q_token_stride, c.q_heads, a.q_head_stride);
  const size_t ob = extent(ab, d, c.tokens, a.out_token_stride, c.q_heads, a.out_head_stride);
  const bool in_place = a.out == a.q && a.out_token_stride == a.q_token_stride && a.out_head_stride == a.q_head_stride;
  if (!in_place && overlaps(a.out, ob, a.q, qb)) return TQ2_ERR_ALIAS;
  if (!apart(d, c.tokens, a.out_token_stride, c.q_heads, a.out_head_stride)) return TQ2_ERR_ALIAS;
  for (const auto& cache : {std::make_pair(c.k, k_extent(c)), std::make_pair(c.v, v_extent(c))})
    if (overlaps(cache.first, cache.second, a.out, ob) ||
        overlaps(cache.first, cache.second, a.workspace, plan.workspace))
      return TQ2_ERR_ALIAS;
  if (overlaps(a.workspace, plan.workspace, a.out, ob) || overlaps(a.workspace, plan.workspace, a.q, qb))
    return TQ2_ERR_ALIAS;
  st = check_device();
  if (st != TQ2_OK) return st;
  tq2::AttnArgs g;
  g.pages = pages_of(c);
  g.q = a.q;
  g.out = a.out;
  g.k_cache = c.k;
  g.v_cache = c.v;
  g.k_scale = c.k_scale;
  g.v_scale = c.v_scale;
  g.q_token = a.q_token_stride;
  g.q_head = a.q_head_stride;
  g.o_token = a.out_token_stride;
  g.o_head = a.out_head_stride;
  g.part = plan.splits > 1 ? static_cast<float*>(a.workspace) : nullptr;
  g.scale = float(scale);
  g.window = int32_t(a.window);
  g.group = uint32_t(c.q_heads / c.kv_heads);
  g.splits = plan.splits;
  g.split_keys = plan.split_keys;
  return launch_status(tq2::launch_paged_attention(g, plan, int(c.act_type), int(c.cache_type),
                                                   static_cast<hipStream_t>(stream)));
}

}  // extern "C"
