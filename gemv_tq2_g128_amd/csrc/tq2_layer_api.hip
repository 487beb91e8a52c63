// C ABI of the operators around the matmuls (tq2_q4.h): argument checks, device
// check, launch.  Same error policy as tq2_api.hip: every failure is a status.
#include "../../include/tq2_q4.h"
#include "tq2_host.h"
#include "tq2_internal.h"
#include "tq2_q4_internal.h"

namespace {

using tq2::aligned;
using tq2::check_device;
using tq2::launch_status;
using tq2::overlaps;

constexpr int64_t kMaxDim = int64_t(1) << 30;

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

}  // extern "C"
