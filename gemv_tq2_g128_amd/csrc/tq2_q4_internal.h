// Launcher of the 4-bit matrix-vector products (not installed).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tq2 {

struct Q4Args {
  const uint8_t* codes;      // [n, k / 2]
  const uint16_t* scales;    // binary16 [n, k / group]
  const float* x;            // [m, k]
  const float* residual;     // [m, n] or nullptr
  float* out;                // [m, n]
  int64_t m, n, k;
};
// Arguments are already validated: 1 <= m <= 16, n >= 1, group 32, 64 or 128.
hipError_t launch_q4_gemv(const Q4Args& a, int group, hipStream_t stream);

}  // namespace tq2
