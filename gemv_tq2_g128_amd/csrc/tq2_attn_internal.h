// Launchers of the paged-cache operators (not installed).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tq2_attn.h"
#include "tq2_pages.h"

namespace tq2 {

struct AppendArgs {
  Pages pages;
  const void* q;                         // nullptr: k and v only
  const void* k;
  const void* v;
  void* q_out;
  void* k_cache;
  void* v_cache;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
  const double* freqs;
  const int32_t* positions;              // nullptr: the place
  const float* q_norm;
  const float* k_norm;
  const float* k_scale;
  const float* v_scale;
  float eps;
  int32_t half;                          // rotated pairs
  int32_t cut[2];                        // first pair of axes 1 and 2
  int32_t interleaved;
};
// Arguments are already validated: tokens >= 1.
hipError_t launch_kv_append(const AppendArgs& a, int act, int cache, hipStream_t stream);

}  // namespace tq2
