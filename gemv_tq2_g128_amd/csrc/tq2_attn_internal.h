// Launchers of the paged-cache operators (not installed).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tq2_attn.h"
#include "tq2_attn_plan.h"
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

struct AttnArgs {
  Pages pages;
  const void* q;
  void* out;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  int64_t q_token, q_head, o_token, o_head;
  float* part;                           // partial outputs, nullptr if splits == 1
  float scale;                           // of the scores, times log2 e
  int32_t window;                        // 0: none
  uint32_t group;                        // query heads of a key head
  int32_t splits;                        // parts of a sequence's keys
  int32_t split_keys;                    // least keys of a part, a multiple of 32
};

// Arguments are already validated: tokens >= 1.
hipError_t launch_attention_tiles(const AttnArgs& a, const AttnPlan& plan, int act, int cache,
                                  hipStream_t stream);
hipError_t launch_paged_attention(const AttnArgs& a, const AttnPlan& plan, int act, int cache,
                                  hipStream_t stream);

}  // namespace tq2
