// Launcher of the token choice (not installed).  Arguments are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tq2_sample.h"

namespace tq2 {

size_t sample_workspace(int64_t rows, int64_t vocab, int64_t type);
hipError_t launch_sample(const tq2_sample_args& a, hipStream_t stream);

}  // namespace tq2
