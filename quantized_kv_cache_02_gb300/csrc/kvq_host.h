// Error reporting and launch accounting shared by the host translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kvq.h"

namespace kvq {

// Set the thread's kvq_last_error message and return ``st``.
kvq_status fail(kvq_status st, const char* fmt, ...);
kvq_status cuda_fail(cudaError_t e, const char* what);
// Add to kvq_kernel_launches.
void count_launches(uint64_t n);

}  // namespace kvq
