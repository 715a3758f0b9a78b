// host.h — what the C entry points of libcolimoe share on the host (internal, not part of the ABI).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace colimoe {

int cuda_fail(cudaError_t e);              // keeps e for coli_moe_last_cuda_error, returns COLI_MOE_ECUDA
int check_device();                        // COLI_MOE_OK if the current device is compute capability 10.3
int num_sms();                             // SMs of the current device (152 where there is none)
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace colimoe
