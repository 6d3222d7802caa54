// q4gsw_api_common.h - what the two files of C entry points share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/q4gsw.h"

namespace q4gsw {

// The calling thread's route string (q4gsw_last_route).
void set_route(const char* s);

// Shape rules shared by every entry point that takes a packed weight.
q4gsw_status check_weight_shape(int N, int K, int gs);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline q4gsw_status from_cuda(cudaError_t e) { return e == cudaSuccess ? Q4GSW_OK : Q4GSW_ERR_CUDA; }

}  // namespace q4gsw
