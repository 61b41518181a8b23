// api.cuh -- what the files of the C ABI share: errors with their detail text, and checks of arguments.
#pragma once
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/moe_nvfp4.h"

namespace moe {

// Set the thread's detail text and return s.
moe_status_t fail(moe_status_t s, const char* fmt, ...);
moe_status_t cuda_fail(cudaError_t e, const char* what);
bool aligned(const void* p, size_t a);
moe_status_t check_device();
moe_status_t check_ws(const void* ws, size_t ws_bytes, size_t need);
bool rows_overlap(const void* a, int64_t ld_a, int64_t width_a, const void* b, int64_t ld_b, int64_t width_b, int T);
bool rows_overlap_bytes(const void* a, int64_t ld_a, int64_t width_a, int T, const void* b, int64_t bytes);
moe_status_t check_rows(const char* name, const void* p, int64_t ld, int64_t width, int elem, int T);

#define MOE_TRY(x)                              \
    do {                                        \
        moe_status_t s_ = (x);                  \
        if (s_ != MOE_OK) return s_;            \
    } while (0)

#define MOE_CUDA(x, what)                       \
    do {                                        \
        cudaError_t e_ = (x);                   \
        if (e_ != cudaSuccess) return cuda_fail(e_, what); \
    } while (0)

}  // namespace moe
