// m2_host.cuh -- argument checks and error mapping shared by the C entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cstdlib>
#include <vector>

#include "m2.h"

namespace m2 {
namespace host {

// Storage dtypes of caches and activations; the post-conv buffer may also be fp16.
inline bool valid_dtype(int32_t d) { return d == M2_F32 || d == M2_BF16; }
inline bool valid_buffer_dtype(int32_t d) { return valid_dtype(d) || d == M2_F16; }
inline int dsize(int32_t d) { return d == M2_F32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool stride_ok(int64_t stride_elems, int elem_size, int64_t min_elems) {
    return stride_elems >= min_elems && (stride_elems * elem_size) % 16 == 0;
}

inline m2_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return M2_OK;
    if (e == cudaErrorMemoryAllocation) return M2_ERR_OOM;
    return M2_ERR_CUDA;
}

// M2_VALIDATE=1: copy the slot indices to the host (synchronising) and reject
// duplicates. Debug aid only; never used on a captured stream.
inline bool validate_mode() {
    const char* v = std::getenv("M2_VALIDATE");
    return v && v[0] == '1';
}

inline m2_status validate_slots(const int32_t* slot_idx, int32_t n, int64_t num_slots, cudaStream_t s) try {
    std::vector<int32_t> h(static_cast<size_t>(n));
    if (cudaMemcpyAsync(h.data(), slot_idx, sizeof(int32_t) * n, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return M2_ERR_CUDA;
    std::vector<char> seen(static_cast<size_t>(num_slots), 0);
    for (int32_t v : h) {
        if (v < 0 || v >= num_slots) continue;  // padding / device-reported
        if (seen[v]) return M2_ERR_INVALID_ARG;
        seen[v] = 1;
    }
    return M2_OK;
} catch (...) {  // no exception leaves a C entry point
    return M2_ERR_OOM;
}

// A cache belongs to the device that was current when it was described; a
// launch on another device would read its buffers through a foreign address.
inline bool on_current_device(int32_t device) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();  // no usable device: the launch reports it
        return true;
    }
    return dev == device;
}

}  // namespace host
}  // namespace m2
