// mxq_check.h -- host-side argument checks shared by the C entry points (mxq_api.cu, mxq_ops_api.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mxq.h"

namespace {

[[maybe_unused]] int elem_bits(mxq_format f) {
    switch (f) {
        case MXQ_AXS6:
        case MXQ_MXFP6_E2M3:
        case MXQ_MXFP6_E3M2: return 6;
        case MXQ_MXFP8_E4M3: return 8;
        case MXQ_MXFP4_E2M1: return 4;
    }
    return -1;
}
[[maybe_unused]] bool fmt_ok(mxq_format f) { return elem_bits(f) > 0; }
[[maybe_unused]] bool dtype_ok(mxq_dtype d) { return d == MXQ_F32 || d == MXQ_BF16; }
[[maybe_unused]] int dtype_bytes(mxq_dtype d) { return d == MXQ_F32 ? 4 : 2; }

constexpr int64_t kMaxElems = (int64_t)1 << 50;

[[maybe_unused]] mxq_status check_shape(int64_t rows, int64_t cols) {
    if (rows < 0 || cols <= 0 || cols % 32 != 0) return MXQ_ERR_SHAPE;
    if (rows > 0 && cols > kMaxElems / rows) return MXQ_ERR_SHAPE;
    return MXQ_OK;
}

// device (or managed) memory of the current device, aligned to `align`
[[maybe_unused]] mxq_status check_ptr(const void* p, uintptr_t align) {
    if (p == nullptr) return MXQ_ERR_INVALID_ARG;
    cudaPointerAttributes a;
    cudaError_t e = cudaPointerGetAttributes(&a, p);
    if (e != cudaSuccess) {
        cudaGetLastError();  // the failed query also sets the (non-sticky) last error: clear it
        return MXQ_ERR_INVALID_ARG;
    }
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) return MXQ_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return MXQ_ERR_CUDA;
    if (a.type == cudaMemoryTypeDevice && a.device != dev) return MXQ_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(p) % align != 0) return MXQ_ERR_ALIGN;
    return MXQ_OK;
}

[[maybe_unused]] bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

[[maybe_unused]] size_t codes_bytes(mxq_format f, int64_t rows, int64_t cols) {
    return (size_t)rows * (size_t)(cols / 32) * (size_t)(4 * elem_bits(f));
}
[[maybe_unused]] size_t scales_bytes(mxq_format f, int64_t rows, int64_t cols) {
    return (size_t)rows * (size_t)(cols / 32) * (f == MXQ_AXS6 ? 2u : 1u);
}
[[maybe_unused]] uintptr_t scales_align(mxq_format f) { return f == MXQ_AXS6 ? 2 : 1; }

[[maybe_unused]] mxq_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return MXQ_OK;
    if (e == cudaErrorNotSupported) return MXQ_ERR_UNSUPPORTED;
    return MXQ_ERR_CUDA;
}

#define MXQ_TRY(x)                         \
    do {                                   \
        mxq_status s_ = (x);               \
        if (s_ != MXQ_OK) return s_;       \
    } while (0)

}  // namespace
