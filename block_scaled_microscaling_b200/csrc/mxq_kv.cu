// mxq_kv.cu -- tokens into and out of a paged MXFP4 key/value cache (sm_100a).
//
// A token's key (and value) of one head is head_dim / 32 blocks along the head's dimension, rounded like any
// other block ("EFQ-Softmax", Jargon: E2M1 codes, one exponent-only scale per 32 values). Page layout: codes
// [pages, heads, page_size, head_dim / 2], scales [pages, heads, page_size, head_dim / 32]: the rows of one head
// in a page are contiguous, which is what its attention reads. One thread per block; the four (two) threads of a
// row read and write neighbouring bytes. Bound by memory, and by one launch where the tokens are few: append and read
// of 16384 tokens (8 heads of 128, bf16) 15 us each (5.6 TB/s), of 61 tokens under 2 us each.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxq_block.cuh"
#include "mxq_ops_internal.h"

namespace mxq {
namespace {

constexpr int kKvThreads = 128;

// row of the cache (of [pages * heads * page_size]) that slot `s` of head `h` is, or -1 outside the cache
__device__ __forceinline__ long long cache_row(const KvCache& c, long long s, int h) {
    if (s < 0 || s >= c.pages * c.page) return -1;
    const uint32_t page = (uint32_t)s / (uint32_t)c.page, off = (uint32_t)s - page * (uint32_t)c.page;  // slots < 2^31
    return ((long long)page * c.heads + h) * c.page + off;
}

// blockIdx.y: 0 keys, 1 values; thread n is block n % DB of head n / DB % heads of token n / (DB * heads)
template <typename T>
__global__ void __launch_bounds__(kKvThreads) k_kv_append(const KvCache c, const void* __restrict__ k, long long k_stride,
                                                          const void* __restrict__ v, long long v_stride, long long tokens,
                                                          const long long* __restrict__ slots, bool a32) {
    const long long n = (long long)blockIdx.x * kKvThreads + threadIdx.x;
    pdl_wait_then_release();
    const int per = c.heads * c.db;
    const long long tok = n / per;
    if (tok >= tokens) return;
    const int rest = (int)(n - tok * per), h = rest / c.db, blk = rest - h * c.db;
    const long long row = cache_row(c, __ldg(slots + tok), h);
    if (row < 0) return;
    const bool val = blockIdx.y != 0;
    const char* src = static_cast<const char*>(val ? v : k) +
                      (tok * (val ? v_stride : k_stride) + (long long)rest * 32) * (long long)sizeof(T);
    uint32_t w[Blk<T>::NW], o[8];
    load_block<T>(src, 0, w, a32);
    const uint32_t byte = scale_byte<F_E2M1>(block_amax<T>(w));
    encode_block<F_E2M1, T>(w, byte, o);
    const long long b = row * c.db + blk;
    *reinterpret_cast<uint4*>((val ? c.vc : c.kc) + b * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    (val ? c.vs : c.ks)[b] = (uint8_t)byte;
}

template <typename T>
__global__ void __launch_bounds__(kKvThreads) k_kv_read(const KvCache c, const long long* __restrict__ slots, long long tokens,
                                                        void* __restrict__ k, void* __restrict__ v, bool a32) {
    const long long n = (long long)blockIdx.x * kKvThreads + threadIdx.x;
    pdl_wait_then_release();
    const int per = c.heads * c.db;
    const long long tok = n / per;
    if (tok >= tokens) return;
    const int rest = (int)(n - tok * per), h = rest / c.db, blk = rest - h * c.db;
    const long long row = cache_row(c, __ldg(slots + tok), h);
    const bool val = blockIdx.y != 0;
    uint32_t o[Blk<T>::NW];
    if (row < 0) {
#pragma unroll
        for (int i = 0; i < Blk<T>::NW; ++i) o[i] = 0;
    } else {
        const long long b = row * c.db + blk;
        const uint4 x = *reinterpret_cast<const uint4*>((val ? c.vc : c.kc) + b * 16);
        const uint32_t pw[4] = {x.x, x.y, x.z, x.w};
        decode_block<F_E2M1, T>(pw, (val ? c.vs : c.ks)[b], o);
    }
    store_block<T>(val ? v : k, n, o, a32);
}

bool both32(const void* a, const void* b, long long sa, long long sb) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | (uintptr_t)sa | (uintptr_t)sb) & 31) == 0;
}

template <typename... KArgs, typename... Args>
cudaError_t launch2(void (*kern)(KArgs...), long long threads, cudaStream_t st, Args... args) {
    const long long grid = (threads + kKvThreads - 1) / kKvThreads;
    if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 2);
    cfg.blockDim = dim3(kKvThreads);
    cfg.stream = st;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_kv_append(const KvCache& c, const void* k, long long k_stride, const void* v, long long v_stride, int dtype,
                             long long tokens, const long long* slots, cudaStream_t st) {
    const int size = dtype == 0 ? 4 : 2;
    const bool a32 = both32(k, v, k_stride * size, v_stride * size);
    const long long n = tokens * c.heads * c.db;
    if (dtype == 0) return launch2(k_kv_append<float>, n, st, c, k, k_stride, v, v_stride, tokens, slots, a32);
    return launch2(k_kv_append<__nv_bfloat16>, n, st, c, k, k_stride, v, v_stride, tokens, slots, a32);
}

cudaError_t launch_kv_read(const KvCache& c, const long long* slots, long long tokens, void* k, void* v, int dtype,
                           cudaStream_t st) {
    const bool a32 = both32(k, v, 0, 0);
    const long long n = tokens * c.heads * c.db;
    if (dtype == 0) return launch2(k_kv_read<float>, n, st, c, slots, tokens, k, v, a32);
    return launch2(k_kv_read<__nv_bfloat16>, n, st, c, slots, tokens, k, v, a32);
}

}  // namespace mxq
