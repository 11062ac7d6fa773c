// mxq_swiglu.cu -- silu(gate) * up with 8-bit checkpoints of its inputs, and its gradients (sm_100a).
//
// Training keeps gate and up between the passes; as MXFP8 E4M3 ("Sonar: Online MXFP6", MXFP8 activations) they
// take 33/64 of their bf16 bytes. Forward: one thread takes a block of 32 values of gate and of up, computes
// the products in fp32 from the unrounded values and encodes both blocks from the same registers. Backward:
// one thread decodes the two blocks and computes, with s = sigmoid(g),
//   dgate = dy * u * s * (1 + g * (1 - s)),   dup = dy * g * s.
// Both are bound by memory: 8.06 bytes per value pair forward and 8.06 backward in bf16 (about 40 instructions
// per pair fit beside that): 16384 x 9728 bf16 takes 190 us forward (6.8 TB/s; 218 with the checkpoint after the products,
// for want of warps) and 188 backward (6.8 TB/s), 8192 x 9728 fp32 181 and 171 (6.2 and 6.6 TB/s). One thread per block needs no shuffle for the block's maximum; a few
// rows are bound by that thread's latency instead (37 x 2560 fp32 4 us a pass). bf16 divides with the
// hardware's approximate reciprocal (2 units in the last place, before the rounding to 2^-8); the exponential is the
// accurate one for both types, since the approximate one loses |x| / 2^24 of its result.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxq_block.cuh"
#include "mxq_ops_internal.h"

namespace mxq {
namespace {

constexpr int kSwThreads = 128;

// 1 / (1 + e^-x) without overflow: with e = e^-|x|, the denominator stays in [1, 2]
template <typename T> __device__ __forceinline__ float sigmoid(float x) {
    const float e = expf(-fabsf(x));
    const float s = sizeof(T) == 4 ? 1.0f / (1.0f + e) : __fdividef(1.0f, 1.0f + e);
    return x < 0.0f ? e * s : s;
}

// first value of block b of a [rows, cols] matrix with row stride ld, kb blocks per row
__device__ __forceinline__ long long block_at(long long b, uint32_t kb, long long ld) {
    long long r;
    if ((unsigned long long)b <= 0xFFFFFFFFull) r = (uint32_t)b / kb;
    else r = b / kb;
    return r * ld + (b - r * kb) * 32;
}

template <typename T>
__global__ void __launch_bounds__(kSwThreads) k_swiglu_forward(const void* __restrict__ gate, const void* __restrict__ up,
                                                               void* __restrict__ out, void* __restrict__ gc,
                                                               uint8_t* __restrict__ gs, void* __restrict__ uc,
                                                               uint8_t* __restrict__ us, long long nblocks, uint32_t kb,
                                                               long long ld, bool in32, bool out32, bool codes32) {
    const long long b = (long long)blockIdx.x * kSwThreads + threadIdx.x;
    pdl_wait_then_release();
    if (b >= nblocks) return;
    const long long at = block_at(b, kb, ld) * (long long)sizeof(T);
    uint32_t g[Blk<T>::NW], u[Blk<T>::NW];
    load_block<T>(static_cast<const char*>(gate) + at, 0, g, in32);
    load_block<T>(static_cast<const char*>(up) + at, 0, u, in32);
    if (gc != nullptr) {  // a checkpoint is asked for; stored before the products, so that few registers are live at a time
        uint32_t code[8];
        uint32_t byte = scale_byte<F_E4M3>(block_amax<T>(g));
        encode_block<F_E4M3, T>(g, byte, code);
        store_payload<F_E4M3>(gc, b, code, codes32);
        gs[b] = (uint8_t)byte;
        byte = scale_byte<F_E4M3>(block_amax<T>(u));
        encode_block<F_E4M3, T>(u, byte, code);
        store_payload<F_E4M3>(uc, b, code, codes32);
        us[b] = (uint8_t)byte;
    }
    char* const to = static_cast<char*>(out) + b * 32 * (long long)sizeof(T);
#pragma unroll
    for (int q = 0; q < Blk<T>::NW / 8; ++q) {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 32 / (int)sizeof(T) / 2; ++j) {
            const int i = q * (32 / (int)sizeof(T) / 2) + j;  // pair of values
            float g0, g1, u0, u1;
            upk(pair<T>(g, i), g0, g1);
            upk(pair<T>(u, i), u0, u1);
            const float y0 = g0 * sigmoid<T>(g0) * u0, y1 = g1 * sigmoid<T>(g1) * u1;
            if constexpr (sizeof(T) == 4) {
                o[2 * j] = __float_as_uint(y0);
                o[2 * j + 1] = __float_as_uint(y1);
            } else {
                o[j] = bf16x2(y0, y1);
            }
        }
        st32(to + 32 * q, o, out32);
    }
}

template <typename T>
__global__ void __launch_bounds__(kSwThreads) k_swiglu_backward(const void* __restrict__ grad, const void* __restrict__ gc,
                                                                const uint8_t* __restrict__ gs, const void* __restrict__ uc,
                                                                const uint8_t* __restrict__ us, void* __restrict__ dgate,
                                                                void* __restrict__ dup, long long nblocks, uint32_t kb,
                                                                long long ld, bool in32, bool out32, bool codes32) {
    const long long b = (long long)blockIdx.x * kSwThreads + threadIdx.x;
    pdl_wait_then_release();
    if (b >= nblocks) return;
    uint32_t cg[8], cu[8], dy[Blk<T>::NW];
    const uint32_t eg = __ldg(gs + b), eu = __ldg(us + b);
    load_payload<F_E4M3>(gc, b, cg, codes32);
    load_payload<F_E4M3>(uc, b, cu, codes32);
    load_block<T>(grad, b, dy, in32);
    const float nan = __uint_as_float(0x7FC00000u);
    const float fg = eg == 0xFFu ? nan : fwd_scale(eg), fu = eu == 0xFFu ? nan : fwd_scale(eu);
    const long long at = block_at(b, kb, ld) * (long long)sizeof(T);
    char* const pg = static_cast<char*>(dgate) + at;
    char* const pu = static_cast<char*>(dup) + at;
    constexpr int NQ = 32 / (int)sizeof(T);  // values in 32 bytes of output
#pragma unroll
    for (int q = 0; q < 32 / NQ; ++q) {
        uint32_t og[8], ou[8];
#pragma unroll
        for (int j = 0; j < NQ / 4; ++j) {
            const int c = q * (NQ / 4) + j;  // word of four codes
            float g[4], u[4], a[4], d[4];
            up4<F_E4M3>(cg[c], g[0], g[1], g[2], g[3]);
            up4<F_E4M3>(cu[c], u[0], u[1], u[2], u[3]);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                float y0, y1;
                upk(pair<T>(dy, 2 * c + i / 2), y0, y1);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float y = e ? y1 : y0, gv = g[i + e] * fg, uv = u[i + e] * fu, s = sigmoid<T>(gv);
                    // s first: for a gate far below zero it is 0, and the other factors' product may be infinite
                    d[i + e] = y * (gv * s);
                    a[i + e] = y * (s * (1.0f + gv * (1.0f - s))) * uv;
                }
            }
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    og[4 * j + i] = __float_as_uint(a[i]);
                    ou[4 * j + i] = __float_as_uint(d[i]);
                }
            } else {
                og[2 * j] = bf16x2(a[0], a[1]);
                og[2 * j + 1] = bf16x2(a[2], a[3]);
                ou[2 * j] = bf16x2(d[0], d[1]);
                ou[2 * j + 1] = bf16x2(d[2], d[3]);
            }
        }
        st32(pg + 32 * q, og, out32);
        st32(pu + 32 * q, ou, out32);
    }
}

bool all32(std::initializer_list<const void*> ps, long long row_bytes) {
    uintptr_t v = (uintptr_t)row_bytes;
    for (const void* p : ps) v |= reinterpret_cast<uintptr_t>(p);
    return (v & 31) == 0;
}

}  // namespace

cudaError_t launch_swiglu_forward(const void* gate, const void* up, int dtype, long long rows, long long cols, long long ld,
                                  void* out, void* gc, void* gs, void* uc, void* us, cudaStream_t st) {
    const long long nb = rows * (cols / 32), grid = (nb + kSwThreads - 1) / kSwThreads;
    if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const bool in32 = all32({gate, up}, ld * (dtype == 0 ? 4 : 2)), out32 = all32({out}, 0), codes32 = all32({gc, uc}, 0);
    auto* a = static_cast<uint8_t*>(gs);
    auto* b = static_cast<uint8_t*>(us);
    if (dtype == 0)
        return launch_pdl(k_swiglu_forward<float>, (unsigned)grid, kSwThreads, st, gate, up, out, gc, a, uc, b, nb,
                          (uint32_t)(cols / 32), ld, in32, out32, codes32);
    return launch_pdl(k_swiglu_forward<__nv_bfloat16>, (unsigned)grid, kSwThreads, st, gate, up, out, gc, a, uc, b, nb,
                      (uint32_t)(cols / 32), ld, in32, out32, codes32);
}

cudaError_t launch_swiglu_backward(const void* grad, int dtype, const void* gc, const void* gs, const void* uc, const void* us,
                                   long long rows, long long cols, void* dgate, void* dup, long long ld, cudaStream_t st) {
    const long long nb = rows * (cols / 32), grid = (nb + kSwThreads - 1) / kSwThreads;
    if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const bool in32 = all32({grad}, 0), out32 = all32({dgate, dup}, ld * (dtype == 0 ? 4 : 2)), codes32 = all32({gc, uc}, 0);
    auto* a = static_cast<const uint8_t*>(gs);
    auto* b = static_cast<const uint8_t*>(us);
    if (dtype == 0)
        return launch_pdl(k_swiglu_backward<float>, (unsigned)grid, kSwThreads, st, grad, gc, a, uc, b, dgate, dup, nb,
                          (uint32_t)(cols / 32), ld, in32, out32, codes32);
    return launch_pdl(k_swiglu_backward<__nv_bfloat16>, (unsigned)grid, kSwThreads, st, grad, gc, a, uc, b, dgate, dup, nb,
                      (uint32_t)(cols / 32), ld, in32, out32, codes32);
}

}  // namespace mxq
