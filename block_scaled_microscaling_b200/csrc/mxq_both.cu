// mxq_both.cu -- one matrix quantized along its rows, its columns or both, as operands of the block-scaled
// product (sm_100a).
//
// A linear layer's training step needs each matrix as an operand along one dimension forward and along the
// other backward (blocks of 32 run along the summed dimension: "Sonar: Online MXFP6", Start a model). One CTA
// takes a tile of 128 x 128 values, so that the tile's scales are exactly one 512-byte tile of the MMA scale
// layout in either direction and its payloads are whole 128-byte (E4M3) or 64-byte (E2M1) runs of a row or of a
// column. The values are read once, through shared memory (rows 16 bytes apart from a multiple of the banks:
// 16-byte reads along a row and 4-byte reads across columns are both free of conflicts); a thread encodes two
// blocks of a row, then two of the columns. Rows past the end count as zeros: the column direction fills its
// last block up with them, and the scale tiles are written whole, padding included.
// Bound by memory: E4M3 both ways of bf16 moves 2 + 2 * 33/32 bytes per value; 8192 x 9728 63 us (5.1 TB/s; the
// shared-memory transposition and the long-scoreboard waits of its loads are what is left, DRAM is half busy). Rows
// alone of whole scale tiles and at least 2^20 values take the quantize kernel of the conversions, which needs no
// transposition (16384 x 2560 MXFP4 15 us); rows that are no multiple of 128 stay here (16383 x 2560 MXFP4 20 us).
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxq_block.cuh"
#include "mxq_ops_internal.h"

namespace mxq {
namespace {

constexpr int kBothThreads = 256;
template <typename T> __host__ __device__ constexpr int both_pitch() { return 128 * (int)sizeof(T) + 16; }

struct BothArgs {
    const void* src;
    long long rows, cols;
    int nct;            // column tiles
    int rfmt, cfmt;     // -1: direction left out
    void *rc, *rs, *cc, *cs;
    bool r32, c32;      // codes 32-byte aligned
};

// payload of one block of values (its words); returns the scale byte
template <typename T> __device__ __forceinline__ uint32_t code_block(int fmt, const uint32_t* w, uint32_t* o) {
    const uint32_t amax = block_amax<T>(w);
    if (fmt == F_E2M1) {
        const uint32_t byte = scale_byte<F_E2M1>(amax);
        encode_block<F_E2M1, T>(w, byte, o);
        return byte;
    }
    const uint32_t byte = scale_byte<F_E4M3>(amax);
    encode_block<F_E4M3, T>(w, byte, o);
    return byte;
}
__device__ __forceinline__ void store16(char* p, const uint32_t* o) { st_stream_v4(p, make_uint4(o[0], o[1], o[2], o[3])); }
// a block's payload to its place; whole 32-byte sectors where the array allows (a32)
__device__ __forceinline__ void put_payload(int fmt, void* codes, long long blk, const uint32_t* o, bool a32) {
    if (fmt == F_E2M1) store16(static_cast<char*>(codes) + blk * 16, o);
    else st32(static_cast<char*>(codes) + blk * 32, o, a32);
}

template <typename T> __global__ void __launch_bounds__(kBothThreads) k_quantize_both(const BothArgs p) {
    constexpr int PITCH = both_pitch<T>(), CH = 128 * (int)sizeof(T) / 16;  // 16-byte chunks of a tile row
    extern __shared__ __align__(16) uint8_t tile[];
    __shared__ __align__(16) uint8_t sc[2][512];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    pdl_wait_then_release();
    const long long rt = blockIdx.x / p.nct;
    const int ct = (int)(blockIdx.x - rt * p.nct);
    const long long row0 = rt * 128, col0 = ct * 128LL;
    const int nrows = (int)min(128LL, p.rows - row0), ncols = (int)min(128LL, p.cols - col0);
    reinterpret_cast<uint32_t*>(sc)[t] = 0;
#pragma unroll
    for (int i = t; i < 128 * CH; i += kBothThreads) {
        const int r = i / CH, c = i % CH;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < nrows && c * (16 / (int)sizeof(T)) < ncols)
            v = ld_stream_v4(static_cast<const char*>(p.src) + ((row0 + r) * p.cols + col0) * (long long)sizeof(T) + 16 * c);
        *reinterpret_cast<uint4*>(tile + r * PITCH + 16 * c) = v;
    }
    __syncthreads();
    if (p.rfmt >= 0) {
        const int r = t & 127, k0 = (t >> 7) * 2;
        const long long kb = p.cols / 32;
        uint32_t o[2][8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = k0 + j;
            if (r < nrows && 32 * k < ncols) {
                uint32_t w[Blk<T>::NW];
#pragma unroll
                for (int i = 0; i < Blk<T>::NW / 4; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4*>(tile + r * PITCH + 32 * k * (int)sizeof(T) + 16 * i);
                    w[4 * i] = v.x;
                    w[4 * i + 1] = v.y;
                    w[4 * i + 2] = v.z;
                    w[4 * i + 3] = v.w;
                }
                sc[0][(r & 31) * 16 + (r >> 5) * 4 + k] = (uint8_t)code_block<T>(p.rfmt, w, o[j]);
            }
        }
        const long long blk = (row0 + r) * kb + ct * 4 + k0;
        if (r < nrows && 32 * k0 < ncols) {
            if (p.rfmt == F_E2M1 && p.r32 && (kb & 1) == 0) {  // two neighbouring payloads of 16 bytes (kb even: both exist)
                const uint32_t both[8] = {o[0][0], o[0][1], o[0][2], o[0][3], o[1][0], o[1][1], o[1][2], o[1][3]};
                st_v8(static_cast<char*>(p.rc) + blk * 16, both);
            } else {
                put_payload(p.rfmt, p.rc, blk, o[0], p.r32);
                if (32 * k0 + 32 < ncols) put_payload(p.rfmt, p.rc, blk + 1, o[1], p.r32);
            }
        }
    }
    if (p.cfmt >= 0) {
        const int rb = warp & 3, half = warp >> 2;
        const long long RB = (p.rows + 31) / 32;
        const bool any = 32 * rb < nrows;
        const uint8_t* base = tile + rb * 32 * PITCH;
        if constexpr (sizeof(T) == 2) {  // columns 2 lane, 2 lane + 1 of the half share a word
            uint32_t w[2][16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t a = *reinterpret_cast<const uint32_t*>(base + 2 * i * PITCH + half * 128 + 4 * lane);
                const uint32_t b = *reinterpret_cast<const uint32_t*>(base + (2 * i + 1) * PITCH + half * 128 + 4 * lane);
                w[0][i] = __byte_perm(a, b, 0x5410);
                w[1][i] = __byte_perm(a, b, 0x7632);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = half * 64 + 2 * lane + j;
                if (any && c < ncols) {
                    uint32_t o[8];
                    sc[1][(c & 31) * 16 + (c >> 5) * 4 + rb] = (uint8_t)code_block<T>(p.cfmt, w[j], o);
                    put_payload(p.cfmt, p.cc, (col0 + c) * RB + rt * 4 + rb, o, p.c32);
                }
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
                const int c = half * 64 + 32 * j + lane;
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = *reinterpret_cast<const uint32_t*>(base + i * PITCH + 4 * c);
                if (any && c < ncols) {
                    uint32_t o[8];
                    sc[1][(c & 31) * 16 + (c >> 5) * 4 + rb] = (uint8_t)code_block<T>(p.cfmt, w, o);
                    put_payload(p.cfmt, p.cc, (col0 + c) * RB + rt * 4 + rb, o, p.c32);
                }
            }
        }
    }
    __syncthreads();
    const int q = t & 127;
    if (t < 128) {
        if (p.rfmt >= 0)
            reinterpret_cast<uint32_t*>(p.rs)[(rt * p.nct + ct) * 128 + q] = reinterpret_cast<const uint32_t*>(sc[0])[q];
    } else if (p.cfmt >= 0) {
        const long long nrt = (p.rows + 127) / 128;
        reinterpret_cast<uint32_t*>(p.cs)[(ct * nrt + rt) * 128 + q] = reinterpret_cast<const uint32_t*>(sc[1])[q];
    }
}

template <typename T> cudaError_t go(const BothArgs& a, unsigned grid, cudaStream_t st) {
    constexpr int SMEM = 128 * both_pitch<T>();
    auto* kern = k_quantize_both<T>;
    if (SMEM > 48 * 1024 - 1024) {
        static std::atomic<unsigned long long> ready{0};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
        if (!(ready.load(std::memory_order_acquire) & bit)) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
            if (e != cudaSuccess) return e;
            ready.fetch_or(bit, std::memory_order_release);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kBothThreads);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_quantize_both(int rfmt, int cfmt, const void* src, int dtype, long long rows, long long cols, void* rc,
                                 void* rs, void* cc, void* cs, cudaStream_t st) {
    // rows alone, in whole scale tiles (no padding to write): the row quantize kernel, which needs no shared memory
    // (8192 x 9728 MXFP8 37 us, 8191 rows with this file's kernel 45); small ones keep this kernel's coarser grid
    if (cfmt < 0 && rows % 128 == 0 && cols % 128 == 0 && rows * cols >= (1LL << 20)) {
        SegTable<1> tab{};
        tab.seg[0] = {src, rc, rs, rows * (cols / 32), 0, cols / 32};
        tab.n = 1;
        return launch_quantize<1>(rfmt, dtype, tab, st);
    }
    BothArgs a{src, rows, cols, (int)((cols + 127) / 128), rfmt, cfmt, rc, rs, cc, cs,
               (reinterpret_cast<uintptr_t>(rc) & 31) == 0, (reinterpret_cast<uintptr_t>(cc) & 31) == 0};
    const long long grid = (rows + 127) / 128 * a.nct;
    if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    return dtype == 0 ? go<float>(a, (unsigned)grid, st) : go<__nv_bfloat16>(a, (unsigned)grid, st);
}

}  // namespace mxq
