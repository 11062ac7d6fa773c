// mxq_matmul.cu -- product of two microscaled matrices on the block-scaled tensor cores (sm_100a).
//
// "Sonar: Online MXFP6", Current limits: converted weights are operands of block-scaled GEMMs. With a [m, k]
// and b [n, k] in one format,
//   out[i, j] = sum over blocks q of 2^(ea[i, q] + eb[j, q]) * sum over l in q of ca[i, l] * cb[j, l];
// tcgen05.mma takes the codes as they are stored and the E8M0 scales from tensor memory, so nothing is
// decoded: kind::mxf4 multiplies 64 values of k per instruction (two scales per row), kind::mxf8f6f4 32 (one).
//
// One CTA computes tiles of 128 rows of X by BN rows of Y, (X, Y) = (a, b), or (b, a) when a has at most 128
// rows: then the weight fills the instruction's 128 rows and the few tokens its narrow side, and the tile is
// written transposed. Three roles: a producer thread fills a ring of stages (TMA boxes of 128-byte rows with
// the 128-byte swizzle; the scales of 128 rows are whole 512-byte tiles in memory, plain bulk copies), one
// thread copies a stage's scale tiles to tensor memory and issues its four MMAs, four warps bring the fp32
// accumulators from tensor memory to `out`. Where the tiles leave SMs idle, the CTAs of a cluster share a
// tile's k range and add their partial tiles through distributed shared memory in rank order: no workspace, no
// atomics, the same bits on every call.
//
// Every wait on an mbarrier is bounded; after a timeout every role leaves, copies and MMAs in flight are waited
// for (bounded too) and tensor memory is freed.
#include <atomic>
#include <cstdint>
#include <mutex>
#include <cuda.h>  // CUtensorMap and its enums (types only: the encoder is fetched through the runtime)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq_tc.cuh"
#include "mxq_tma.cuh"

namespace mxq {
namespace {

constexpr int kMmThreads = 192;  // producer warp, MMA warp, four epilogue warps
constexpr int kMmRows = 128;     // rows of X per tile
constexpr int kMmSplitMax = 8;   // portable cluster size

// per format: values of k in a staged 128-byte row, values per MMA, 512-byte scale tiles per 128 rows and stage
template <int F> struct MmFmt;
template <> struct MmFmt<F_E2M1> { static constexpr int VALS = 256, KI = 64, TS = 2; };
template <> struct MmFmt<F_E4M3> { static constexpr int VALS = 128, KI = 32, TS = 1; };

template <int F, int BN> struct MmCfg {
    static constexpr int TS = MmFmt<F>::TS;
    static constexpr int NB = (BN + 127) / 128;  // scale tiles along Y's rows
    static constexpr int A_BYTES = kMmRows * 128, B_BYTES = BN * 128;
    static constexpr int SFA = A_BYTES + B_BYTES, SFB = SFA + TS * 512;
    static constexpr int STAGE = (SFB + NB * TS * 512 + 1023) / 1024 * 1024;
    static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 6 : 8;
    static constexpr int SMEM = STAGES * STAGE + 1024;  // + alignment slack
    // tensor memory: BN accumulator columns, then two buffers of scale columns (a stage's copies never write
    // the buffer that the stage before reads)
    static constexpr int SF_COLS = TS * 4 * (1 + NB);
    static constexpr int COLS = BN + 2 * SF_COLS;
    static constexpr int ALLOC = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static_assert(SMEM <= 227 * 1024 && BN * kMmRows * 4 <= STAGES * STAGE, "the stages fit, and the partial tile in them");
};

struct MmArgs {
    const uint8_t* sx;  // scale tiles of X and Y
    const uint8_t* sy;
    void* out;
    int rx, ry;        // rows of X and Y
    int k;             // values of k
    int kt4;           // scale tiles along k
    int tiles, xtiles; // output tiles; xtiles along X (the fast direction)
    int split;         // CTAs (of one cluster) per tile
    long long ld;      // row length of out
};

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_get(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

template <typename T> __device__ __forceinline__ T round_to(float v);
template <> __device__ __forceinline__ float round_to<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 32 bytes (as words) of one output row from column c on, `left` columns of the row remaining
template <typename T>
__device__ __forceinline__ void store_run(T* p, const uint32_t* w, int left, bool a32) {
    constexpr int N = 32 / (int)sizeof(T);
    if (a32 && left >= N) {
        st_v8(p, w);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) {
                if constexpr (sizeof(T) == 4) p[i] = __uint_as_float(w[i]);
                else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
    }
}
// eight words of output from fp32 accumulators: 8 fp32 values or 16 bf16
template <typename T>
__device__ __forceinline__ void pack_run(const float* v, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
        else w[i] = bf16x2(v[2 * i], v[2 * i + 1]);
    }
}

template <int F, int BN, bool SWAP, typename T>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_matmul(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my, const MmArgs p, unsigned int* err) {
    using C = MmCfg<F, BN>;
    using FM = MmFmt<F>;
    constexpr int ST = C::STAGES;
    extern __shared__ uint8_t dsm[];
    uint8_t* const stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) unsigned long long bars[2 * ST + 3];  // full[ST], empty[ST], acc full, acc empty, drained
    __shared__ uint32_t tmem_addr;
    __shared__ int abort_flag;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const uint32_t s0 = smem_u32(stages);
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[ST + s]); };
    const uint32_t acc_full = smem_u32(&bars[2 * ST]), acc_empty = smem_u32(&bars[2 * ST + 1]),
                   drained = smem_u32(&bars[2 * ST + 2]);
    if (t == 0) {
        for (int s = 0; s < 2 * ST; ++s) mbar_init(full(s), 1);
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 4);
        mbar_init(drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc<C::ALLOC>(smem_u32(&tmem_addr));
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t acc = tmem_addr;
    volatile int* ab = &abort_flag;
    // the grids before this one in the stream are complete before anything is read or written
    pdl_wait_then_release();

    const int nks = (p.k + FM::VALS - 1) / FM::VALS;
    const int rank = p.split > 1 ? (int)(blockIdx.x % p.split) : 0;
    const int ks0 = (int)((long long)nks * rank / p.split), ks1 = (int)((long long)nks * (rank + 1) / p.split);
    const int tile0 = blockIdx.x / p.split, tile_step = gridDim.x / p.split;  // split > 1: one tile per cluster

    if (warp == 0) {
        if (lane == 0) {
            long long n = 0;  // stages issued
            bool ok = true;
            for (int tile = tile0; ok && tile < p.tiles; tile += tile_step) {
                const int xt = tile % p.xtiles, yt = tile / p.xtiles;
                for (int ks = ks0; ks < ks1; ++ks, ++n) {
                    const int s = (int)(n % ST);
                    if (n >= ST && !mbar_wait(empty(s), (uint32_t)((n / ST - 1) & 1), ab, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t base = s0 + s * C::STAGE;
                    const int c0 = ks * FM::TS;
                    const uint32_t sf = (uint32_t)min(FM::TS, p.kt4 - c0) * 512u;
                    int nb = (p.ry + 127) / 128 - yt * BN / 128;  // Y's scale tiles that exist
                    nb = nb < C::NB ? nb : C::NB;
                    mbar_expect_tx(full(s), C::A_BYTES + C::B_BYTES + sf * (1 + nb));
                    tma_box(base, &mx, ks * 128, xt * kMmRows, full(s));
                    tma_box(base + C::A_BYTES, &my, ks * 128, yt * BN, full(s));
                    bulk_get(base + C::SFA, p.sx + ((long long)xt * p.kt4 + c0) * 512, sf, full(s));
                    for (int i = 0; i < nb; ++i)
                        bulk_get(base + C::SFB + i * FM::TS * 512, p.sy + ((long long)(yt * BN / 128 + i) * p.kt4 + c0) * 512, sf,
                                 full(s));
                }
            }
            // after a timeout: copies in flight land before shared memory goes away
            if (*ab)
                for (long long q = n > ST ? n - ST : 0; q < n; ++q) {
                    const unsigned long long t0 = global_ns();
                    while (!mbar_test(full((int)(q % ST)), (uint32_t)(q / ST) & 1u) && global_ns() - t0 < kWaitLimitNs) {
                    }
                }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_block_scaled<F>(kMmRows, BN);
            long long n = 0;
            int it = 0;
            bool ok = true;
            for (int tile = tile0; ok && tile < p.tiles; tile += tile_step, ++it) {
                if (it > 0 && !mbar_wait(acc_empty, (uint32_t)(it - 1) & 1u, ab, err)) break;
                tc_fence_after();
                for (int ks = ks0; ks < ks1; ++ks, ++n) {
                    const int s = (int)(n % ST);
                    if (!mbar_wait(full(s), (uint32_t)(n / ST) & 1u, ab, err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t base = s0 + s * C::STAGE;
                    const uint32_t sfa = acc + BN + (uint32_t)(n & 1) * C::SF_COLS, sfb = sfa + FM::TS * 4;
#pragma unroll
                    for (int c = 0; c < FM::TS; ++c) {
                        tc_copy_scales(sfa + 4 * c, desc_scales(base + C::SFA + c * 512));
#pragma unroll
                        for (int i = 0; i < C::NB; ++i)
                            tc_copy_scales(sfb + 4 * (c * C::NB + i), desc_scales(base + C::SFB + (i * FM::TS + c) * 512));
                    }
                    const int left = p.k - ks * FM::VALS;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j * FM::KI < left) {
                            const int c = F == F_E2M1 ? j >> 1 : 0;                          // scale tile
                            const uint32_t id = F == F_E2M1 ? 2u * (j & 1) : (uint32_t)j;    // first byte of its columns
                            tc_mma_block_scaled<F>(acc, desc_sw128(base + 32 * j), desc_sw128(base + C::A_BYTES + 32 * j),
                                                   idesc | (id << 4) | (id << 29), sfa + 4 * c, sfb + 4 * c * C::NB,
                                                   ks > ks0 || j > 0);
                        }
                    tc_commit(empty(s));
                }
                if (ok) tc_commit(acc_full);
            }
            if (*ab) {  // MMAs in flight end before their shared and tensor memory goes away
                tc_commit(drained);
                const unsigned long long t0 = global_ns();
                while (!mbar_test(drained, 0) && global_ns() - t0 < kWaitLimitNs) {
                }
            }
        }
    } else {
        const int quad = warp & 3;  // the warp's lanes of tensor memory
        const uint32_t mine = acc + ((uint32_t)(quad * 32) << 16);
        T* const out = static_cast<T*>(p.out);
        const bool a32 = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.ld * (long long)sizeof(T))) & 31) == 0;
        int it = 0;
        for (int tile = tile0; tile < p.tiles; tile += tile_step, ++it) {
            // lane 0 waits for the warp (bounded); its verdict is the warp's
            bool ok = lane != 0 || mbar_wait(acc_full, (uint32_t)it & 1u, ab, err);
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            tc_fence_after();
            const int xt = tile % p.xtiles, yt = tile / p.xtiles;
            const int x = xt * kMmRows + quad * 32 + lane, y0 = yt * BN;
            if (p.split > 1) {
                // partial tile to shared memory (the stages are consumed), [BN][128]
                float* const red = reinterpret_cast<float*>(stages);
#pragma unroll 1
                for (int c = 0; c < BN; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(mine + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) red[(c + i) * 128 + quad * 32 + lane] = __uint_as_float(v[i]);
                }
                break;
            }
            if constexpr (SWAP) {
#pragma unroll 1
                for (int c = 0; c < BN; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(mine + c, v);
                    tmem_wait_ld();
                    if (x < p.rx)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (y0 + c + i < p.ry) out[(long long)(y0 + c + i) * p.ld + x] = round_to<T>(__uint_as_float(v[i]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty);
            } else if constexpr (sizeof(T) == 2) {
                // 128 columns at a time to registers, rounded; after the last of them the accumulators are free
                // for the next tile's MMAs, before the stores
                T* const row = out + (long long)x * p.ld + y0;
#pragma unroll 1
                for (int h = 0; h < BN; h += 128) {
                    uint32_t w[64];
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(mine + h + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[c / 2 + i] = bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    }
                    if (h + 128 == BN) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acc_empty);
                    }
                    if (x < p.rx)
#pragma unroll
                        for (int c = 0; c < 128; c += 16)
                            if (y0 + h + c < p.ry) store_run<T>(row + h + c, w + c / 2, p.ry - y0 - h - c, a32);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < BN; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(mine + c, v);
                    tmem_wait_ld();
                    if (x < p.rx) {
                        T* const row = out + (long long)x * p.ld + y0 + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            if (y0 + c + i < p.ry) store_run<T>(row + i, v + i, p.ry - y0 - c - i, a32);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty);
            }
        }
    }
    if (p.split > 1) {
        // each CTA adds its share of the columns over the cluster, in rank order
        __syncwarp();
        cluster_sync();
        if (t >= 64) {
            const int r = t - 64, xt = tile0 % p.xtiles, y0 = tile0 / p.xtiles * BN, x = xt * kMmRows + r;
            T* const out = static_cast<T*>(p.out);
            const int per = BN / p.split < 1 ? 1 : BN / p.split;
            const bool a32 = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.ld * (long long)sizeof(T))) & 31) == 0;
            constexpr int RUN = 32 / (int)sizeof(T);
            for (int c = rank * per; c < (rank + 1) * per && c < BN && y0 + c < p.ry; c += SWAP ? 1 : RUN) {
                float v[RUN];
#pragma unroll
                for (int i = 0; i < (SWAP ? 1 : RUN); ++i) {
                    float sum = 0.f;
                    for (int q = 0; q < p.split; ++q) sum += ld_peer_f32(s0 + 4u * (uint32_t)((c + i) * 128 + r), (uint32_t)q);
                    v[i] = sum;
                }
                if (x < p.rx) {
                    if constexpr (SWAP) {
                        out[(long long)(y0 + c) * p.ld + x] = round_to<T>(v[0]);
                    } else {
                        uint32_t w[8];
                        pack_run<T>(v, w);
                        store_run<T>(out + (long long)x * p.ld + y0 + c, w, p.ry - y0 - c, a32);
                    }
                }
            }
        }
        __syncwarp();
        cluster_sync();  // peers have read this CTA's partial tile
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<C::ALLOC>(acc);
    }
}

// tensor map of an operand's codes, [rows, row_bytes]: boxes of box_rows rows x 128 bytes, 128-byte swizzle
bool encode_codes_map(CUtensorMap* m, const void* base, long long rows, long long row_bytes, int box_rows) {
    static PFN_cuTensorMapEncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* q = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &q, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled>(q);
        else
            cudaGetLastError();
    });
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct MmCall {
    const void *xc, *xs, *yc, *ys;  // codes and scales of X and Y
    long long rx, ry, k, ld;
    void* out;
    int dev, sms;
    unsigned int* err;
    cudaStream_t st;
};

template <int F, int BN, bool SWAP, typename T> cudaError_t go(const MmCall& c) {
    using C = MmCfg<F, BN>;
    auto* kern = k_matmul<F, BN, SWAP, T>;
    static std::atomic<unsigned long long> ready{0};  // devices whose shared-memory limit is raised
    const unsigned long long bit = c.dev < 64 ? 1ull << c.dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    const long long row_bytes = F == F_E2M1 ? c.k / 2 : c.k;
    CUtensorMap mx, my;
    if (!encode_codes_map(&mx, c.xc, c.rx, row_bytes, kMmRows) || !encode_codes_map(&my, c.yc, c.ry, row_bytes, BN))
        return cudaErrorUnknown;
    MmArgs a{};
    a.sx = static_cast<const uint8_t*>(c.xs);
    a.sy = static_cast<const uint8_t*>(c.ys);
    a.out = c.out;
    a.rx = (int)c.rx;
    a.ry = (int)c.ry;
    a.k = (int)c.k;
    a.kt4 = (int)((c.k / 32 + 3) / 4);
    const long long xt = (c.rx + kMmRows - 1) / kMmRows, yt = (c.ry + BN - 1) / BN;
    if (xt * yt > 0x7FFFFFFFLL / kMmSplitMax) return cudaErrorInvalidValue;
    a.xtiles = (int)xt;
    a.tiles = (int)(xt * yt);
    a.ld = c.ld;
    // idle SMs take part of a tile's k range, at least two stages each
    const int nks = (int)((c.k + MmFmt<F>::VALS - 1) / MmFmt<F>::VALS);
    a.split = 1;
    if (BN <= 128)
        while (a.split < kMmSplitMax && a.tiles * a.split * 2 <= c.sms && nks >= a.split * 4) a.split *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.split > 1 ? a.tiles * a.split : (a.tiles < c.sms ? a.tiles : c.sms)));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = c.st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.split;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, mx, my, (const MmArgs)a, c.err);
}

template <int F, typename T> cudaError_t pick(MmCall c, const void* ac, const void* as, const void* bc, const void* bs,
                                              long long m, long long n) {
    if (m <= 128) {  // few tokens: the weight's rows on the 128-row side
        c.xc = bc; c.xs = bs; c.rx = n;
        c.yc = ac; c.ys = as; c.ry = m;
        if (m <= 16) return go<F, 16, true, T>(c);
        if (m <= 32) return go<F, 32, true, T>(c);
        if (m <= 64) return go<F, 64, true, T>(c);
        return go<F, 128, true, T>(c);
    }
    c.xc = ac; c.xs = as; c.rx = m;
    c.yc = bc; c.ys = bs; c.ry = n;
    // tiles of 128 x 256 move the fewest operand bytes; narrower ones where those would leave SMs idle
    if (((m + 127) / 128) * ((n + 255) / 256) >= c.sms) return go<F, 256, false, T>(c);
    return go<F, 128, false, T>(c);
}

}  // namespace

cudaError_t launch_matmul(int fmt, const void* ac, const void* as, const void* bc, const void* bs, long long m, long long n,
                          long long k, void* out, int dtype, cudaStream_t st) {
    MmCall c{};
    c.k = k;
    c.ld = n;
    c.out = out;
    c.st = st;
    cudaError_t e = cudaGetDevice(&c.dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, c.dev);
    if (e != cudaSuccess) return e;
    e = device_error_word(&c.err);
    if (e != cudaSuccess) return e;
    if (fmt == F_E2M1)
        return dtype == 0 ? pick<F_E2M1, float>(c, ac, as, bc, bs, m, n) : pick<F_E2M1, __nv_bfloat16>(c, ac, as, bc, bs, m, n);
    return dtype == 0 ? pick<F_E4M3, float>(c, ac, as, bc, bs, m, n) : pick<F_E4M3, __nv_bfloat16>(c, ac, as, bc, bs, m, n);
}

}  // namespace mxq
