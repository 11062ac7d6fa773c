// mxq_matmul.cu -- product of two microscaled matrices on the block-scaled tensor cores (sm_100a).
//
// "Sonar: Online MXFP6", Current limits: converted weights are operands of block-scaled GEMMs. With a [m, k]
// and b [n, k] in one format,
//   out[i, j] = sum over blocks q of 2^(ea[i, q] + eb[j, q]) * sum over l in q of ca[i, l] * cb[j, l];
// tcgen05.mma takes the codes as they are stored and the E8M0 scales from tensor memory, so nothing is
// decoded: kind::mxf4 multiplies 64 values of k per instruction (two scales per row), kind::mxf8f6f4 32 (one).
//
// Three roles: a producer warp fills a ring of stages (TMA boxes of 128-byte rows with the 128-byte swizzle; the
// scales of 128 rows are whole 512-byte tiles in memory), a second warp copies a stage's scale tiles to tensor
// memory and issues its four MMAs, eight warps bring the fp32 accumulators from tensor memory to `out`. Both
// issuing warps run converged with one elected thread, on operands that are uniform over the warp: with the whole
// loop under one lane and descriptors built per instruction, issuing took longer than the MMAs (8192 x 9728 x 2560
// MXFP8 177 us, now 153).
// - Large products: a pair of CTAs computes 256 x 256 of out (k_matmul_pair).
// - Others: a CTA computes 128 rows of X by up to 128 rows of Y, (X, Y) = (a, b), or (b, a) when a has at most 128
//   rows: then the weight fills the instruction's 128 rows, the few tokens its narrow side, in steps of 16, and the
//   tile is written transposed. Two CTAs fit an SM. Where the tiles leave SMs idle, the CTAs of a cluster share a
//   tile's k range and add their partial tiles through distributed shared memory in rank order: no workspace, no
//   atomics, the same bits on every call.
//
// Every wait on an mbarrier is bounded; after a timeout every role leaves, copies and MMAs in flight are waited
// for (bounded too) and tensor memory is freed.
#include <atomic>
#include <cstdint>
#include <mutex>
#include <type_traits>
#include <cuda.h>  // CUtensorMap and its enums (types only: the encoder is fetched through the runtime)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "mxq_device.cuh"
#include "mxq_ops_internal.h"
#include "mxq_tc.cuh"
#include "mxq_tma.cuh"

namespace mxq {
namespace {

constexpr int kMmThreads = 320;  // producer warp, MMA warp, eight epilogue warps
constexpr int kMmRows = 128;     // rows of X per tile
constexpr int kMmSplitMax = 8;   // portable cluster size

// output of rows that are not aligned: 32 rows of two 32-byte pieces for each epilogue warp, 17 words apart
constexpr int kMmPitch = 17, kMmStaging = 8 * 32 * kMmPitch * 4;
// per format: values of k in a staged 128-byte row, values per MMA, 512-byte scale tiles per 128 rows and stage
template <int F> struct MmFmt;
template <> struct MmFmt<F_E2M1> { static constexpr int VALS = 256, KI = 64, TS = 2; };
template <> struct MmFmt<F_E4M3> { static constexpr int VALS = 128, KI = 32, TS = 1; };

// a tile of 128 x bn, bn <= 128 and a multiple of 16
template <int F> struct MmCfg {
    static constexpr int TS = MmFmt<F>::TS;
    static constexpr int A_BYTES = kMmRows * 128;
    static constexpr int SF_BYTES = 2 * TS * 512;  // X's scale tiles, then Y's
    static constexpr int MAX_STAGES = 8;
    __host__ __device__ static constexpr int stage_bytes(int bn) { return A_BYTES + bn * 128 + (SF_BYTES + 1023) / 1024 * 1024; }
    // as many stages as fit the SM, or half of it
    static constexpr int stages(int bn, bool two, bool staged) {
        const int n = ((two ? 112 : 224) * 1024 - 1024 - (staged ? kMmStaging : 0)) / stage_bytes(bn);
        return n < MAX_STAGES ? n : MAX_STAGES;
    }
    // the ring; a partial tile takes its place
    __host__ __device__ static constexpr int ring_bytes(int bn, int stages) {
        const int ring = stages * stage_bytes(bn), part = bn * kMmRows * 4;
        return ring > part ? ring : part;
    }
    static int smem(int bn, int stages, bool staged) {
        return ring_bytes(bn, stages) + (staged ? kMmStaging : 0) + 1024;  // + alignment slack
    }
    // tensor memory: 128 accumulator columns, then two buffers of scale columns (a stage's copies never write the
    // buffer that the stage before reads)
    static constexpr int SF_COLS = TS * 4 * 2;
    static constexpr int ALLOC = 256;
    static_assert(128 + 2 * SF_COLS <= ALLOC && stages(128, true, false) >= 3, "tensor memory of two CTAs, a ring of three stages");
};

// position in a ring of n stages: stage and the parity of its current use (counters, since one thread's divisions
// by a stage count that is no power of two took longer than a stage's MMAs)
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) {
            s = 0;
            phase ^= 1u;
        }
    }
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
    int bn, stages;    // rows of Y per tile, stages of the ring
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

// rows of out begin on 32 bytes
template <typename T> __host__ __device__ __forceinline__ bool rows_aligned(const void* out, long long ld) {
    return ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(ld * (long long)sizeof(T))) & 31) == 0;
}
// 32 bytes (as words) of one output row from column c on, `left` columns of the row remaining
template <typename T>
__device__ __forceinline__ void store_run(T* p, const uint32_t* w, int left) {
    constexpr int N = 32 / (int)sizeof(T);
    if (left >= N) {
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

// Rows that do not start on 32 bytes (row lengths that are not a multiple of 16 bf16 or 8 fp32 values): the warp's 32 rows
// go through shared memory, 32 bytes at a time, and two lanes write a row from one whole 32-byte sector of the output to
// the next, wherever in the row it starts; the ring of two pieces holds what such a sector can reach. With one lane per
// row, value by value, 16384 x 9725 x 2560 (MXFP4) took 1615 us, with words of pieces that straddle sectors 510, with
// whole sectors word by word 354, and so 227 (n = 9720 180, n = 9728, stored from registers, 164).
template <typename T, int N>
__device__ __forceinline__ void store_staged(const uint32_t* w, uint32_t* stage, T* out, long long ld, int x0, int rx, int y0, int ry) {
    const int lane = threadIdx.x & 31;
    constexpr int P = 32 / (int)sizeof(T), H = P / 2;  // values in a piece, in a lane's half of a sector
    const int lim = ry - y0 < N ? ry - y0 : N;
    using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
#pragma unroll
    for (int j = 0; j <= N / P; ++j) {
        if ((j - 1) * P >= lim) break;  // the same for the warp: no row's window j holds a value
        if (j < N / P)
#pragma unroll
            for (int i = 0; i < 8; ++i) stage[lane * kMmPitch + (j & 1) * 8 + i] = w[j * 8 + i];
        __syncwarp();
#pragma unroll
        for (int r = lane >> 1; r < 32; r += 16) {
            if (x0 + r >= rx) continue;
            Bits* const row = reinterpret_cast<Bits*>(out + (long long)(x0 + r) * ld + y0);
            const int skew = (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & (P - 1);
            const int c = j * P - skew + H * (lane & 1);  // the lane's first value; all lie in pieces j - 1 and j
            const uint32_t* const from = stage + r * kMmPitch;
            uint32_t v[5];
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = from[(c + i) & 15];
            } else {
#pragma unroll
                for (int i = 0; i < 5; ++i) v[i] = from[((c >> 1) + i) & 15];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(v[i], v[i + 1], 16 * (c & 1));
            }
            if (c >= 0 && c + H <= lim) {
                *reinterpret_cast<uint4*>(row + c) = make_uint4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i)
                    if (c + i >= 0 && c + i < lim) row[c + i] = (Bits)(sizeof(T) == 4 ? v[i & 3] : v[i >> 1] >> (16 * (i & 1)));
            }
        }
        __syncwarp();
    }
}

// N accumulator columns of the warp's 32 rows (tensor-memory address `mine`) to rows x0 .. of out, columns y0 ..; calls
// `release` once all of them are in registers (bf16: rounded), before the first store
template <typename T, int N, typename R>
__device__ __forceinline__ void store_rows(uint32_t mine, uint32_t* stage, T* out, long long ld, int x0, int rx, int y0, int ry,
                                           bool a32, R release) {
    constexpr int PER = 32 / (int)sizeof(T);  // columns in 32 bytes
    uint32_t w[N * (int)sizeof(T) / 4];
#pragma unroll
    for (int c = 0; c < N; c += 32) {
        if constexpr (sizeof(T) == 4) {
            tmem_ld32(mine + c, w + c);
        } else {
            uint32_t v[32];
            tmem_ld32(mine + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) w[c / 2 + i] = bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        }
    }
    if constexpr (sizeof(T) == 4) tmem_wait_ld();
    release();
    if (!a32) {
        store_staged<T, N>(w, stage, out, ld, x0, rx, y0, ry);
        return;
    }
    const int x = x0 + (threadIdx.x & 31);
    T* const row = out + (long long)x * ld + y0;
    if (x < rx)
#pragma unroll
        for (int c = 0; c < N; c += PER)
            if (y0 + c < ry) store_run<T>(row + c, w + c / PER * 8, ry - y0 - c);
}

// the partial tiles [bn][128] of S CTAs, at `part` in each, added in rank order: this CTA's share of the columns to
// out. 256 threads: in the transposed form (rows of out are columns of the tile) four rows of a column each, 16 bytes
// from every CTA; else row e % 128, a run of columns in two halves
template <int S, bool SWAP, typename T>
__device__ __forceinline__ void add_parts(uint32_t part, int e, int rank, int bn, int x, int y0, const MmArgs& p, T* out, uint32_t* stage,
                                          bool a32) {
    const int per = bn / S;  // bn is a multiple of 16, S at most 8
    if constexpr (SWAP) {
        const int r = 4 * (e & 31);
        if (x + r >= p.rx) return;
        const bool whole = a32 && x + r + 4 <= p.rx;
#pragma unroll 2
        for (int c = rank * per + (e >> 5); c < (rank + 1) * per && y0 + c < p.ry; c += 8) {
            float4 v[S];
#pragma unroll
            for (int q = 0; q < S; ++q) v[q] = ld_peer_f32x4(part + 4u * (uint32_t)(c * 128 + r), (uint32_t)q);
#pragma unroll
            for (int q = 1; q < S; ++q) {
                v[0].x += v[q].x;
                v[0].y += v[q].y;
                v[0].z += v[q].z;
                v[0].w += v[q].w;
            }
            T* const to = out + (long long)(y0 + c) * p.ld + x + r;
            if (whole) {
                if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(to) = v[0];
                else *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2(v[0].x, v[0].y), bf16x2(v[0].z, v[0].w));
            } else {
                const float f[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (x + r + i < p.rx) to[i] = round_to<T>(f[i]);
            }
        }
    } else {
        constexpr int RUN = 32 / (int)sizeof(T);  // columns at a time
        const int r = e & 127;
        for (int c = rank * per + (e >> 7) * RUN; c < (rank + 1) * per && y0 + c < p.ry; c += 2 * RUN) {
            float v[RUN][S], sum[RUN];
#pragma unroll
            for (int i = 0; i < RUN; ++i)
#pragma unroll
                for (int q = 0; q < S; ++q) v[i][q] = ld_peer_f32(part + 4u * (uint32_t)((c + i) * 128 + r), (uint32_t)q);
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                sum[i] = v[i][0];
#pragma unroll
                for (int q = 1; q < S; ++q) sum[i] += v[i][q];
            }
            uint32_t w[8];
            pack_run<T>(sum, w);
            if (!a32) store_staged<T, RUN>(w, stage, out, p.ld, x + (r & ~31), p.rx, y0 + c, p.ry);
            else if (x + r < p.rx) store_run<T>(out + (long long)(x + r) * p.ld + y0 + c, w, p.ry - y0 - c);
        }
    }
}

template <int F, bool SWAP, typename T>
__global__ void __launch_bounds__(kMmThreads, 2)
    k_matmul(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my, const MmArgs p, unsigned int* err) {
    using C = MmCfg<F>;
    using FM = MmFmt<F>;
    constexpr int MS = C::MAX_STAGES;
    const int bn = SWAP ? p.bn : 128, ST = p.stages, STAGE = C::stage_bytes(bn);
    const uint32_t sf_at = C::A_BYTES + bn * 128;  // X's scale tiles in a stage
    extern __shared__ uint8_t dsm[];
    uint8_t* const stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) unsigned long long bars[2 * MS + 3];  // full[MS], empty[MS], acc full, acc empty, drained
    __shared__ uint32_t tmem_addr;
    __shared__ int abort_flag;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const uint32_t s0 = smem_u32(stages);
    T* const out = static_cast<T*>(p.out);
    const bool a32 = rows_aligned<T>(out, p.ld);
    // an epilogue warp's staging; only there if !SWAP && !a32
    uint32_t* const stage = reinterpret_cast<uint32_t*>(stages + C::ring_bytes(bn, ST)) + (warp - 2) * 32 * kMmPitch;
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[MS + s]); };
    const uint32_t acc_full = smem_u32(&bars[2 * MS]), acc_empty = smem_u32(&bars[2 * MS + 1]),
                   drained = smem_u32(&bars[2 * MS + 2]);
    if (t == 0) {
        for (int s = 0; s < 2 * MS; ++s) mbar_init(full(s), 1);
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 8);
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
        const bool one = elect_one();
        Ring at;
        long long n = 0;  // stages issued
        bool ok = true;
        for (int tile = tile0; ok && tile < p.tiles; tile += tile_step) {
            const int xt = tile % p.xtiles, yt = tile / p.xtiles;
            const uint8_t* const sx = p.sx + (long long)xt * p.kt4 * 512;
            const uint8_t* const sy = p.sy + (long long)yt * p.kt4 * 512;  // bn < 128: one tile of Y
            for (int ks = ks0; ks < ks1; ++ks, ++n, at.next(ST)) {
                if (n >= ST && !mbar_wait(empty(at.s), at.phase ^ 1u, ab, err)) {
                    ok = false;
                    break;
                }
                if (!one) continue;
                const uint32_t base = s0 + at.s * STAGE, bar = full(at.s);
                const int c0 = ks * FM::TS;
                const uint32_t sf = (uint32_t)min(FM::TS, p.kt4 - c0) * 512u;
                mbar_expect_tx(bar, C::A_BYTES + bn * 128 + 2 * sf);
                tma_box(base, &mx, ks * 128, xt * kMmRows, bar);
                tma_box(base + C::A_BYTES, &my, ks * 128, yt * bn, bar);
                bulk_get(base + sf_at, sx + (long long)c0 * 512, sf, bar);
                bulk_get(base + sf_at + FM::TS * 512, sy + (long long)c0 * 512, sf, bar);
            }
        }
        // after a timeout: copies in flight land before shared memory goes away
        if (one && *ab)
            for (long long q = n > ST ? n - ST : 0; q < n; ++q) {
                const unsigned long long t0 = global_ns();
                while (!mbar_test(full((int)(q % ST)), (uint32_t)(q / ST) & 1u) && global_ns() - t0 < kWaitLimitNs) {
                }
            }
    } else if (warp == 1) {
        const bool one = elect_one();
        const uint32_t idesc = idesc_block_scaled<F>(kMmRows, bn);
        const SmemDesc dop = desc_sw128(s0), dsf = desc_scales(s0);
        Ring at;
        uint32_t odd = 0;
        int it = 0;
        bool ok = true;
        for (int tile = tile0; ok && tile < p.tiles; tile += tile_step, ++it) {
            if (it > 0 && !mbar_wait(acc_empty, (uint32_t)(it - 1) & 1u, ab, err)) break;
            tc_fence_after();
            for (int ks = ks0; ks < ks1; ++ks, at.next(ST), odd ^= 1u) {
                if (!mbar_wait(full(at.s), at.phase, ab, err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!one) continue;
                const uint32_t step = at.s * STAGE;
                const uint32_t sfa = acc + 128 + odd * C::SF_COLS, sfb = sfa + FM::TS * 4;
#pragma unroll
                for (int c = 0; c < FM::TS; ++c) {
                    tc_copy_scales(sfa + 4 * c, dsf + (step + sf_at + c * 512));
                    tc_copy_scales(sfb + 4 * c, dsf + (step + sf_at + (FM::TS + c) * 512));
                }
                const int left = p.k - ks * FM::VALS;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j * FM::KI < left) {
                        const int c = F == F_E2M1 ? j >> 1 : 0;                        // scale tile
                        const uint32_t id = F == F_E2M1 ? 2u * (j & 1) : (uint32_t)j;  // first byte of its columns
                        tc_mma_block_scaled<F>(acc, dop + (step + 32 * j), dop + (step + C::A_BYTES + 32 * j),
                                               idesc | (id << 4) | (id << 29), sfa + 4 * c, sfb + 4 * c, ks > ks0 || j > 0);
                    }
                tc_commit(empty(at.s));
            }
            if (ok && one) tc_commit(acc_full);
        }
        if (one && *ab) {  // MMAs in flight end before their shared and tensor memory goes away
            tc_commit(drained);
            const unsigned long long t0 = global_ns();
            while (!mbar_test(drained, 0) && global_ns() - t0 < kWaitLimitNs) {
            }
        }
    } else {
        const int quad = warp & 3, half = (warp - 2) >> 2;  // the warp's lanes of tensor memory, its part of the columns
        const uint32_t mine = acc + ((uint32_t)(quad * 32) << 16);
        int it = 0;
        for (int tile = tile0; tile < p.tiles; tile += tile_step, ++it) {
            // lane 0 waits for the warp (bounded); its verdict is the warp's
            bool ok = lane != 0 || mbar_wait(acc_full, (uint32_t)it & 1u, ab, err);
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            tc_fence_after();
            const int xt = tile % p.xtiles, yt = tile / p.xtiles;
            const int x = xt * kMmRows + quad * 32 + lane, y0 = yt * bn;
            if (p.split > 1) {
                // partial tile to shared memory (the stages are consumed), [bn][128]
                float* const red = reinterpret_cast<float*>(stages);
#pragma unroll 1
                for (int c = 16 * half; c < bn; c += 32) {
                    uint32_t v[16];
                    tmem_ld16(mine + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) red[(c + i) * 128 + quad * 32 + lane] = __uint_as_float(v[i]);
                }
                break;
            }
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty);
            };
            if constexpr (SWAP) {
#pragma unroll 1
                for (int c = 16 * half; c < bn; c += 32) {
                    uint32_t v[16];
                    tmem_ld16(mine + c, v);
                    tmem_wait_ld();
                    if (x < p.rx)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (y0 + c + i < p.ry) out[(long long)(y0 + c + i) * p.ld + x] = round_to<T>(__uint_as_float(v[i]));
                }
                release();
            } else {
                store_rows<T, 64>(mine + half * 64, stage, out, p.ld, x - lane, p.rx, y0 + half * 64, p.ry, a32, release);
            }
        }
    }
    if (p.split > 1) {
        __syncwarp();
        cluster_sync();
        if (t >= 64) {
            const int e = t - 64, x = tile0 % p.xtiles * kMmRows, y0 = tile0 / p.xtiles * bn;
            if (p.split == 2) add_parts<2, SWAP, T>(s0, e, rank, bn, x, y0, p, out, stage, a32);
            else if (p.split == 4) add_parts<4, SWAP, T>(s0, e, rank, bn, x, y0, p, out, stage, a32);
            else add_parts<8, SWAP, T>(s0, e, rank, bn, x, y0, p, out, stage, a32);
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

// ---- two CTAs on one tile ---------------------------------------------------------------------
//
// The CTAs of a pair compute 256 x 256 of out: each stages 128 rows of a and 128 of b, the tensor cores of both
// read b's rows from both, and each keeps the 128 x 256 accumulators of its rows. A stage moves 32 KB of codes
// into an SM for the same MMAs that take 48 KB in a tile of 128 x 256; an SM takes about 60 bytes a cycle from L2,
// so that transfer (0.30 us a stage) and the MMAs (0.27 us) are level. The leader (rank 0) issues the MMAs and owns
// the barriers that count the stages' bytes; its commits arrive in both CTAs. Eight epilogue warps, so that a tile's
// accumulators leave tensor memory in one go and the next tile's MMAs start before the stores (four warps: 159 us,
// eight: 153 at 8192 x 9728 x 2560 MXFP8).
// Measured, values N(0, 1): 8192 x 9728 x 2560 MXFP8 150 us (2.7 PFLOP/s; one CTA per tile of 128 x 256 163 us),
// 16384 x 9728 x 2560 MXFP4 165 us (4.9 PFLOP/s; 180 us). The board's power limit bounds them: with all codes zero
// the same launches take 126 us, and k = 9728 reaches 3.8 (MXFP8) and 7.3 (MXFP4) PFLOP/s.
template <int F> struct PairCfg {
    static constexpr int TS = MmFmt<F>::TS;
    static constexpr int HALF = 128 * 128;  // bytes of 128 staged rows
    static constexpr int SFA = 2 * HALF, SFB = SFA + TS * 512, BYTES = SFB + 2 * TS * 512;
    static constexpr int STAGE = (BYTES + 1023) / 1024 * 1024;
    static constexpr int MAX_STAGES = 6;
    static constexpr int stages(bool staged) { return MAX_STAGES - (staged && MAX_STAGES * STAGE + kMmStaging > 226 * 1024 - 512); }
    static constexpr int smem(bool staged) { return stages(staged) * STAGE + (staged ? kMmStaging : 0) + 1024; }
    static constexpr int SF_COLS = TS * 4 * 3;  // a's scales of the CTA's 128 rows, b's of 256
    static_assert(smem(false) <= 227 * 1024 - 512 && smem(true) <= 227 * 1024 - 512 && 256 + 2 * SF_COLS <= 512, "shared and tensor memory");
};

// 2-D / 3-D boxes into this CTA, their bytes counted on a barrier of the pair (a cluster address)
__device__ __forceinline__ void pair_box2(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void pair_box3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

template <int F, typename T>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_matmul_pair(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                  const __grid_constant__ CUtensorMap msa, const __grid_constant__ CUtensorMap msb, const MmArgs p,
                  unsigned int* err) {
    using C = PairCfg<F>;
    using FM = MmFmt<F>;
    constexpr int MS = C::MAX_STAGES;
    const int ST = p.stages;
    extern __shared__ uint8_t dsm[];
    uint8_t* const stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) unsigned long long bars[2 * MS + 3];  // full[MS], empty[MS], acc full, acc empty, drained
    __shared__ uint32_t tmem_addr;
    __shared__ int abort_flag;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const uint32_t rank = cluster_rank(), s0 = smem_u32(stages);
    auto full = [&](int s) { return smem_u32(&bars[s]); };          // the leader's counts both CTAs' bytes
    auto empty = [&](int s) { return smem_u32(&bars[MS + s]); };
    const uint32_t acc_full = smem_u32(&bars[2 * MS]), acc_empty = smem_u32(&bars[2 * MS + 1]),
                   drained = smem_u32(&bars[2 * MS + 2]);
    if (t == 0) {
        for (int s = 0; s < 2 * MS; ++s) mbar_init(full(s), 1);
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 16);  // the epilogue warps of both CTAs
        mbar_init(drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tmem_alloc<512, true>(smem_u32(&tmem_addr));
        tc_fence_before();
    }
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    const uint32_t acc = tmem_addr;
    volatile int* ab = &abort_flag;
    pdl_wait_then_release();

    const int nks = (p.k + FM::VALS - 1) / FM::VALS;
    const int tile0 = blockIdx.x >> 1, tile_step = gridDim.x >> 1;

    if (warp == 0) {
        {
            const bool one = elect_one();
            Ring at;
            long long n = 0;  // stages issued
            bool ok = true;
            const uint32_t full0 = peer_addr(full(0), 0);
            for (int tile = tile0; ok && tile < p.tiles; tile += tile_step) {
                const int xt = tile % p.xtiles, yt = tile / p.xtiles;
                for (int ks = 0; ks < nks; ++ks, ++n, at.next(ST)) {
                    const int s = at.s;
                    if (n >= ST && !mbar_wait<true>(empty(s), at.phase ^ 1u, ab, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t base = s0 + s * C::STAGE, bar = full0 + 8u * (uint32_t)s;
                    if (!one) continue;
                    if (rank == 0) mbar_expect_tx(full(s), 2 * C::BYTES);
                    pair_box2(base, &ma, ks * 128, xt * 256 + (int)rank * 128, bar);
                    pair_box2(base + C::HALF, &mb, ks * 128, yt * 256 + (int)rank * 128, bar);
                    pair_box3(base + C::SFA, &msa, 0, ks * FM::TS, xt * 2 + (int)rank, bar);
                    pair_box3(base + C::SFB, &msb, 0, ks * FM::TS, yt * 2, bar);
                }
            }
            if (one && *ab) {  // after a timeout: copies in flight land before shared memory goes away
                const unsigned long long t0 = global_ns();
                if (rank == 0)
                    for (long long q = n > ST ? n - ST : 0; q < n; ++q)
                        while (!mbar_test(full((int)(q % ST)), (uint32_t)(q / ST) & 1u) && global_ns() - t0 < kWaitLimitNs) {
                        }
                else  // their bytes are counted in the leader: give them time
                    while (global_ns() - t0 < kWaitLimitNs / 100) {
                    }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const bool one = elect_one();
            constexpr uint32_t idesc = idesc_block_scaled<F>(256, 256);
            Ring at;
            const SmemDesc dop = desc_sw128(s0), dsf = desc_scales(s0);
            uint32_t odd = 0;
            int it = 0;
            bool ok = true;
            for (int tile = tile0; ok && tile < p.tiles; tile += tile_step, ++it) {
                if (it > 0 && !mbar_wait<true>(acc_empty, (uint32_t)(it - 1) & 1u, ab, err)) break;
                tc_fence_after();
                for (int ks = 0; ks < nks; ++ks, at.next(ST), odd ^= 1u) {
                    const int s = at.s;
                    if (!mbar_wait<true>(full(s), at.phase, ab, err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (!one) continue;
                    const uint32_t step = s * C::STAGE;
                    const uint32_t sfa = acc + 256 + odd * C::SF_COLS, sfb = sfa + FM::TS * 4;
#pragma unroll
                    for (int c = 0; c < FM::TS; ++c) {
                        tc_copy_scales<true>(sfa + 4 * c, dsf + (step + C::SFA + c * 512));
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            tc_copy_scales<true>(sfb + 4 * (c * 2 + i), dsf + (step + C::SFB + (i * FM::TS + c) * 512));
                    }
                    const int left = p.k - ks * FM::VALS;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j * FM::KI < left) {
                            const int c = F == F_E2M1 ? j >> 1 : 0;
                            const uint32_t id = F == F_E2M1 ? 2u * (j & 1) : (uint32_t)j;
                            tc_mma_block_scaled<F, true>(acc, dop + (step + 32 * j), dop + (step + C::HALF + 32 * j),
                                                         idesc | (id << 4) | (id << 29), sfa + 4 * c, sfb + 8 * c, ks > 0 || j > 0);
                        }
                    tc_commit<true>(empty(s));
                }
                if (ok && one) tc_commit<true>(acc_full);
            }
            if (one && *ab) {  // MMAs in flight end before their shared and tensor memory goes away
                tc_commit<true>(drained);
                const unsigned long long t0 = global_ns();
                while (!mbar_test(drained, 0) && global_ns() - t0 < kWaitLimitNs) {
                }
            }
        }
    } else {
        const int quad = warp & 3, half = (warp - 2) >> 2;
        uint32_t* const stage = reinterpret_cast<uint32_t*>(stages + ST * C::STAGE) + (warp - 2) * 32 * kMmPitch;
        const uint32_t mine = acc + ((uint32_t)(quad * 32) << 16), leader_empty = peer_addr(acc_empty, 0);
        T* const out = static_cast<T*>(p.out);
        const bool a32 = rows_aligned<T>(p.out, p.ld);
        int it = 0;
        for (int tile = tile0; tile < p.tiles; tile += tile_step, ++it) {
            bool ok = lane != 0 || mbar_wait<true>(acc_full, (uint32_t)it & 1u, ab, err);
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            tc_fence_after();
            const int xt = tile % p.xtiles, yt = tile / p.xtiles;
            const int x0 = xt * 256 + (int)rank * 128 + quad * 32, y0 = yt * 256 + half * 128;
            store_rows<T, 128>(mine + half * 128, stage, out, p.ld, x0, p.rx, y0, p.ry, a32, [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(leader_empty);
            });
        }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // neither CTA is signalled or read by the other any more
    if (warp == 1) {
        tc_fence_after();
        tmem_free<512, true>(acc);
    }
}

// the driver's tensor-map encoder, fetched once through the runtime (null if it cannot be had)
PFN_cuTensorMapEncodeTiled map_encoder() {
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
    return fn;
}
// tensor map of an operand's codes, [rows, row_bytes]: boxes of box_rows rows x 128 bytes, 128-byte swizzle
bool encode_codes_map(CUtensorMap* m, const void* base, long long rows, long long row_bytes, int box_rows) {
    const PFN_cuTensorMapEncodeTiled fn = map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// tensor map of an operand's scale tiles, [tile rows, kt4, 128 words]: boxes of tile_rows x ts tiles
bool encode_scales_map(CUtensorMap* m, const void* base, long long rows, long long kt4, int ts, int tile_rows) {
    const PFN_cuTensorMapEncodeTiled fn = map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {128, (cuuint64_t)kt4, (cuuint64_t)((rows + 127) / 128)};
    const cuuint64_t strides[2] = {512, (cuuint64_t)kt4 * 512};
    const cuuint32_t box[3] = {128, (cuuint32_t)ts, (cuuint32_t)tile_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

// raise a kernel's shared-memory limit, once per device (`ready`: the kernel's devices done)
template <typename K> cudaError_t allow_smem(K* kern, int bytes, int dev, std::atomic<unsigned long long>& ready) {
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
    return e;
}

template <int F, typename T> cudaError_t go_pair(const MmCall& c) {
    using C = PairCfg<F>;
    auto* kern = k_matmul_pair<F, T>;
    static std::atomic<unsigned long long> ready{0};
    const cudaError_t e = allow_smem(kern, C::smem(false) > C::smem(true) ? C::smem(false) : C::smem(true), c.dev, ready);
    if (e != cudaSuccess) return e;
    const long long row_bytes = F == F_E2M1 ? c.k / 2 : c.k;
    MmArgs a{};
    a.out = c.out;
    a.rx = (int)c.rx;
    a.ry = (int)c.ry;
    a.k = (int)c.k;
    a.kt4 = (int)((c.k / 32 + 3) / 4);
    const long long xt = (c.rx + 255) / 256, yt = (c.ry + 255) / 256;
    if (xt * yt > 0x3FFFFFFFLL) return cudaErrorInvalidValue;
    a.xtiles = (int)xt;
    a.tiles = (int)(xt * yt);
    a.split = 1;
    a.ld = c.ld;
    const bool staged = !rows_aligned<T>(c.out, c.ld);
    a.stages = C::stages(staged);
    CUtensorMap ma, mb, msa, msb;
    if (!encode_codes_map(&ma, c.xc, c.rx, row_bytes, 128) || !encode_codes_map(&mb, c.yc, c.ry, row_bytes, 128) ||
        !encode_scales_map(&msa, c.xs, c.rx, a.kt4, C::TS, 1) || !encode_scales_map(&msb, c.ys, c.ry, a.kt4, C::TS, 2))
        return cudaErrorUnknown;
    cudaLaunchConfig_t cfg = {};
    const int pairs = c.sms / 2;
    cfg.gridDim = dim3((unsigned)(2 * (a.tiles < pairs ? a.tiles : pairs)));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = C::smem(staged);
    cfg.stream = c.st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, ma, mb, msa, msb, (const MmArgs)a, c.err);
}

template <int F, bool SWAP, typename T> cudaError_t go(const MmCall& c, int bn) {
    using C = MmCfg<F>;
    auto* kern = k_matmul<F, SWAP, T>;
    static std::atomic<unsigned long long> ready{0};
    const cudaError_t e = allow_smem(kern, 225 * 1024, c.dev, ready);
    if (e != cudaSuccess) return e;
    const long long row_bytes = F == F_E2M1 ? c.k / 2 : c.k;
    CUtensorMap mx, my;
    if (!encode_codes_map(&mx, c.xc, c.rx, row_bytes, kMmRows) || !encode_codes_map(&my, c.yc, c.ry, row_bytes, bn))
        return cudaErrorUnknown;
    MmArgs a{};
    a.sx = static_cast<const uint8_t*>(c.xs);
    a.sy = static_cast<const uint8_t*>(c.ys);
    a.out = c.out;
    a.rx = (int)c.rx;
    a.ry = (int)c.ry;
    a.k = (int)c.k;
    a.kt4 = (int)((c.k / 32 + 3) / 4);
    const long long xt = (c.rx + kMmRows - 1) / kMmRows, yt = (c.ry + bn - 1) / bn;
    if (xt * yt > 0x7FFFFFFFLL / kMmSplitMax) return cudaErrorInvalidValue;
    a.xtiles = (int)xt;
    a.tiles = (int)(xt * yt);
    a.ld = c.ld;
    a.bn = bn;
    // Idle SMs take part of a tile's k range, at least two stages each. One CTA per SM with the whole ring is faster than
    // two with half each (MXFP8 77 x 9728 x 2560 10.7 us against 12.4, 333 x 1024 x 2560 7.8 against 11.0), except where
    // more tiles than SMs would take a second wave of several stages (2048 x 2048 x 2048 12.9 against 11.3; with three
    // stages, 1024 x 2560 x 352, 5.6 against 6.1).
    const int nks = (int)((c.k + MmFmt<F>::VALS - 1) / MmFmt<F>::VALS);
    const bool staged = !SWAP && !rows_aligned<T>(c.out, c.ld);
    const bool two = !staged && a.tiles > c.sms && nks > 4;  // two rings and their staging would have two stages each
    a.split = 1;
    while (!two && a.split < kMmSplitMax && a.tiles * a.split * 2 <= c.sms && nks >= a.split * 4) a.split *= 2;
    a.stages = C::stages(bn, two, staged);
    const int places = two ? 2 * c.sms : c.sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.split > 1 ? a.tiles * a.split : (a.tiles < places ? a.tiles : places)));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = C::smem(bn, a.stages, staged);
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
        return go<F, true, T>(c, (int)((m + 15) / 16 * 16));
    }
    c.xc = ac; c.xs = as; c.rx = m;
    c.yc = bc; c.ys = bs; c.ry = n;
    // 256 x 256 per pair of SMs moves the fewest operand bytes, if that gives every pair a tile (MXFP8, pairs against single
    // CTAs: 2048 x 2560 x 2560, 80 tiles and so a second wave of six, 18.4 us and 18.7; 100 tiles 19.2 and 22.0, 1000 x 9728
    // x 2560 26.5 and 28.8, 8192 x 9728 x 2560 154 and 188; 64 tiles, 2048 x 2048 x 2048, 10.5 and 11.4)
    if (((m + 255) / 256) * ((n + 255) / 256) >= c.sms / 2) return go_pair<F, T>(c);
    return go<F, false, T>(c, 128);
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

