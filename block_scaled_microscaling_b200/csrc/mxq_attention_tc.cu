// mxq_attention_tc.cu -- attention over the paged MXFP4 cache for many queries, on the 5th-generation tensor cores
// (sm_100a).
//
// A CTA takes two tiles of 128 rows (query x head of one key head's group) and walks blocks of 128 keys:
//   S = Q K^T (fp32 in tensor memory),  P = 2^(S - m) (f16, over S),  O += P V (fp32, tensor memory),
// with the formulas, the masks and the roundings of mxq_attention.cu. Block scales are relative to the largest K of a block of
// keys (blocks 2^28 below it are 0) and to the largest V so far (0 from 2^24 to 2^28 below it on). Decoding 128 keys then serves 256
// rows, not 32 as in a warp's registers there. Roles:
// - two warps bring the blocks' codes to a ring in shared memory (16-byte asynchronous copies), one finds their largest
//   scales.
// - four decoding warps turn the codes into f16 operands in the 128-byte swizzle: K as [key][dimension], V transposed,
//   [dimension][key], by interleaving the nibbles of two keys before the conversion, so that both products have the
//   summed index contiguous. The places of the raw codes are permuted so that these reads, like the 16-byte writes,
//   touch every bank once. K is a block ahead of V.
// - four softmax warps per tile, a row per thread: its 128 scores come from tensor memory, the weights go back as the A
//   operand of the second product. The maximum is raised (and O rescaled, in tensor memory) only when a score exceeds
//   it by 2^8, or when a value block exceeds 2^13 of the reference scale.
// - one warp issues the MMAs: O of a tile's block, then S of its next block, while the other tile is in its softmax.
// Measured: 128 queries of 32 heads over 32768 keys (8 heads of 128) 81 us, 0.85 PFLOP/s; 512 over 8192 keys 93 us, a prompt of
// 2048 on itself 82 us; of head_dim 64, 128 over 16384 keys 44 us. A block
// of 128 keys for 256 rows takes about 4300 cycles: a tile's softmax (2500 to 3000) and its two products (1400) follow
// each other, while the other tile is half a block away; decoding is busy for 3000 cycles, the tensor cores for 42% of the
// time. Other divisions were slower: one tile per CTA with S in two buffers (163 us when this took 120), blocks of 64 keys
// with S in two buffers (119 for 98: products of 64 columns take as long as those of 128), and weights handed over in
// halves changed nothing. Beside the blocks stand about 13 us for the first block, the sums and joining the splits.
//
// Every wait on an mbarrier is bounded; after a timeout every role runs to its end without waiting.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "mxq_attention.cuh"
#include "mxq_tc.cuh"

namespace mxq {
namespace {

// warpgroups: softmax of the two tiles, decoding, and one of single warps: MMA, two of copies, scales. Registers are moved between them: 128 a thread
// at launch = (184 + 184 + 104 + 40) / 4
constexpr int kTcThreads = 512, kTcDecode = 8, kTcMma = 12, kTcCopy = 13, kTcScales = 15;
template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// K is decoded to 2^-13 of the largest block of its 128 keys, V to 2^-10 of the largest that set its reference or less, and
// blocks 2^14 below that are exact: so are those 2^16 below what a row sees while the others of its tile see this much more
constexpr int kTcRoomK = 11, kTcRoomV = 8;
constexpr int kTcRaw = 3;        // blocks in the ring of raw codes

template <int D> struct TcCfg {
    static constexpr int ROW = D / 2, SROW = D / 32;
    static constexpr int Q = 128 * D * 2, K = 128 * D * 2, V = K;  // bytes of an operand
    static constexpr int RV = 128 * ROW, RKS = 2 * RV, RVS = RKS + 128 * SROW, RAW = RVS + 128 * SROW;
    static constexpr int AT_K = 2 * Q, AT_V = AT_K + 2 * K, AT_RAW = AT_V + V, BYTES = AT_RAW + kTcRaw * RAW;
    static constexpr int SMEM = BYTES + 1024;  // + alignment slack
    static_assert(SMEM <= 224 * 1024, "shared memory");
    // place of 16-byte piece c of row r of the raw codes of K and of V
    static __device__ __forceinline__ uint32_t k_at(int r, int c) {
        return D == 128 ? (uint32_t)(r * ROW + 16 * (c ^ ((r >> 1) & 3))) : (uint32_t)(r * ROW + 16 * (c ^ ((r >> 2) & 1)));
    }
    static __device__ __forceinline__ uint32_t v_at(int r, int c) {
        const int kg = r >> 3;
        return D == 128 ? (uint32_t)((r ^ ((kg >> 2) & 1)) * ROW + 16 * (c ^ (kg & 3)))
                        : (uint32_t)((r ^ (kg & 3)) * ROW + 16 * (c ^ ((kg >> 2) & 1)));
    }
};
// tensor memory columns
constexpr int kColS = 0, kColO = 256;  // + 128 for the second tile

// what the scales' warp tells the others about a block
struct BlockInfo {
    int kref, vref;      // reference scale bytes
    uint32_t pages;      // bit j: keys 16 j .. are in a page of the cache
    uint32_t nan;        // a value block of the block of keys is NaN: nan_keys holds which
};

// position in a ring of n places: place and the parity of its current use
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// f16 factors 2^(byte - ref) of two scale bytes (in the halves of x), 0 below 2^-14: the exponent fields byte - ref + 15,
// with floor2 = ref - 15 in both halves and minus2 the number that takes it off both
__device__ __forceinline__ uint32_t scale_pair(uint32_t x, uint32_t floor2, uint32_t minus2) {
    uint32_t m;
    asm("max.s16x2 %0, %1, %2;" : "=r"(m) : "r"(x), "r"(floor2));
    return (m + minus2) << 10;
}
// largest scale byte of the 16 bytes w that are not NaN (0xFF), or -1; sets `nan` if one is
__device__ __forceinline__ int max_byte(const uint32_t* w, bool& nan) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t bad = __vcmpeq4(w[i], 0xFFFFFFFFu);
        nan |= bad != 0;
        m = __vmaxu4(m, w[i] & ~bad);
    }
    m = __vmaxu4(m, m >> 16);
    m = __vmaxu4(m, m >> 8);
    return (int)(m & 0xFFu);
}

template <int D> __global__ void __launch_bounds__(kTcThreads, 1) k_kv_attention_tiles(const __grid_constant__ AtArgs p, unsigned int* err) {
    using C = TcCfg<D>;
    extern __shared__ uint8_t dsm8[];
    uint8_t* const base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm8) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(base);
    __shared__ __align__(8) unsigned long long bars[22];
    __shared__ uint32_t tmem_addr;
    __shared__ int abort_flag;
    __shared__ BlockInfo infos[8];  // eight blocks: more than the roles can be apart
    __shared__ uint32_t there[8][2];      // groups of 16 keys of a block that are in pages: even and odd ones
    __shared__ Spread spreads[4][2];      // noted by the decoding warps, where the rows see different keys
    __shared__ uint8_t nan_keys[8][128];  // of a block with NaN values: bit b of key's byte: its block b is NaN
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto k_full = [&](int i) { return bar(i & 1); };
    auto k_empty = [&](int i) { return bar(2 + (i & 1)); };
    const uint32_t v_full = bar(4), v_empty = bar(5), drained = bar(6);
    auto q_full = [&](int x) { return bar(7 + x); };   // of tile x
    auto s_full = [&](int x) { return bar(9 + x); };   // S of a block, and everything issued before it; at the end, O
    auto p_full = [&](int x) { return bar(11 + x); };  // P of a block
    auto raw_full = [&](int i) { return bar(13 + i); };   // of a place in the ring of raw codes
    auto raw_empty = [&](int i) { return bar(16 + i); };
    auto info_full = [&](int i) { return bar(19 + i); };
    if (t == 0) {
        for (int i = 0; i < kTcRaw; ++i) {
            mbar_init(raw_full(i), 66);  // the copies of 64 threads, and two that tell of the pages
            mbar_init(raw_empty(i), 128);
            mbar_init(info_full(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full(i), 128);
            mbar_init(k_empty(i), 1);
            mbar_init(q_full(i), 128);
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 128);
        }
        mbar_init(v_full, 128);
        mbar_init(v_empty, 1);
        mbar_init(drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kTcMma) {
        tmem_alloc<512>(smem_u32(&tmem_addr));
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_addr;
    volatile int* ab = &abort_flag;
    pdl_wait_then_release();

    const int tile = p.by_splits(blockIdx.x), sp = blockIdx.x - tile * p.splits;
    const int bh = p.by_tiles(tile), rt = tile - bh * p.row_tiles;
    const int b = p.by_heads(bh), head = bh - b * p.c.heads;
    const Span s = span_of(p, b);
    const int rows = s.nq * p.group, r0 = rt * kTileRows;
    if (p.fill && rt == 0 && sp == 0) fill_rows<D>(p, s, b, head * p.group, p.group);
    Groups gr{0, 0, 1};
    KeyRange some{0, 0};  // the keys that a row of the CTA sees: the bytes of others count as zeros
    int i0 = 0, i1 = 0;   // the CTA's queries
    if (r0 < rows) {
        i0 = p.by_group(r0), i1 = p.by_group(min(r0 + kTileRows, rows) - 1);
        gr = groups_of<kTileKeysShift, kTileMinBlocks>(p, s, i0, i1);
        some = keys_seen(p, s, i0, i1);
    }
    const int first = gr.lo + sp * gr.per, n = max(min(first + gr.per, gr.hi) - first, 0);  // blocks of this CTA
    const bool alone = gr.hi - gr.lo <= gr.per;  // one split holds all keys
    const bool work = r0 < rows && (n > 0 || sp == 0), two = r0 + 128 < rows;  // two: the second tile has rows

    if (warp < kTcDecode) {
        regs_up<184>();
        const int x = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        if (work && (x == 0 || two)) {
            // ---- softmax: thread's row r0 + 128 x + row ----
            const int r = r0 + 128 * x + row, i = p.by_group(min(r, rows - 1)), h = head * p.group + (min(r, rows - 1) - i * p.group);
            const int pos = r < rows ? max(s.len - s.n + i, -1) : -1;  // (-1 at least, so that pos - window is an int)
            const int see_hi = min(pos + 1, s.len), see_lo = p.window > 0 ? pos - p.window + 1 : 0;  // keys see_lo .. see_hi - 1
            const uint32_t ts = tm + ((uint32_t)(quad * 32) << 16) + kColS + 128 * x, to = ts + kColO - kColS;
            constexpr int LANES = D / 8, RPI = 32 / LANES;  // lanes that read or write a row, rows at a time
            const int ch = lane % LANES, sub = lane / LANES;
            float mul = 0.f;
            if (n > 0) {  // (without keys the rows' place of Q is used for the output alone)
                // Q's rows over a power of two, in f16; D / 8 lanes read a row
                uint4 q[LANES];
#pragma unroll
                for (int k = 0; k < LANES; ++k) {
                    const int rk = min(r0 + 128 * x + quad * 32 + k * RPI + sub, rows - 1), ik = p.by_group(rk);
                    const int hk = head * p.group + (rk - ik * p.group);
                    q[k] = __ldg(reinterpret_cast<const uint4*>(p.q + (s.q0 + ik) * p.q_row_stride + hk * p.q_head_stride) + ch);
                }
                int mine = 0;
#pragma unroll
                for (int k = 0; k < LANES; ++k) {
                    const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
                    uint32_t top = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) top = max(top, max((w[j] & 0x7FFFu) << 16, w[j] & 0x7FFF0000u));
#pragma unroll
                    for (int j = 1; j < LANES; j *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, j));
                    const int e = min(max((int)(top >> 23), 1), 253) - 127;
                    const float down = pow2i(-e);
                    uint32_t f[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f[j] = pack_h2(__uint_as_float(w[j] << 16) * down, __uint_as_float(w[j] & 0xFFFF0000u) * down);
                    const int to_row = quad * 32 + k * RPI + sub;
                    sts128(sb + x * C::Q + (ch >> 3) * 16384 + to_row * 128 + (((ch & 7) ^ (to_row & 7)) << 4), f[0], f[1], f[2], f[3]);
                    const int theirs = __shfl_sync(0xFFFFFFFFu, e, lane % RPI * LANES);  // of row k * RPI + lane % RPI
                    if (lane / RPI == k) mine = theirs;
                }
                mul = p.scale * pow2i(mine);
                fence_proxy_async();
                mbar_arrive(q_full(x));
            }
            float m = 0.f, thr = -INFINITY, l = 0.f;
            int vref = 0;
            uint32_t vnan = 0;  // bit j: dimensions 32 j .. of the row are NaN
            bool ok = true;
            for (int it = 0; it < n; ++it) {
                // S of this block, and with it the products before: O of block it - 1 is complete
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(s_full(x), (uint32_t)it & 1u, ab, err));
                if (!ok) break;
                tc_fence_after();
                const BlockInfo bi = infos[it & 7];
                const int key0 = (first + it) * 128;
                union {
                    uint32_t u[128];
                    float f[128];
                    unsigned long long d[64];
                } e;
#pragma unroll
                for (int c = 0; c < 128; c += 32) tmem_ld32(ts + c, e.u + c);
                tmem_wait_ld();
                if (bi.nan) {
                    for (int j = 0; j < 128; ++j) {
                        const uint32_t bits = nan_keys[it & 7][j];
                        if (key0 + j < see_hi && key0 + j >= see_lo) vnan |= bits;
                    }
                }
                float mk = mul * pow2i(bi.kref - 127);
                if (bi.kref <= 0) mk = mul * 0x1p-64f * pow2i(bi.kref - 63);  // 2^(kref - 127) is a subnormal
                const unsigned long long mk2 = dup2(mk), m2 = dup2(-m);
#pragma unroll
                for (int j = 0; j < 64; ++j) e.d[j] = f2fma(e.d[j], mk2, m2);
                // keys that the row does not see
                if (!__all_sync(0xFFFFFFFFu, bi.pages == 0xFFu && key0 >= see_lo && key0 + 128 <= see_hi)) {
                    const int lo = see_lo - key0, hi = see_hi - key0;
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (j >= hi || j < lo || !((bi.pages >> (j >> 4)) & 1u)) e.f[j] = -INFINITY;
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 128; j += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) top[k] = max3(top[k], e.f[j + 2 * k], e.f[j + 2 * k + 1]);
                const float y = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // raise the maximum, or follow the reference scale of V
                const bool raise = y > thr, follow = it > 0 && bi.vref != vref;
                if (__any_sync(0xFFFFFFFFu, raise || follow)) {
                    float f = 1.f, dx = 0.f;
                    if (raise) {
                        f = thr > 0.f ? ex2(-y) : 0.f;
                        dx = y;
                        m += y;
                        thr = 8.f;
                    }
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (raise && e.f[j] != -INFINITY) e.f[j] -= dx;
                    l *= f;
                    if (it > 0) {
                        if (follow) f *= pow2i(vref - bi.vref);
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(to + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st16(to + c, o);
                        }
                    }
                }
                vref = bi.vref;
                // weights over S: two keys per column
                unsigned long long sum2 = dup2(0.f);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float a = ex2(e.f[32 * c + 2 * j]), b2 = ex2(e.f[32 * c + 2 * j + 1]);
                        sum2 = f2add(sum2, pk(a, b2));
                        w[j] = pack_h2(a, b2);
                    }
                    tmem_st16(ts + 16 * c, w);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full(x));
                float sa, sc;
                upk(sum2, sa, sc);
                l += sa + sc;
            }
            if (n > 0 && ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(s_full(x), (uint32_t)n & 1u, ab, err));
            tc_fence_after();
            if (!(thr > 0.f)) m = -INFINITY;
            if (ok && n > 0 && i1 > i0 && spread_beyond<4>(spreads, kTcRoomK, kTcRoomV)) {
                const int t0 = 128 * x + quad * 32;
                for (int k = t0; k < t0 + 32 && r0 + k < rows; ++k)
                    exact_row<D>(p, s, b, head, r0 + k, first * 128, (first + n) * 128, alone, (long long)blockIdx.x * kTileRows + k);
            } else if (ok) {
                const long long at = (long long)(s.q0 + i) * p.heads + h, slot0 = (long long)blockIdx.x * kTileRows + 128 * x + quad * 32;
                const float vtrue = scale_of(vref), f = alone ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                const float nan = __uint_as_float(0x7FC00000u);
                // through the rows' place of Q, which nothing reads any more: whole rows, 16 bytes a lane
                const uint32_t stage = sb + x * C::Q + quad * (C::Q / 4), mine = stage + lane * (2 * D);
                const int cols = alone ? D : D / 2, left = rows - (r0 + 128 * x + quad * 32);  // columns at a time
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += cols) {
#pragma unroll 1
                    for (int c = c0; c < c0 + cols; c += 16) {
                        uint32_t o[16];
                        if (n > 0) {
                            tmem_ld16(to + c, o);
                            tmem_wait_ld();
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = 0;
                        }
                        const float g = (vnan >> (c >> 5)) & 1u ? nan : f;
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * g * vtrue);
                        if (alone) {
                            uint32_t w[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) w[j] = bf16x2(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                sts128(mine + ((((c >> 3) + j) ^ (lane & 7)) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                sts128(mine + (((((c - c0) >> 2) + j) ^ (lane & 7)) << 4), o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        }
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int k = 0; k < LANES; ++k) {
                        const int rk = k * RPI + sub;
                        const uint4 v = lds128u(stage + rk * (2 * D) + ((ch ^ (rk & 7)) << 4));
                        if (rk >= left) continue;
                        if (alone) {
                            const int row_k = r0 + 128 * x + quad * 32 + rk, ik = p.by_group(row_k);
                            const long long at_k = (long long)(s.q0 + ik) * p.heads + head * p.group + (row_k - ik * p.group);
                            reinterpret_cast<uint4*>(p.out + at_k * D)[ch] = v;
                        } else {
                            reinterpret_cast<uint4*>(p.part + (slot0 + rk) * D + c0)[ch] = v;
                        }
                    }
                    __syncwarp();
                }
                if (r < rows) {
                    if (!alone) *reinterpret_cast<float2*>(p.part + p.part_ml + (slot0 + lane) * 2) = make_float2(m, l);
                    else if (p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                }
            }
        }
    } else if (warp < kTcMma) {
        regs_down<104>();
        // ---- decoding: K of block it, then V of block it - 1 (K's two buffers let it run ahead of the products that
        // still read V) ----
        const int w = warp - kTcDecode, d = 32 * w + lane;
        Ring at, at_v;
        uint32_t pages_v = 0;
        int vref_v = 0;
        bool nan_v = false, live = work && n > 0;
        // while Q and the first codes are on their way; the softmax warps read it when O, and so all of K, is done
        if (live && i1 > i0) note_spread<D>(p, s, b, head, i0, i1, first * 128, (first + n) * 128, d, 128, spreads);
        for (int it = 0; live && it <= n; ++it) {
            const int key0 = (first + it) * 128;
            BlockInfo bi{0, 0, 0, 0};
            if (it < n) {
                live = mbar_wait(raw_full(at.s), at.phase, ab, err) && mbar_wait(info_full(at.s), at.phase, ab, err);
                if (!live) break;
                const uint32_t raw = sb + C::AT_RAW + (uint32_t)at.s * C::RAW;
                bi = infos[it & 7];
                // K: thread d decodes key d
                uint32_t sw, kx[C::SROW][4];
                if constexpr (D == 128) sw = lds32(raw + C::RKS + 4 * d);
                else sw = (lds32(raw + C::RKS + 4 * (d >> 1)) >> (16 * (d & 1))) & 0xFFFFu;
#pragma unroll
                for (int j = 0; j < C::SROW; ++j) {
                    const uint4 y = lds128u(raw + C::k_at(d, j));
                    kx[j][0] = y.x;
                    kx[j][1] = y.y;
                    kx[j][2] = y.z;
                    kx[j][3] = y.w;
                }
                if (bi.nan) {
                    // value blocks that are NaN, of key d
                    uint32_t bits = 0;
#pragma unroll
                    for (int j = 0; j < C::SROW; ++j)
                        if (lds8(raw + C::RVS + d * C::SROW + j) == 0xFFu) bits |= 1u << j;
                    if (key0 + d >= some.hi || !((bi.pages >> (d >> 4)) & 1u)) bits = 0;
                    nan_keys[it & 7][d] = (uint8_t)bits;
                }
                const int c0 = bi.kref - 15;
                const uint32_t floor2 = (uint32_t)(c0 & 0xFFFF) * 0x10001u, minus2 = (uint32_t)(-c0 * 0x10001);
                const uint32_t kb = sb + C::AT_K + (uint32_t)(it & 1) * C::K + d * 128;
                if (it > 1) live = mbar_wait(k_empty(it), (uint32_t)((it >> 1) - 1) & 1u, ab, err);
                if (!live) break;
#pragma unroll
                for (int j = 0; j < C::SROW; ++j) {
                    const uint32_t byte = (sw >> (8 * j)) & 0xFFu;
                    uint32_t f = scale_pair(byte * 0x10001u, floor2, minus2);
                    if (byte == 0xFFu) f = 0x7E007E00u;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[4];
                        e2m1_to_h2(kx[j][k], o);
                        const int ch = (j & 1) * 4 + k;
                        sts128(kb + (j >> 1) * 16384 + ((ch ^ (d & 7)) << 4), mul_h2(o[0], f), mul_h2(o[1], f), mul_h2(o[2], f),
                               mul_h2(o[3], f));
                    }
                }
                fence_proxy_async();
                mbar_arrive(k_full(it));
            }
            if (it > 0) {
                // V: keys 64 u + 8 kg .. + 7, eight dimensions of one 32-value block
                const uint32_t raw = sb + C::AT_RAW + (uint32_t)at_v.s * C::RAW;
                const int key0v = key0 - 128;
                const bool edge = pages_v != 0xFFu || key0v + 128 > some.hi || key0v < some.lo || nan_v;
                const int c0 = vref_v - 15;
                const uint32_t floor2 = (uint32_t)(c0 & 0xFFFF) * 0x10001u, minus2 = (uint32_t)(-c0 * 0x10001);
                const int kg = lane & 7, dg = lane >> 3, blk = D == 128 ? w : w & 1;
                constexpr int UNITS = D == 128 ? 2 : 1;
                uint32_t x[UNITS][8], sc[UNITS][4];
#pragma unroll
                for (int uu = 0; uu < UNITS; ++uu) {
                    const int k0 = (D == 128 ? uu : w >> 1) * 64 + kg * 8;
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[uu][j] = lds32(raw + C::RV + C::v_at(k0 + j, blk) + 4 * dg);
                    uint32_t sw[8];  // the keys' scale of the block
                    if constexpr (D == 128) {
                        const uint4 a = lds128u(raw + C::RVS + 4 * k0), c = lds128u(raw + C::RVS + 4 * k0 + 16);
                        const uint32_t y[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) sw[j] = (y[j] >> (8 * blk)) & 0xFFu;
                    } else {
                        const uint4 a = lds128u(raw + C::RVS + 2 * k0);
                        const uint32_t y[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) sw[j] = (y[j >> 1] >> (16 * (j & 1) + 8 * blk)) & 0xFFu;
                    }
                    if (edge) {
                        const bool in = (pages_v >> (k0 >> 4)) & 1u;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (!in || key0v + k0 + j >= some.hi || key0v + k0 + j < some.lo || sw[j] == 0xFFu) sw[j] = 0;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[uu][j] = scale_pair(sw[2 * j] | (sw[2 * j + 1] << 16), floor2, minus2);
                }
                mbar_arrive(raw_empty(at_v.s));
                if (it > 1) live = mbar_wait(v_empty, (uint32_t)(it - 2) & 1u, ab, err);
                if (!live) break;
#pragma unroll
                for (int uu = 0; uu < UNITS; ++uu) {
                    const int u = D == 128 ? uu : w >> 1;
                    uint32_t ev[4][4], od[4][4];  // [pair of keys][dimension / 2]
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e2m1_to_h2((x[uu][2 * j] & 0x0F0F0F0Fu) | ((x[uu][2 * j + 1] << 4) & 0xF0F0F0F0u), ev[j]);
                        e2m1_to_h2(((x[uu][2 * j] >> 4) & 0x0F0F0F0Fu) | (x[uu][2 * j + 1] & 0xF0F0F0F0u), od[j]);
                    }
                    const uint32_t row = sb + C::AT_V + (uint32_t)u * (D * 128) + (uint32_t)(blk * 32 + dg * 8) * 128;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        sts128(row + (2 * k) * 128 + ((kg ^ (2 * k)) << 4), mul_h2(ev[0][k], sc[uu][0]), mul_h2(ev[1][k], sc[uu][1]),
                               mul_h2(ev[2][k], sc[uu][2]), mul_h2(ev[3][k], sc[uu][3]));
                        sts128(row + (2 * k + 1) * 128 + ((kg ^ (2 * k + 1)) << 4), mul_h2(od[0][k], sc[uu][0]),
                               mul_h2(od[1][k], sc[uu][1]), mul_h2(od[2][k], sc[uu][2]), mul_h2(od[3][k], sc[uu][3]));
                    }
                }
                fence_proxy_async();
                mbar_arrive(v_full);
            }
            at_v = at;
            at.next(kTcRaw);
            pages_v = bi.pages;
            vref_v = bi.vref;
            nan_v = bi.nan != 0;
        }
    } else {
        regs_down<40>();
        if (work && (warp == kTcCopy || warp == kTcCopy + 1)) {
            // ---- copies: this warp takes four of a block's eight groups of 16 keys ----
            const int c0 = 4 * (warp - kTcCopy);
            constexpr int PIECES = C::ROW / 16, STEPS = 16 * PIECES / 32;  // 16-byte pieces of a row; of a group per lane
            const long long page_rows = (long long)p.c.heads * p.c.page, head_row = (long long)head * p.c.page;
            int pg = -1, off = 0;  // lane j < 4: page and first row of group c0 + j of the next block, as loaded
            auto lookup = [&](int blk) {
                const int key = (first + blk) * 128 + 16 * (c0 + lane);
                pg = -1;
                if (lane < 4 && blk < n && key < some.hi) {
                    const int at = p.by_page(key);
                    off = key - at * p.c.page;
                    pg = __ldg(p.table + b * p.table_stride + at);
                }
            };
            Ring at;
            lookup(0);
            for (int it = 0; it < n; ++it, at.next(kTcRaw)) {
                // one verdict for the warp: the shuffles below need every lane
                if (it >= kTcRaw && !__all_sync(0xFFFFFFFFu, mbar_wait(raw_empty(at.s), at.phase ^ 1u, ab, err))) break;
                const uint32_t raw = sb + C::AT_RAW + (uint32_t)at.s * C::RAW;
                if (pg >= p.c.pages) pg = -1;
                uint32_t bits = 0;
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    const int x = __shfl_sync(0xFFFFFFFFu, pg, j), o = __shfl_sync(0xFFFFFFFFu, off, j), g = c0 + j;
                    if (x < 0) continue;
                    bits |= 1u << g;
                    const long long row = x * page_rows + head_row + o;
#pragma unroll
                    for (int i = 0; i < STEPS; ++i) {
                        const int e = 32 * i + lane, r = 16 * g + e / PIECES;
                        copy16(raw + C::k_at(r, e % PIECES), p.c.kc + row * C::ROW + 16 * e);
                        copy16(raw + C::RV + C::v_at(r, e % PIECES), p.c.vc + row * C::ROW + 16 * e);
                    }
                    if (lane < 2 * C::SROW) {  // scales: SROW pieces each of K and V
                        const bool v = lane >= C::SROW;
                        const int e = lane - (v ? C::SROW : 0);
                        copy16(raw + (v ? C::RVS : C::RKS) + 16 * (C::SROW * g + e), (v ? p.c.vs : p.c.ks) + row * C::SROW + 16 * e);
                    }
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(raw_full(at.s)) : "memory");
                if (lane == 0) {
                    there[it & 7][warp - kTcCopy] = bits;
                    mbar_arrive(raw_full(at.s));
                }
                lookup(it + 1);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (work && warp == kTcScales) {
            // ---- reference scales ----
            int vref = -1000;
            Ring at;
            for (int it = 0; it < n; ++it, at.next(kTcRaw)) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(raw_full(at.s), at.phase, ab, err))) break;
                const uint32_t raw = sb + C::AT_RAW + (uint32_t)at.s * C::RAW;
                const int key0 = (first + it) * 128;
                const uint32_t pages = there[it & 7][0] | there[it & 7][1];
                const bool edge = pages != 0xFFu || key0 + 128 > some.hi || key0 < some.lo;
                constexpr int PER = 16 / C::SROW;  // keys of the lane's 16 bytes
                const int mine = min(lane, 128 / PER - 1);
                bool nan = false;
                int top[2];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const uint4 y = lds128u(raw + (v ? C::RVS : C::RKS) + 16 * mine);
                    uint32_t x[4] = {y.x, y.y, y.z, y.w};
                    if (edge) {
                        const int key = key0 + mine * PER;
                        const bool in = (pages >> (mine * PER >> 4)) & 1u;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (D == 128) {
                                if (!in || key + i >= some.hi || key + i < some.lo) x[i] = 0;
                            } else {  // two keys to a word
                                if (!in || key + 2 * i >= some.hi || key + 2 * i < some.lo) x[i] &= 0xFFFF0000u;
                                if (!in || key + 2 * i + 1 >= some.hi || key + 2 * i + 1 < some.lo) x[i] &= 0xFFFFu;
                            }
                        }
                    }
                    top[v] = (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)max_byte(x, nan));
                }
                nan = __any_sync(0xFFFFFFFFu, nan);
                if (top[1] > vref + 13) vref = top[1] - 10;
                if (lane == 0) {
                    infos[it & 7] = {top[0] - 13, vref, pages, nan ? 1u : 0u};
                    mbar_arrive(info_full(at.s));
                }
            }
        } else if (warp == kTcMma && work && n > 0) {
            // ---- MMAs ----
            const bool one = elect_one();
            constexpr uint32_t id_s = idesc_f16(128, 128), id_o = idesc_f16(128, D);
            const SmemDesc dq = desc_sw128(sb);
            bool ok = true;
            auto scores = [&](int x, int it) {  // S of tile x
                if (one) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t at = (k >> 2) * 16384 + (k & 3) * 32;
                        tc_mma_f16(tm + kColS + 128 * x, dq + (x * C::Q + at), dq + (C::AT_K + (it & 1) * C::K + at), id_s, k > 0);
                    }
                    if (x == two) tc_commit(k_empty(it));
                    tc_commit(s_full(x));
                }
            };
            ok = mbar_wait(k_full(0), 0, ab, err);
            for (int x = 0; ok && x <= two; ++x) {
                ok = mbar_wait(q_full(x), 0, ab, err);
                tc_fence_after();
                if (ok) scores(x, 0);
            }
            for (int it = 0; ok && it < n; ++it)
                for (int x = 0; ok && x <= two; ++x) {
                    if (x == 0) ok = mbar_wait(v_full, (uint32_t)it & 1u, ab, err);
                    ok = ok && mbar_wait(p_full(x), (uint32_t)it & 1u, ab, err);
                    if (!ok) break;
                    tc_fence_after();
                    if (one) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc_mma_f16_ts(tm + kColO + 128 * x, tm + kColS + 128 * x + 8 * k, dq + (C::AT_V + (k >> 2) * (D * 128) + (k & 3) * 32),
                                          id_o, it > 0 || k > 0);
                        if (x == two) tc_commit(v_empty);
                    }
                    if (it + 1 < n) {
                        // S of the next block over P, which the product before has read (they execute in order)
                        if (x == 0) ok = mbar_wait(k_full(it + 1), (uint32_t)((it + 1) >> 1) & 1u, ab, err);
                        tc_fence_after();
                        if (ok) scores(x, it + 1);
                    } else if (one) {
                        tc_commit(s_full(x));
                    }
                }
            if (one && *ab) {  // MMAs in flight end before their shared and tensor memory goes away
                tc_commit(drained);
                const unsigned long long t0 = global_ns();
                while (!mbar_test(drained, 0) && global_ns() - t0 < kWaitLimitNs) {
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kTcMma) {
        tc_fence_after();
        tmem_free<512>(tm);
    }
}

template <int D> cudaError_t go(const AtArgs& a, long long tiles, int dev, cudaStream_t st) {
    auto* kern = k_kv_attention_tiles<D>;
    static std::atomic<unsigned long long> ready{0};
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TcCfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    unsigned int* err = nullptr;
    cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * a.splits));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = TcCfg<D>::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, err);
}

}  // namespace

cudaError_t launch_kv_attention_tiles(const AtArgs& a, long long tiles, int dev, cudaStream_t st) {
    return a.c.db == 4 ? go<128>(a, tiles, dev, st) : go<64>(a, tiles, dev, st);
}

}  // namespace mxq
