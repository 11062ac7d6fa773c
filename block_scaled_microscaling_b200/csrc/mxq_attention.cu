// mxq_attention.cu -- attention over the paged MXFP4 key/value cache (sm_100a).
//
// For the queries of one sequence that share a key/value head (rows = query x head of the group),
//   s[j, r] = scale * log2(e) * sum_d K[j, d] Q[r, d],   o[r, d] = sum_j 2^(s[j, r] - m_r) V[j, d] / sum_j 2^(s[j, r] - m_r)
// over the keys j that row r sees. 17 bytes hold 32 cached values, so at the copy bandwidth 12 values arrive per
// picosecond and the SMs have about three lane instructions for each: what bounds the kernel is turning codes into
// operands. Hence:
// - each warp takes groups of 16 keys (a group lies within a page) through its own ring of stages in shared memory,
//   filled by 16-byte asynchronous copies two groups ahead: no registers hold data in flight and no warp waits for
//   another. Codes leave the stage in the layout of mma.sync's fragments. The summed index may be permuted freely,
//   so the lane that holds key g's part of an operand owns a contiguous quarter of the key (16 bytes of codes and one
//   scale at head_dim 128), and four lanes share it; for V, whose operand pairs two keys, a lane takes the same 8
//   bytes of four neighbouring keys and interleaves the nibbles of two keys with shifts and masks before the
//   conversion. V's rows are stored permuted, so that these reads touch every bank once.
// - cvt.rn.f16x2.e2m1x2 converts two codes; one f16x2 product applies the block scale. Both products run in f16
//   with fp32 sums (m16n8k16): keys (then head dimensions) fill the instruction's 16 rows and the queries its 8
//   columns, so one query of up to 8 heads per key head (a decoding step) wastes nothing.
// - f16 holds a code times 2^x exactly for -23 <= x <= 13, so block scales are taken relative to a reference per
//   warp (K and V each), 2^6 below the largest block when it was set and raised by a vote when a block exceeds 2^13
//   of it; codes of blocks more than 2^29 below the largest that the warp's rows see lose bits (mxq_attention.cuh has what
//   happens where rows see different keys). Rows of Q are divided by a power of two for the same reason: values 2^17
//   below a row's largest lose bits, those 2^25 below it are 0. Scores return to their true size in fp32.
// - the running maximum m_r is raised only when a score exceeds it by 2^8 (one vote per 16 keys); the weights
//   then are at most 2^8 and round to f16 for the second product (relative error 2^-11; below 2^-14 absolute, 2^-25): the
//   tensor cores take 16-bit operands, and f16 is the one with the most digits. Their sum is that of the fp32 values,
//   since the rounding is even on average. 2^x is the hardware's (relative error 2^-22, far below that rounding).
// The four warps of a CTA take every fourth group (page numbers are fetched 32 groups at a time); their results are
// joined through shared memory. Where one row tile holds a sequence's queries (decoding), the groups of all sequences
// and heads are cut into equal shares, one per resident CTA, whatever the lengths: a CTA walks the pieces of its
// share, and the at most two of them that are part of a split sequence leave their sums to a second kernel, which
// joins them in order. Otherwise a long sequence is split over a fixed number of CTAs, joined the same way.
// Measured (32 heads on 8 of 128, one query each): 16 sequences of 24 .. 32 thousand keys 137 us (3.7 TB/s of cache; the
// issue slots are 63% busy, the arithmetic pipe 52%, and the waits of dependent conversions fill the rest: with three
// CTAs to an SM, 183 us; five, with spilled registers, 158; two groups at a time, 143), one sequence of 4000 keys 9
// us, of 32768 keys 20; of head_dim 64, 16 sequences of 16384 keys 63. At head_dim 128 the limits of 128 and 168 registers
// make the compiler spill (72 and 180 bytes of stores a thread for 8 and 16 rows).
#include <atomic>
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "mxq_attention.cuh"

namespace mxq {
namespace {

constexpr int kAtWarps = 4, kAtThreads = 32 * kAtWarps;
constexpr int kAtStages = 3;       // groups in a warp's ring (four: as fast, six: 146 us for 141 at 16 sequences of 24..32 thousand keys)
constexpr int kAtMaxSplits = 256;
constexpr long long kJoinRows = 2048;  // below, the warps of a CTA share the splits of a row (4096 rows of 9 splits: 92 us so, 85 with a warp each)
// a reference is at most 2^6 below the largest block, and blocks 2^23 below a reference are exact: so are those 2^16 below
// what a row sees while the others of its tile see 2^13 of it
constexpr int kAtRoom = 13;
constexpr int kEvenGroups = 8;     // groups that an equal share has at least, if there are fewer sequences
constexpr int kAtMaxEven = 512;    // sequences whose shares are worked out by every CTA

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// log2 of a weight: score * mk - m
__device__ __forceinline__ float weight_exponent(float score, float mk, float m) { return fmaf(score, mk, -m); }
// byte 0x4440 + j of x, zero-extended
__device__ __forceinline__ uint32_t prmt(uint32_t x, uint32_t sel) { return __byte_perm(x, 0u, sel); }
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
// 2^(byte - ref) as fp32 (2^-126 far below 1, which the conversion to f16 makes 0; it rounds small ones)
__device__ __forceinline__ float rel_scale(int byte, int ref) {
    return __uint_as_float((uint32_t)(max(byte, ref - 126) - (ref - 127)) << 23);
}
// a stage: codes of 16 keys and values, then their scales
template <int D> struct AtStage {
    static constexpr int ROW = D / 2, SROW = D / 32;  // bytes of a key's codes, of its scales
    static constexpr int K = 0, V = 16 * ROW, KS = 2 * V, VS = KS + 16 * SROW, BYTES = VS + 16 * SROW;
    // place of 16-byte piece c of V's row r: a lane quad's four rows 4t + i fall on different banks
    static __device__ __forceinline__ uint32_t v_at(int r, int c) {
        if (D == 128) return (uint32_t)(V + (r ^ ((r >> 2) & 1)) * ROW + 16 * (c ^ ((r >> 3) << 1)));
        return (uint32_t)(V + (r ^ (r >> 2)) * ROW + 16 * c);
    }
};
// the lane's share of the copies of a group
template <int D> struct Fetch {
    using S = AtStage<D>;
    static constexpr int PIECES = S::ROW / 16;  // 16-byte pieces of a row
    const char *k, *v;
    const uint8_t* scales;
    uint32_t at, at_v[PIECES / 2], at_s;
    bool scaled;
    __device__ __forceinline__ Fetch(const KvCache& c, int lane) {
        k = c.kc + 16 * lane;
        v = c.vc + 16 * lane;
        at = S::K + 16 * lane;
#pragma unroll
        for (int i = 0; i < PIECES / 2; ++i) at_v[i] = S::v_at((i * 32 + lane) / PIECES, lane % PIECES);
        const bool of_v = lane >= S::SROW;  // scales: SROW pieces of 16 bytes each of K and V
        const int j = lane - (of_v ? S::SROW : 0);
        scaled = lane < 2 * S::SROW;
        scales = (of_v ? c.vs : c.ks) + 16 * j;
        at_s = (of_v ? S::VS : S::KS) + 16 * j;
    }
    // group: its place in the cache, in groups (2^31 of them would be 2 TB at head_dim 64)
    __device__ __forceinline__ void copy(int group, uint32_t stage) const {
        const long long from = (long long)group * (16 * S::ROW);
#pragma unroll
        for (int i = 0; i < PIECES / 2; ++i) {
            copy16(stage + at + 512 * i, k + from + 512 * i);
            copy16(stage + at_v[i], v + from + 512 * i);
        }
        if (scaled) copy16(stage + at_s, scales + (long long)group * (16 * S::SROW));
    }
};

// float offset of dimension d of row r in a warp's result: rows D + 4 floats apart, so that the lanes' 16-byte
// writes (dimensions g D/8 .., rows 2t, 2t + 1) meet in a bank at most in pairs
template <int D> __device__ __forceinline__ int res_off(int r, int d) { return r * (D + 4) + d; }

// keys 16 first .. 16 last of one sequence and head for the rows of a tile
struct Piece {
    Span s;
    int b, head, r0;
    int first, last;
    bool alone;       // all of the tile's keys: the output itself is written
    long long slot;   // else the place of the partial sums
};

// NQ: groups of eight rows that a warp handles together (their Q operands in shared memory when NQ is 4)
// MIXED: the rows may see different keys (several queries)
template <int D, int NQ, bool MIXED> __device__ __forceinline__ void attend(const AtArgs& p, const Piece& w) {
    constexpr int ROWS = 8 * NQ, STEPS = D / 16, TILES = D / 16;
    constexpr bool QS = NQ == 4;
    using S = AtStage<D>;
    extern __shared__ __align__(16) float dsm[];  // stages of the warps, Q's operands; later the warps' results
    __shared__ float sm_m[kAtWarps][ROWS], sm_l[kAtWarps][ROWS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const Span& s = w.s;
    const int b = w.b, head = w.head, r0 = w.r0, rows = s.nq * p.group, first = w.first, last = w.last;
    const int i0 = p.by_group(r0), i1 = p.by_group(min(r0 + ROWS, rows) - 1);

    // ---- the rows' queries: lane (g, t) holds row g of each eight, dimensions t D/4 .., divided by 2^e ----
    uint32_t qf[QS ? 1 : NQ][STEPS][2];
    uint2* const qsm = reinterpret_cast<uint2*>(reinterpret_cast<char*>(dsm) + kAtWarps * kAtStages * S::BYTES);
    int q_exp[NQ][2];  // e per column of the score tiles (rows 2t, 2t + 1)
    int pos[NQ][2];    // last key that the row sees (-1: no row, or none; never less, so that pos - window is an int)
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int r = r0 + 8 * n + g;
        uint32_t x8[D / 8];
        if (r < rows) {
            const int i = p.by_group(r), h = head * p.group + (r - i * p.group);
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (s.q0 + i) * p.q_row_stride + h * p.q_head_stride + t * (D / 4));
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const uint4 x = __ldg(src + j);
                x8[4 * j] = x.x;
                x8[4 * j + 1] = x.y;
                x8[4 * j + 2] = x.z;
                x8[4 * j + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < D / 8; ++j) x8[j] = 0;
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) top = max(top, max((x8[j] & 0x7FFFu) << 16, x8[j] & 0x7FFF0000u));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const int e = min(max((int)(top >> 23), 1), 253) - 127;
        const float down = pow2i(-e);
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            uint32_t f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t x = x8[2 * st + k];
                f[k] = pack_h2(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xFFFF0000u) * down);
            }
            if constexpr (QS) {
                if (warp == n) qsm[(n * STEPS + st) * 32 + lane] = make_uint2(f[0], f[1]);
            } else {
                qf[n][st][0] = f[0];
                qf[n][st][1] = f[1];
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int col = 2 * t + k, rr = r0 + 8 * n + col;
            q_exp[n][k] = __shfl_sync(0xFFFFFFFFu, e, 4 * col);
            pos[n][k] = rr < rows ? max(s.len - s.n + p.by_group(rr), -1) : -1;
        }
    }
    if constexpr (QS) __syncthreads();

    float o[NQ][TILES][4], l[NQ][2];
    float m[NQ][2], thr[NQ][2];  // running maximum (0 before the first key) and what a score may exceed it by
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int u = 0; u < TILES; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[n][u][k] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            m[n][k] = l[n][k] = 0.f;
            thr[n][k] = -INFINITY;
        }
    }
    int kref = -1000, vref = -1000;   // block scales are taken relative to these bytes
    int klim = -1, vlim = -1;         // and may be at most these
    float mk[NQ][2];                  // scale * log2(e) * 2^(q_exp + kref - 127)
#pragma unroll
    for (int n = 0; n < NQ; ++n) mk[n][0] = mk[n][1] = 0.f;
    uint32_t vnan = 0;                // bit 2n + k: a value block that row sees is NaN

    // groups of which every row sees every key (in a page of the cache)
    const int pos_lo = s.len - s.n + i0, pos_hi = s.len - s.n + i1;
    const int whole_hi = min(s.len, pos_lo + 1) >> 4, whole_lo = p.window > 0 ? ((max(pos_hi, -1) - p.window) >> 4) + 1 : 0;
    const KeyRange seen_by_some = keys_seen(p, s, i0, i1);
    const uint32_t ring = smem_u32(dsm) + warp * kAtStages * S::BYTES;
    int places = -1;            // lane j: place in the cache (in groups; -1: none) of the warp's group 32 * (issued / 32) + j
    int issued = 0;             // groups of this warp whose copies are issued
    uint32_t there = 0;         // bit j: the group issued j before the last is in a page of the cache
    uint32_t put = ring;
    const Fetch<D> from(p.c, lane);
    auto issue = [&] {
        if ((issued & 31) == 0) {
            const int grp = first + warp + (issued + lane) * kAtWarps;
            places = -1;
            if (grp < last) {
                const int key = 16 * grp, at = p.by_page(key);
                const int pg = __ldg(p.table + b * p.table_stride + at);
                if (pg >= 0 && pg < p.c.pages)
                    places = (int)((((long long)pg * p.c.heads + head) * p.c.page + (key - at * p.c.page)) >> 4);
            }
        }
        const int place = __shfl_sync(0xFFFFFFFFu, places, issued & 31);
        if (place >= 0) from.copy(place, put);
        there = (there << 1) | (place >= 0 ? 1u : 0u);
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++issued;
        put = put + S::BYTES == ring + kAtStages * S::BYTES ? ring : put + S::BYTES;
    };
#pragma unroll
    for (int i = 0; i < kAtStages - 1; ++i) issue();
    __shared__ Spread spreads[MIXED ? kAtWarps : 1][2];
    const bool mixed = MIXED && i1 > i0;
    if (mixed) note_spread<D>(p, s, b, head, i0, i1, 16 * first, 16 * last, threadIdx.x, kAtThreads, spreads);
    uint32_t stage = ring;
    const int kr = 4 * (g >> 1) + (g & 1);  // the lane's keys of the score tiles: kr, kr + 2
    const uint32_t k_at = S::K + kr * S::ROW + t * (S::ROW / 4), ks_at = S::KS + kr * S::SROW + (D == 128 ? t : t >> 1);
    const uint32_t vs_at = S::VS + 4 * t * S::SROW, v_sel = 0x4440u + (D == 128 ? g >> 1 : g >> 2);
    for (int grp = first + warp; grp < last; grp += kAtWarps) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAtStages - 2) : "memory");
        __syncwarp();  // every lane's copies of this group have landed, and the group before is read by every lane
        issue();
        const bool in_page = (there >> (kAtStages - 1)) & 1u;
        const int key0 = 16 * grp;
        uint32_t ks[2], vs[4];
        ks[0] = lds8(stage + ks_at);
        ks[1] = lds8(stage + ks_at + 2 * S::SROW);
        if constexpr (D == 128) {
            const uint4 w = lds128u(stage + vs_at);
            vs[0] = prmt(w.x, v_sel);
            vs[1] = prmt(w.y, v_sel);
            vs[2] = prmt(w.z, v_sel);
            vs[3] = prmt(w.w, v_sel);
        } else {
            const uint2 w = lds64(stage + vs_at);
            vs[0] = prmt(w.x, v_sel);
            vs[1] = prmt(w.x, v_sel + 2);
            vs[2] = prmt(w.y, v_sel);
            vs[3] = prmt(w.y, v_sel + 2);
        }
        const bool whole = in_page && grp < whole_hi && grp >= whole_lo;
        if (!whole) {  // bytes of keys that no row of the tile sees count as zeros
            const int end = in_page ? seen_by_some.hi - key0 : 0, begin = seen_by_some.lo - key0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (kr + 2 * i >= end || kr + 2 * i < begin) ks[i] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * t + i >= end || 4 * t + i < begin) vs[i] = 0;
        }
        if (__any_sync(0xFFFFFFFFu, (int)max(ks[0], ks[1]) > klim || (int)max(max(vs[0], vs[1]), max(vs[2], vs[3])) > vlim)) {
            // raise the references where a block (NaN blocks aside) exceeds 2^13 of them
            int kt = -1, vt = -1;
#pragma unroll
            for (int i = 0; i < 2; ++i) kt = max(kt, ks[i] == 0xFFu ? -1 : (int)ks[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) vt = max(vt, vs[i] == 0xFFu ? -1 : (int)vs[i]);
            kt = __reduce_max_sync(0xFFFFFFFFu, kt);
            if (kt > kref + 13) {
                kref = kt - 6;
                klim = min(kref + 13, 254);
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) mk[n][k] = p.scale * pow2i(min(q_exp[n][k] + kref - 127, 127));
            }
            vt = __reduce_max_sync(0xFFFFFFFFu, vt);
            if (vt > vref + 13) {
                const float f = pow2i(vref - (vt - 6));  // 0 the first time: the sums are 0
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int u = 0; u < TILES; ++u)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[n][u][k] *= f;
                vref = vt - 6;
                vlim = min(vref + 13, 254);
            }
            // a NaN block of V makes its 32 dimensions NaN for the rows that see its key, and for no others
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                    const bool bad = __shfl_sync(0xFFFFFFFFu, vs[i], (lane & ~3) | tt) == 0xFFu;
                    const int key = key0 + 4 * tt + i;
                    if (bad)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                if (key <= pos[n][k] && (p.window <= 0 || key > pos[n][k] - p.window)) vnan |= 1u << (2 * n + k);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (vs[i] == 0xFFu) vs[i] = 0;
        }
        // ---- scores: keys x rows ----
        float sc[NQ][4];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[n][k] = 0.f;
        {
            uint32_t f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = ks[i] == 0xFFu ? __uint_as_float(0x7FC00000u) : rel_scale((int)ks[i], kref);
                f[i] = pack_h2(x, x);
            }
            uint32_t kw[2][D / 32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (D == 128) {
                    const uint4 x = lds128u(stage + k_at + 2 * i * S::ROW);
                    kw[i][0] = x.x;
                    kw[i][1] = x.y;
                    kw[i][2] = x.z;
                    kw[i][3] = x.w;
                } else {
                    const uint2 x = lds64(stage + k_at + 2 * i * S::ROW);
                    kw[i][0] = x.x;
                    kw[i][1] = x.y;
                }
            }
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                uint32_t a[4], c[4];
                e2m1_to_h2(kw[0][j], a);
                e2m1_to_h2(kw[1][j], c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[k] = mul_h2(a[k], f[0]);
                    c[k] = mul_h2(c[k], f[1]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        uint32_t b0, b1;
                        if constexpr (QS) {
                            const uint2 x = qsm[(n * STEPS + 2 * j + h) * 32 + lane];
                            b0 = x.x;
                            b1 = x.y;
                        } else {
                            b0 = qf[n][2 * j + h][0];
                            b1 = qf[n][2 * j + h][1];
                        }
                        mma16816(sc[n], a[2 * h], c[2 * h], a[2 * h + 1], c[2 * h + 1], b0, b1);
                    }
            }
        }
        // ---- weights ----
        float e[NQ][4];
        bool up = false;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                e[n][k] = weight_exponent(sc[n][k], mk[n][k & 1], m[n][k & 1]);
                if (!whole) {
                    const int key = key0 + kr + (k & 2);
                    const bool seen = in_page && key <= pos[n][k & 1] && (p.window <= 0 || key > pos[n][k & 1] - p.window);
                    if (!seen) e[n][k] = -INFINITY;
                }
            }
            up |= fmaxf(e[n][0], e[n][2]) > thr[n][0] || fmaxf(e[n][1], e[n][3]) > thr[n][1];
        }
        if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float x = fmaxf(e[n][k], e[n][k + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
                    // x is relative to the maximum so far; before the first key there is none
                    const bool begun = thr[n][k] > 0.f;
                    if (x == -INFINITY || (begun && x <= 0.f)) continue;
                    const float f = begun ? ex2(-x) : 0.f;
                    m[n][k] += x;
                    thr[n][k] = 8.f;
                    l[n][k] *= f;
#pragma unroll
                    for (int u = 0; u < TILES; ++u) {
                        o[n][u][k] *= f;
                        o[n][u][k + 2] *= f;
                    }
                    if (e[n][k] != -INFINITY) e[n][k] = weight_exponent(sc[n][k], mk[n][k], m[n][k]);
                    if (e[n][k + 2] != -INFINITY) e[n][k + 2] = weight_exponent(sc[n][k + 2], mk[n][k], m[n][k]);
                }
            }
        }
        uint32_t pb[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int k = 0; k < 4; ++k) e[n][k] = ex2(e[n][k]);
            l[n][0] += e[n][0] + e[n][2];
            l[n][1] += e[n][1] + e[n][3];
            pb[n][0] = transpose8x8(pack_h2(e[n][0], e[n][1]));
            pb[n][1] = transpose8x8(pack_h2(e[n][2], e[n][3]));
        }
        // ---- sums: dimensions x rows ----
        {
            const uint32_t f0 = pack_h2(rel_scale((int)vs[0], vref), rel_scale((int)vs[1], vref));
            const uint32_t f1 = pack_h2(rel_scale((int)vs[2], vref), rel_scale((int)vs[3], vref));
            uint32_t vw[4][D / 64];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == 128) {
                    const uint2 x = lds64(stage + S::v_at(4 * t + i, g >> 1) + 8 * (g & 1));
                    vw[i][0] = x.x;
                    vw[i][1] = x.y;
                } else {
                    vw[i][0] = lds32(stage + S::v_at(4 * t + i, g >> 2) + 4 * (g & 3));
                }
            }
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                uint32_t e0[4], e1[4], d0[4], d1[4];  // even, odd dimensions of keys 4t, 4t + 1 and 4t + 2, 4t + 3
                e2m1_to_h2((vw[0][j] & 0x0F0F0F0Fu) | ((vw[1][j] << 4) & 0xF0F0F0F0u), e0);
                e2m1_to_h2((vw[2][j] & 0x0F0F0F0Fu) | ((vw[3][j] << 4) & 0xF0F0F0F0u), e1);
                e2m1_to_h2(((vw[0][j] >> 4) & 0x0F0F0F0Fu) | (vw[1][j] & 0xF0F0F0F0u), d0);
                e2m1_to_h2(((vw[2][j] >> 4) & 0x0F0F0F0Fu) | (vw[3][j] & 0xF0F0F0F0u), d1);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a0 = mul_h2(e0[k], f0), a1 = mul_h2(d0[k], f0), a2 = mul_h2(e1[k], f1), a3 = mul_h2(d1[k], f1);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) mma16816(o[n][4 * j + k], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                }
            }
        }
        stage = stage + S::BYTES == ring + kAtStages * S::BYTES ? ring : stage + S::BYTES;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // (the last ones are empty)
    // from here on a row without a key has the maximum -inf
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (!(thr[n][k] > 0.f)) m[n][k] = -INFINITY;

    // ---- join the warps ----
    const float vtrue = scale_of(vref);
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int d = 4; d < 32; d *= 2) l[n][k] += __shfl_xor_sync(0xFFFFFFFFu, l[n][k], d);
            if (g == 0) {
                sm_m[warp][8 * n + 2 * t + k] = m[n][k];
                sm_l[warp][8 * n + 2 * t + k] = l[n][k];
            }
        }
    __syncthreads();
    if (mixed && spread_beyond<MIXED ? kAtWarps : 1>(spreads, kAtRoom, kAtRoom)) {
        for (int r = warp; r < min(ROWS, rows - r0); r += kAtWarps)
            exact_row<D>(p, s, b, head, r0 + r, 16 * first, 16 * last, w.alone, w.slot * ROWS + r);
        return;
    }
    float* const mine = dsm + warp * ROWS * (D + 4);
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = 8 * n + 2 * t + k;
            float top = sm_m[0][r];
#pragma unroll
            for (int q = 1; q < kAtWarps; ++q) top = fmaxf(top, sm_m[q][r]);
            // a warp without a visible key has sums of 0 (or NaN, which stays)
            float f = m[n][k] == -INFINITY ? 1.f : ex2(m[n][k] - top);
            if (vnan & (1u << (2 * n + k))) f = __uint_as_float(0x7FC00000u);
            // the lane's dimensions g D/8 ..: tile 4j + q holds 8j + 2q (first eight rows of the tile) and the next
#pragma unroll
            for (int j = 0; j < TILES; j += 2)
                *reinterpret_cast<float4*>(mine + res_off<D>(r, g * (D / 8) + 2 * j)) =
                    make_float4(o[n][j][k] * f * vtrue, o[n][j][k + 2] * f * vtrue, o[n][j + 1][k] * f * vtrue, o[n][j + 1][k + 2] * f * vtrue);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * (D / 4); i += kAtThreads) {
        const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
        if (r0 + r >= rows) break;
        float top = sm_m[0][r];
#pragma unroll
        for (int q = 1; q < kAtWarps; ++q) top = fmaxf(top, sm_m[q][r]);
        float total = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < kAtWarps; ++q) {
            total += sm_l[q][r] * (sm_m[q][r] == -INFINITY ? 1.f : ex2(sm_m[q][r] - top));
            const float4 x = *reinterpret_cast<const float4*>(dsm + q * ROWS * (D + 4) + res_off<D>(r, d));
            a.x += x.x;
            a.y += x.y;
            a.z += x.z;
            a.w += x.w;
        }
        if (w.alone) {
            const float inv = total == 0.f ? 0.f : 1.f / total;
            const int tok = p.by_group(r0 + r), h = head * p.group + (r0 + r - tok * p.group);
            const long long at = (long long)(s.q0 + tok) * p.heads + h;
            *reinterpret_cast<uint2*>(p.out + at * D + d) = make_uint2(bf16x2(a.x * inv, a.y * inv), bf16x2(a.z * inv, a.w * inv));
            if (p.lse && d == 0) p.lse[at] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
        } else {
            const long long at = w.slot * ROWS + r;
            *reinterpret_cast<float4*>(p.part + at * D + d) = a;
            if (d == 0) *reinterpret_cast<float2*>(p.part + p.part_ml + at * 2) = make_float2(top, total);
        }
    }
}

// groups that the queries of sequence b see
__device__ __forceinline__ Groups groups_in(const AtArgs& p, const Span& s) {
    if (s.nq > 0) return groups_of(p, s, 0, s.nq - 1);
    return {0, 0, 0};
}

// the share of CTA blockIdx.x of all groups, (sequence, head, group) in order
template <int D, int NQ, bool MIXED> __device__ __forceinline__ void attend_share(const AtArgs& p) {
    __shared__ long long pre[kAtMaxEven + 1];  // groups of the sequences before, one head
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    constexpr int PER = kAtMaxEven / kAtThreads;
    int n[PER], sum = 0;  // 2^27 groups a sequence at most; the sums below are 64-bit where they can pass 32
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = t * PER + i;
        n[i] = 0;
        if (b < p.batch) {
            const Groups g = groups_in(p, span_of(p, b));
            n[i] = g.hi - g.lo;
        }
        sum += n[i];
    }
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += x;
    }
    __shared__ long long warp_total[kAtWarps];
    __shared__ int warp_filled[kAtWarps];
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    long long at = incl - sum;
    for (int w = 0; w < warp; ++w) at += warp_total[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = t * PER + i;
        if (b <= p.batch) pre[b] = at;
        at += n[i];
    }
    if (t == kAtThreads - 1 && p.batch == kAtMaxEven) pre[kAtMaxEven] = at;
    int filled = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) filled += n[i] > 0;
    filled = __reduce_add_sync(0xFFFFFFFFu, filled);
    if (lane == 0) warp_filled[warp] = filled;
    __syncthreads();
    int some = 0;  // sequences with a key
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) some += warp_filled[w];
    // sequences without a key, and rows that nobody computes
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        const bool none = pre[b + 1] == pre[b];
        if (none || p.fill) {
            const Span s = span_of(p, b);
            if (none) zero_rows<D>(p, s.q0, s.q0 + s.nq, 0, p.heads);
            if (p.fill) fill_rows<D>(p, s, b, 0, p.heads);
        }
    }
    const long long total = pre[p.batch] * p.c.heads;
    // kEvenGroups groups a share, but a share for each sequence and head with a key if the grid has them (a piece takes as
    // long as several groups); never more shares than groups: each has one
    const long long want = max((total + kEvenGroups - 1) / kEvenGroups, (long long)some * p.c.heads);
    const long long shares = min((long long)gridDim.x, want), c = blockIdx.x;
    int4 info = make_int4(-1, 0, 0, 0);
    if (c < shares) {
        const long long end = total * (c + 1) / shares;
        long long u = total * c / shares;
        for (bool begin = true; u < end; begin = false) {
            int lo = 0, hi = p.batch - 1;  // the last sequence that begins at or before u (those without a group lie before it)
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pre[mid] * p.c.heads <= u) lo = mid;
                else hi = mid - 1;
            }
            Piece w;
            w.b = lo;
            const int len = (int)(pre[lo + 1] - pre[lo]);
            const long long rel = u - pre[lo] * p.c.heads;
            w.head = (int)(rel / len);
            const int g0 = (int)(rel - (long long)w.head * len), g1 = (int)min((long long)len, g0 + (end - u));
            w.s = span_of(p, lo);
            w.r0 = 0;
            const Groups g = groups_in(p, w.s);
            w.first = g.lo + g0;
            w.last = g.lo + g1;
            w.alone = g0 == 0 && g1 == len;
            w.slot = 2 * c + (g0 > 0 ? 0 : 1);
            if (begin && g0 > 0) {
                const long long t0 = u - g0, t1 = t0 + len;  // the tile's units; shares c' with total c' / shares <= unit
                info = make_int4(lo, w.head, total * (c - 1) / shares <= t0, (int)((t1 * shares - 1) / total));
            }
            if (!begin) __syncthreads();  // the piece before is out of shared memory
            attend<D, NQ, MIXED>(p, w);
            u += g1 - g0;
        }
    }
    if (t == 0) p.info[c] = info;
}

template <int D, int NQ, bool MIXED> __global__ void __launch_bounds__(kAtThreads, NQ == 4 ? 2 : NQ == 2 ? 3 : 4) k_kv_attention(const __grid_constant__ AtArgs p) {
    pdl_wait_then_release();
    if (NQ < 4 && p.even) {
        attend_share<D, NQ, MIXED>(p);
        return;
    }
    Piece w;
    const int tile = p.by_splits(blockIdx.x), sp = blockIdx.x - tile * p.splits;
    const int bh = p.by_tiles(tile), rt = tile - bh * p.row_tiles;
    w.b = p.by_heads(bh);
    w.head = bh - w.b * p.c.heads;
    w.s = span_of(p, w.b);
    const int rows = w.s.nq * p.group;
    w.r0 = rt * 8 * NQ;
    if (p.fill && rt == 0 && sp == 0) fill_rows<D>(p, w.s, w.b, w.head * p.group, p.group);
    if (w.r0 >= rows) return;
    const Groups gr = groups_of(p, w.s, p.by_group(w.r0), p.by_group(min(w.r0 + 8 * NQ, rows) - 1));
    w.first = gr.lo + sp * gr.per;
    w.last = min(w.first + gr.per, gr.hi);
    w.alone = gr.hi - gr.lo <= gr.per;  // one split holds all keys
    w.slot = blockIdx.x;
    if (w.first >= w.last && sp > 0) return;
    attend<D, NQ, MIXED>(p, w);
}

// ---- joining ------------------------------------------------------------------------------------

template <int D> struct Joined {
    static constexpr int PER = D / 32;  // dimensions of a lane
    float top, total, sum[PER];
};
// the sum of a row's pieces: its maximum, total and the lane's D / 32 dimensions. `at(q)` is piece q's row of the partial
// sums; this warp takes the pieces lo .. hi - 1 of n (the maximum is over all)
template <int D, typename At> __device__ __forceinline__ Joined<D> join_pieces(const AtArgs& p, int n, int lo, int hi, At at) {
    constexpr int PER = D / 32, AHEAD = 8;  // loads in flight
    using Vec = std::conditional_t<PER == 4, float4, float2>;
    const int lane = threadIdx.x & 31;
    const float2* const ml = reinterpret_cast<const float2*>(p.part + p.part_ml);
    const Vec* const part = reinterpret_cast<const Vec*>(p.part) + lane;
    Joined<D> r;
    r.top = -INFINITY;
    for (int q = lane; q < n; q += 32) r.top = fmaxf(r.top, __ldcg(&ml[at(q)]).x);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) r.top = fmaxf(r.top, __shfl_xor_sync(0xFFFFFFFFu, r.top, d));
    r.total = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) r.sum[k] = 0.f;
    for (int q0 = lo; q0 < hi; q0 += 32) {
        float f = 0.f;
        if (q0 + lane < hi) {
            const float2 x = __ldcg(&ml[at(q0 + lane)]);
            f = x.x == -INFINITY ? 1.f : ex2(x.x - r.top);
            r.total += x.y * f;
        }
        const int m = min(32, hi - q0);
        for (int q1 = 0; q1 < m; q1 += AHEAD) {
            Vec x[AHEAD];
#pragma unroll
            for (int q = 0; q < AHEAD; ++q)
                if (q1 + q < m) x[q] = __ldcg(part + at(q0 + q1 + q) * 32);
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                const float fq = __shfl_sync(0xFFFFFFFFu, f, (q1 + q) & 31);
                if (q1 + q >= m) continue;
                r.sum[0] += x[q].x * fq;
                r.sum[1] += x[q].y * fq;
                if constexpr (PER == 4) {
                    r.sum[2] += x[q].z * fq;
                    r.sum[3] += x[q].w * fq;
                }
            }
        }
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) r.total += __shfl_xor_sync(0xFFFFFFFFu, r.total, d);
    return r;
}
template <int D> __device__ __forceinline__ void write_joined(const AtArgs& p, const Joined<D>& r, long long at) {
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const float inv = r.total == 0.f ? 0.f : 1.f / r.total;
    uint32_t out[PER / 2];
#pragma unroll
    for (int k = 0; k < PER / 2; ++k) out[k] = bf16x2(r.sum[2 * k] * inv, r.sum[2 * k + 1] * inv);
    if constexpr (PER == 4) reinterpret_cast<uint2*>(p.out + at * D)[lane] = make_uint2(out[0], out[1]);
    else reinterpret_cast<uint32_t*>(p.out + at * D)[lane] = out[0];
    if (p.lse && lane == 0) p.lse[at] = r.total == 0.f ? -INFINITY : (r.top + log2f(r.total)) * kLn2;
}
// adds what the other warps of a row summed, in their order: warp `w` of W; `others` is the row's, [W][D + 1]. All of the
// CTA's threads call it; warp 0 has the result.
template <int D, int W> __device__ __forceinline__ void join_warps(Joined<D>& r, int w, float* others) {
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < PER; ++k) others[w * (D + 1) + PER * lane + k] = r.sum[k];
    if (lane == 0) others[w * (D + 1) + D] = r.total;
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int v = 1; v < W; ++v) {
        r.total += others[v * (D + 1) + D];
#pragma unroll
        for (int k = 0; k < PER; ++k) r.sum[k] += others[v * (D + 1) + PER * lane + k];
    }
}

// the sequences that shares split: share c's first piece names one; the share where it was split first joins it. Four
// warps take a row, two rows to a CTA.
template <int D, int NQ> __global__ void __launch_bounds__(256) k_kv_attention_join_shares(const AtArgs p) {
    constexpr int ROWS = 8 * NQ, W = 4;
    __shared__ float others[2][W][D + 1];
    pdl_wait_then_release();
    const int c = blockIdx.x + 1;
    const int4 info = __ldcg(p.info + c);
    if (info.x < 0 || !info.z) return;
    const int warp = threadIdx.x >> 5, w = warp & 3, row = blockIdx.y * 2 + (warp >> 2);
    const Span s = span_of(p, info.x);
    const bool there = row < s.nq * p.group;
    // pieces: the last of share c - 1, the first of shares c .. info.w
    const int n = there ? info.w - c + 2 : 0, per = (n + W - 1) / W;
    Joined<D> r = join_pieces<D>(p, n, w * per, min((w + 1) * per, n),
                                 [&](int q) { return (q == 0 ? 2LL * c - 1 : 2LL * (c - 1 + q)) * ROWS + row; });
    join_warps<D, W>(r, w, &others[warp >> 2][0][0]);
    if (w > 0 || !there) return;
    const int i = p.by_group(row), h = info.y * p.group + row - i * p.group;
    write_joined<D>(p, r, (long long)(s.q0 + i) * p.heads + h);
}

// the splits of each row (sequence, query, head); W: warps that share a row's splits (4 where rows are few, else 1)
template <int D, int ROWS, int W> __global__ void __launch_bounds__(kAtThreads) k_kv_attention_join(const AtArgs p) {
    __shared__ float others[W][D + 1];
    const int w = W == 1 ? 0 : threadIdx.x >> 5;
    pdl_wait_then_release();
    int id = W == 1 ? blockIdx.x * kAtWarps + (threadIdx.x >> 5) : blockIdx.x;
    const int h = id % p.heads;
    id /= p.heads;
    const int i = id % p.max_q, b = id / p.max_q;
    if (b >= p.batch) return;
    const Span s = span_of(p, b);
    if (i >= s.nq) return;
    const int head = h / p.group, row = i * p.group + h - head * p.group, rt = row / ROWS, r0 = rt * ROWS;
    constexpr bool TC = ROWS == kTileRows;
    const Groups gr = groups_of<TC ? kTileKeysShift : 4, TC ? kTileMinBlocks : kAtMinGroups>(
        p, s, p.by_group(r0), p.by_group(min(r0 + ROWS, s.nq * p.group) - 1));
    const int n = (gr.hi - gr.lo + gr.per - 1) / gr.per;
    if (n <= 1) return;  // written by its split
    const long long first = (((long long)b * p.c.heads + head) * p.row_tiles + rt) * p.splits * ROWS + (row - r0);
    const int per = (n + W - 1) / W;
    Joined<D> r = join_pieces<D>(p, n, w * per, min((w + 1) * per, n), [&](int q) { return first + (long long)q * ROWS; });
    if constexpr (W > 1) {
        join_warps<D, W>(r, w, &others[0][0]);
        if (w > 0) return;
    }
    write_joined<D>(p, r, (long long)(s.q0 + i) * p.heads + h);
}

// eights of rows per tile; more than 32 rows: the kernel that decodes a block of keys for 256 of them at once
constexpr int kNqTiles = kTileRows / 8;
int nq_of(long long rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : kNqTiles; }

// Splits of many-query tiles: those whose waves are over first; a CTA's start and end take about as long as kTileEnds
// blocks of keys.
constexpr long long kTileWaves = 4, kTileEnds = 4;
// No number of blocks up to `blocks` gets more splits than this. In w waves there are at most c = w sms / tiles splits,
// which end after w (ends + b / c) or later; in v < w waves, d = v sms / tiles splits end before v (ends + 1 + b / d). So w
// can win at b only if the first is below the second, and since v (ends + 1) <= w ends, then also at every larger b.
long long most_splits(long long tiles, long long blocks, int sms) {
    long long most = 1;
    for (long long w = 1; w <= kTileWaves; ++w) {
        const long long c = w * sms / tiles;
        bool wins = c > most;
        for (long long v = 1; v < w && wins; ++v) {
            const long long d = v * sms / tiles;
            wins = d == 0 || w * (kTileEnds * c + blocks) * d < v * ((kTileEnds + 1) * d + blocks) * c;
        }
        if (wins) most = c;
    }
    return most;
}

struct Plan {
    int nq, row_tiles, splits, shares;  // shares > 0: equal shares instead of splits
    long long tiles, pieces;            // places for partial sums
};
// Rows of a key head in eights. One row tile per sequence: equal shares, one per place (16 sequences of 24576 to 32768
// keys: 145 us, 156 with splits). Otherwise, and for one sequence, where working out the shares only takes time (4000
// keys: 14.4 us against 20.2), the keys in splits of at least kAtMinGroups groups of 16 keys for one wave of CTAs, or of
// 32 groups or more for about two.
// at_most: the workspace that any smaller max_keys needs too.
Plan plan_of(const KvCache& c, long long batch, int max_q, int heads, long long max_keys, int sms, bool at_most = false) {
    Plan p{};
    const long long rows = (long long)max_q * (heads / c.heads);
    p.nq = nq_of(rows);
    p.row_tiles = (int)((rows + 8 * p.nq - 1) / (8 * p.nq));
    p.tiles = batch * c.heads * p.row_tiles;
    p.splits = 1;
    const long long groups = (max_keys + 15) / 16, tiles = p.tiles > 0 ? p.tiles : 1;
    const long long places = (long long)sms * (p.nq == 4 ? 2 : p.nq == 2 ? 3 : 4);  // resident CTAs
    if (p.nq < 4 && batch > 1 && batch <= kAtMaxEven && groups > kAtMinGroups) {
        const long long by_groups = (tiles * groups + kEvenGroups - 1) / kEvenGroups, most = by_groups > tiles ? by_groups : tiles;
        p.shares = (int)(most < places ? most : places);
        p.pieces = 2LL * p.shares;
        return p;
    }
    if (p.nq == kNqTiles) {
        // one CTA per SM
        const long long blocks = (max_keys + 127) / 128;
        long long most = blocks / kTileMinBlocks, best = 0;
        if (most > kAtMaxSplits) most = kAtMaxSplits;
        if (at_most) {
            p.splits = (int)most_splits(tiles, blocks, sms);
            if (p.splits > most) p.splits = most > 1 ? (int)most : 1;
            p.pieces = p.splits > 1 ? p.tiles * p.splits : 0;
            return p;
        }
        for (long long n = 1; n <= most || n == 1; ++n) {
            const long long waves = (tiles * n + sms - 1) / sms, time = waves * (kTileEnds + (blocks + n - 1) / n);
            if (n > 1 && waves > kTileWaves) break;
            if (n == 1 || time < best) {
                best = time;
                p.splits = (int)n;
            }
        }
        p.pieces = p.splits > 1 ? p.tiles * p.splits : 0;
        return p;
    }
    long long one = places / tiles, two = 2 * places / tiles;
    if (one > groups / kAtMinGroups) one = groups / kAtMinGroups;
    if (two > groups / 32) two = groups / 32;
    long long want = one > two ? one : two;
    if (want > kAtMaxSplits) want = kAtMaxSplits;
    if (want > 1) p.splits = (int)want;
    p.pieces = p.splits > 1 ? p.tiles * p.splits : 0;
    return p;
}

template <int D, int ROWS> cudaError_t join(const AtArgs& a, cudaStream_t st) {
    const long long rows = (long long)a.batch * a.max_q * a.heads;
    if (rows > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    if (rows < kJoinRows) return launch_pdl(k_kv_attention_join<D, ROWS, kAtWarps>, (unsigned)rows, kAtThreads, st, a);
    return launch_pdl(k_kv_attention_join<D, ROWS, 1>, (unsigned)((rows + kAtWarps - 1) / kAtWarps), kAtThreads, st, a);
}

template <int D, int NQ, bool MIXED> cudaError_t go(const AtArgs& a, const Plan& pl, int dev, cudaStream_t st) {
    constexpr int RES = kAtWarps * 8 * NQ * (D + 4) * 4;
    constexpr int IN = kAtWarps * kAtStages * AtStage<D>::BYTES + (NQ == 4 ? NQ * (D / 16) * 32 * 8 : 0);
    constexpr int SMEM = RES > IN ? RES : IN;
    auto* kern = k_kv_attention<D, NQ, MIXED>;
    static std::atomic<unsigned long long> ready{0};
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    if (pl.tiles * a.splits > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pl.shares > 0 ? pl.shares : pl.tiles * a.splits));
    cfg.blockDim = dim3(kAtThreads);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e != cudaSuccess || pl.pieces == 0 || pl.shares == 1) return e;
    cfg.dynamicSmemBytes = 0;
    if (pl.shares == 0) return join<D, 8 * NQ>(a, st);
    cfg.gridDim = dim3((unsigned)(pl.shares - 1), (unsigned)((a.max_q * a.group + 1) / 2));
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, k_kv_attention_join_shares<D, NQ>, a);
}
template <int D> cudaError_t go_tiles(const AtArgs& a, const Plan& pl, int dev, cudaStream_t st) {
    if (pl.tiles * a.splits > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    const cudaError_t e = launch_kv_attention_tiles(a, pl.tiles, dev, st);
    return e != cudaSuccess || pl.pieces == 0 ? e : join<D, kTileRows>(a, st);
}

int sm_count(int dev) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        sms = 148;
    }
    return sms;
}

}  // namespace

long long kv_attention_workspace(const KvCache& c, long long batch, int max_q, int heads, long long max_keys, bool at_most) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
    const Plan p = plan_of(c, batch, max_q, heads, max_keys, sm_count(dev), at_most);
    return p.pieces * 8 * p.nq * (c.db * 32 + 2) * 4 + p.shares * (long long)sizeof(int4);
}

cudaError_t launch_kv_attention(const KvAttention& x, cudaStream_t st) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const Plan pl = plan_of(x.c, x.batch, x.max_q, x.heads, x.max_keys, sm_count(dev));
    AtArgs a{};
    a.c = x.c;
    a.q = static_cast<const __nv_bfloat16*>(x.q);
    a.q_rows = x.q_rows;
    a.q_row_stride = x.q_row_stride;
    a.q_head_stride = x.q_head_stride;
    a.starts = x.starts;
    a.lens = x.lens;
    a.table = x.table;
    a.table_stride = x.table_stride;
    a.max_keys = x.max_keys;
    a.batch = (int)x.batch;
    a.heads = x.heads;
    a.group = x.heads / x.c.heads;
    a.max_q = x.max_q;
    a.window = x.window;
    a.fill = x.fill;
    a.splits = pl.splits;
    a.row_tiles = pl.row_tiles;
    a.scale = x.scale * kLog2e;
    a.out = static_cast<__nv_bfloat16*>(x.out);
    a.lse = x.lse;
    a.part = static_cast<float*>(x.workspace);
    a.part_ml = pl.pieces * 8 * pl.nq * (x.c.db * 32);
    a.even = pl.shares > 0;
    a.info = reinterpret_cast<int4*>(a.part + pl.pieces * 8 * pl.nq * (x.c.db * 32 + 2));
    a.by_group = FastDiv((uint32_t)a.group);
    a.by_page = FastDiv((uint32_t)x.c.page);
    a.by_splits = FastDiv((uint32_t)pl.splits);
    a.by_tiles = FastDiv((uint32_t)pl.row_tiles);
    a.by_heads = FastDiv((uint32_t)x.c.heads);
    if (x.c.db == 4) {
        if (pl.nq == 1) return a.max_q > 1 ? go<128, 1, true>(a, pl, dev, st) : go<128, 1, false>(a, pl, dev, st);
        if (pl.nq == 2) return a.max_q > 1 ? go<128, 2, true>(a, pl, dev, st) : go<128, 2, false>(a, pl, dev, st);
        if (pl.nq == 4) return a.max_q > 1 ? go<128, 4, true>(a, pl, dev, st) : go<128, 4, false>(a, pl, dev, st);
        return go_tiles<128>(a, pl, dev, st);
    }
    if (pl.nq == 1) return a.max_q > 1 ? go<64, 1, true>(a, pl, dev, st) : go<64, 1, false>(a, pl, dev, st);
    if (pl.nq == 2) return a.max_q > 1 ? go<64, 2, true>(a, pl, dev, st) : go<64, 2, false>(a, pl, dev, st);
    if (pl.nq == 4) return a.max_q > 1 ? go<64, 4, true>(a, pl, dev, st) : go<64, 4, false>(a, pl, dev, st);
    return go_tiles<64>(a, pl, dev, st);
}

}  // namespace mxq
