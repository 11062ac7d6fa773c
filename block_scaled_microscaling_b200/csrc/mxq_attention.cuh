// mxq_attention.cuh -- what the two kernels of attention over the MXFP4 cache share (sm_100a): arguments, the keys
// that rows see, decoding helpers.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mxq_device.cuh"
#include "mxq_ops_internal.h"
#include "mxq_tma.cuh"

namespace mxq {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kAtMinGroups = 8;    // groups of 16 keys that a split has at least

// n / d for 0 <= n < 2^31: with l = ceil(log2 d) and mul = ceil(2^(31 + l) / d), n * mul >> (31 + l) is exact
struct FastDiv {
    uint32_t mul, sh;
    FastDiv() : mul(1u << 31), sh(31) {}
    explicit FastDiv(uint32_t d) {
        uint32_t l = 0;
        while ((1ull << l) < d) ++l;
        sh = 31 + l;
        mul = (uint32_t)(((1ull << sh) + d - 1) / d);
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)(((unsigned long long)(uint32_t)n * mul) >> sh); }
};

struct AtArgs {
    KvCache c;
    FastDiv by_group, by_page, by_splits, by_tiles, by_heads;
    const __nv_bfloat16* q;
    long long q_rows, q_row_stride, q_head_stride;
    const int* starts;
    const int* lens;
    const int* table;
    long long table_stride;
    long long max_keys;
    int batch, heads, group, max_q, window, splits, row_tiles;
    bool fill;
    bool even;     // equal shares of all groups (one row tile per sequence and head)
    int4* info;    // even: of each share's first piece if its sequence began in an earlier share: sequence, head, whether
                   // that was the share just before, last share of the sequence; else sequence -1
    float scale;   // already times log2(e)
    __nv_bfloat16* out;
    float* lse;
    float* part;   // pieces' [rows][D] sums, then their [rows][2] maximum and total; piece of split s of tile t: t * splits
                   // + s; even: 2 c for the first piece of share c if its sequence began earlier, 2 c + 1 for its last
    long long part_ml;  // offset of the latter
};

// what a CTA (and the joining kernel) works out about its sequence and rows
struct Span {
    int q0, n, nq;   // first row of q, queries of the sequence, of which computed
    int len;         // keys
};
__device__ __forceinline__ Span span_of(const AtArgs& p, int b) {
    Span s;
    if (p.starts) {
        const int rows = (int)p.q_rows;
        s.q0 = min(max(__ldg(p.starts + b), 0), rows);
        s.n = min(max(__ldg(p.starts + b + 1), s.q0), rows) - s.q0;
    } else {
        s.q0 = b * p.max_q;
        s.n = p.max_q;
    }
    s.nq = min(s.n, p.max_q);
    s.len = (int)min((long long)max(__ldg(p.lens + b), 0), p.max_keys);
    return s;
}
// the keys lo .. hi - 1 are those that at least one of the queries i0 .. i1 sees
struct KeyRange {
    int lo, hi;
};
__device__ __forceinline__ KeyRange keys_seen(const AtArgs& p, const Span& s, int i0, int i1) {
    KeyRange k;
    k.hi = min(s.len, max(s.len - s.n + i1 + 1, 0));
    // 64 bits: the first query may stand far before the first key, and the window may be any int
    k.lo = p.window > 0 ? (int)min(max((long long)(s.len - s.n + i0 + 1) - p.window, 0LL), (long long)k.hi) : 0;
    return k;
}
// their groups of 2^SHIFT keys, and groups per split (MIN at least)
struct Groups {
    int lo, hi, per;
};
template <int SHIFT = 4, int MIN = kAtMinGroups> __device__ __forceinline__ Groups groups_of(const AtArgs& p, const Span& s, int i0, int i1) {
    const KeyRange k = keys_seen(p, s, i0, i1);
    Groups g;
    g.lo = k.lo >> SHIFT;
    g.hi = (k.hi + (1 << SHIFT) - 1) >> SHIFT;
    const int n = g.hi - g.lo;
    g.per = max((n + p.splits - 1) / p.splits, MIN);
    return g;
}

// zeros (and -inf) for rows lo .. hi of out, `nh` heads from h0 on
template <int D> __device__ void zero_rows(const AtArgs& p, int lo, int hi, int h0, int nh) {
    for (int r = lo; r < hi; ++r) {
        const long long at = (long long)r * p.heads + h0;
        for (int i = threadIdx.x; i < nh * (D / 8); i += blockDim.x)
            reinterpret_cast<uint4*>(p.out + at * D)[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int i = threadIdx.x; i < nh; i += blockDim.x) p.lse[at + i] = -INFINITY;
    }
}
// the rows that no CTA computes: beyond max_q in each sequence, before the first sequence, behind the last
template <int D> __device__ void fill_rows(const AtArgs& p, const Span& s, int b, int h0, int nh) {
    zero_rows<D>(p, s.q0 + s.nq, s.q0 + s.n, h0, nh);
    if (b == 0) zero_rows<D>(p, 0, s.q0, h0, nh);
    if (b == p.batch - 1) zero_rows<D>(p, s.q0 + s.n, (int)p.q_rows, h0, nh);
}

__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// the four bytes of x, each two E2M1 codes, as f16 pairs (low nibble in the low half)
__device__ __forceinline__ void e2m1_to_h2(uint32_t x, uint32_t* r) {
    asm("{ .reg .b8 c0, c1, c2, c3;\n mov.b32 {c0, c1, c2, c3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, c0;\n cvt.rn.f16x2.e2m1x2 %1, c1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c2;\n cvt.rn.f16x2.e2m1x2 %3, c3; }"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(x));
}
// 2^e for any integer e (clamped to the fp32 range, subnormals flushed)
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)min(max(e + 127, 0), 255) << 23); }
// 2^(byte - 127) of a reference scale byte of -149 .. 254: below 1 a subnormal, whose product with a normal sum is exact
__device__ __forceinline__ float scale_of(int byte) {
    return __uint_as_float(byte > 0 ? (uint32_t)byte << 23 : byte > -23 ? 1u << (byte + 22) : 0u);
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}


__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// ---- keys that only some rows of a tile see -------------------------------------------------------
//
// The rows of a tile share the powers of two that keys and values are decoded to. A key that only some of them see (the
// causal edge of a chunk, the lower edge of a window) may hold far larger blocks than the others see, and would cost
// those bits. So the kernels look at the scales of these keys, which are few (two for each query at most), and of up to
// kSpreadKeys keys that every row sees: the largest block of the former (`edge`), of the latter (`whole`), and the smallest
// of the former keys' largest blocks (`least`, keys of zeros aside). Every row that sees a key sees a block of `whole`, or of
// `least` where no key is seen by all: where `edge` exceeds that by more than `room`, the tile's rows are computed anew by
// exact_row, which shares nothing. That is slow (4 queries of 32 heads
// over 3000 keys 92 us for 18, 128 over 32768 keys 21 ms for 0.08) and does not happen with keys and values of one kind;
// the look itself takes up to 1 us a call (8 sequences of 4 queries over 8000 keys 47.5 us for 47.1, 4 prompts of 2000 tokens
// with a window of 512, whose CTAs are short, 181 for 175).
struct Spread {
    int whole, edge, least;
    __device__ __forceinline__ bool beyond(int room) const { return edge > (whole >= 0 ? whole : least) + room; }
};
constexpr int kSpreadKeys = 64;
// `out` [warps][2]: of K and V, for the queries i0 .. i1 (i1 > i0) over the keys first .. last - 1; `t` of `threads` threads,
// whole warps, call it
template <int D> __device__ __forceinline__ void note_spread(const AtArgs& p, const Span& s, int b, int head, int i0, int i1, int first, int last, int t, int threads, Spread (*out)[2]) {
    const KeyRange some = keys_seen(p, s, i0, i1);
    const int pos_lo = max(s.len - s.n + i0, -1), pos_hi = max(s.len - s.n + i1, -1);
    const int lo = max(some.lo, first), hi = max(min(some.hi, last), lo);
    // every row sees the keys all_lo .. all_hi - 1
    const int all_lo = min(max(p.window > 0 ? pos_hi - p.window + 1 : 0, lo), hi), all_hi = max(min(pos_lo + 1, hi), all_lo);
    const int below = all_lo - lo, edges = below + (hi - all_hi), n = edges + min(all_hi - all_lo, kSpreadKeys);
    int whole[2] = {-1, -1}, edge[2] = {-1, -1}, least[2] = {256, 256};
    constexpr int AHEAD = 2;  // keys of a thread whose loads are in flight
    for (int e0 = t; e0 < n; e0 += AHEAD * threads) {
        int at[AHEAD], off[AHEAD], pg[AHEAD];
        uint32_t w[AHEAD][2];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int e = e0 + u * threads;
            const int key = e < below ? lo + e : e < edges ? all_hi + (e - below) : all_hi - 1 - (e - edges);
            at[u] = p.by_page(key);
            off[u] = key - at[u] * p.c.page;
            pg[u] = -1;
            if (e < n) pg[u] = __ldg(p.table + b * p.table_stride + at[u]);
            if (pg[u] >= p.c.pages) pg[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const long long row = ((long long)max(pg[u], 0) * p.c.heads + head) * p.c.page + off[u];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const uint8_t* const scales = (v ? p.c.vs : p.c.ks) + row * (D / 32);
                w[u][v] = 0;
                if (pg[u] >= 0) w[u][v] = D == 128 ? *reinterpret_cast<const uint32_t*>(scales) : (uint32_t)*reinterpret_cast<const uint16_t*>(scales);
            }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (pg[u] < 0) continue;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                uint32_t x = w[u][v] & ~__vcmpeq4(w[u][v], 0xFFFFFFFFu);  // NaN blocks aside
                x = __vmaxu4(x, x >> 16);
                const int most = (int)max(x & 0xFFu, (x >> 8) & 0xFFu);
                if (e0 + u * threads >= edges) {
                    whole[v] = max(whole[v], most);
                } else {
                    edge[v] = max(edge[v], most);
                    if (most > 0) least[v] = min(least[v], most);
                }
            }
        }
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const Spread x{__reduce_max_sync(0xFFFFFFFFu, whole[v]), __reduce_max_sync(0xFFFFFFFFu, edge[v]), __reduce_min_sync(0xFFFFFFFFu, least[v])};
        if ((t & 31) == 0) out[t >> 5][v] = x;
    }
}
// whether the notes of W warps call for exact_row
template <int W> __device__ __forceinline__ bool spread_beyond(const Spread (*notes)[2], int room_k, int room_v) {
    bool beyond = false;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        Spread x = notes[0][v];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            x.whole = max(x.whole, notes[w][v].whole);
            x.edge = max(x.edge, notes[w][v].edge);
            x.least = min(x.least, notes[w][v].least);
        }
        beyond |= x.beyond(v ? room_v : room_k);
    }
    return beyond;
}
// by one warp: the row of rows (query x head of the group) `row` of a sequence over the keys first .. last - 1, in fp32
// throughout, to out (alone) or to row `part_row` of the partial sums. Lane d / (D / 32) holds dimension d.
template <int D> __device__ __forceinline__ void exact_row(const AtArgs& p, const Span s, int b, int head, int row, int first, int last, bool alone, long long part_row) {
    constexpr int PER = D / 32, KEYS = 8;  // keys at a time
    const int lane = threadIdx.x & 31;
    const int i = p.by_group(row), h = head * p.group + (row - i * p.group), pos = s.len - s.n + i;
    const int lo = p.window > 0 && pos >= p.window ? max(first, pos - p.window + 1) : first, hi = min(last, pos + 1);
    const uint16_t* const q16 = reinterpret_cast<const uint16_t*>(p.q + (s.q0 + i) * p.q_row_stride + h * p.q_head_stride) + lane * PER;
    float q[PER], o[PER], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int d = 0; d < PER; ++d) {
        q[d] = __uint_as_float((uint32_t)__ldg(q16 + d) << 16);
        o[d] = 0.f;
    }
    auto decode = [&](const char* codes, const uint8_t* scales, long long at, float* v) {
        const char* const c = codes + at * (D / 2) + lane * (PER / 2);
        const uint32_t byte = scales[at * (D / 32) + lane * PER / 32];
        const float f = byte == 0xFFu ? __uint_as_float(0x7FC00000u) : fwd_scale(byte);
        const uint32_t x = PER == 4 ? (uint32_t)*reinterpret_cast<const uint16_t*>(c) : (uint32_t)*reinterpret_cast<const uint8_t*>(c);
#pragma unroll
        for (int d = 0; d < PER; ++d) {  // twice the value of codes 0 .. 7: 0 1 2 3 4 6 8 12, a byte each
            const uint32_t code = x >> (4 * d), twice = __byte_perm(0x03020100u, 0x0C080604u, code & 7u) & 0xFFu;
            v[d] = (code & 8u ? -0.5f : 0.5f) * (float)twice * f;
        }
    };
    for (int j = lo; j < hi;) {
        const int at = p.by_page(j), off = j - at * p.c.page, n = min(hi - j, p.c.page - off);
        const int pg = __ldg(p.table + b * p.table_stride + at);
        j += n;
        if (pg < 0 || pg >= p.c.pages) continue;
        const long long place = ((long long)pg * p.c.heads + head) * p.c.page + off;
        for (int r = 0; r < n; r += KEYS) {  // (beyond the last key: the last again, which does not count)
            float v[KEYS][PER], x[KEYS];
#pragma unroll
            for (int u = 0; u < KEYS; ++u) {
                float k[PER];
                decode(p.c.kc, p.c.ks, place + min(r + u, n - 1), k);
                decode(p.c.vc, p.c.vs, place + min(r + u, n - 1), v[u]);
                x[u] = 0.f;
#pragma unroll
                for (int d = 0; d < PER; ++d) x[u] = fmaf(q[d], k[d], x[u]);
            }
#pragma unroll
            for (int d = 1; d < 32; d *= 2)
#pragma unroll
                for (int u = 0; u < KEYS; ++u) x[u] += __shfl_xor_sync(0xFFFFFFFFu, x[u], d);
            float top = m;
#pragma unroll
            for (int u = 0; u < KEYS; ++u) {
                x[u] = r + u < n ? x[u] * p.scale : -INFINITY;
                top = fmaxf(top, x[u]);
            }
            if (top > m) {
                const float f = ex2(m - top);
                m = top;
                l *= f;
#pragma unroll
                for (int d = 0; d < PER; ++d) o[d] *= f;
            }
#pragma unroll
            for (int u = 0; u < KEYS; ++u) {
                if (x[u] == -INFINITY) continue;
                const float w = ex2(x[u] - m);
                l += w;
#pragma unroll
                for (int d = 0; d < PER; ++d) o[d] = fmaf(w, v[u][d], o[d]);
            }
        }
    }
    if (alone) {
        const long long at = (long long)(s.q0 + i) * p.heads + h;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int d = 0; d < PER; ++d) p.out[at * D + lane * PER + d] = __float2bfloat16_rn(o[d] * inv);
        if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
#pragma unroll
        for (int d = 0; d < PER; ++d) p.part[part_row * D + lane * PER + d] = o[d];
        if (lane == 0) *reinterpret_cast<float2*>(p.part + p.part_ml + part_row * 2) = make_float2(m, l);
    }
}

// many rows of a sequence and key head: 256 at a time, keys in blocks of 128 (mxq_attention_tc.cu)
constexpr int kTileRows = 256, kTileKeysShift = 7, kTileMinBlocks = 1;
cudaError_t launch_kv_attention_tiles(const AtArgs& a, long long tiles, int dev, cudaStream_t st);

}  // namespace mxq
