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

// many rows of a sequence and key head: 256 at a time, keys in blocks of 128 (mxq_attention_tc.cu)
constexpr int kTileRows = 256, kTileKeysShift = 7, kTileMinBlocks = 1;
cudaError_t launch_kv_attention_tiles(const AtArgs& a, long long tiles, int dev, cudaStream_t st);

}  // namespace mxq
