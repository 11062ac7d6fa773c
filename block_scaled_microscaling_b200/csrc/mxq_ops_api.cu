// mxq_ops_api.cu -- the C ABI of the operators (declared in include/mxq_ops.h): argument checks on the host before
// any launch, size queries and dispatch to the launchers of mxq_matmul.cu, mxq_both.cu, mxq_swiglu.cu, mxq_kv.cu
// and mxq_attention.cu.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mxq_ops.h"
#include "mxq_check.h"
#include "mxq_ops_internal.h"

namespace {

constexpr int64_t kMaxInt = 0x7FFFFFFF;
// keys of a sequence: the kernels step over blocks of 128 in 32 bits, some blocks past the last
constexpr int64_t kMaxKeys = kMaxInt - 511;

bool product_format(mxq_format f) { return f == MXQ_MXFP4_E2M1 || f == MXQ_MXFP8_E4M3; }

bool product_shape_ok(int64_t m, int64_t n, int64_t k) {
    if (m < 0 || n < 0 || m >= kMaxInt - 256 || n >= kMaxInt - 256 || k >= kMaxInt - 512) return false;
    if (check_shape(m, k) != MXQ_OK || check_shape(n, k) != MXQ_OK) return false;
    return n == 0 || m <= kMaxElems / n;
}

struct Range {
    const void* p;
    size_t n;
};
// outputs may overlap neither an input nor one another
template <int NI, int NO> bool disjoint(const Range (&in)[NI], const Range (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (out[i].n && in[j].n && overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return false;
        for (int j = i + 1; j < NO; ++j)
            if (out[i].n && out[j].n && overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return false;
    }
    return true;
}

// bytes from the first value to the last of `rows` rows of `cols` values, `ld` apart
size_t span_bytes(int64_t rows, int64_t cols, int64_t ld, mxq_dtype d) {
    return rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * (size_t)dtype_bytes(d) : 0;
}
bool stride_ok(int64_t ld, int64_t cols, int64_t rows, mxq_dtype d) {
    return ld >= cols && ld <= kMaxElems / (rows > 0 ? rows : 1) && ld * dtype_bytes(d) % 16 == 0;
}
// two interleaved matrices of one row stride (halves of one): no row of one touches a row of the other
bool strided_disjoint(const void* a, const void* b, int64_t rows, int64_t cols, int64_t ld, mxq_dtype d) {
    const size_t n = span_bytes(rows, cols, ld, d);
    if (!overlap(a, n, b, n)) return true;
    const int64_t row = ld * dtype_bytes(d), w = cols * dtype_bytes(d);
    const int64_t x = (int64_t)((uintptr_t)a % (uintptr_t)row), y = (int64_t)((uintptr_t)b % (uintptr_t)row);
    const int64_t gap = x > y ? x - y : y - x;
    return gap >= w && row - gap >= w;
}

mxq_status check_cache(const mxq_kv_cache* c) {
    if (c == nullptr) return MXQ_ERR_INVALID_ARG;
    if (c->pages < 0 || c->kv_heads < 1 || c->page_size < 16 || c->page_size % 16 != 0 || c->page_size > 65536 || c->head_dim < 1)
        return MXQ_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128) return MXQ_ERR_UNSUPPORTED;
    if (c->kv_heads > 65536 || c->pages > kMaxInt / c->page_size) return MXQ_ERR_SHAPE;
    return MXQ_OK;
}
mxq_status check_cache_memory(const mxq_kv_cache* c) {
    if (c->pages == 0) return MXQ_OK;
    MXQ_TRY(check_ptr(c->k_codes, 16));
    MXQ_TRY(check_ptr(c->k_scales, 16));
    MXQ_TRY(check_ptr(c->v_codes, 16));
    MXQ_TRY(check_ptr(c->v_scales, 16));
    return MXQ_OK;
}
struct CacheRanges {
    Range r[4];
};
CacheRanges cache_ranges(const mxq_kv_cache* c) {
    const size_t blocks = (size_t)c->pages * (size_t)c->kv_heads * (size_t)c->page_size * (size_t)(c->head_dim / 32);
    return {{{c->k_codes, blocks * 16}, {c->k_scales, blocks}, {c->v_codes, blocks * 16}, {c->v_scales, blocks}}};
}
mxq::KvCache cache_of(const mxq_kv_cache* c) {
    return {static_cast<char*>(c->k_codes), static_cast<char*>(c->v_codes), static_cast<uint8_t*>(c->k_scales),
            static_cast<uint8_t*>(c->v_scales), c->pages, c->kv_heads, c->page_size, c->head_dim / 32};
}

}  // namespace

extern "C" {

mxq_status mxq_matmul(mxq_format fmt, const void* a_codes, const void* a_scales, const void* b_codes, const void* b_scales,
                      int64_t m, int64_t n, int64_t k, void* out, mxq_dtype dtype, mxq_stream stream) {
    if (!fmt_ok(fmt) || !dtype_ok(dtype)) return MXQ_ERR_INVALID_ARG;
    if (!product_format(fmt)) return MXQ_ERR_UNSUPPORTED;
    if (!product_shape_ok(m, n, k)) return MXQ_ERR_SHAPE;
    if (m == 0 || n == 0) return MXQ_OK;
    MXQ_TRY(check_ptr(a_codes, 16));
    MXQ_TRY(check_ptr(a_scales, 16));
    MXQ_TRY(check_ptr(b_codes, 16));
    MXQ_TRY(check_ptr(b_scales, 16));
    MXQ_TRY(check_ptr(out, 16));
    const Range in[] = {{a_codes, codes_bytes(fmt, m, k)},
                        {a_scales, mxq_mma_scales_bytes(m, k)},
                        {b_codes, codes_bytes(fmt, n, k)},
                        {b_scales, mxq_mma_scales_bytes(n, k)}};
    const Range res[] = {{out, (size_t)m * (size_t)n * dtype_bytes(dtype)}};
    if (!disjoint(in, res)) return MXQ_ERR_INVALID_ARG;
    return from_cuda(mxq::launch_matmul((int)fmt, a_codes, a_scales, b_codes, b_scales, m, n, k, out, (int)dtype,
                                        (cudaStream_t)stream));
}

mxq_status mxq_quantize_both(mxq_format row_fmt, mxq_format col_fmt, const void* src, mxq_dtype dtype, int64_t rows,
                             int64_t cols, void* row_codes, void* row_scales, void* col_codes, void* col_scales,
                             mxq_stream stream) {
    const bool r = row_codes != nullptr || row_scales != nullptr, c = col_codes != nullptr || col_scales != nullptr;
    if (!dtype_ok(dtype) || (r && !fmt_ok(row_fmt)) || (c && !fmt_ok(col_fmt))) return MXQ_ERR_INVALID_ARG;
    if ((r && !product_format(row_fmt)) || (c && !product_format(col_fmt))) return MXQ_ERR_UNSUPPORTED;
    MXQ_TRY(check_shape(rows, cols));
    if (rows >= kMaxInt - 128 || cols >= kMaxInt - 128) return MXQ_ERR_SHAPE;
    if (rows == 0) return MXQ_OK;
    if (!r && !c) return MXQ_ERR_INVALID_ARG;
    const int64_t rows32 = (rows + 31) / 32 * 32;
    MXQ_TRY(check_ptr(src, 16));
    if (r) {
        MXQ_TRY(check_ptr(row_codes, 16));
        MXQ_TRY(check_ptr(row_scales, 16));
    }
    if (c) {
        MXQ_TRY(check_ptr(col_codes, 16));
        MXQ_TRY(check_ptr(col_scales, 16));
    }
    const Range in[] = {{src, (size_t)rows * (size_t)cols * dtype_bytes(dtype)}};
    const Range res[] = {{row_codes, r ? codes_bytes(row_fmt, rows, cols) : 0},
                         {row_scales, r ? mxq_mma_scales_bytes(rows, cols) : 0},
                         {col_codes, c ? codes_bytes(col_fmt, cols, rows32) : 0},
                         {col_scales, c ? mxq_mma_scales_bytes(cols, rows32) : 0}};
    if (!disjoint(in, res)) return MXQ_ERR_INVALID_ARG;
    return from_cuda(mxq::launch_quantize_both(r ? (int)row_fmt : -1, c ? (int)col_fmt : -1, src, (int)dtype, rows, cols,
                                               row_codes, row_scales, col_codes, col_scales, (cudaStream_t)stream));
}

size_t mxq_linear_workspace_bytes(mxq_format fmt, int64_t m, int64_t k) {
    if (!fmt_ok(fmt) || !product_format(fmt) || check_shape(m, k) != MXQ_OK) return 0;
    return codes_bytes(fmt, m, k) + mxq_mma_scales_bytes(m, k);  // codes: whole blocks, so the scales are 16-byte aligned
}

mxq_status mxq_linear(mxq_format fmt, const void* x, mxq_dtype dtype, int64_t m, int64_t k, const void* b_codes,
                      const void* b_scales, int64_t n, void* out, void* workspace, size_t workspace_bytes,
                      mxq_stream stream) {
    if (!fmt_ok(fmt) || !dtype_ok(dtype)) return MXQ_ERR_INVALID_ARG;
    if (!product_format(fmt)) return MXQ_ERR_UNSUPPORTED;
    if (!product_shape_ok(m, n, k)) return MXQ_ERR_SHAPE;
    if (m == 0 || n == 0) return MXQ_OK;
    for (const void* p : {x, b_codes, b_scales, (const void*)out, (const void*)workspace}) MXQ_TRY(check_ptr(p, 16));
    const size_t nc = codes_bytes(fmt, m, k), need = nc + mxq_mma_scales_bytes(m, k);
    if (workspace_bytes < need) return MXQ_ERR_INVALID_ARG;
    const Range in[] = {{x, (size_t)m * (size_t)k * dtype_bytes(dtype)},
                        {b_codes, codes_bytes(fmt, n, k)},
                        {b_scales, mxq_mma_scales_bytes(n, k)}};
    const Range res[] = {{out, (size_t)m * (size_t)n * dtype_bytes(dtype)}, {workspace, need}};
    if (!disjoint(in, res)) return MXQ_ERR_INVALID_ARG;
    void* const scales = static_cast<char*>(workspace) + nc;
    MXQ_TRY(from_cuda(mxq::launch_quantize_both((int)fmt, -1, x, (int)dtype, m, k, workspace, scales, nullptr, nullptr,
                                                (cudaStream_t)stream)));
    return from_cuda(mxq::launch_matmul((int)fmt, workspace, scales, b_codes, b_scales, m, n, k, out, (int)dtype,
                                        (cudaStream_t)stream));
}

mxq_status mxq_swiglu_forward(const void* gate, const void* up, mxq_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                              void* out, void* gate_codes, void* gate_scales, void* up_codes, void* up_scales,
                              mxq_stream stream) {
    if (!dtype_ok(dtype)) return MXQ_ERR_INVALID_ARG;
    MXQ_TRY(check_shape(rows, cols));
    if (ld < cols || ld > kMaxElems / (rows > 0 ? rows : 1)) return MXQ_ERR_SHAPE;
    if (!stride_ok(ld, cols, rows, dtype)) return MXQ_ERR_ALIGN;
    if (rows == 0) return MXQ_OK;
    const bool keep = gate_codes || gate_scales || up_codes || up_scales;
    for (const void* p : {gate, up, (const void*)out}) MXQ_TRY(check_ptr(p, 16));
    if (keep) {
        MXQ_TRY(check_ptr(gate_codes, 16));
        MXQ_TRY(check_ptr(up_codes, 16));
        MXQ_TRY(check_ptr(gate_scales, 1));
        MXQ_TRY(check_ptr(up_scales, 1));
    }
    const size_t n = span_bytes(rows, cols, ld, dtype), nc = keep ? codes_bytes(MXQ_MXFP8_E4M3, rows, cols) : 0,
                 ns = keep ? scales_bytes(MXQ_MXFP8_E4M3, rows, cols) : 0;
    const Range in[] = {{gate, n}, {up, n}};
    const Range res[] = {{out, span_bytes(rows, cols, cols, dtype)}, {gate_codes, nc}, {gate_scales, ns}, {up_codes, nc}, {up_scales, ns}};
    if (!disjoint(in, res)) return MXQ_ERR_INVALID_ARG;
    return from_cuda(mxq::launch_swiglu_forward(gate, up, (int)dtype, rows, cols, ld, out, gate_codes, gate_scales, up_codes,
                                                up_scales, (cudaStream_t)stream));
}

mxq_status mxq_swiglu_backward(const void* grad, mxq_dtype dtype, const void* gate_codes, const void* gate_scales,
                               const void* up_codes, const void* up_scales, int64_t rows, int64_t cols, void* dgate,
                               void* dup, int64_t ld, mxq_stream stream) {
    if (!dtype_ok(dtype)) return MXQ_ERR_INVALID_ARG;
    MXQ_TRY(check_shape(rows, cols));
    if (ld < cols || ld > kMaxElems / (rows > 0 ? rows : 1)) return MXQ_ERR_SHAPE;
    if (!stride_ok(ld, cols, rows, dtype)) return MXQ_ERR_ALIGN;
    if (rows == 0) return MXQ_OK;
    for (const void* p : {grad, gate_codes, up_codes, (const void*)dgate, (const void*)dup}) MXQ_TRY(check_ptr(p, 16));
    MXQ_TRY(check_ptr(gate_scales, 1));
    MXQ_TRY(check_ptr(up_scales, 1));
    const size_t n = span_bytes(rows, cols, ld, dtype), nc = codes_bytes(MXQ_MXFP8_E4M3, rows, cols),
                 ns = scales_bytes(MXQ_MXFP8_E4M3, rows, cols);
    const Range in[] = {{grad, span_bytes(rows, cols, cols, dtype)}, {gate_codes, nc}, {gate_scales, ns}, {up_codes, nc}, {up_scales, ns}};
    const Range one[] = {{dgate, n}}, two[] = {{dup, n}};
    if (!disjoint(in, one) || !disjoint(in, two) || !strided_disjoint(dgate, dup, rows, cols, ld, dtype)) return MXQ_ERR_INVALID_ARG;
    return from_cuda(mxq::launch_swiglu_backward(grad, (int)dtype, gate_codes, gate_scales, up_codes, up_scales, rows, cols,
                                                 dgate, dup, ld, (cudaStream_t)stream));
}

mxq_status mxq_kv_append(const mxq_kv_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         mxq_dtype dtype, int64_t tokens, const int64_t* slots, mxq_stream stream) {
    if (!dtype_ok(dtype)) return MXQ_ERR_INVALID_ARG;
    MXQ_TRY(check_cache(cache));
    const int64_t cols = (int64_t)cache->kv_heads * cache->head_dim;
    if (tokens < 0 || tokens > kMaxElems / cols) return MXQ_ERR_SHAPE;
    const int64_t most = kMaxElems / (tokens > 0 ? tokens : 1);
    if (k_stride < cols || v_stride < cols || k_stride > most || v_stride > most) return MXQ_ERR_SHAPE;
    if (!stride_ok(k_stride, cols, tokens, dtype) || !stride_ok(v_stride, cols, tokens, dtype)) return MXQ_ERR_ALIGN;
    if (tokens == 0 || cache->pages == 0) return MXQ_OK;
    MXQ_TRY(check_cache_memory(cache));
    MXQ_TRY(check_ptr(k, 16));
    MXQ_TRY(check_ptr(v, 16));
    MXQ_TRY(check_ptr(slots, 8));
    const CacheRanges c = cache_ranges(cache);
    const Range in[] = {{k, span_bytes(tokens, cols, k_stride, dtype)}, {v, span_bytes(tokens, cols, v_stride, dtype)},
                        {slots, (size_t)tokens * 8}};
    if (!disjoint(in, c.r)) return MXQ_ERR_INVALID_ARG;
    return from_cuda(mxq::launch_kv_append(cache_of(cache), k, k_stride, v, v_stride, (int)dtype, tokens,
                                           reinterpret_cast<const long long*>(slots), (cudaStream_t)stream));
}

mxq_status mxq_kv_read(const mxq_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v, mxq_dtype dtype,
                       mxq_stream stream) {
    if (!dtype_ok(dtype)) return MXQ_ERR_INVALID_ARG;
    MXQ_TRY(check_cache(cache));
    const int64_t cols = (int64_t)cache->kv_heads * cache->head_dim;
    if (tokens < 0 || tokens > kMaxElems / cols) return MXQ_ERR_SHAPE;
    if (tokens == 0) return MXQ_OK;
    MXQ_TRY(check_cache_memory(cache));
    MXQ_TRY(check_ptr(k, 16));
    MXQ_TRY(check_ptr(v, 16));
    MXQ_TRY(check_ptr(slots, 8));
    const CacheRanges c = cache_ranges(cache);
    const size_t n = span_bytes(tokens, cols, cols, dtype);
    const Range in[] = {c.r[0], c.r[1], c.r[2], c.r[3], {slots, (size_t)tokens * 8}}, res[] = {{k, n}, {v, n}};
    if (!disjoint(in, res)) return MXQ_ERR_INVALID_ARG;
    return from_cuda(mxq::launch_kv_read(cache_of(cache), reinterpret_cast<const long long*>(slots), tokens, k, v, (int)dtype,
                                         (cudaStream_t)stream));
}

size_t mxq_kv_attention_workspace_bytes(const mxq_kv_cache* cache, int64_t batch, int64_t q_rows, int32_t max_q,
                                        int32_t q_heads, int64_t max_keys) {
    if (check_cache(cache) != MXQ_OK || batch <= 0 || q_rows <= 0 || max_q <= 0 || q_heads <= 0 ||
        q_heads % cache->kv_heads != 0 || max_keys <= 0 || batch > kMaxInt)
        return 0;
    if (max_q > q_rows) max_q = (int32_t)q_rows;
    if (max_keys > kMaxKeys) max_keys = kMaxKeys;
    return (size_t)mxq::kv_attention_workspace(cache_of(cache), batch, max_q, q_heads, max_keys, true);
}

mxq_status mxq_kv_attention(const mxq_kv_cache* cache, const void* q, int64_t q_rows, int64_t q_row_stride,
                            int64_t q_head_stride, int32_t q_heads, int64_t batch, const int32_t* q_starts, int32_t max_q,
                            const int32_t* seq_lens, int64_t max_keys, const int32_t* block_table, int64_t table_stride,
                            float scale, int32_t window, int32_t fill, void* out, float* lse, void* workspace, size_t workspace_bytes,
                            mxq_stream stream) {
    MXQ_TRY(check_cache(cache));
    if (q_heads < 1 || q_heads % cache->kv_heads != 0 || batch < 0 || batch > kMaxInt || q_rows < 0 || q_rows > kMaxInt - 1 ||
        max_q < 0 || max_keys < 0 || table_stride < 0 || window < 0 || table_stride > kMaxElems || q_rows > kMaxElems / q_heads / 128)
        return MXQ_ERR_SHAPE;
    if (q_starts == nullptr && (max_q == 0 ? q_rows != 0 : q_rows % max_q != 0 || q_rows / max_q != batch)) return MXQ_ERR_SHAPE;
    const int d = cache->head_dim;
    if (q_row_stride < 0 || q_head_stride < 0 || q_row_stride > kMaxElems || q_head_stride > kMaxElems / q_heads ||
        (q_rows > 0 && q_row_stride > kMaxElems / q_rows))
        return MXQ_ERR_SHAPE;
    if (q_row_stride % 8 != 0 || q_head_stride % 8 != 0) return MXQ_ERR_ALIGN;
    if (q_rows == 0 || batch == 0 || max_q == 0) return MXQ_OK;
    MXQ_TRY(check_ptr(q, 16));
    MXQ_TRY(check_ptr(out, 16));
    if (lse) MXQ_TRY(check_ptr(lse, 4));
    if (q_starts) MXQ_TRY(check_ptr(q_starts, 4));
    MXQ_TRY(check_ptr(seq_lens, 4));
    const int64_t cap = table_stride > kMaxInt / cache->page_size ? kMaxInt : table_stride * cache->page_size;
    if (max_keys > cap) max_keys = cap;
    if (max_keys > kMaxKeys) max_keys = kMaxKeys;
    if (max_keys > 0) MXQ_TRY(check_ptr(block_table, 4));
    MXQ_TRY(check_cache_memory(cache));
    if (max_q > q_rows) max_q = (int32_t)q_rows;  // no sequence has more
    mxq::KvAttention x{};
    x.c = cache_of(cache);
    const size_t need = (size_t)mxq::kv_attention_workspace(x.c, batch, max_q, q_heads, max_keys, false);
    if (need > 0) {
        if (workspace_bytes < need) return MXQ_ERR_INVALID_ARG;
        MXQ_TRY(check_ptr(workspace, 16));
    }
    const CacheRanges c = cache_ranges(cache);
    const size_t nout = (size_t)q_rows * (size_t)q_heads;
    const Range in[] = {c.r[0], c.r[1], c.r[2], c.r[3],
                        {q, (size_t)((q_rows - 1) * q_row_stride + (q_heads - 1) * q_head_stride + d) * 2},
                        {q_starts, q_starts ? ((size_t)batch + 1) * 4 : 0},
                        {seq_lens, (size_t)batch * 4},
                        {block_table, max_keys > 0 ? (size_t)batch * (size_t)table_stride * 4 : 0}};
    const Range res[] = {{out, nout * (size_t)d * 2}, {lse, lse ? nout * 4 : 0}, {workspace, need}};
    if (!disjoint(in, res)) return MXQ_ERR_INVALID_ARG;
    x.q = q;
    x.q_rows = q_rows;
    x.q_row_stride = q_row_stride;
    x.q_head_stride = q_head_stride;
    x.batch = batch;
    x.max_keys = max_keys;
    x.table_stride = table_stride;
    x.starts = q_starts;
    x.lens = seq_lens;
    x.table = block_table;
    x.heads = q_heads;
    x.max_q = max_q;
    x.window = window;
    x.fill = fill != 0;
    x.scale = scale;
    x.out = out;
    x.lse = lse;
    x.workspace = workspace;
    return from_cuda(mxq::launch_kv_attention(x, (cudaStream_t)stream));
}

}  // extern "C"
