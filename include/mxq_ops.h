/*
 * mxq_ops.h -- C ABI of libmxq, language-model operators on the microscaled
 * formats of mxq.h (NVIDIA B200, sm_100a):
 *   - the product of two microscaled matrices on the block-scaled tensor cores,
 *     and a quantize that writes both operand directions of one matrix;
 *   - silu(gate) * up with an 8-bit checkpoint of its inputs, and its gradients;
 *   - a paged key/value cache in MXFP4: append, read back, attention.
 *
 * The formats, block rule, layouts, special values, statuses and calling rules
 * (asynchronous on `stream`, nothing allocated or synchronized, argument errors
 * reported before any launch) are those of mxq.h.
 */
#ifndef MXQ_OPS_H
#define MXQ_OPS_H

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Product of two microscaled matrices:
 *   out[i, j] = sum_l a[i, l] * b[j, l]      i < m, j < n, l < k
 * where a [m, k] and b [n, k] are the values their codes and scales stand for
 * (blocks of 32 along k), accumulated in fp32 by the block-scaled tensor-core
 * instruction and rounded once into `dtype`.
 *   fmt      MXQ_MXFP4_E2M1 or MXQ_MXFP8_E4M3, of both operands
 *            (MXQ_ERR_UNSUPPORTED otherwise).
 *   *_codes  as mxq_quantize / mxq_quantize_mma write them, 16-byte aligned.
 *   *_scales in the tile layout of mxq_quantize_mma (mxq_mma_scales_bytes(rows, k)
 *            bytes), 16-byte aligned.
 *   out      [m, n] row-major, 16-byte aligned; may not overlap an operand.
 * m, n >= 0 (0: no-op; m, n < 2^31 - 256), k > 0, k % 32 == 0, k < 2^31 - 512. A scale
 * byte 0xFF or an E4M3 NaN code makes every output that its block enters NaN.
 * The kernel's waits are bounded (mxq_check_device).
 */
MXQ_API mxq_status mxq_matmul(mxq_format fmt, const void* a_codes, const void* a_scales, const void* b_codes,
                              const void* b_scales, int64_t m, int64_t n, int64_t k, void* out, mxq_dtype dtype,
                              mxq_stream stream);

/*
 * Quantize src [rows, cols] in one pass along either or both directions, as
 * operands of mxq_matmul:
 *   row_codes [rows, cols/32 * P], row_scales: what mxq_quantize_mma(row_fmt) writes;
 *   col_codes [cols, rows32/32 * P], col_scales: what mxq_quantize_mma(col_fmt)
 *     writes for the transpose of src, its rows filled up with zeros to
 *     rows32 = the next multiple of 32.
 * Both *_codes and *_scales of a direction may be NULL: that direction is left
 * out (one of the two is needed). Formats as in mxq_matmul. cols % 32 == 0,
 * any rows >= 0 (< 2^31 - 128), cols < 2^31 - 128; pointers 16-byte aligned; no
 * output may overlap src or another output. Scale arrays are written in full
 * (mxq_mma_scales_bytes(rows, cols) and (cols, rows32) bytes, padding 0).
 */
MXQ_API mxq_status mxq_quantize_both(mxq_format row_fmt, mxq_format col_fmt, const void* src, mxq_dtype dtype,
                                     int64_t rows, int64_t cols, void* row_codes, void* row_scales, void* col_codes,
                                     void* col_scales, mxq_stream stream);

/*
 * Linear layer on a converted weight: x [m, k] of type dtype rounded to fmt along
 * its rows (as mxq_quantize_mma), times b [n, k] (as mxq_matmul):
 *   out [m, n] of type dtype.
 * workspace: mxq_linear_workspace_bytes(fmt, m, k) bytes, 16-byte aligned, for x's
 * codes and scales; used by this call alone until it has finished. Other rules
 * and errors, and bounded waits (mxq_check_device), as mxq_quantize_mma and
 * mxq_matmul.
 */
MXQ_API size_t mxq_linear_workspace_bytes(mxq_format fmt, int64_t m, int64_t k);
MXQ_API mxq_status mxq_linear(mxq_format fmt, const void* x, mxq_dtype dtype, int64_t m, int64_t k,
                              const void* b_codes, const void* b_scales, int64_t n, void* out, void* workspace,
                              size_t workspace_bytes, mxq_stream stream);

/*
 * out = silu(gate) * up, with gate and up kept as MXFP8 E4M3 checkpoints (as
 * mxq_quantize writes them: codes [rows, cols], scales [rows, cols/32]):
 *   out[i, j] = g * sigmoid(g) * u, computed in fp32 from the unrounded inputs.
 * gate, up: [rows, cols] with row stride ld values (ld >= cols; the two may be
 * halves of one matrix); out [rows, cols] contiguous. All of type dtype.
 * cols % 32 == 0; pointers and row strides in bytes 16-byte aligned. No output
 * may overlap an input or another output. All four checkpoint pointers NULL: none
 * is kept.
 */
MXQ_API mxq_status mxq_swiglu_forward(const void* gate, const void* up, mxq_dtype dtype, int64_t rows, int64_t cols,
                                      int64_t ld, void* out, void* gate_codes, void* gate_scales, void* up_codes,
                                      void* up_scales, mxq_stream stream);
/*
 * Gradients of that call from its checkpoints: with g, u the values the codes
 * stand for and s = sigmoid(g),
 *   dgate = grad * u * s * (1 + g * (1 - s)),   dup = grad * g * s.
 * grad [rows, cols] contiguous; dgate, dup with row stride ld (ld >= cols; they
 * may be halves of one matrix, whose other bytes stay as they are). Rules as
 * above. A block with scale 0xFF gives NaN gradients.
 */
MXQ_API mxq_status mxq_swiglu_backward(const void* grad, mxq_dtype dtype, const void* gate_codes,
                                       const void* gate_scales, const void* up_codes, const void* up_scales,
                                       int64_t rows, int64_t cols, void* dgate, void* dup, int64_t ld,
                                       mxq_stream stream);

/*
 * Paged key/value cache in MXFP4: each token's key and value of each head is
 * head_dim / 32 blocks along the head's dimension. Codes are [pages, kv_heads,
 * page_size, head_dim / 2] bytes, scales [pages, kv_heads, page_size,
 * head_dim / 32] bytes, both as mxq_quantize writes a row of head_dim values.
 * Token slot s is row s % page_size of page s / page_size. head_dim is 64 or
 * 128 (MXQ_ERR_UNSUPPORTED otherwise); page_size a multiple of 16, at most 65536;
 * pages * page_size < 2^31; all four arrays 16-byte aligned.
 */
typedef struct {
    void* k_codes;
    void* k_scales;
    void* v_codes;
    void* v_scales;
    int64_t pages;
    int32_t kv_heads;
    int32_t page_size;
    int32_t head_dim;
} mxq_kv_cache;

/*
 * Round keys and values of `tokens` tokens to MXFP4 and write them to the cache:
 * token t goes to slot slots[t] (int64, device memory). A slot outside
 * [0, pages * page_size) is skipped (padding). Slots of one call must differ:
 * what a slot named twice holds afterwards is unspecified (other slots are not
 * affected). k, v: token t, head h, dimension d at t * stride + h * head_dim + d,
 * of type dtype, 16-byte aligned, strides in values with stride * size a
 * multiple of 16 bytes and stride >= kv_heads * head_dim.
 */
MXQ_API mxq_status mxq_kv_append(const mxq_kv_cache* cache, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, mxq_dtype dtype, int64_t tokens, const int64_t* slots,
                                 mxq_stream stream);
/*
 * Read tokens back: k, v [tokens, kv_heads, head_dim] contiguous, of type dtype,
 * 16-byte aligned, hold the values of slots[t]; zeros for a slot outside the
 * cache. Exact (an E2M1 value times its scale is a bf16 value).
 */
MXQ_API mxq_status mxq_kv_read(const mxq_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
                               mxq_dtype dtype, mxq_stream stream);

/*
 * Attention of bf16 queries over the cache. Sequence b (b < batch) has
 * seq_lens[b] keys (int32), key j being row j % page_size of page
 * block_table[b * table_stride + j / page_size] (int32); its n_b queries are the
 * rows q_starts[b] .. q_starts[b + 1] of q (int32 [batch + 1]; NULL: every
 * sequence has max_q queries, q_rows = batch * max_q). The i-th of them stands
 * at position p = seq_lens[b] - n_b + i and sees the keys j <= p, with
 * window > 0 only those j > p - window:
 *   out = sum_j w_j v_j,  w = softmax over the keys seen of scale * (q . k_j)
 *   lse = log sum_j exp(scale * (q . k_j))           (natural logarithm)
 * q head h reads key/value head h / (q_heads / kv_heads). A query that sees no
 * key gives out = 0 and lse = -inf. Keys that a query does not see do not enter
 * it, whatever bytes they hold; a key whose page number is outside [0,
 * pages) is seen by no query. Starts do not decrease; each is clamped to [0, q_rows].
 * Rows of q that belong to no sequence, and queries of a sequence beyond max_q,
 * are not computed: with fill == 0 they are left as they are in out and lse,
 * otherwise they get 0 and -inf.
 *   q      row r, head h at r * q_row_stride + h * q_head_stride (values; strides
 *          multiples of 8, q 16-byte aligned); out [q_rows, q_heads, head_dim]
 *          bf16 contiguous, 16-byte aligned; lse fp32 [q_rows, q_heads] or NULL.
 *   max_keys  an upper bound of seq_lens that the host knows (longer sequences
 *          are cut to it); at most table_stride * page_size counts. It sets how
 *          the keys are split over CTAs.
 *   workspace  mxq_kv_attention_workspace_bytes(...) bytes (may be 0: then NULL),
 *          16-byte aligned, used by this call alone until it has finished. What
 *          a max_keys asks for is enough for every smaller one, and for tables
 *          of any width.
 * Keys, values and rows of q are brought to half precision (f16), exactly up to a
 * power of two: a block more than 2^16 below the largest that the query sees (of
 * the keys; of the values), and values of q more than 2^17 below the largest of
 * their row, may lose bits or count as zero. Scores and sums are fp32 (a row's sum
 * of weights of up to 2^8 times its values must stay below 2^128), 2^x has an
 * error of 2^-22; the weights w enter the second product in f16 (2^-11). Where a
 * key that only some queries of a chunk see is far larger than the others, the
 * chunk's rows are computed one by one in fp32, many times slower.
 * Where max_q * (q_heads / kv_heads) exceeds 32, the kernel's waits are bounded
 * (mxq_check_device).
 */
MXQ_API size_t mxq_kv_attention_workspace_bytes(const mxq_kv_cache* cache, int64_t batch, int64_t q_rows,
                                                int32_t max_q, int32_t q_heads, int64_t max_keys);
MXQ_API mxq_status mxq_kv_attention(const mxq_kv_cache* cache, const void* q, int64_t q_rows, int64_t q_row_stride,
                                    int64_t q_head_stride, int32_t q_heads, int64_t batch, const int32_t* q_starts,
                                    int32_t max_q, const int32_t* seq_lens, int64_t max_keys,
                                    const int32_t* block_table, int64_t table_stride, float scale, int32_t window,
                                    int32_t fill, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                    mxq_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_OPS_H */
