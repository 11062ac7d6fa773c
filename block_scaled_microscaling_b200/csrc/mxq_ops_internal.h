// mxq_ops_internal.h -- launch interface between the C ABI of the operators (mxq_ops_api.cu) and their kernels
// (mxq_matmul.cu, mxq_both.cu, mxq_swiglu.cu, mxq_kv.cu, mxq_attention.cu). Not part of the public header.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "mxq_internal.h"

namespace mxq {

// out[m, n] = a b^T of two microscaled operands (fmt F_E4M3 or F_E2M1, scales in the MMA tile layout)
cudaError_t launch_matmul(int fmt, const void* ac, const void* as, const void* bc, const void* bs, long long m, long long n,
                          long long k, void* out, int dtype, cudaStream_t st);
// formats -1: direction left out
cudaError_t launch_quantize_both(int rfmt, int cfmt, const void* src, int dtype, long long rows, long long cols, void* rc,
                                 void* rs, void* cc, void* cs, cudaStream_t st);
cudaError_t launch_swiglu_forward(const void* gate, const void* up, int dtype, long long rows, long long cols, long long ld,
                                  void* out, void* gc, void* gs, void* uc, void* us, cudaStream_t st);
cudaError_t launch_swiglu_backward(const void* grad, int dtype, const void* gc, const void* gs, const void* uc, const void* us,
                                   long long rows, long long cols, void* dgate, void* dup, long long ld, cudaStream_t st);
// paged MXFP4 cache: page rows per head, db = head_dim / 32 blocks per row
struct KvCache {
    char *kc, *vc;
    uint8_t *ks, *vs;
    long long pages;
    int heads, page, db;
};
cudaError_t launch_kv_append(const KvCache& c, const void* k, long long k_stride, const void* v, long long v_stride, int dtype,
                             long long tokens, const long long* slots, cudaStream_t st);
cudaError_t launch_kv_read(const KvCache& c, const long long* slots, long long tokens, void* k, void* v, int dtype,
                           cudaStream_t st);
struct KvAttention {
    KvCache c;
    const void* q;
    long long q_rows, q_row_stride, q_head_stride, batch, max_keys, table_stride;
    const int *starts, *lens, *table;
    int heads, max_q, window;
    bool fill;  // rows that no query of a sequence computes get zeros
    float scale;
    void* out;
    float* lse;
    void* workspace;
};
// at_most: enough for any smaller max_keys too
long long kv_attention_workspace(const KvCache& c, long long batch, int max_q, int heads, long long max_keys, bool at_most);
cudaError_t launch_kv_attention(const KvAttention& x, cudaStream_t st);

}  // namespace mxq
