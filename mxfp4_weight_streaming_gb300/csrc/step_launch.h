// Host interface of the step's attention-side kernels (norm.cu, rope.cu,
// attention.cu, kv_cache.cu). Arguments are checked by step_capi.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mxfp4 {

struct CacheView;
struct BatchView;

struct ResidualNormArgs {
    const void *x, *residual, *post_weight, *post_bias, *gate, *weight, *bias;
    void *y, *r_out;
    uint8_t* ys;  // null: y is bf16; otherwise y takes microscaled codes and this their scales
    int64_t tokens, n, gate_stride;
    float scale, eps, weight_offset;
    bool layer;
    bool e2m1;    // type of the codes
};
cudaError_t launch_residual_norm(const ResidualNormArgs& a, int num_sms, cudaStream_t stream);

struct RopeArgs {
    const void* qkv;  // bf16 rows of (q_heads + 2 kv_heads) * head_dim, qkv_stride elements apart
    int64_t qkv_stride;
    const int* positions;  // null: the cache index
    const float* inv_freq;
    void* q_out;
    int q_heads, rotary_dim;
    bool interleaved, e4m3;
    float factor;
};
cudaError_t launch_rope_append(const RopeArgs& a, const CacheView& cache, const BatchView& batch,
                               cudaStream_t stream);

struct AttentionArgs {
    const void* q;  // bf16 rows of q_heads * head_dim, q_stride elements apart
    int64_t q_stride;
    const unsigned long long* tree_mask;
    const int* positions;  // null: a window counts cache indices
    void* out;   // bf16 [tokens, q_heads, head_dim]
    float* lse;  // null or [tokens, q_heads]
    void* workspace;
    unsigned* status;
    int q_heads;
    int max_q, max_seq;
    bool e4m3;
    float scale, softcap;
    int window;
};
size_t attention_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q, bool e4m3, int num_sms);
// K or V pool of a layer as the tensor map attention_tc.cu copies from: (D,
// page, kv_heads, pages): bf16 in boxes of 64 elements x min(page, 128)
// tokens with the 128-byte swizzle, E4M3 in boxes of D bytes, not swizzled.
// (capi.cu).
cudaError_t encode_kv_map(CUtensorMap* map, const void* pool, const CacheView& cache, bool e4m3);
cudaError_t launch_attention(const AttentionArgs& a, const CacheView& cache, const BatchView& batch, int num_sms,
                             cudaStream_t stream);

// Pools of several layers: the same block table holds for each.
struct PoolView {
    void* k;
    void* v;
    int64_t page_stride, layer_stride;  // bytes
    int layers, num_pages, kv_heads, page_shift;
    int row_bytes;  // of one token's row of one head
};

struct CacheUpdateArgs {
    const int* table;
    int64_t table_stride;
    const int* seq_lens;
    const int* parent;
    const int* keep;  // null: everything
    const int* grow;
    int* table_out;   // [sequences][table_width], dense
    int* lens_out;
    int* copies;      // [sequences][3]
    int* info;        // [2]
    void* workspace;
    int old_sequences, sequences, table_width, num_pages, page_shift;
};
size_t cache_workspace_bytes(int64_t sequences, int64_t num_pages);
cudaError_t launch_cache_update(const CacheUpdateArgs& a, cudaStream_t stream);
cudaError_t launch_cache_copy(const PoolView& pool, const int* copies, int sequences, cudaStream_t stream);
cudaError_t launch_cache_accept(const PoolView& pool, const BatchView& batch, const int* path, int path_len,
                                const int* n_accept, int* lens_out, cudaStream_t stream);

}  // namespace mxfp4
