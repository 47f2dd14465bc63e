// C ABI of the step's attention side: argument checks, then the launches of
// norm.cu, rope.cu, attention.cu and kv_cache.cu.
#include <cmath>

#include "step_common.cuh"
#include "step_launch.h"

namespace {

using mxfp4::BatchView;
using mxfp4::CacheView;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launched(cudaError_t e) { return e == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA; }

int elem_bytes(const mxfp4_kv_cache_t& c) { return c.dtype == MXFP4_KV_E4M3 ? 1 : 2; }

int64_t page_stride_of(const mxfp4_kv_cache_t& c) {
    return c.page_stride ? c.page_stride : static_cast<int64_t>(c.kv_heads) * c.page_size * c.head_dim;
}

int64_t layer_stride_of(const mxfp4_kv_cache_t& c) {
    return c.layer_stride ? c.layer_stride : c.num_pages * page_stride_of(c);
}

int cache_status(const mxfp4_kv_cache_t* c) {
    if (!c || !c->k || !c->v || c->num_pages <= 0 || c->layers <= 0 || c->kv_heads <= 0 || c->page_size <= 0 ||
        c->head_dim <= 0 || c->page_stride < 0 || c->layer_stride < 0 || c->reserved != 0)
        return MXFP4_ERR_INVALID_ARG;
    if (c->dtype != MXFP4_KV_BF16 && c->dtype != MXFP4_KV_E4M3) return MXFP4_ERR_INVALID_ARG;
    if (c->num_pages >= (1 << 24) || c->layers > 1024 || c->kv_heads > 1024 || c->page_size < 16 ||
        c->page_size > 1024 || mxfp4::log2_exact(c->page_size) < 0 || (c->head_dim != 64 && c->head_dim != 128))
        return MXFP4_ERR_SHAPE;
    const int64_t dense = static_cast<int64_t>(c->kv_heads) * c->page_size * c->head_dim;
    if (page_stride_of(*c) < dense || page_stride_of(*c) >= (int64_t(1) << 36)) return MXFP4_ERR_SHAPE;
    const int e = elem_bytes(*c);
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
        page_stride_of(*c) * e % 16 != 0 || layer_stride_of(*c) * e % 16 != 0)
        return MXFP4_ERR_ALIGN;
    return MXFP4_OK;
}

int batch_status(const mxfp4_kv_batch_t* b) {
    if (!b || !b->q_start || !b->seq_lens || !b->block_table || b->batch <= 0 || b->tokens <= 0 ||
        b->table_width <= 0 || b->table_stride < 0 || b->max_q <= 0 || b->max_seq <= 0 || b->reserved != 0)
        return MXFP4_ERR_INVALID_ARG;
    if (b->batch > 1024 || b->tokens > (1 << 24) || b->table_width > (1 << 24) ||
        (b->table_stride && b->table_stride < b->table_width))
        return MXFP4_ERR_SHAPE;
    if (!aligned(b->q_start, 4) || !aligned(b->seq_lens, 4) || !aligned(b->block_table, 4)) return MXFP4_ERR_ALIGN;
    return MXFP4_OK;
}

CacheView cache_view(const mxfp4_kv_cache_t& c) {
    CacheView v{};
    v.k = c.k;
    v.v = c.v;
    v.k_scale = c.dtype == MXFP4_KV_E4M3 ? c.k_scale : nullptr;
    v.v_scale = c.dtype == MXFP4_KV_E4M3 ? c.v_scale : nullptr;
    v.page_stride = page_stride_of(c);
    v.num_pages = static_cast<int>(c.num_pages);
    v.kv_heads = c.kv_heads;
    v.page_shift = mxfp4::log2_exact(c.page_size);
    v.head_dim = c.head_dim;
    return v;
}

BatchView batch_view(const mxfp4_kv_batch_t& b, int page_size) {
    BatchView v{};
    v.q_start = b.q_start;
    v.seq_lens = b.seq_lens;
    v.block_table = b.block_table;
    v.table_stride = b.table_stride ? b.table_stride : b.table_width;
    v.table_width = b.table_width;
    const int64_t room = static_cast<int64_t>(b.table_width) * page_size;
    v.room = static_cast<int>(room < (int64_t(1) << 30) ? room : (int64_t(1) << 30));
    v.batch = b.batch;
    v.tokens = b.tokens;
    return v;
}

mxfp4::PoolView pool_view(const mxfp4_kv_cache_t& c) {
    mxfp4::PoolView v{};
    const int e = elem_bytes(c);
    v.k = c.k;
    v.v = c.v;
    v.page_stride = page_stride_of(c) * e;
    v.layer_stride = layer_stride_of(c) * e;
    v.layers = c.layers;
    v.num_pages = static_cast<int>(c.num_pages);
    v.kv_heads = c.kv_heads;
    v.page_shift = mxfp4::log2_exact(c.page_size);
    v.row_bytes = c.head_dim * e;
    return v;
}

int caps_of(mxfp4::DeviceCaps* caps) { return mxfp4::device_caps(caps); }

int attention(const void* q, int64_t q_stride, int q_heads, const mxfp4_kv_cache_t* cache,
              const mxfp4_kv_batch_t* batch, float scale, float softcap, int window, const uint64_t* tree_mask,
              const int32_t* positions, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (positions && !tree_mask) return MXFP4_ERR_INVALID_ARG;
    if (!q || !out || q_heads <= 0 || window < 0 || !(softcap >= 0.f) || std::isinf(softcap) || !std::isfinite(scale))
        return MXFP4_ERR_INVALID_ARG;
    if (int rc = cache_status(cache)) return rc;
    if (int rc = batch_status(batch)) return rc;
    // The kernels count a request's rows, rounded up to a row tile, in an int.
    if (q_heads % cache->kv_heads || q_heads > 128 * cache->kv_heads || (tree_mask && batch->max_q > 64) ||
        static_cast<int64_t>(batch->tokens) * (q_heads / cache->kv_heads) > (int64_t(1) << 31) - 256)
        return MXFP4_ERR_SHAPE;
    if (q_stride < static_cast<int64_t>(q_heads) * cache->head_dim) return MXFP4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || q_stride % 8 || !aligned(out, 16) || !aligned(lse, 4) || !aligned(tree_mask, 8) ||
        !aligned(positions, 4))
        return MXFP4_ERR_ALIGN;
    if (!workspace) return MXFP4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MXFP4_ERR_ALIGN;
    if (workspace_bytes < mxfp4_attention_workspace_size(q_heads, cache, batch)) return MXFP4_ERR_WORKSPACE;
    mxfp4::DeviceCaps caps;
    if (int rc = caps_of(&caps)) return rc;
    mxfp4::AttentionArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.tree_mask = reinterpret_cast<const unsigned long long*>(tree_mask);
    a.positions = positions;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    a.status = caps.status;
    a.q_heads = q_heads;
    a.max_q = batch->max_q;
    a.max_seq = batch->max_seq;
    a.e4m3 = cache->dtype == MXFP4_KV_E4M3;
    a.scale = scale;
    a.softcap = softcap;
    // Sequences are cut to 2^30 tokens (batch_view), which a longer window never
    // leaves; the kernels' differences with it then stay within an int.
    a.window = window < (1 << 30) ? window : 0;
    return launched(mxfp4::launch_attention(a, cache_view(*cache), batch_view(*batch, cache->page_size), caps.num_sms,
                                            static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int mxfp4_residual_norm(const void* x, const void* residual, int64_t tokens, int64_t n, const void* post_weight,
                        const void* post_bias, const void* gate, int64_t gate_stride, float scale,
                        const void* weight, const void* bias, float weight_offset, float eps, int layer, void* y,
                        void* r_out, void* stream) {
    if (!x || !residual || !weight || !y || !r_out || tokens <= 0 || n <= 0 || (post_bias && !post_weight) ||
        gate_stride < 0 || (gate_stride && gate_stride < n) || !(eps >= 0.f))
        return MXFP4_ERR_INVALID_ARG;
    if (n > 32768 || tokens >= (int64_t(1) << 31)) return MXFP4_ERR_SHAPE;
    for (const void* p : {x, residual, post_weight, post_bias, gate, weight, bias, static_cast<const void*>(y),
                          static_cast<const void*>(r_out)})
        if (!aligned(p, 2)) return MXFP4_ERR_ALIGN;
    if (y == r_out) return MXFP4_ERR_INVALID_ARG;
    mxfp4::DeviceCaps caps;
    if (int rc = caps_of(&caps)) return rc;
    mxfp4::ResidualNormArgs a{};
    a.x = x;
    a.residual = residual;
    a.post_weight = post_weight;
    a.post_bias = post_bias;
    a.gate = gate;
    a.weight = weight;
    a.bias = bias;
    a.y = y;
    a.r_out = r_out;
    a.tokens = tokens;
    a.n = n;
    a.gate_stride = gate_stride;
    a.scale = scale;
    a.eps = eps;
    a.weight_offset = weight_offset;
    a.layer = layer != 0;
    return launched(mxfp4::launch_residual_norm(a, caps.num_sms, static_cast<cudaStream_t>(stream)));
}

int mxfp4_rope_append(const void* qkv, int64_t qkv_stride, int q_heads, const int32_t* positions,
                      const float* inv_freq, int rotary_dim, int interleaved, float factor,
                      const mxfp4_kv_cache_t* cache, const mxfp4_kv_batch_t* batch, void* q_out, void* stream) {
    if (!qkv || !q_out || q_heads <= 0 || rotary_dim < 0 || (rotary_dim && !inv_freq)) return MXFP4_ERR_INVALID_ARG;
    if (int rc = cache_status(cache)) return rc;
    if (int rc = batch_status(batch)) return rc;
    if (rotary_dim % 2 || rotary_dim > cache->head_dim || q_heads > 128 * cache->kv_heads) return MXFP4_ERR_SHAPE;
    if (qkv_stride < static_cast<int64_t>(q_heads + 2 * cache->kv_heads) * cache->head_dim)
        return MXFP4_ERR_INVALID_ARG;
    if (!aligned(qkv, 16) || !aligned(q_out, 16) || qkv_stride % 8 || !aligned(positions, 4) || !aligned(inv_freq, 4))
        return MXFP4_ERR_ALIGN;
    mxfp4::DeviceCaps caps;
    if (int rc = caps_of(&caps)) return rc;
    mxfp4::RopeArgs a{};
    a.qkv = qkv;
    a.qkv_stride = qkv_stride;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.q_out = q_out;
    a.q_heads = q_heads;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved != 0;
    a.e4m3 = cache->dtype == MXFP4_KV_E4M3;
    a.factor = factor;
    return launched(
        mxfp4::launch_rope_append(a, cache_view(*cache), batch_view(*batch, cache->page_size), static_cast<cudaStream_t>(stream)));
}

size_t mxfp4_attention_workspace_size(int q_heads, const mxfp4_kv_cache_t* cache, const mxfp4_kv_batch_t* batch) {
    if (!cache || !batch || q_heads <= 0 || cache->kv_heads <= 0 || batch->max_q <= 0 || cache->head_dim <= 0 ||
        q_heads % cache->kv_heads)
        return 0;
    mxfp4::DeviceCaps caps;
    const int sms = mxfp4::device_caps(&caps) == MXFP4_OK ? caps.num_sms : 152;
    return mxfp4::attention_workspace_bytes(q_heads, cache->kv_heads, cache->head_dim, batch->max_q,
                                             cache->dtype == MXFP4_KV_E4M3, sms);
}

int mxfp4_attention(const void* q, int64_t q_stride, int q_heads, const mxfp4_kv_cache_t* cache,
                    const mxfp4_kv_batch_t* batch, float scale, float softcap, int window,
                    const uint64_t* tree_mask, void* out, float* lse, void* workspace, size_t workspace_bytes,
                    void* stream) {
    return attention(q, q_stride, q_heads, cache, batch, scale, softcap, window, tree_mask, nullptr, out, lse, workspace,
                     workspace_bytes, stream);
}

int mxfp4_attention_at(const void* q, int64_t q_stride, int q_heads, const mxfp4_kv_cache_t* cache,
                       const mxfp4_kv_batch_t* batch, float scale, float softcap, int window,
                       const uint64_t* tree_mask, const int32_t* positions, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream) {
    return attention(q, q_stride, q_heads, cache, batch, scale, softcap, window, tree_mask, positions, out, lse,
                     workspace, workspace_bytes, stream);
}

size_t mxfp4_cache_workspace_size(int64_t sequences, int64_t num_pages) {
    if (sequences <= 0 || num_pages <= 0) return 0;
    return mxfp4::cache_workspace_bytes(sequences, num_pages);
}

int mxfp4_cache_update(const int32_t* table, int64_t table_stride, int table_width, const int32_t* seq_lens,
                       int old_sequences, const int32_t* parent, const int32_t* keep, const int32_t* grow,
                       int sequences, int64_t num_pages, int page_size, int32_t* table_out, int32_t* lens_out,
                       int32_t* copies, int32_t* info, void* workspace, size_t workspace_bytes, void* stream) {
    if (!table || !seq_lens || !parent || !grow || !table_out || !lens_out || !copies || !info || table_width <= 0 ||
        table_stride < 0 || old_sequences <= 0 || sequences <= 0 || num_pages <= 0 || page_size <= 0 ||
        table_out == table || lens_out == seq_lens || lens_out == keep)
        return MXFP4_ERR_INVALID_ARG;
    if (sequences > 65536 || old_sequences > 65536 || num_pages >= (1 << 24) || table_width > (1 << 24) ||
        page_size < 16 || page_size > 1024 || mxfp4::log2_exact(page_size) < 0 ||
        static_cast<int64_t>(table_width) * page_size >= (int64_t(1) << 31) ||
        (table_stride && table_stride < table_width))
        return MXFP4_ERR_SHAPE;
    for (const void* p : {static_cast<const void*>(table), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(parent), static_cast<const void*>(keep),
                          static_cast<const void*>(grow), static_cast<const void*>(table_out),
                          static_cast<const void*>(lens_out), static_cast<const void*>(copies),
                          static_cast<const void*>(info)})
        if (!aligned(p, 4)) return MXFP4_ERR_ALIGN;
    if (!workspace) return MXFP4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MXFP4_ERR_ALIGN;
    if (workspace_bytes < mxfp4::cache_workspace_bytes(sequences, num_pages)) return MXFP4_ERR_WORKSPACE;
    mxfp4::DeviceCaps caps;
    if (int rc = caps_of(&caps)) return rc;
    mxfp4::CacheUpdateArgs a{};
    a.table = table;
    a.table_stride = table_stride ? table_stride : table_width;
    a.seq_lens = seq_lens;
    a.parent = parent;
    a.keep = keep;
    a.grow = grow;
    a.table_out = table_out;
    a.lens_out = lens_out;
    a.copies = copies;
    a.info = info;
    a.workspace = workspace;
    a.old_sequences = old_sequences;
    a.sequences = sequences;
    a.table_width = table_width;
    a.num_pages = static_cast<int>(num_pages);
    a.page_shift = mxfp4::log2_exact(page_size);
    return launched(mxfp4::launch_cache_update(a, static_cast<cudaStream_t>(stream)));
}

int mxfp4_cache_copy(const mxfp4_kv_cache_t* cache, const int32_t* copies, int sequences, void* stream) {
    if (!copies || sequences <= 0) return MXFP4_ERR_INVALID_ARG;
    if (int rc = cache_status(cache)) return rc;
    if (sequences > 65536) return MXFP4_ERR_SHAPE;
    if (!aligned(copies, 4)) return MXFP4_ERR_ALIGN;
    mxfp4::DeviceCaps caps;
    if (int rc = caps_of(&caps)) return rc;
    return launched(mxfp4::launch_cache_copy(pool_view(*cache), copies, sequences, static_cast<cudaStream_t>(stream)));
}

int mxfp4_cache_accept(const mxfp4_kv_cache_t* cache, const mxfp4_kv_batch_t* batch, const int32_t* path,
                       int path_len, const int32_t* n_accept, int32_t* lens_out, void* stream) {
    if (!path || !n_accept || !lens_out || path_len <= 0) return MXFP4_ERR_INVALID_ARG;
    if (int rc = cache_status(cache)) return rc;
    if (int rc = batch_status(batch)) return rc;
    if (lens_out == batch->seq_lens || lens_out == n_accept) return MXFP4_ERR_INVALID_ARG;
    if (path_len > 64) return MXFP4_ERR_SHAPE;
    if (!aligned(path, 4) || !aligned(n_accept, 4) || !aligned(lens_out, 4)) return MXFP4_ERR_ALIGN;
    mxfp4::DeviceCaps caps;
    if (int rc = caps_of(&caps)) return rc;
    return launched(mxfp4::launch_cache_accept(pool_view(*cache), batch_view(*batch, cache->page_size), path, path_len, n_accept,
                                               lens_out, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
