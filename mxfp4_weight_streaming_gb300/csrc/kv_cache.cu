// The paged cache's bookkeeping between steps: which pages each sequence
// holds (update), the rows of partly filled pages that forked sequences take
// along (copy), and the rows of an accepted draft path (accept).
//
// Update is whole-number work over a few tables, all latency: one block, whose
// barriers cost less than more launches would. Copy and accept move
// contiguous 16-byte vectors, a block per page or request, head and K or V of
// a layer. Update and copy of 32 beams in 24 layers (93 MB moved each way) take
// 21 us together, accept and update of 8 requests in 16 layers 13 us. Update
// alone: 5 us with a pool of 654 pages, 21 with 16,384, 72 with 65,536 (its two
// passes over the pool).
#include <climits>

#include "step_launch.h"

#include "step_common.cuh"

namespace mxfp4 {
namespace {

constexpr int kUpdateThreads = 1024;

// Workspace of cache_update: per page its references, writers and lowest
// writer, and the free pages by rank; per sequence what it keeps.
struct UpdateSpace {
    int *refs, *writers, *lowest, *by_rank;  // [num_pages]
    int *base, *want, *last, *offset;        // [sequences]
};

__host__ __device__ UpdateSpace update_space(void* ws, int64_t sequences, int64_t num_pages) {
    int* p = static_cast<int*>(ws);
    UpdateSpace s;
    s.refs = p;
    s.writers = s.refs + num_pages;
    s.lowest = s.writers + num_pages;
    s.by_rank = s.lowest + num_pages;
    s.base = s.by_rank + num_pages;
    s.want = s.base + sequences;
    s.last = s.want + sequences;
    s.offset = s.last + sequences;
    return s;
}

// Exclusive sum over the block, and the block's total.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* total, T* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    T w = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T t = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += t;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const T before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
    return inc - v + (warp ? before : 0);
}

// One block. All counts are whole numbers, so the order of the atomics does
// not show in the result.
__global__ void __launch_bounds__(kUpdateThreads) cache_update_kernel(CacheUpdateArgs a) {
    __shared__ int part[32];
    __shared__ int64_t part64[32];
    const UpdateSpace s = update_space(a.workspace, a.sequences, a.num_pages);
    const int page = 1 << a.page_shift, tid = threadIdx.x;
    pdl_wait_previous();
    pdl_launch_dependents();
    for (int p = tid; p < a.num_pages; p += kUpdateThreads) {
        s.refs[p] = 0;
        s.writers[p] = 0;
        s.lowest[p] = a.sequences;
    }
    __syncthreads();
    for (int i = tid; i < a.sequences; i += kUpdateThreads) {
        const int par = a.parent[i];
        const bool has = par >= 0 && par < a.old_sequences;
        const int64_t room = static_cast<int64_t>(a.table_width) << a.page_shift;
        const int old = has ? static_cast<int>(min(static_cast<int64_t>(max(a.seq_lens[par], 0)), room)) : 0;
        const int base = a.keep ? min(max(a.keep[i], 0), old) : old;
        const int64_t want = min(static_cast<int64_t>(base) + max(a.grow[i], 0), room);
        int last = -1;
        if ((base & (page - 1)) && want > base) {
            last = a.table[par * a.table_stride + (base >> a.page_shift)];
            if (last < 0 || last >= a.num_pages) last = -1;
        }
        s.base[i] = base;
        s.want[i] = static_cast<int>(want);
        s.last[i] = last;
        if (last >= 0) {
            atomicAdd(&s.writers[last], 1);
            atomicMin(&s.lowest[last], i);
        }
    }
    __syncthreads();
    // Kept entries, one warp per sequence.
    for (int i = tid >> 5; i < a.sequences; i += kUpdateThreads / 32) {
        const int kept = (s.base[i] + page - 1) >> a.page_shift;
        const int* from = a.table + a.parent[i] * a.table_stride;
        for (int c = tid & 31; c < a.table_width; c += 32) {
            int e = -1;
            if (c < kept) {
                e = from[c];
                if (e < 0 || e >= a.num_pages) e = -1;
                else atomicAdd(&s.refs[e], 1);
            }
            a.table_out[static_cast<int64_t>(i) * a.table_width + c] = e;
        }
    }
    __syncthreads();
    // Pages each sequence asks for, and where its share of the free ones begins
    // (at the pool's size at most, where none are left). The sum is 64 bits:
    // 65,536 sequences may ask for 2^24 pages each.
    int64_t need_total = 0;
    for (int i0 = 0; i0 < a.sequences; i0 += kUpdateThreads) {
        const int i = i0 + tid;
        int need = 0, copy = 0;
        if (i < a.sequences) {
            const int last = s.last[i];
            if (last >= 0) copy = !(s.refs[last] == s.writers[last] && s.lowest[last] == i);
            need = copy + ((s.want[i] + page - 1) >> a.page_shift) - ((s.base[i] + page - 1) >> a.page_shift);
        }
        int64_t total;
        const int64_t off = need_total + block_scan<int64_t>(need, &total, part64);
        if (i < a.sequences) {
            s.offset[i] = static_cast<int>(min(off, static_cast<int64_t>(a.num_pages)));
            if (!copy) s.last[i] = -1;
        }
        need_total += total;
    }
    // The free pages by rank, as many as are asked for; all are counted.
    int free_total = 0;
    for (int p0 = 0; p0 < a.num_pages; p0 += kUpdateThreads) {
        const int p = p0 + tid;
        const int is_free = p < a.num_pages && s.refs[p] == 0;
        int total;
        const int rank = free_total + block_scan<int>(is_free, &total, part);
        if (is_free) s.by_rank[rank] = p;
        free_total += total;
    }
    __syncthreads();
    for (int i = tid; i < a.sequences; i += kUpdateThreads) {
        const int base = s.base[i], want = s.want[i], src = s.last[i], off = s.offset[i];
        const int copy = src >= 0;
        const int kept = (base + page - 1) >> a.page_shift;
        const int need = copy + ((want + page - 1) >> a.page_shift) - kept;
        const int got = min(max(free_total - off, 0), need);
        const int copied = copy && got > 0;
        const int pages = kept + got - copied;
        int* row = a.table_out + static_cast<int64_t>(i) * a.table_width;
        for (int j = copied; j < got; ++j) row[kept + j - copied] = s.by_rank[off + j];
        int dst = -1;
        if (copied) {
            dst = s.by_rank[off];
            row[kept - 1] = dst;
        }
        const int64_t holds = static_cast<int64_t>(pages) << a.page_shift;
        a.lens_out[i] = copy && !copied ? base : static_cast<int>(min(static_cast<int64_t>(want), holds));
        a.copies[3 * i] = copied ? src : -1;
        a.copies[3 * i + 1] = dst;
        a.copies[3 * i + 2] = copied ? base & (page - 1) : 0;
    }
    if (tid == 0) {
        const int64_t given = min(need_total, static_cast<int64_t>(free_total));
        a.info[0] = free_total - static_cast<int>(given);
        a.info[1] = static_cast<int>(min(need_total - given, static_cast<int64_t>(INT_MAX)));
    }
}

constexpr int kMoveThreads = 128;

// One block per (sequence, head, K or V of a layer): the rows to take along
// are contiguous within a page and head.
__global__ void __launch_bounds__(kMoveThreads) cache_copy_kernel(PoolView pool, const int* copies) {
    pdl_wait_previous();
    pdl_launch_dependents();
    const int i = blockIdx.x;
    const int src = copies[3 * i], dst = copies[3 * i + 1], rows = copies[3 * i + 2];
    if (src < 0 || dst < 0 || src >= pool.num_pages || dst >= pool.num_pages) return;
    const int layer = blockIdx.z >> 1;
    char* base = static_cast<char*>((blockIdx.z & 1) ? pool.v : pool.k) + layer * pool.layer_stride +
                 ((static_cast<int64_t>(blockIdx.y) << pool.page_shift) * pool.row_bytes);
    const uint4* from = reinterpret_cast<const uint4*>(base + src * pool.page_stride);
    uint4* to = reinterpret_cast<uint4*>(base + dst * pool.page_stride);
    const int n = min(rows, 1 << pool.page_shift) * (pool.row_bytes / 16);
    for (int v = threadIdx.x; v < n; v += kMoveThreads) to[v] = from[v];
}

// One block per (request, head, K or V of a layer). Rows are all read before
// any is written, so a path may name them in any order.
constexpr int kMaxPath = 64;
__global__ void __launch_bounds__(kMoveThreads) cache_accept_kernel(PoolView pool, BatchView bt, const int* path,
                                                                     int path_len, const int* n_accept,
                                                                     int* lens_out) {
    pdl_wait_previous();
    pdl_launch_dependents();
    const int b = blockIdx.x;
    int first, n, seq;
    request_extent(bt, b, first, n, seq);
    const int start = seq - n;  // of new token 0; below 0 it is not in the cache
    const int took = min(max(n_accept[b], 0), min(path_len, n));
    if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) lens_out[b] = max(start + took, 0);
    const int layer = blockIdx.z >> 1;
    char* base = static_cast<char*>((blockIdx.z & 1) ? pool.v : pool.k) + layer * pool.layer_stride +
                 ((static_cast<int64_t>(blockIdx.y) << pool.page_shift) * pool.row_bytes);
    const int vecs = pool.row_bytes / 16;  // of one row; at most 32
    constexpr int kHold = kMaxPath * 32 / kMoveThreads;
    uint4 held[kHold];
    uint32_t have = 0;
    const int mask = (1 << pool.page_shift) - 1;
    auto row_ptr = [&](int at) -> uint4* {
        const int page = at < 0 ? -1 : page_of(bt, b, at, pool.page_shift, pool.num_pages);
        return page < 0 ? nullptr
                        : reinterpret_cast<uint4*>(base + page * pool.page_stride +
                                                   static_cast<int64_t>(at & mask) * pool.row_bytes);
    };
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        const int v = h * kMoveThreads + threadIdx.x, i = v / vecs;
        if (i >= took) continue;
        const int from = path[static_cast<int64_t>(b) * path_len + i];
        if (from < 0 || from >= n || from == i) continue;
        const uint4* p = row_ptr(start + from);
        if (!p) continue;
        held[h] = p[v % vecs];
        have |= 1u << h;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        if (!(have >> h & 1)) continue;
        const int v = h * kMoveThreads + threadIdx.x;
        uint4* p = row_ptr(start + v / vecs);
        if (p) p[v % vecs] = held[h];
    }
}

}  // namespace

size_t cache_workspace_bytes(int64_t sequences, int64_t num_pages) {
    return static_cast<size_t>(4 * num_pages + 4 * sequences) * sizeof(int);
}

cudaError_t launch_cache_update(const CacheUpdateArgs& a, cudaStream_t stream) {
    PdlLaunch l(dim3(1), dim3(kUpdateThreads), 0, stream);
    return cudaLaunchKernelEx(&l.cfg, cache_update_kernel, a);
}

cudaError_t launch_cache_copy(const PoolView& pool, const int* copies, int sequences, cudaStream_t stream) {
    PdlLaunch l(dim3(sequences, pool.kv_heads, 2 * pool.layers), dim3(kMoveThreads), 0, stream);
    return cudaLaunchKernelEx(&l.cfg, cache_copy_kernel, pool, copies);
}

cudaError_t launch_cache_accept(const PoolView& pool, const BatchView& batch, const int* path, int path_len,
                                const int* n_accept, int* lens_out, cudaStream_t stream) {
    PdlLaunch l(dim3(batch.batch, pool.kv_heads, 2 * pool.layers), dim3(kMoveThreads), 0, stream);
    return cudaLaunchKernelEx(&l.cfg, cache_accept_kernel, pool, batch, path, path_len, n_accept, lens_out);
}

}  // namespace mxfp4
