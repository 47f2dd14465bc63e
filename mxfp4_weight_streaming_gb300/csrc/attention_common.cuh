// What the attention kernels share: how the step's work is cut, the
// workspace of partial results, and the join of the parts.
//
// The rows of a KV head's queries in one request are its (token, head of the
// group) pairs, row = token * G + head: all of them read the same K and V. A
// row tile of R rows and its visible keys are an item; an item is cut into
// key tiles, and the key tiles of all items of the step, counted in order
// (request, row tile, KV head, key tile), are dealt to the CTAs in equal
// runs. So a long sequence is shared by many CTAs and many short ones share
// a CTA, whatever the lengths on the device are. A CTA whose run begins or
// ends inside an item leaves that item's part in the workspace (at most two
// per CTA); items that lie whole in a run are finished by their CTA.
#pragma once

#include "step_common.cuh"

namespace mxfp4 {
namespace attn {

// Requests are counted in at most this many groups of neighbours (one request
// each up to that many), so the sums fit beside full-size tiles.
constexpr int kGroups = 64;
constexpr float kLog2e = 1.4426950408889634f;

// n / d for n < 2^31 by a multiplication: with s = ceil(log2 d) and m =
// ceil(2^(31 + s) / d), m d - 2^(31 + s) < d <= 2^s keeps the quotient exact.
struct Divisor {
    uint32_t d, m, s;
    __host__ __device__ __forceinline__ int div(int n) const {
#ifdef __CUDA_ARCH__
        return s == 0 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), m) >> (s - 1));
#else
        return static_cast<int>(static_cast<uint32_t>(n) / d);
#endif
    }
};

inline Divisor divisor(int d) {
    Divisor v{};
    v.d = static_cast<uint32_t>(d);
    while ((1u << v.s) < v.d) ++v.s;
    v.m = v.s == 0 ? 0 : static_cast<uint32_t>(((uint64_t(1) << (31 + v.s)) + v.d - 1) / v.d);
    return v;
}

// Cut of one call. Rows of a request, n * group, are at most 2^31 - 256 (the
// entry point refuses more).
struct Cut {
    int group;       // query heads per KV head
    Divisor by_group;
    int kv_heads;
    int row_shift;   // R = 1 << row_shift
    int key_shift;   // keys per unit of work
    int window;      // 0: none
    bool tree;
    bool placed;     // windows count from Params::positions, not from the cache index
    int min_share;   // units a CTA takes at least
};

// Keys [begin, end) that some row of row tile rt of a request sees; begin is
// rounded down to a key tile only where tiles are counted.
__device__ __forceinline__ void item_keys(const Cut& c, int n, int seq, int rt, int& begin, int& end) {
    const int tok0 = c.by_group.div(rt << c.row_shift);
    const int tok1 = min(n - 1, c.by_group.div((rt << c.row_shift) + (1 << c.row_shift) - 1));
    end = c.tree ? seq : max(seq - n + tok1 + 1, 0);
    begin = c.window ? max(seq - n + (c.placed ? 0 : tok0) - c.window + 1, 0) : 0;
    end = max(end, begin);
}

__device__ __forceinline__ int item_tiles(const Cut& c, int n, int seq, int rt) {
    int begin, end;
    item_keys(c, n, seq, rt, begin, end);
    return max(((end + (1 << c.key_shift) - 1) >> c.key_shift) - (begin >> c.key_shift), 1);
}

__device__ __forceinline__ int row_tiles(const Cut& c, int n) {
    return (n * c.group + (1 << c.row_shift) - 1) >> c.row_shift;
}

__device__ __forceinline__ int64_t request_units(const Cut& c, const BatchView& bt, int b) {
    int first, n, seq;
    request_extent(bt, b, first, n, seq);
    int64_t u = 0;
    for (int rt = row_tiles(c, n) - 1; rt >= 0; --rt) u += item_tiles(c, n, seq, rt);
    return u * c.kv_heads;
}

__device__ __forceinline__ int requests_per_group(const BatchView& bt) { return (bt.batch + kGroups - 1) / kGroups; }

// Units of work before each group of requests; returns their sum. Called by
// THREADS threads (a warp, or the whole block), t = 0 .. THREADS - 1.
template <int THREADS>
__device__ __forceinline__ int64_t count_units(const Cut& c, const BatchView& bt, int t, int64_t* before) {
    const int per = requests_per_group(bt), groups = (bt.batch + per - 1) / per;
    auto sync = [] {
        if constexpr (THREADS == 32) __syncwarp();
        else __syncthreads();
    };
#pragma unroll 2
    for (int i = t; i < groups; i += THREADS) {
        int64_t u = 0;
        for (int b = i * per; b < min((i + 1) * per, bt.batch); ++b) u += request_units(c, bt, b);
        before[i + 1] = u;
    }
    sync();
    if (t < 32) {
        int64_t carry = 0;
        for (int i0 = 0; i0 < groups; i0 += 32) {
            const int i = i0 + t;
            int64_t v = i < groups ? before[i + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
                if (t >= o) v += x;
            }
            v += carry;
            if (i < groups) before[i + 1] = v;
            carry = __shfl_sync(0xffffffffu, v, 31);
        }
        if (t == 0) before[0] = 0;
    }
    sync();
    return before[groups];
}

struct Item {
    int b, rt, head;        // request, row tile, KV head
    int first, n, seq;      // the request's extent
    int begin, end;         // visible keys
    int tile, tiles;        // the unit's key tile within the item, and the item's count
};

__device__ __forceinline__ Item locate(const Cut& c, const BatchView& bt, const int64_t* before,
                                       int64_t unit) {
    Item it;
    const int per = requests_per_group(bt);
    int lo = 0, hi = (bt.batch + per - 1) / per;  // before[lo] <= unit < before[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= unit) lo = mid;
        else hi = mid;
    }
    int64_t rem = unit - before[lo];
    it.b = lo * per;
    if (per > 1)
        for (int64_t u; rem >= (u = request_units(c, bt, it.b)); ++it.b) rem -= u;
    request_extent(bt, it.b, it.first, it.n, it.seq);
    it.rt = 0;
    while (true) {
        it.tiles = item_tiles(c, it.n, it.seq, it.rt);
        const int64_t block = static_cast<int64_t>(it.tiles) * c.kv_heads;
        if (rem < block) break;
        rem -= block;
        ++it.rt;
    }
    const uint32_t tiles = it.tiles;
    it.head = static_cast<int>(rem >> 32 ? rem / tiles : static_cast<uint32_t>(rem) / tiles);
    it.tile = static_cast<int>(rem - it.head * static_cast<int64_t>(tiles));
    item_keys(c, it.n, it.seq, it.rt, it.begin, it.end);
    return it;
}

__device__ __forceinline__ int64_t share_of(const Cut& c, int64_t total, int ctas) {
    // 64-bit divisions are long: taken only where they are needed.
    const int64_t share = total >> 31 ? (total + ctas - 1) / ctas
                                      : (static_cast<uint32_t>(total) + static_cast<uint32_t>(ctas) - 1u) /
                                            static_cast<uint32_t>(ctas);
    return max(share, static_cast<int64_t>(c.min_share));
}

// Partial results: two slots per CTA, slot 2c for a part that began before
// the CTA's run and 2c + 1 for one that begins in it.
struct alignas(32) Split {
    int parts;     // 0: there is none
    int row0, rows;  // its row tile's first row in the request, and its rows
    int first;     // the request's first row of q
    int head;      // KV head
};
struct Parts {
    float* o;        // [2 ctas], not divided by the sum: [R][D], or from attention_tc.cu [D / 4][R][4]
    float2* ml;      // [2 ctas][R]: running maximum (of log2 scores) and sum
    Split* split;    // [ctas]: the item that begins in CTA c and ends beyond it
};

__host__ __device__ inline size_t parts_bytes(int ctas, int rows, int d) {
    return static_cast<size_t>(ctas) * (2 * rows * (d * sizeof(float) + sizeof(float2)) + sizeof(Split));
}

__host__ __device__ inline Parts parts_in(void* ws, int ctas, int rows, int d) {
    Parts p;
    p.split = static_cast<Split*>(ws);
    p.ml = reinterpret_cast<float2*>(p.split + ctas);
    p.o = reinterpret_cast<float*>(p.ml + static_cast<size_t>(2) * ctas * rows);
    return p;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The smaller one, NaN where either is (fminf gives the other).
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Scores in the log2 domain: s * scale * log2(e), or with a cap
// cap * tanh(s * scale / cap) * log2(e). tanh x = 1 - 2 / (1 + e^2x): off by
// a few 1e-7 of the cap (the hardware's tanh, off by 5e-4 of it, would cost
// percents of a probability).
struct ScoreMap {
    float mul;      // scale * log2(e), or 2 * scale / cap * log2(e)
    float cap;      // cap * log2(e); 0: no cap
    __device__ __forceinline__ float operator()(float s) const {
        if (cap == 0.f) return s * mul;
        const float e = exp2_fast(min_nan(s * mul, 80.f));
        return cap - __fdividef(2.f * cap, 1.f + e);
    }
};

// Where a query's window counts from, by its position (cut to the cache indices
// of the new tokens [start, seq), and so that it leaves none of those out).
__device__ __forceinline__ int window_from(const int* position, int start, int seq, int window) {
    return min(min(max(load_word(position), start), seq - 1), start + window - 1);
}

// What the kernels take.
struct Params {
    const __nv_bfloat16* q;
    int64_t q_stride;
    const unsigned long long* tree_mask;
    const int* positions;  // of the queries, where a window counts from them: null unless cut.placed
    __nv_bfloat16* out;
    float* lse;
    void* ws;
    unsigned* status;
    int q_heads;
    bool negate;  // attention_tc.cu: the scale is negative (map has its magnitude)
    ScoreMap map;
    Cut cut;
    CacheView cache;
    BatchView batch;
};

// Joins the parts that `ctas` CTAs left in the workspace (attention.cu).
cudaError_t launch_join(const Params& p, bool e4m3, bool from_tc, int ctas, cudaStream_t stream);

// CTAs for a call: no more than it has key tiles if the caller's bounds hold
// (and no less work is done if they do not: each CTA's run is longer then). A
// token over 1,000 has 128 tiles for 304 CTAs.
inline int ctas_for(const Params& p, int64_t max_rows, int max_seq, int most) {
    const int64_t rows = (max_rows + (1 << p.cut.row_shift) - 1) >> p.cut.row_shift;
    const int64_t keys = (static_cast<int64_t>(max_seq) >> p.cut.key_shift) + 2;
    // Any int32 bounds will do, so the product is cut on the way.
    int64_t tiles = rows;
    for (const int64_t f : {keys, static_cast<int64_t>(p.cut.kv_heads), static_cast<int64_t>(p.batch.batch)})
        tiles = tiles < most ? tiles * f : most;
    return tiles < most ? static_cast<int>(tiles) : most;
}

// The tensor-core kernel (attention_tc.cu): any number of rows.
size_t tc_workspace_bytes(int64_t rows, int d, int num_sms);
cudaError_t launch_tc(const Params& p, bool e4m3, int64_t rows, int max_seq, int num_sms, cudaStream_t stream);

inline ScoreMap score_map(float scale, float softcap) {
    ScoreMap m;
    m.cap = softcap > 0.f ? softcap * kLog2e : 0.f;
    m.mul = softcap > 0.f ? 2.f * scale / softcap * kLog2e : scale * kLog2e;
    return m;
}

}  // namespace attn
}  // namespace mxfp4
