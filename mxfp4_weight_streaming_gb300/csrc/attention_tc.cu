// Attention of a step's new tokens over the paged cache, for many rows per KV
// head (verify steps of several tokens, prompt chunks): both products on the
// fifth-generation tensor cores.
//
// One CTA per SM works through its run of key tiles (128 keys, see
// attention_common.cuh). Two streams of work alternate on the tensor cores,
// each with a score tile S [128 rows][128 keys] and an output accumulator O
// [128 rows][D] in TMEM: while one stream's scores become probabilities, the
// other's products run.
//   SPLIT (at most 128 rows): both streams take the same rows, stream s the
//         key tiles of parity s; their accumulators are joined at the end.
//   otherwise: stream s takes rows 128 s .. of a 256-row tile; both read the
//         same K and V tiles.
// Warps:
//   0-3, 4-7  turn the scores of stream 0 and 1 into probabilities, one
//             thread per row (TMEM lane), so maxima and sums need no exchange;
//             P goes back to TMEM in bf16 over the first half of S and is the
//             A operand of P V
//   8         issues the products
//   9, 10     copy the K and the V pages (TMA, 128-byte swizzle) into a ring
//             of [128 keys][64 elements] boxes: K is a K-major B operand of
//             Q K^T, V as it lies in memory an N-major B operand of P V.
//             Warp 9 finds the CTA's parts of items and tells the others
//   11        copies the rows of q
//   12-15     E4M3 caches only: turn the copied bytes into f16 tiles of the
//             ring (exact; the scales go to the scores and the outputs), and
//             q into f16, each row by a power of two that keeps it in range
// Operands are bf16, with an E4M3 cache f16. Probabilities are rounded to that
// type too, since a product takes both operands in one type: each is off by up
// to 2^-8 (2^-11) of itself, the outputs by 2.0e-3 to 2.4e-3 in the rms against
// 1.7e-3 by their own rounding to bf16; with f16 it does not show (but ones
// below 2^-25 of the largest are 0 there). Their sum is of the unrounded ones.
// Elements of q below 2^-17 of their row's largest lose bits in f16, 2^-25 of
// the largest at most: as little as the scores' fp32 sums.
//
// A row's running maximum is raised only when a score exceeds it by 2^8, so
// O is seldom rescaled (by the row's own thread, after the stream's last
// product). Score maxima, sums and accumulators are fp32. (Running maximum and
// sum: Milakov and Gimelshein, 2018; two tiles that take turns between products
// and softmax: Shah et al., 2024.)
#include <cuda.h>
#include <cuda_fp16.h>

#include "attention_common.cuh"
#include "step_launch.h"
#include "tc_common.cuh"

namespace mxfp4 {
namespace attn {
namespace {

// 12 warps, and 4 more where an E4M3 cache is to be converted.
__host__ __device__ constexpr int tc_threads(bool e4m3) { return e4m3 ? 512 : 384; }
constexpr int kTcKeys = 128;   // keys per tile
constexpr int kMmaWarp = 8, kLoadWarp = 9, kLoadVWarp = 10, kConvertWarp = 12;
constexpr float kTcSlack = 8.f;

template <int D, bool SPLIT, bool E4M3>
struct Layout {
    static constexpr int kTile = kTcKeys * D * 2;  // bytes of a bf16 K or V tile, or of a 128-row q tile
    static constexpr int kHalf = 128 * 128;        // bytes of [128 rows][64 elements]
    static constexpr int kQ = (SPLIT ? 1 : 2) * kTile;
    // bf16: 5 tiles of 32 KB, or 8 of 16 KB: three or more in flight beside
    // the two in use. E4M3: the tiles in flight are the raw ones.
    static constexpr int kSlots = D == 128 ? (E4M3 ? 3 : 5) : (E4M3 ? 5 : 8);
    static constexpr int kRawTile = E4M3 ? kTcKeys * D : 0;
    static constexpr int kRawSlots = !E4M3 ? 1 : D == 64 ? 8 : SPLIT ? 5 : 4;
    static constexpr int kRing = kQ;               // offsets
    static constexpr int kRaw = kRing + kSlots * kTile;
    static constexpr int kBytes = kRaw + kRawSlots * kRawTile + 1024;  // and alignment
};

// A part of an item, key tiles [tile0, tile0 + steps) of its keys, as the
// warps need it.
struct alignas(16) Segment {
    int steps;         // 0: no more
    int q0, rows;      // the request's first row of q; rows of the row tile
    int row0;          // its first row, counted in the request
    int start;         // cache index of the request's first new token
    int begin, end;    // keys that some row sees
    int tile0;
    int head;
    int whole, begins; // the whole item; its first tile
    int b;             // request
    int parts;         // of an item that begins here and ends in another CTA
};

// Everything the warps tell one another.
template <bool SPLIT, bool E4M3>
struct Shared {
    int64_t before[kGroups + 1];
    uint64_t kv_full[8], kv_empty[8], raw_full[8], raw_empty[8], patch, q_full[2], q_empty, s_full[2], p_full[2][2],
        pv_done[2], vote[2], meet, drain, seg_full[2], seg_empty[2];
    Segment seg[2];
    float m[2][SPLIT ? 128 : 1], l[2][SPLIT ? 128 : 1];  // of the two streams' rows
    int8_t q_exp[2][E4M3 ? (SPLIT ? 128 : 256) : 4];     // of q's rows, by turns
    uint32_t tmem;
    uint32_t bad[2];   // last tile (counted from 1) of each stream whose V is not finite
    uint32_t skip[2];  // the stream's product with V has been taken by its warps
    int abort;
};

__device__ __forceinline__ uint32_t idesc_f16(uint32_t n, bool b_n_major, bool negate_a, bool f16) {
    // fp32 accumulators, types of A and B, sign of A, B's major, N / 8, M / 16 (M = 128).
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(negate_a) << 13) |
           (static_cast<uint32_t>(b_n_major) << 16) | ((n >> 3) << 17) | (8u << 24);
}

// D[128 x N] (+)= A[128 x 16] B[N x 16]^T, bf16, A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// The same with A in TMEM (two bf16 a column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

__device__ __forceinline__ void tmem_load32(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
}

// A TMEM load's registers hold nothing before the wait that follows it: no use
// of them may move above this (to be placed after the wait).
__device__ __forceinline__ void loaded32(float* r) {
    asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                 "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
                 "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
                 :: "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Four E4M3 bytes -> four f16, exact.
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t w) {
    uint2 r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(w));
    return r;
}

__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

// Whether any of this thread's share (1 of 128) of a V tile is an infinity or a NaN.
template <int D, bool F16>
__device__ __forceinline__ bool v_not_finite(uint32_t v, int r) {
    constexpr uint32_t kExp = F16 ? 0x7c007c00u : 0x7f807f80u;
    uint32_t bad = 0;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint4 w = lds128(v + (c * 128 + r) * 16);
        bad |= __vcmpeq2(w.x & kExp, kExp) | __vcmpeq2(w.y & kExp, kExp) |
               __vcmpeq2(w.z & kExp, kExp) | __vcmpeq2(w.w & kExp, kExp);
    }
    return bad != 0;
}

template <bool F16>
__device__ __forceinline__ float half_of(uint32_t pair, int h) {
    if constexpr (F16) return __half2float(__ushort_as_half(static_cast<uint16_t>(h ? pair >> 16 : pair)));
    return __uint_as_float(h ? pair & 0xffff0000u : pair << 16);
}

// O += P V of one tile by the rows' own threads, leaving out the keys whose
// probability is 0. Warp-wide.
template <int D, bool F16>
__device__ __noinline__ void add_tile_by_rows(uint32_t ot, uint32_t pt, uint32_t v, uint32_t half_bytes, bool first) {
#pragma unroll 1
    for (int col = 0; col < D; col += 32) {
        float o[32];
        tmem_load32(ot + col, o);
        tc::tmem_wait_ld();
        loaded32(o);
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = first ? 0.f : o[x];
#pragma unroll 1
        for (int k2 = 0; k2 < kTcKeys / 2; ++k2) {
            uint32_t pair;
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(pair) : "r"(pt + k2) : "memory");
            tc::tmem_wait_ld();
            asm volatile("" : "+r"(pair)::"memory");
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float f = half_of<F16>(pair, h);
                if (f == 0.f) continue;
                const int k = 2 * k2 + h;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int chunk = (col >> 3) + c;
                    const uint4 w = lds128(v + (chunk >> 3) * half_bytes + k * 128 + (((chunk & 7) ^ (k & 7)) << 4));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        o[8 * c + 2 * x] += f * half_of<F16>(u[x], 0);
                        o[8 * c + 2 * x + 1] += f * half_of<F16>(u[x], 1);
                    }
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
            tc::tmem_store16(ot + col + 16 * c, *reinterpret_cast<const uint32_t(*)[16]>(&o[16 * c]));
        tc::tmem_wait_st();
    }
}

// Rows [lo, hi) of key tile t of a segment hold its keys.
__device__ __forceinline__ void tile_rows(const Segment& g, int step, int& lo, int& hi) {
    const int key0 = (g.tile0 + step) * kTcKeys;
    lo = max(g.begin - key0, 0);
    hi = min(g.end - key0, kTcKeys);
}

// The i-th tile of a segment of n steps in the order in which the products
// need them: K0 V0 K1 V1 ..., or (SPLIT, where scores run two tiles ahead)
// K0 K1 V0 K2 V1 ...
template <bool SPLIT>
__device__ __forceinline__ int ring_order(int i, int n, bool& v) {
    if (!SPLIT) {
        v = i & 1;
        return i >> 1;
    }
    v = i == 2 * n - 1 || (i && !(i & 1));
    return i == 2 * n - 1 ? n - 1 : v ? (i >> 1) - 1 : (i + 1) >> 1;
}

// Where K tile j and V tile j of a segment of n steps come in that order.
template <bool SPLIT>
__device__ __forceinline__ uint32_t k_place(int j) {
    return SPLIT ? (j < 2 ? j : 2 * j - 1) : 2 * j;
}
template <bool SPLIT>
__device__ __forceinline__ uint32_t v_place(int j, int n) {
    return SPLIT ? min(n, j + 2) + j : 2 * j + 1;
}

// Row r of a segment's row tile in q, or null.
__device__ __forceinline__ const __nv_bfloat16* q_row(const Params& p, const Segment& g, int r) {
    if (r >= g.rows) return nullptr;
    const int tok = p.cut.by_group.div(g.row0 + r);
    return p.q + (g.q0 + tok) * p.q_stride + (g.head * p.cut.group + g.row0 + r - tok * p.cut.group) * p.cache.head_dim;
}

// How a warp takes the segments that the load warp hands out.
template <class S>
__device__ __forceinline__ bool take_segment(S& sh, uint32_t& turn, Segment& g, const WaitCtx& wait) {
    const uint32_t i = turn & 1;
    const bool ok = mbar_wait(smem_addr(&sh.seg_full[i]), (turn >> 1) & 1, wait);
    if (!__all_sync(0xffffffffu, ok)) return false;
    g = sh.seg[i];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&sh.seg_empty[i]));
    ++turn;
    return g.steps > 0;
}

// ------------------------------------------------------------------ copies
// A load warp. What does not change from tile to tile is kept, since at full
// bandwidth a K and a V tile have 1.4 us together. Lane b finds the page of
// the tile's box b; one lane issues the copies (an instruction that lanes
// issue one by one takes as long for each).
template <int D, bool SPLIT, bool E4M3>
struct Loader {
    using L = Layout<D, SPLIT, E4M3>;
    static constexpr uint32_t kRingSlots = E4M3 ? L::kRawSlots : L::kSlots;
    static constexpr uint32_t kBytes = E4M3 ? L::kRawTile : L::kTile;
    static constexpr int kHalves = E4M3 ? 1 : D / 64;  // copies per box
    const Params& p;
    Shared<SPLIT, E4M3>& sh;
    WaitCtx wait;
    uint32_t ring, full, empty;  // shared addresses
    uint32_t last = 0;           // ring tiles issued, by the highest number
    uint32_t patches = 0;
    int lane, box_rows, boxes, page_mask, page_shift;
    bool one, ok = true;
    // The segment.
    const int* table;
    int begin, end, key_base, steps, head;

    __device__ Loader(const Params& p_, Shared<SPLIT, E4M3>& sh_, WaitCtx w, uint32_t base, int lane_)
        : p(p_), sh(sh_), wait(w), lane(lane_) {
        ring = base + (E4M3 ? L::kRaw : L::kRing);
        full = smem_addr(E4M3 ? sh.raw_full : sh.kv_full);
        empty = smem_addr(E4M3 ? sh.raw_empty : sh.kv_empty);
        page_shift = p.cache.page_shift;
        page_mask = (1 << page_shift) - 1;
        box_rows = min(1 << page_shift, kTcKeys);
        boxes = kTcKeys / box_rows;
        one = elect_one();
    }

    __device__ __forceinline__ void begin_segment(const Segment& g) {
        table = p.batch.block_table + g.b * p.batch.table_stride;
        begin = g.begin;
        end = g.end;
        key_base = g.tile0 * kTcKeys;
        steps = g.steps;
        head = __shfl_sync(0xffffffffu, g.head, 0);
    }

    // This lane's box of a tile: its page, or the pool's size, which reads as
    // zeros. Read well before the copy that needs it (a table read takes as
    // long as a copy).
    __device__ __forceinline__ int page_for(int step) const {
        const int key = key_base + step * kTcKeys + lane * box_rows;
        int pg = -1;
        if (step < steps && lane < boxes && key < end && key + box_rows > begin) pg = load_word(table + (key >> page_shift));
        return static_cast<uint32_t>(pg) < static_cast<uint32_t>(p.cache.num_pages) ? pg : p.cache.num_pages;
    }

    // Ring tile n (counted over the CTA's life) from key tile `step`.
    __device__ __forceinline__ void tile(const CUtensorMap* map, uint32_t n, int step, bool v, int pg) {
        const uint32_t slot = n % kRingSlots, turn = n / kRingSlots;
        ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * slot, (turn & 1) ^ 1, wait));
        if (!ok) return;
        if (withhold_stage(n)) return;  // test builds only
        const int key0 = key_base + step * kTcKeys;
        // Rows of V that hold no key of this item but lie in a page that
        // does: whatever is there must not meet the products (0 * NaN).
        const int lo = max(begin - key0, 0), hi = min(end - key0, kTcKeys);
        const bool ragged = !E4M3 && v && ((lo | hi) & (box_rows - 1));
        const uint32_t bar = ragged ? smem_addr(&sh.patch) : full + 8 * slot;
        const uint32_t dst = ring + slot * kBytes;
        if (one) mbar_arrive_expect_tx(bar, kBytes);
        const int y = key0 & page_mask;
        for (int b = 0; b < boxes; ++b) {
            const int page = __shfl_sync(0xffffffffu, pg, b);
            if (one) {
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    tma_load_4d(dst + h * L::kHalf + b * box_rows * (E4M3 ? D : 128), map, h * 64, y, head, page, bar);
            }
        }
        last = n + 1;
        if (ragged) patch(dst, full + 8 * slot, lo, hi);
    }

    __device__ __noinline__ void patch(uint32_t dst, uint32_t full_bar, int lo, int hi) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&sh.patch), patches & 1, wait));
        if (!ok) return;
        ++patches;
        const int lo0 = lo & ~(box_rows - 1), hi1 = (hi + box_rows - 1) & ~(box_rows - 1);
#pragma unroll 1
        for (int i = lane; i < kTcKeys * (D / 8); i += 32) {
            const int r = i / (D / 8), c = i % (D / 8);
            if ((r >= lo0 && r < lo) || (r >= hi && r < hi1))
                sts128(dst + (c >> 3) * L::kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4), 0, 0, 0, 0);
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(full_bar);
    }

    // After a wait ran out: the copies in flight land before the CTA ends.
    __device__ __noinline__ void drain() {
        const uint64_t t0 = global_timer_ns();
        for (uint32_t n = last > kRingSlots ? last - kRingSlots : 0; n < last; ++n)
            while (!mbar_try_wait(full + 8 * (n % kRingSlots), (n / kRingSlots) & 1) &&
                   !mbar_try_wait(smem_addr(&sh.patch), patches & 1) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
    }
};

template <int D, bool SPLIT, bool CAP, bool E4M3>
__global__ void __launch_bounds__(tc_threads(E4M3), 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ Params p) {
    using L = Layout<D, SPLIT, E4M3>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared<SPLIT, E4M3> sh;
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cut& cut = p.cut;
    constexpr int R = SPLIT ? 128 : 256;  // rows of a row tile
    const Parts parts = parts_in(p.ws, gridDim.x, R, D);
    const WaitCtx wait{p.status, &sh.abort};

    if (warp == kMmaWarp) {
        tc::tmem_alloc(smem_addr(&sh.tmem), 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 32 * kLoadWarp) {
        for (const CUtensorMap* m : {&kmap, &vmap})
            asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
        sh.abort = 0;
        for (int i = 0; i < 8; ++i) {
            mbar_init(smem_addr(&sh.kv_full[i]), E4M3 ? 128 : 1);
            mbar_init(smem_addr(&sh.kv_empty[i]), 1);
            mbar_init(smem_addr(&sh.raw_full[i]), 1);
            mbar_init(smem_addr(&sh.raw_empty[i]), 128);
        }
        mbar_init(smem_addr(&sh.patch), 1);
        mbar_init(smem_addr(&sh.q_empty), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&sh.q_full[s]), E4M3 ? 128 : 288);
            mbar_init(smem_addr(&sh.s_full[s]), 1);
            mbar_init(smem_addr(&sh.p_full[s][0]), 128);
            mbar_init(smem_addr(&sh.p_full[s][1]), 128);
            mbar_init(smem_addr(&sh.pv_done[s]), 1);
            mbar_init(smem_addr(&sh.vote[s]), 128);
            mbar_init(smem_addr(&sh.seg_full[s]), 1);
            mbar_init(smem_addr(&sh.seg_empty[s]), E4M3 ? 14 : 11);  // warps
            sh.bad[s] = sh.skip[s] = 0;
        }
        mbar_init(smem_addr(&sh.meet), 256);
        mbar_init(smem_addr(&sh.drain), 1);
        fence_barrier_init();
    }
    pdl_wait_previous();
    if (threadIdx.x == 0) parts.split[blockIdx.x].parts = 0;
    tc::fence_before_sync();
    const int64_t total = count_units<tc_threads(E4M3)>(cut, p.batch, threadIdx.x, sh.before);  // ends with a block barrier
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);

    // 384 threads start with 168 registers each; the two groups that hold a
    // row of scores per thread take 200, the third keeps 104. 512 threads start
    // with 128: 168, and 88 for the others. (The sums are the same.)
    if (warp >= 8) {
        if constexpr (E4M3) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kLoadWarp) {
        const int64_t share = share_of(cut, total, gridDim.x);
        int64_t unit = share * blockIdx.x;
        const int64_t unit_end = min(unit + share, total);
        Loader<D, SPLIT, E4M3> ld(p, sh, wait, base, lane);
        uint32_t used = 0;  // ring tiles before this segment
        for (uint32_t turn = 0;; ++turn) {
            Segment g{};
            if (unit < unit_end && ld.ok) {
                const Item it = locate(cut, p.batch, sh.before, unit);
                g.steps = static_cast<int>(min(unit_end - unit, static_cast<int64_t>(it.tiles - it.tile)));
                g.q0 = it.first;
                g.row0 = it.rt * R;
                g.rows = min(R, it.n * cut.group - g.row0);
                g.start = it.seq - it.n;
                g.begin = it.begin;
                g.end = it.end;
                g.tile0 = (it.begin >> 7) + it.tile;
                g.head = it.head;
                g.begins = it.tile == 0;
                g.whole = g.begins && g.steps == it.tiles;
                g.b = it.b;
                const int64_t last = unit + it.tiles - 1;
                g.parts = g.begins && !g.whole ? static_cast<int>(last >> 31 ? last / share
                                                                             : static_cast<uint32_t>(last) /
                                                                                   static_cast<uint32_t>(share)) -
                                                     static_cast<int>(blockIdx.x) + 1
                                               : 0;
                unit += g.steps;
            }
            if (turn >= 2)
                ld.ok = __all_sync(0xffffffffu, ld.ok && mbar_wait(smem_addr(&sh.seg_empty[turn & 1]),
                                                                   ((turn >> 1) - 1) & 1, wait));
            if (!ld.ok) break;
            if (lane == 0) {
                sh.seg[turn & 1] = g;
                mbar_arrive(smem_addr(&sh.seg_full[turn & 1]));
            }
            if (g.steps == 0) break;
            ld.begin_segment(g);
            const int n = __shfl_sync(0xffffffffu, g.steps, 0);
            // K; the other load warp copies V.
            int p0 = ld.page_for(0), p1 = ld.page_for(1);
#pragma unroll 1
            for (int j = 0; j < n && ld.ok; ++j) {
                ld.tile(&kmap, used + k_place<SPLIT>(j), j, false, p0);
                p0 = p1;
                p1 = ld.page_for(j + 2);
            }
            used += 2 * n;
        }
        if (!ld.ok && lane == 0) ld.drain();
    } else if (warp == kMmaWarp) {
        // All lanes walk through the tiles, so that what the products are
        // given stays in uniform registers; one lane issues.
        const uint32_t idesc_qk = idesc_f16(kTcKeys, false, p.negate, E4M3),
                       idesc_pv = idesc_f16(D, true, false, E4M3);
        const uint64_t q_desc = tc::operand_desc(base), k_desc = tc::operand_desc(base + L::kRing);
        const uint64_t v_desc = tc::smem_desc(base + L::kRing, L::kHalf, 1024, tc::kLayoutSwizzle128);
        const bool one = elect_one();
        uint32_t used = 0;          // ring tiles taken
        uint32_t turn = 0;          // segments taken
        uint32_t done[2] = {0, 0};  // probabilities taken, per stream
        bool ok = true;
        Segment g;
        auto wait_for = [&](uint64_t& bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(smem_addr(&bar), parity, wait));
            return ok;
        };
        auto full = [&](uint32_t n) -> uint64_t& { return sh.kv_full[n % L::kSlots]; };
        auto parity = [&](uint32_t n) { return (n / L::kSlots) & 1; };
        auto qk = [&](int s, uint32_t n, bool frees_k, bool frees_q) {
            const uint64_t q = q_desc + (SPLIT ? 0 : (s * L::kTile) >> 4);
            const uint64_t k = k_desc + (n % L::kSlots) * (L::kTile >> 4);
            tc::fence_after_sync();
            if (one) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t off = ((i >> 2) * L::kHalf + (i & 3) * 32) >> 4;
                    mma_ss(tmem + s * 128, q + off, k + off, idesc_qk, i > 0);
                }
                tc::commit_to(smem_addr(&sh.s_full[s]));
                if (frees_k) tc::commit_to(smem_addr(&sh.kv_empty[n % L::kSlots]));
                if (frees_q) tc::commit_to(smem_addr(&sh.q_empty));
            }
            __syncwarp();
        };
        // Two barriers in one test where both are through (a test takes 90 ns).
        auto wait_both = [&](uint64_t& b1, uint32_t p1, uint64_t& b2, uint32_t p2) {
            if (__all_sync(0xffffffffu, mbar_test2(smem_addr(&b1), p1, smem_addr(&b2), p2))) return true;
            return wait_for(b1, p1) && wait_for(b2, p2);
        };
        // P V of tile n. The second half of the probabilities comes while the
        // first half's product runs. v_new, k_new: tile n, and K tile k, which
        // the stream's next scores take, have not been waited for yet.
        auto pv = [&](int s, uint32_t n, bool first, bool frees, bool v_new, uint32_t k, bool k_new) {
            const uint64_t v = v_desc + (n % L::kSlots) * (L::kTile >> 4);
            auto issue = [&](int i0, int i1) {
                tc::fence_after_sync();
                if (one && !lds_u32_volatile(smem_addr(&sh.skip[s]))) {
#pragma unroll
                    for (int i = i0; i < i1; ++i)
                        mma_ts(tmem + 256 + s * D, tmem + s * 128 + i * 8, v + i * (2048 >> 4), idesc_pv,
                               !(first && i == 0));
                }
            };
            if (!wait_both(sh.p_full[s][0], done[s] & 1, v_new ? full(n) : sh.p_full[s][0], v_new ? parity(n) : done[s] & 1))
                return false;
            issue(0, kTcKeys / 32);
            if (!wait_both(sh.p_full[s][1], done[s] & 1, k_new ? full(k) : sh.p_full[s][1], k_new ? parity(k) : done[s] & 1))
                return false;
            issue(kTcKeys / 32, kTcKeys / 16);
            if (one) {
                tc::commit_to(smem_addr(&sh.pv_done[s]));
                if (frees) tc::commit_to(smem_addr(&sh.kv_empty[n % L::kSlots]));
            }
            __syncwarp();
            ++done[s];
            return true;
        };
        while (ok && take_segment(sh, turn, g, wait)) {
            const int n = __shfl_sync(0xffffffffu, g.steps, 0);
            if (!wait_for(sh.q_full[(turn - 1) & 1], ((turn - 1) >> 1) & 1)) break;
            if constexpr (SPLIT) {
                // Ring order: K0 K1 V0 K2 V1 K3 ...
                auto k_at = [&](int j) { return used + k_place<SPLIT>(j); };
                auto v_at = [&](int j) { return used + v_place<SPLIT>(j, n); };
                for (int j = 0; j < min(n, 2) && wait_for(full(k_at(j)), parity(k_at(j))); ++j)
                    qk(j, k_at(j), true, j == n - 1);
                for (int j = 0; j < n && ok; ++j) {
                    const int s = j & 1;
                    const uint32_t k = k_at(j + 2);
                    if (!pv(s, v_at(j), j < 2, true, true, k, j + 2 < n)) break;
                    if (j + 2 < n) qk(s, k, true, j + 2 == n - 1);
                }
            } else {
                if (!wait_for(full(used), parity(used))) break;
                qk(0, used, false, false);
                qk(1, used, true, n == 1);
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t v = used + 2 * j + 1, k = v + 1;
                    const bool more = j + 1 < n;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (!pv(s, v, j == 0, s == 1, s == 0, k, more && s == 0)) break;
                        if (more) qk(s, k, s == 1, s == 1 && j + 2 == n);
                    }
                }
            }
            used += 2 * n;
        }
        if (!ok && one) {  // products in flight end before TMEM is given back
            tc::commit_to(smem_addr(&sh.drain));
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(smem_addr(&sh.drain), 0) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
    } else if (warp == kLoadVWarp) {
        Loader<D, SPLIT, E4M3> ld(p, sh, wait, base, lane);
        uint32_t turn = 0, used = 0;
        Segment g;
        while (ld.ok && take_segment(sh, turn, g, wait)) {
            ld.begin_segment(g);
            const int n = __shfl_sync(0xffffffffu, g.steps, 0);
            int p0 = ld.page_for(0), p1 = ld.page_for(1);
#pragma unroll 1
            for (int j = 0; j < n && ld.ok; ++j) {
                ld.tile(&vmap, used + v_place<SPLIT>(j, n), j, true, p0);
                p0 = p1;
                p1 = ld.page_for(j + 2);
            }
            used += 2 * n;
        }
        if (!ld.ok && lane == 0) ld.drain();
    } else if (!E4M3) {
        uint32_t turn = 0;
        bool ok = true;
        Segment g;
        while (ok && take_segment(sh, turn, g, wait)) {
            // The first segment's rows come from the softmax warps, idle then (one
            // warp takes 10,000 cycles over 256 rows); later ones while those are
            // at work, once the last segment's products have read theirs.
            if (turn == 1) {
                mbar_arrive(smem_addr(&sh.q_full[0]));
                continue;
            }
            ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&sh.q_empty), turn & 1, wait));
            if (!ok) break;
            // A lane copies one 16-byte chunk of every S-th row; the row's place
            // in q (head of the group, then the next token) moves along with it.
            constexpr int S = 32 / (D / 8);
            const int c = lane % (D / 8), r0 = lane / (D / 8);
            const int tok = cut.by_group.div(g.row0 + r0);
            int h = g.row0 + r0 - tok * cut.group;
            const __nv_bfloat16* src = p.q + (g.q0 + tok) * p.q_stride + (g.head * cut.group + h) * D + 8 * c;
            const int64_t wrap = p.q_stride - static_cast<int64_t>(cut.group) * D;
            const uint32_t to = base + (c >> 3) * L::kHalf;
#pragma unroll 4
            for (int r = r0; r < R; r += S) {
                const uint32_t dst = to + (r >> 7) * L::kTile + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4);
                const bool in = r < g.rows;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(in ? src : p.q),
                             "r"(in ? 16 : 0)
                             : "memory");
                src += S * D;
                h += S;
                for (int k = 0; k < S && h >= cut.group; ++k) {
                    h -= cut.group;
                    src += wrap;
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_shared();
            // 9 arrivals a lane stand for the 288 of the first segment.
            asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], 9;\n\t}" ::"r"(
                             smem_addr(&sh.q_full[(turn - 1) & 1]))
                         : "memory");
        }
    } else if (warp >= kConvertWarp) {
        uint32_t turn = 0, count = 0;
        bool ok = true;
        Segment g;
        const int t = threadIdx.x - 32 * kConvertWarp;
        auto convert = [&](int step) {
            const uint32_t rs = count % L::kRawSlots, slot = count % L::kSlots;
            const uint32_t turns = count / L::kSlots;
            ok = ok && mbar_wait(smem_addr(&sh.raw_full[rs]), (count / L::kRawSlots) & 1, wait) &&
                 (!turns || mbar_wait(smem_addr(&sh.kv_empty[slot]), (turns - 1) & 1, wait));
            if (!ok) return;
            int lo, hi;
            tile_rows(g, step, lo, hi);
            // A thread takes the same 16 elements of every 2048 / D-th row, so its
            // addresses (and its place in the swizzle) move by constants.
            constexpr int kRows = 2048 / D, kTurns = kTcKeys / kRows;
            const int r0 = t / (D / 16), c = t % (D / 16), x = 2 * (c & 3);
            const uint32_t src = base + L::kRaw + rs * L::kRawTile + t * 16;
            const uint32_t dst = base + L::kRing + slot * L::kTile + (c >> 2) * L::kHalf + r0 * 128;
            const uint32_t d0 = dst + ((x ^ (r0 & 7)) << 4), d1 = dst + (((x + 1) ^ (r0 & 7)) << 4);
            const bool whole = lo == 0 && hi == kTcKeys;
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                uint4 w = lds128(src + k * 2048);
                if (!whole && (r0 + k * kRows < lo || r0 + k * kRows >= hi)) w = make_uint4(0, 0, 0, 0);
                const uint2 a = e4m3x4_to_f16x4(w.x), b = e4m3x4_to_f16x4(w.y), d = e4m3x4_to_f16x4(w.z),
                            e = e4m3x4_to_f16x4(w.w);
                sts128(d0 + k * kRows * 128, a.x, a.y, b.x, b.y);
                sts128(d1 + k * kRows * 128, d.x, d.y, e.x, e.y);
            }
            fence_proxy_async_shared();
            mbar_arrive(smem_addr(&sh.raw_empty[rs]));
            mbar_arrive(smem_addr(&sh.kv_full[slot]));
            ++count;
        };
        // q; 2^-e brings a row's largest magnitude to [1, 2). The sign of its KV
        // head's scale goes with it (or a NaN): the factor of the scores has to
        // be positive, since masked ones are -inf.
        auto convert_q = [&]() {
            ok = ok && (turn < 2 || mbar_wait(smem_addr(&sh.q_empty), turn & 1, wait));
            if (!ok) return;
#pragma unroll 1
            for (int r = t; r < R; r += 128) {
                const uint4* src = reinterpret_cast<const uint4*>(q_row(p, g, r));
                const uint32_t row = base + (r >> 7) * L::kTile + (r & 127) * 128;
                const float ks = p.cache.k_scale ? p.cache.k_scale[g.head] : 1.f;
                float top = 0.f;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 w = src ? src[c] : make_uint4(0, 0, 0, 0);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        top = fmaxf(top, fmaxf(fabsf(half_of<false>(u[x], 0)), fabsf(half_of<false>(u[x], 1))));
                }
                const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -120), 120);
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) *
                                   (ks == ks ? copysignf(1.f, ks) : ks);
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 w = src ? src[c] : make_uint4(0, 0, 0, 0);
                    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        u[x] = pack_f16x2(half_of<false>(u[x], 0) * down, half_of<false>(u[x], 1) * down);
                    sts128(row + (c >> 3) * L::kHalf + (((c & 7) ^ (r & 7)) << 4), u[0], u[1], u[2], u[3]);
                }
                sh.q_exp[(turn - 1) & 1][r] = static_cast<int8_t>(e);
            }
            fence_proxy_async_shared();
            mbar_arrive(smem_addr(&sh.q_full[(turn - 1) & 1]));
        };
        while (ok && take_segment(sh, turn, g, wait)) {
#pragma unroll 1
            for (int i = 0; i < 2 * g.steps && ok; ++i) {
                bool v;
                convert(ring_order<SPLIT>(i, g.steps, v));
                if (i == 0) convert_q();
            }
            __syncwarp();
        }
    }
    } else {
        if constexpr (E4M3) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int wg = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_at = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t st = tmem + wg * 128 + lane_at;      // S, then P
        const uint32_t ot = tmem + 256 + wg * D + lane_at;  // O
        uint32_t tiles[2] = {0, 0};  // tiles of each stream before this segment
        uint32_t meets = 0, votes = 0, turn_seg = 0;
        uint32_t used = 0;           // ring tiles before this segment
        bool ok = true, skipped = false;
        Segment g;
        // A warp gives up as one: what follows are warp-wide TMEM accesses.
        auto wait_all = [&](uint64_t& bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(smem_addr(&bar), parity, wait));
            return ok;
        };
        auto meet = [&]() {  // both groups of warps
            mbar_arrive(smem_addr(&sh.meet));
            wait_all(sh.meet, meets & 1);
            ++meets;
        };

        while (ok && take_segment(sh, turn_seg, g, wait)) {
            if (!E4M3 && turn_seg == 1) {
#pragma unroll 4
                for (int i = threadIdx.x; i < R * (D / 8); i += 256) {
                    const int row = i / (D / 8), c = i % (D / 8);
                    const __nv_bfloat16* src = q_row(p, g, row);
                    const uint32_t dst = base + (row >> 7) * L::kTile + (c >> 3) * L::kHalf + (row & 127) * 128 +
                                         (((c & 7) ^ (row & 7)) << 4);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                                 "l"(src ? src + 8 * c : p.q), "r"(src ? 16 : 0)
                                 : "memory");
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_shared();
                mbar_arrive(smem_addr(&sh.q_full[0]));
            }
            const int tr = (SPLIT ? 0 : wg * 128) + r;  // row in the row tile
            const bool in = tr < g.rows;
            const int tok = cut.by_group.div(g.row0 + (in ? tr : 0));
            int pos = g.start + tok;
            if (cut.placed && in) pos = window_from(p.positions + g.q0 + tok, g.start, g.end, cut.window);
            // Keys below `open` are visible to every row of the stream (without
            // a window); keys from `all_from` on have left no row's window.
            const int open = cut.tree ? g.start : g.start + cut.by_group.div(g.row0 + (SPLIT ? 0 : wg * 128)) + 1;
            const int all_from = g.end - cut.window, open_end = min(open, g.end);
            // This row's first and last visible key.
            const int first = max(g.begin, cut.window ? pos - cut.window + 1 : 0);
            const int last = in ? min(cut.tree ? g.end - 1 : pos, g.end - 1) : -1;
            const int n_all = g.steps, n_my = SPLIT ? (n_all + 1 - wg) / 2 : n_all;
            float mul = p.map.mul;
            // q_full alternates between two barriers: q of the segment after next
            // waits for this one's last probabilities, so no group with tiles can
            // still be here when its barrier's phase comes round again (on one
            // barrier the next segment's q would do that, from the moment this
            // one's last scores are taken). A group without tiles has no use for
            // it. A count of these warps in q_empty instead measured the same or
            // slower (256 requests x 8 tokens over 300: 205 us against 194).
            if (E4M3 && n_my) {
                if (!wait_all(sh.q_full[(turn_seg - 1) & 1], ((turn_seg - 1) >> 1) & 1)) break;
                const int e = sh.q_exp[(turn_seg - 1) & 1][(SPLIT ? 0 : wg * 128) + r];
                const float ks = p.cache.k_scale ? p.cache.k_scale[g.head] : 1.f;
                mul = fmaxf(fabsf(mul * ks * __uint_as_float(static_cast<uint32_t>(127 + e) << 23)), 1e-36f);
            }
            float m = -INFINITY, l = 0.f;

            for (int jj = 0; jj < n_my; ++jj) {
                const int j = SPLIT ? 2 * jj + wg : jj;
                const uint32_t turn = tiles[wg] + jj;
                if (!wait_all(sh.s_full[wg], turn & 1)) break;
                tc::fence_after_sync();
                float s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_load32(st + c * 32, s + c * 32);
                tc::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) loaded32(s + c * 32);
                if constexpr (CAP) {
                    // ScoreMap's formula, two scores an instruction where there is one.
                    const uint64_t cmul = f32x2_pack(mul, mul), one = f32x2_pack(1.f, 1.f);
                    const uint64_t cap = f32x2_pack(p.map.cap, p.map.cap), cap2 = f32x2_pack(-2.f * p.map.cap, -2.f * p.map.cap);
#pragma unroll
                    for (int c = 0; c < 128; c += 2) {
                        const float2 x = f32x2_unpack(f32x2_mul(f32x2_pack(s[c], s[c + 1]), cmul));
                        const float2 d = f32x2_unpack(f32x2_add(f32x2_pack(exp2_fast(x.x), exp2_fast(x.y)), one));
                        const float2 t = f32x2_unpack(f32x2_fma(f32x2_pack(rcp_fast(d.x), rcp_fast(d.y)), cap2, cap));
                        s[c] = t.x;
                        s[c + 1] = t.y;
                    }
                }
                const int key0 = (g.tile0 + j) * kTcKeys;
                // Some row does not see some key of this tile.
                const bool edge = key0 + kTcKeys > open_end || (cut.window && key0 < all_from);
                if (edge) {
                    uint32_t see[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int lo = max(first - key0 - 32 * w, 0), hi = min(last - key0 - 32 * w, 31);
                        see[w] = hi >= lo ? (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo) : 0u;
                    }
                    if (cut.tree && in && key0 + kTcKeys > g.start) {
                        const unsigned long long word = p.tree_mask[g.q0 + tok];
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            // Bit b of this word is new token key0 + 32 w + b - start.
                            const int d = key0 + 32 * w - g.start;
                            uint32_t allow;
                            if (d >= 64) allow = 0;
                            else if (d >= 0) allow = static_cast<uint32_t>(word >> d);
                            else if (d <= -32) allow = 0xffffffffu;
                            else allow = (static_cast<uint32_t>(word) << -d) | ((1u << -d) - 1);
                            see[w] &= allow;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (!(see[c >> 5] >> (c & 31) & 1)) s[c] = -INFINITY;
                }
                float top4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c < 124; c += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x) top4[x] = max3(top4[x], s[c + x], s[c + 4 + x]);
                float top = max3(max3(top4[0], top4[1], top4[2]), top4[3], max3(s[124], s[125], fmaxf(s[126], s[127])));
                if constexpr (!CAP) top *= mul;
                if (__any_sync(0xffffffffu, top > m + kTcSlack)) {
                    const float up = fmaxf(m, top);
                    const float f = up == m ? 1.f : exp2_fast(m - up);
                    m = up;
                    l *= f;
                    if (jj) {  // the first product of a segment overwrites O
                        if (!wait_all(sh.pv_done[wg], (turn - 1) & 1)) break;
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tmem_load32(ot + c, o);
                            tc::tmem_wait_ld();
                            loaded32(o);
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] *= f;
                            tc::tmem_store16(ot + c, *reinterpret_cast<const uint32_t(*)[16]>(&o[0]));
                            tc::tmem_store16(ot + c + 16, *reinterpret_cast<const uint32_t(*)[16]>(&o[16]));
                        }
                    }
                }
                if (skipped && !edge) {  // before this tile's first half is handed over
                    if (r == 0) sts_u32_volatile(smem_addr(&sh.skip[wg]), 0);
                    skipped = false;
                }
                const float base_m = m == -INFINITY ? 0.f : m;
                uint64_t sum2[2] = {0, 0};
                const uint64_t mul2 = f32x2_pack(mul, mul), one2 = f32x2_pack(1.f, 1.f);
                const uint64_t neg2 = f32x2_pack(-base_m, -base_m);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const uint64_t pair = f32x2_pack(s[c * 32 + 2 * x], s[c * 32 + 2 * x + 1]);
                        const float2 t = f32x2_unpack(f32x2_fma(pair, CAP ? one2 : mul2, neg2));
                        const float a = exp2_fast(t.x), b = exp2_fast(t.y);
                        sum2[x & 1] = f32x2_add(sum2[x & 1], f32x2_pack(a, b));
                        w[x] = E4M3 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
                    }
                    tc::tmem_store16(st + c * 16, w);
                    if (c == 1 && !edge) {
                        tc::tmem_wait_st();
                        tc::fence_before_sync();
                        mbar_arrive(smem_addr(&sh.p_full[wg][0]));
                    }
                }
                const float2 sums = f32x2_unpack(f32x2_add(sum2[0], sum2[1]));
                l += sums.x + sums.y;
                tc::tmem_wait_st();
                // V of a key that some rows see and others do not may hold an
                // infinity or a NaN, and 0 * NaN is NaN: then the rows' own
                // threads take the product, without the keys they do not see.
                bool bad = false;
                if (edge) {
                    const uint32_t n = used + v_place<SPLIT>(j, n_all);
                    const uint32_t v = base + L::kRing + (n % L::kSlots) * L::kTile;
                    if (!wait_all(sh.kv_full[n % L::kSlots], (n / L::kSlots) & 1)) break;
                    if (v_not_finite<D, E4M3>(v, r)) sts_u32_volatile(smem_addr(&sh.bad[wg]), turn + 1);
                    mbar_arrive(smem_addr(&sh.vote[wg]));
                    if (!wait_all(sh.vote[wg], votes & 1)) break;
                    ++votes;
                    bad = lds_u32_volatile(smem_addr(&sh.bad[wg])) == turn + 1;
                    if (bad) {
                        if (jj && !wait_all(sh.pv_done[wg], (turn - 1) & 1)) break;
                        tc::fence_after_sync();
                        add_tile_by_rows<D, E4M3>(ot, st, v, L::kHalf, jj == 0);
                    }
                    if (r == 0) sts_u32_volatile(smem_addr(&sh.skip[wg]), bad);
                    skipped = bad;
                }
                tc::fence_before_sync();
                if (edge) mbar_arrive(smem_addr(&sh.p_full[wg][0]));
                mbar_arrive(smem_addr(&sh.p_full[wg][1]));
            }
            // The end of this segment.
            float f_own = 1.f, f_other = 0.f, sum = l, topm = m;
            if constexpr (SPLIT) {
                sh.m[wg][r] = m;
                sh.l[wg][r] = l;
                meet();
                const float m2 = sh.m[wg ^ 1][r], l2 = sh.l[wg ^ 1][r];
                topm = fmaxf(m, m2);
                const float b = topm == -INFINITY ? 0.f : topm;
                f_own = l == 0.f ? 0.f : exp2_fast(m - b);
                f_other = l2 == 0.f ? 0.f : exp2_fast(m2 - b);
                sum = f_own * l + f_other * l2;
            }
            const uint32_t after[2] = {tiles[0] + (SPLIT ? (n_all + 1) / 2 : n_all),
                                       tiles[1] + (SPLIT ? n_all / 2 : n_all)};
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if ((SPLIT || s == wg) && after[s] != tiles[s])
                    wait_all(sh.pv_done[s], (after[s] - 1) & 1);
            tc::fence_after_sync();
            const int slot = 2 * blockIdx.x + g.begins;
            if (g.parts && threadIdx.x == 0)
                parts.split[blockIdx.x] = Split{g.parts, g.row0, g.rows, g.q0, g.head};
            if (ok) {
                const int64_t to = static_cast<int64_t>(g.q0 + tok) * p.q_heads + g.head * cut.group + g.row0 + tr -
                                   tok * cut.group;
                const float vs = E4M3 && p.cache.v_scale ? p.cache.v_scale[g.head] : 1.f;
                const float inv = sum == 0.f ? 0.f : vs / sum;
                // SPLIT: each group takes half of the columns of both accumulators.
                constexpr int CH = SPLIT ? D / 64 : D / 32;
#pragma unroll 1
                for (int c = 0; c < CH; ++c) {
                    float o[32];
                    const int col = ((SPLIT ? wg * CH : 0) + c) * 32;
                    tmem_load32(ot + col, o);
                    if constexpr (SPLIT) {
                        float o2[32];
                        tmem_load32(tmem + 256 + (wg ^ 1) * D + lane_at + col, o2);
                        tc::tmem_wait_ld();
                        loaded32(o);
                        loaded32(o2);
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            o[x] = l == 0.f ? 0.f : f_own * o[x];
                            o[x] = f_other == 0.f ? o[x] : fmaf(f_other, o2[x], o[x]);
                        }
                    } else {
                        tc::tmem_wait_ld();
                        loaded32(o);
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = l == 0.f ? 0.f : o[x];
                    }
                    if (in && g.whole) {
                        uint4* dst = reinterpret_cast<uint4*>(p.out + to * D + col);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            dst[x] = make_uint4(pack_bf16x2(o[8 * x] * inv, o[8 * x + 1] * inv),
                                                pack_bf16x2(o[8 * x + 2] * inv, o[8 * x + 3] * inv),
                                                pack_bf16x2(o[8 * x + 4] * inv, o[8 * x + 5] * inv),
                                                pack_bf16x2(o[8 * x + 6] * inv, o[8 * x + 7] * inv));
                    } else if (in) {  // [D / 4][R]: a warp writes 512 bytes in a row
                        float4* dst = reinterpret_cast<float4*>(parts.o) +
                                      (static_cast<int64_t>(slot) * (D / 4) + (col >> 2)) * R + tr;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            dst[x * R] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                    }
                    __syncwarp();
                }
                if (in && (!SPLIT || wg == 0)) {
                    if (!g.whole) parts.ml[slot * R + tr] = make_float2(topm, sum);
                    else if (p.lse) p.lse[to] = sum == 0.f ? -INFINITY : (topm + log2f(sum)) / kLog2e;
                }
            }
            tiles[0] = after[0];
            tiles[1] = after[1];
            used += 2 * n_all;
            tc::fence_before_sync();
            if constexpr (SPLIT) meet();  // both accumulators have been read
        }
    }
    __syncthreads();
    pdl_launch_dependents();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

template <int D, bool SPLIT, bool CAP, bool E4M3>
cudaError_t launch(const Params& p, const CUtensorMap& k, const CUtensorMap& v, int ctas, cudaStream_t stream) {
    constexpr int smem = Layout<D, SPLIT, E4M3>::kBytes;
    static_assert(smem + sizeof(Shared<SPLIT, E4M3>) <= 227 * 1024, "shared memory");
    static thread_local int ready_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (ready_device != dev) {
        e = cudaFuncSetAttribute(attention_tc_kernel<D, SPLIT, CAP, E4M3>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready_device = dev;
    }
    PdlLaunch l(dim3(ctas), dim3(tc_threads(E4M3)), smem, stream);
    return cudaLaunchKernelEx(&l.cfg, attention_tc_kernel<D, SPLIT, CAP, E4M3>, k, v, p);
}

template <int D, bool E4M3>
cudaError_t launch_d(const Params& p, bool split, const CUtensorMap& k, const CUtensorMap& v, int ctas,
                     cudaStream_t stream) {
    const bool cap = p.map.cap != 0.f;
    if (split)
        return cap ? launch<D, true, true, E4M3>(p, k, v, ctas, stream)
                   : launch<D, true, false, E4M3>(p, k, v, ctas, stream);
    return cap ? launch<D, false, true, E4M3>(p, k, v, ctas, stream)
               : launch<D, false, false, E4M3>(p, k, v, ctas, stream);
}

bool is_split(int64_t rows) { return rows <= 128; }

// Tensor maps of recent pools, per host thread: they depend on addresses and
// shapes only.
struct PoolMaps {
    int dev = -1;
    CacheView view{};
    bool e4m3 = false;
    CUtensorMap k, v;
};
cudaError_t pool_maps(int dev, const CacheView& c, bool e4m3, const PoolMaps** out) {
    static thread_local PoolMaps slots[64];
    static thread_local int next = 0;
    for (const PoolMaps& s : slots)
        if (s.view.k == c.k && s.view.v == c.v && s.dev == dev && s.view.page_stride == c.page_stride &&
            s.view.num_pages == c.num_pages && s.view.kv_heads == c.kv_heads && s.view.page_shift == c.page_shift &&
            s.view.head_dim == c.head_dim && s.e4m3 == e4m3) {
            *out = &s;
            return cudaSuccess;
        }
    PoolMaps& s = slots[next];
    s.dev = -1;
    cudaError_t e = encode_kv_map(&s.k, c.k, c, e4m3);
    if (e == cudaSuccess) e = encode_kv_map(&s.v, c.v, c, e4m3);
    if (e != cudaSuccess) return e;
    s.view = c;
    s.e4m3 = e4m3;
    s.dev = dev;
    next = (next + 1) % 64;
    *out = &s;
    return cudaSuccess;
}

}  // namespace

size_t tc_workspace_bytes(int64_t rows, int d, int num_sms) {
    return parts_bytes(num_sms, is_split(rows) ? 128 : 256, d);
}

cudaError_t launch_tc(const Params& in, bool e4m3, int64_t rows, int max_seq, int num_sms, cudaStream_t stream) {
    Params p = in;
    const bool split = is_split(rows);
    p.cut.row_shift = split ? 7 : 8;
    p.cut.key_shift = 7;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const PoolMaps* maps = nullptr;
    if (e == cudaSuccess) e = pool_maps(dev, p.cache, e4m3, &maps);
    if (e != cudaSuccess) return e;
    const CUtensorMap &k = maps->k, &v = maps->v;
    const int ctas = ctas_for(p, rows, max_seq, num_sms);
    if (p.cache.head_dim == 64)
        e = e4m3 ? launch_d<64, true>(p, split, k, v, ctas, stream)
                 : launch_d<64, false>(p, split, k, v, ctas, stream);
    else
        e = e4m3 ? launch_d<128, true>(p, split, k, v, ctas, stream)
                 : launch_d<128, false>(p, split, k, v, ctas, stream);
    return e == cudaSuccess ? launch_join(p, e4m3, true, ctas, stream) : e;
}

}  // namespace attn
}  // namespace mxfp4
