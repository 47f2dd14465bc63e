// Attention of a step's new tokens over the paged cache, for many rows per KV
// head (verify steps of several tokens, prompt chunks): both products on the
// fifth-generation tensor cores, bf16 cache.
//
// One CTA per SM works through its run of key tiles (128 keys, see
// attention_common.cuh). Two streams of work alternate on the tensor cores,
// each with a score tile S [128 rows][128 keys] and an output accumulator O
// [128 rows][D] in TMEM: while one stream's scores become probabilities, the
// other's products run.
//   more than 128 rows: stream s is rows 128 s .. of a 256-row tile; both
//                       read the same K and V tiles.
//   at most 128 rows:   both streams take the same rows, stream s the key
//                       tiles of parity s; their accumulators are joined at the end.
// Warps: 0-3 and 4-7 turn the scores of stream 0 and 1 into probabilities,
// one thread per row (TMEM lane), so maxima and sums need no exchange; P goes
// back to TMEM in bf16 over the first half of S and is the A operand of P V.
// Warp 8 issues the products, warp 9 the TMA copies of K and V pages into a
// ring of [128 keys][64 elements] boxes (128-byte swizzle): K is a K-major B
// operand of Q K^T, V as it lies in memory an N-major B operand of P V.
//
// A row's running maximum is raised only when a score exceeds it by 2^8, so
// O is seldom rescaled (by the row's own thread, after the stream's last
// product). Score maxima, sums and accumulators are fp32.
#include <cuda.h>

#include "attention_common.cuh"
#include "step_launch.h"
#include "tc_common.cuh"

namespace mxfp4 {
namespace attn {
namespace {

constexpr int kTcThreads = 384;  // 12 warps, 10 of them at work: registers are dealt by groups of 4 warps
constexpr int kTcKeys = 128;   // keys per tile
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr float kTcSlack = 8.f;

template <int D, bool SPLIT>
struct Layout {
    static constexpr int kTile = kTcKeys * D * 2;      // bytes of a K or V tile, or of a 128-row q tile
    static constexpr int kHalf = 128 * 128;            // bytes of [128 rows][64 elements]
    static constexpr int kQ = (SPLIT ? 1 : 2) * kTile;
    // 5 tiles of 32 KB, or 8 of 16 KB: three or more in flight beside the two in use.
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr int kRing = kQ;                   // offset of the ring
    static constexpr int kBytes = kQ + kSlots * kTile + 1024;  // and alignment
};

// Everything the warps tell one another.
template <bool SPLIT>
struct Shared {
    int64_t before[kGroups + 1];
    uint64_t kv_full[8], kv_empty[8], patch, q_full[2], s_full[2], p_full[2][2], pv_done[2], vote[2], meet, drain;
    float m[2][SPLIT ? 128 : 1], l[2][SPLIT ? 128 : 1];  // of the two streams' rows
    uint32_t tmem;
    uint32_t bad[2];   // last tile (counted from 1) of each stream whose V is not finite
    uint32_t skip[2];  // the stream's product with V has been taken by its warps
    int abort;
};

__device__ __forceinline__ uint32_t idesc_f16(uint32_t n, bool b_n_major) {
    // fp32 accumulators, bf16 operands, B's major, N / 8, M / 16 (M = 128).
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(b_n_major) << 16) | ((n >> 3) << 17) | (8u << 24);
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
template <int D>
__device__ __forceinline__ bool v_not_finite(uint32_t v, int r) {
    uint32_t bad = 0;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint4 w = lds128(v + (c * 128 + r) * 16);
        bad |= __vcmpeq2(w.x & 0x7f807f80u, 0x7f807f80u) | __vcmpeq2(w.y & 0x7f807f80u, 0x7f807f80u) |
               __vcmpeq2(w.z & 0x7f807f80u, 0x7f807f80u) | __vcmpeq2(w.w & 0x7f807f80u, 0x7f807f80u);
    }
    return bad != 0;
}

// O += P V of one tile by the rows' own threads, leaving out the keys whose
// probability is 0. Warp-wide.
template <int D>
__device__ __noinline__ void add_tile_by_rows(uint32_t ot, uint32_t pt, uint32_t v, uint32_t half_bytes, bool first) {
#pragma unroll 1
    for (int col = 0; col < D; col += 32) {
        float o[32];
        tmem_load32(ot + col, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = first ? 0.f : o[x];
#pragma unroll 1
        for (int k2 = 0; k2 < kTcKeys / 2; ++k2) {
            uint32_t pair;
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(pair) : "r"(pt + k2) : "memory");
            tc::tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float f = __uint_as_float(h ? pair & 0xffff0000u : pair << 16);
                if (f == 0.f) continue;
                const int k = 2 * k2 + h;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int chunk = (col >> 3) + c;
                    const uint4 w = lds128(v + (chunk >> 3) * half_bytes + k * 128 + (((chunk & 7) ^ (k & 7)) << 4));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        o[8 * c + 2 * x] += f * __uint_as_float(u[x] << 16);
                        o[8 * c + 2 * x + 1] += f * __uint_as_float(u[x] & 0xffff0000u);
                    }
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c)
            tc::tmem_store16(ot + col + 16 * c, *reinterpret_cast<const uint32_t(*)[16]>(&o[16 * c]));
        tc::tmem_wait_st();
    }
}

// A part of an item: key tiles [tile, tile + steps).
struct Segment {
    Item it;
    int steps;
    int rows;   // of the row tile
    bool whole;
    int64_t unit;
};

__device__ __forceinline__ bool next_segment(const Params& p, const int64_t* before, int64_t& unit, int64_t unit_end,
                                             Segment& g) {
    if (unit >= unit_end) return false;
    g.it = locate(p.cut, p.batch, p.cache.page_shift, before, unit);
    g.steps = static_cast<int>(min(unit_end - unit, static_cast<int64_t>(g.it.tiles - g.it.tile)));
    g.rows = min(1 << p.cut.row_shift, g.it.n * p.cut.group - (g.it.rt << p.cut.row_shift));
    g.whole = g.it.tile == 0 && g.steps == g.it.tiles;
    g.unit = unit;
    unit += g.steps;
    return true;
}

// ------------------------------------------------------------------ copies
template <int D, bool SPLIT>
struct Loader {
    using L = Layout<D, SPLIT>;
    const Params& p;
    Shared<SPLIT>& sh;
    const CUtensorMap *kmap, *vmap;
    WaitCtx wait;
    uint32_t base;
    int lane;
    uint32_t count = 0, patches = 0;
    bool ok = true;

    // This lane's box of a tile: its page, or -1. Read well before the copy
    // that needs it (a table read takes as long as a copy).
    __device__ int page_for(const Segment& g, int step) const {
        const CacheView& cv = p.cache;
        const int box = min(1 << cv.page_shift, kTcKeys), boxes = kTcKeys / box;
        const int key = (g.it.begin / kTcKeys + g.it.tile + step) * kTcKeys + (lane & (boxes - 1)) * box;
        if (step >= g.steps || key >= g.it.end || key + box <= g.it.begin) return -1;
        return page_of(p.batch, g.it.b, key, cv.page_shift, cv.num_pages);
    }

    __device__ void tile(const Segment& g, int step, bool v, int pg) {
        if (!ok) return;
        const CacheView& cv = p.cache;
        const uint32_t slot = count % L::kSlots, turn = count / L::kSlots;
        const uint32_t full = smem_addr(&sh.kv_full[slot]);
        if (turn && !mbar_wait(smem_addr(&sh.kv_empty[slot]), (turn - 1) & 1, wait)) {
            ok = false;
            return;
        }
        const int key0 = (g.it.begin / kTcKeys + g.it.tile + step) * kTcKeys;
        const int page = 1 << cv.page_shift;
        const int box = min(page, kTcKeys), boxes = kTcKeys / box;
        // Rows of V that hold no key of this item but lie in a page that
        // does: whatever is there must not meet the products (0 * NaN).
        const int lo = g.it.begin > key0 ? g.it.begin - key0 : 0, hi = min(g.it.end - key0, kTcKeys);
        const bool ragged = v && ((lo & (box - 1)) || (hi < kTcKeys && (hi & (box - 1))));
        const uint32_t bar = ragged ? smem_addr(&sh.patch) : full;
        if (lane == 0) mbar_arrive_expect_tx(bar, L::kTile);
        __syncwarp();
        const uint32_t dst = base + L::kRing + slot * L::kTile;
        if (lane < boxes * (D / 64)) {
            const int half = lane / boxes, b = lane & (boxes - 1), key = key0 + b * box;
            // A page coordinate past the pool reads as zeros.
            tma_load_4d(dst + half * L::kHalf + b * box * 128, v ? vmap : kmap, half * 64, key & (page - 1), g.it.head,
                        pg < 0 ? cv.num_pages : pg, bar);
        }
        __syncwarp();
        if (ragged) {
            if (!mbar_wait(bar, patches & 1, wait)) {
                ok = false;
                return;
            }
            ++patches;
            const int lo0 = lo & ~(box - 1), hi1 = (hi + box - 1) & ~(box - 1);
            for (int i = lane; i < kTcKeys * (D / 8); i += 32) {
                const int r = i / (D / 8), c = i % (D / 8);
                if ((r >= lo0 && r < lo) || (r >= hi && r < hi1))
                    sts128(dst + (c >> 3) * L::kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4), 0, 0, 0, 0);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
        }
        ++count;
    }

    // After a wait ran out: the copies in flight land before the CTA ends.
    __device__ void drain() {
        const uint64_t t0 = global_timer_ns();
        for (uint32_t c = count > L::kSlots ? count - L::kSlots : 0; c < count; ++c)
            while (!mbar_try_wait(smem_addr(&sh.kv_full[c % L::kSlots]), (c / L::kSlots) & 1) &&
                   global_timer_ns() - t0 < kWaitLimitNs) {
            }
    }
};

template <int D, bool SPLIT, bool CAP>
__global__ void __launch_bounds__(kTcThreads, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ Params p) {
    using L = Layout<D, SPLIT>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared<SPLIT> sh;
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
    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int i = 0; i < 8; ++i) {
            mbar_init(smem_addr(&sh.kv_full[i]), 1);
            mbar_init(smem_addr(&sh.kv_empty[i]), 1);
        }
        mbar_init(smem_addr(&sh.patch), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&sh.q_full[s]), SPLIT ? 256 : 128);
            mbar_init(smem_addr(&sh.s_full[s]), 1);
            mbar_init(smem_addr(&sh.p_full[s][0]), 128);
            mbar_init(smem_addr(&sh.p_full[s][1]), 128);
            mbar_init(smem_addr(&sh.pv_done[s]), 1);
            mbar_init(smem_addr(&sh.vote[s]), 128);
            sh.bad[s] = sh.skip[s] = 0;
        }
        mbar_init(smem_addr(&sh.meet), 256);
        mbar_init(smem_addr(&sh.drain), 1);
        fence_barrier_init();
    }
    pdl_wait_previous();
    if (threadIdx.x == 0) parts.split[blockIdx.x] = make_int4(0, 0, 0, 0);
    tc::fence_before_sync();
    const int64_t total = count_units(cut, p.batch, p.cache.page_shift, sh.before);  // ends with a block barrier
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const int64_t share = share_of(cut, total, gridDim.x);
    int64_t unit = share * blockIdx.x;
    const int64_t unit_end = min(unit + share, total);
    Segment g;

    // 384 threads start with 168 registers each; the two groups that hold a
    // row of scores per thread take 208, the third keeps 88 (the sum is the same).
    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kLoadWarp) {
        Loader<D, SPLIT> ld{p, sh, &kmap, &vmap, wait, base, lane};
        while (next_segment(p, sh.before, unit, unit_end, g)) {
            int p0 = ld.page_for(g, 0), p1 = ld.page_for(g, 1), p2 = ld.page_for(g, 2);
            if constexpr (SPLIT) {  // the order in which the products need them
                ld.tile(g, 0, false, p0);
                if (g.steps > 1) ld.tile(g, 1, false, p1);
            }
            for (int j = 0; j < g.steps; ++j) {
                if constexpr (!SPLIT) ld.tile(g, j, false, p0);
                ld.tile(g, j, true, p0);
                if (SPLIT && j + 2 < g.steps) ld.tile(g, j + 2, false, p2);
                p0 = p1;
                p1 = p2;
                p2 = ld.page_for(g, j + 3);
            }
        }
        if (!ld.ok && lane == 0) ld.drain();
    } else if (warp == kMmaWarp) {
        // All lanes walk through the tiles, so that what the products are
        // given stays in uniform registers; one lane issues.
        const uint32_t idesc_qk = idesc_f16(kTcKeys, false), idesc_pv = idesc_f16(D, true);
        const uint64_t q_desc = tc::operand_desc(base), k_desc = tc::operand_desc(base + L::kRing);
        const uint64_t v_desc = tc::smem_desc(base + L::kRing, L::kHalf, 1024, tc::kLayoutSwizzle128);
        const bool one = elect_one();
        uint32_t used = 0;         // ring tiles taken
        uint32_t q_turn = 0;       // items begun
        uint32_t done[2] = {0, 0}; // probabilities taken, per stream
        bool ok = true;
        auto wait_for = [&](uint64_t& bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(smem_addr(&bar), parity, wait));
            return ok;
        };
        auto tile_ready = [&](uint32_t n) { return wait_for(sh.kv_full[n % L::kSlots], (n / L::kSlots) & 1); };
        auto qk = [&](int s, uint32_t n, bool frees) {
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
                if (frees) tc::commit_to(smem_addr(&sh.kv_empty[n % L::kSlots]));
            }
            __syncwarp();
        };
        // The two halves of a tile's keys: the second half's probabilities
        // come while the first half's product runs.
        auto pv = [&](int s, uint32_t n, bool first, bool frees) {
            const uint64_t v = v_desc + (n % L::kSlots) * (L::kTile >> 4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!wait_for(sh.p_full[s][h], done[s] & 1)) return false;
                tc::fence_after_sync();
                const bool skip = lds_u32_volatile(smem_addr(&sh.skip[s])) != 0;
                if (one && !skip) {
#pragma unroll
                    for (int i = h * kTcKeys / 32; i < (h + 1) * kTcKeys / 32; ++i)
                        mma_ts(tmem + 256 + s * D, tmem + s * 128 + i * 8, v + i * (2048 >> 4), idesc_pv,
                               !(first && i == 0));
                }
            }
            if (one) {
                tc::commit_to(smem_addr(&sh.pv_done[s]));
                if (frees) tc::commit_to(smem_addr(&sh.kv_empty[n % L::kSlots]));
            }
            __syncwarp();
            ++done[s];
            return true;
        };
        while (ok && next_segment(p, sh.before, unit, unit_end, g)) {
            const int n = __shfl_sync(0xffffffffu, g.steps, 0);
            if constexpr (SPLIT) {
                if (!wait_for(sh.q_full[0], q_turn & 1)) break;
                // Ring order: K0 K1 V0 K2 V1 K3 ...
                auto k_at = [&](int j) { return used + (j < 2 ? j : 2 * j - 1); };
                auto v_at = [&](int j) { return used + min(n, j + 2) + j; };
                for (int j = 0; j < min(n, 2) && tile_ready(k_at(j)); ++j) qk(j, k_at(j), true);
                for (int j = 0; j < n && ok; ++j) {
                    const int s = j & 1;
                    if (!tile_ready(v_at(j)) || !pv(s, v_at(j), j < 2, true)) break;
                    if (j + 2 < n && tile_ready(k_at(j + 2))) qk(s, k_at(j + 2), true);
                }
            } else {
                if (!tile_ready(used)) break;
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (wait_for(sh.q_full[s], q_turn & 1)) qk(s, used, s == 1);
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t v = used + 2 * j + 1, k = v + 1;
                    const bool more = j + 1 < n;
                    if (!tile_ready(v)) break;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (!pv(s, v, j == 0, s == 1)) break;
                        if (more && (s == 1 || tile_ready(k))) qk(s, k, s == 1);
                    }
                }
            }
            used += 2 * n;
            ++q_turn;
        }
        if (!ok && one) {  // products in flight end before TMEM is given back
            tc::commit_to(smem_addr(&sh.drain));
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(smem_addr(&sh.drain), 0) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int wg = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_at = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t st = tmem + wg * 128 + lane_at;            // S, then P
        const uint32_t ot = tmem + 256 + wg * D + lane_at;        // O
        uint32_t tiles[2] = {0, 0};  // tiles of each stream before this segment
        uint32_t meets = 0, votes = 0;
        uint32_t used = 0;           // ring tiles before this segment
        bool ok = true, skipped = false;
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
        // q rows of a segment into shared memory: this stream's 128 rows, or
        // (SPLIT) half of the elements of the one 128-row tile.
        auto load_q = [&](const Segment& s) {
            const int row = s.it.rt * R + (SPLIT ? 0 : wg * 128) + r;
            const bool in = (SPLIT ? 0 : wg * 128) + r < s.rows;
            const int i = in ? cut.by_group.div(row) : 0;
            const uint4* src = reinterpret_cast<const uint4*>(
                p.q + (s.it.first + i) * p.q_stride + (s.it.head * cut.group + (in ? row - i * cut.group : 0)) * D);
            const uint32_t dst = base + (SPLIT ? 0 : wg * L::kTile);
            constexpr int N = SPLIT ? D / 16 : D / 8;
            const int c0 = SPLIT ? wg * N : 0;
            uint4 w[N];
#pragma unroll
            for (int c = 0; c < N; ++c) w[c] = in ? src[c0 + c] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < N; ++c) {
                const int at = c0 + c;
                sts128(dst + (at >> 3) * L::kHalf + r * 128 + (((at & 7) ^ (r & 7)) << 4), w[c].x ^ p.q_flip,
                       w[c].y ^ p.q_flip, w[c].z ^ p.q_flip, w[c].w ^ p.q_flip);
            }
            fence_proxy_async_shared();
            mbar_arrive(smem_addr(&sh.q_full[SPLIT ? 0 : wg]));
        };

        bool more = next_segment(p, sh.before, unit, unit_end, g);
        if (more) load_q(g);
        while (more && ok) {
            const Item& it = g.it;
            const int row = it.rt * R + (SPLIT ? 0 : wg * 128) + r;
            const bool in = (SPLIT ? 0 : wg * 128) + r < g.rows;
            const int tok = in ? cut.by_group.div(row) : 0;
            const int start = it.seq - it.n, pos = start + tok;
            // Keys below `open` are visible to every row of the tile (without a window).
            const int open = cut.tree ? start : start + cut.by_group.div(it.rt * R) + 1;
            // Keys from `all_from` on have left no row's window.
            const int all_from = start + min(it.n - 1, cut.by_group.div((it.rt + 1) * R - 1)) - cut.window + 1;
            // This row's first and last visible key.
            const int first = max(it.begin, cut.window ? pos - cut.window + 1 : 0);
            const int last = in ? min(cut.tree ? it.seq - 1 : pos, it.end - 1) : -1;
            float m = -INFINITY, l = 0.f;
            const int n_all = g.steps, n_my = SPLIT ? (n_all + 1 - wg) / 2 : n_all;

            for (int jj = 0; jj < n_my; ++jj) {
                const int j = SPLIT ? 2 * jj + wg : jj;
                const uint32_t turn = tiles[wg] + jj;
                if (!wait_all(sh.s_full[wg], turn & 1)) break;
                tc::fence_after_sync();
                float s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_load32(st + c * 32, s + c * 32);
                tc::tmem_wait_ld();
                if constexpr (CAP) {
                    // ScoreMap's formula, two scores an instruction where there is one.
                    const uint64_t mul = f32x2_pack(p.map.mul, p.map.mul), one = f32x2_pack(1.f, 1.f);
                    const uint64_t cap = f32x2_pack(p.map.cap, p.map.cap), cap2 = f32x2_pack(-2.f * p.map.cap, -2.f * p.map.cap);
#pragma unroll
                    for (int c = 0; c < 128; c += 2) {
                        const float2 x = f32x2_unpack(f32x2_mul(f32x2_pack(s[c], s[c + 1]), mul));
                        const float2 d = f32x2_unpack(f32x2_add(f32x2_pack(exp2_fast(x.x), exp2_fast(x.y)), one));
                        const float2 t = f32x2_unpack(f32x2_fma(f32x2_pack(rcp_fast(d.x), rcp_fast(d.y)), cap2, cap));
                        s[c] = t.x;
                        s[c + 1] = t.y;
                    }
                }
                const int key0 = (it.begin / kTcKeys + it.tile + j) * kTcKeys;
                // Some row does not see some key of this tile.
                const bool edge = key0 + kTcKeys > min(open, it.end) || (cut.window && key0 < all_from);
                if (edge) {
                    uint32_t see[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int lo = max(first - key0 - 32 * w, 0), hi = min(last - key0 - 32 * w, 31);
                        see[w] = hi >= lo ? (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo) : 0u;
                    }
                    if (cut.tree && in && key0 + kTcKeys > start) {
                        const unsigned long long word = p.tree_mask[it.first + tok];
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            // Bit b of this word is new token key0 + 32 w + b - start.
                            const int d = key0 + 32 * w - start;
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
                if constexpr (!CAP) top *= p.map.mul;
                if (__any_sync(0xffffffffu, top > m + kTcSlack)) {
                    const float up = fmaxf(m, top);
                    const float f = up == m ? 1.f : exp2_fast(m - up);
                    m = up;
                    l *= f;
                    if (jj) {  // the first product of a segment overwrites O
                        if (!wait_all(sh.pv_done[wg], (turn - 1) & 1)) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tc::TmemLd<16>::load(ot + c * 16, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            tc::tmem_store16(ot + c * 16, o);
                        }
                    }
                }
                if (skipped && !edge) {  // before this tile's first half is handed over
                    if (r == 0) sts_u32_volatile(smem_addr(&sh.skip[wg]), 0);
                    skipped = false;
                }
                const float base_m = m == -INFINITY ? 0.f : m;
                uint64_t sum2[2] = {0, 0};
                const uint64_t mul2 = f32x2_pack(p.map.mul, p.map.mul), one2 = f32x2_pack(1.f, 1.f);
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
                        w[x] = pack_bf16x2(a, b);
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
                    const uint32_t n = used + (SPLIT ? min(n_all, j + 2) + j : 2 * j + 1);
                    const uint32_t v = base + L::kRing + (n % L::kSlots) * L::kTile;
                    if (!wait_all(sh.kv_full[n % L::kSlots], (n / L::kSlots) & 1)) break;
                    if (v_not_finite<D>(v, r)) sts_u32_volatile(smem_addr(&sh.bad[wg]), turn + 1);
                    mbar_arrive(smem_addr(&sh.vote[wg]));
                    if (!wait_all(sh.vote[wg], votes & 1)) break;
                    ++votes;
                    bad = lds_u32_volatile(smem_addr(&sh.bad[wg])) == turn + 1;
                    if (bad) {
                        if (jj && !wait_all(sh.pv_done[wg], (turn - 1) & 1)) break;
                        tc::fence_after_sync();
                        add_tile_by_rows<D>(ot, st, v, L::kHalf, jj == 0);
                    }
                    if (r == 0) sts_u32_volatile(smem_addr(&sh.skip[wg]), bad);
                    skipped = bad;
                }
                tc::fence_before_sync();
                if (edge) mbar_arrive(smem_addr(&sh.p_full[wg][0]));
                mbar_arrive(smem_addr(&sh.p_full[wg][1]));
            }
            if constexpr (SPLIT) {
                sh.m[wg][r] = m;
                sh.l[wg][r] = l;
                meet();  // both streams have taken their last scores: q may go
            }
            const Segment cur = g;
            more = next_segment(p, sh.before, unit, unit_end, g);
            if (more && ok) load_q(g);

            // The end of this segment.
            float f_own = 1.f, f_other = 0.f, sum = l, topm = m;
            if constexpr (SPLIT) {
                const float m2 = sh.m[wg ^ 1][r], l2 = sh.l[wg ^ 1][r];
                topm = fmaxf(m, m2);
                const float b = topm == -INFINITY ? 0.f : topm;
                f_own = l == 0.f ? 0.f : exp2_fast(m - b);
                f_other = l2 == 0.f ? 0.f : exp2_fast(m2 - b);
                sum = f_own * l + f_other * l2;
            }
            const uint32_t after[2] = {tiles[0] + (SPLIT ? (cur.steps + 1) / 2 : cur.steps),
                                       tiles[1] + (SPLIT ? cur.steps / 2 : cur.steps)};
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if ((SPLIT || s == wg) && after[s] != tiles[s])
                    wait_all(sh.pv_done[s], (after[s] - 1) & 1);
            tc::fence_after_sync();
            const int slot = 2 * blockIdx.x + (cur.it.tile == 0);
            const int tr = (SPLIT ? 0 : wg * 128) + r;  // row in the row tile
            if (!cur.whole && cur.it.tile == 0 && threadIdx.x == 0) {
                const int64_t end = cur.unit + cur.it.tiles - 1;
                parts.split[blockIdx.x] =
                    make_int4(static_cast<int>(end / share) - blockIdx.x + 1, cur.it.b, cur.it.rt, cur.it.head);
            }
            if (ok) {
                const int64_t to = static_cast<int64_t>(cur.it.first + tok) * p.q_heads + cur.it.head * cut.group +
                                   (in ? row - tok * cut.group : 0);
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                // SPLIT: each group takes half of the columns of both accumulators.
                constexpr int CH = SPLIT ? D / 64 : D / 32;
                const int c0 = SPLIT ? wg * CH : 0;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    float o[32];
                    const int col = (c0 + c) * 32;
                    tmem_load32(ot + col, o);
                    if constexpr (SPLIT) {
                        float o2[32];
                        tmem_load32(tmem + 256 + (wg ^ 1) * D + lane_at + col, o2);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            const float a = f_own == 0.f ? 0.f : f_own * o[x];
                            o[x] = f_other == 0.f ? a : fmaf(f_other, o2[x], a);
                        }
                    } else {
                        tc::tmem_wait_ld();
                        if (l == 0.f) {
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] = 0.f;
                        }
                    }
                    if (!in) continue;
                    if (cur.whole) {
                        uint4* dst = reinterpret_cast<uint4*>(p.out + to * D + col);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            dst[x] = make_uint4(pack_bf16x2(o[8 * x] * inv, o[8 * x + 1] * inv),
                                                pack_bf16x2(o[8 * x + 2] * inv, o[8 * x + 3] * inv),
                                                pack_bf16x2(o[8 * x + 4] * inv, o[8 * x + 5] * inv),
                                                pack_bf16x2(o[8 * x + 6] * inv, o[8 * x + 7] * inv));
                    } else {
                        float4* dst = reinterpret_cast<float4*>(
                            parts.o + (static_cast<int64_t>(slot) * R + tr) * D + col);
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            dst[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                    }
                }
                if (in && (!SPLIT || wg == 0)) {
                    if (!cur.whole) parts.ml[slot * R + tr] = make_float2(topm, sum);
                    else if (p.lse) p.lse[to] = sum == 0.f ? -INFINITY : (topm + log2f(sum)) / kLog2e;
                }
            }
            tiles[0] = after[0];
            tiles[1] = after[1];
            used += 2 * cur.steps;
            tc::fence_before_sync();
            if constexpr (SPLIT) meet();  // both accumulators have been read
        }
    }
    __syncthreads();
    pdl_launch_dependents();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

template <int D, bool SPLIT, bool CAP>
cudaError_t launch(const Params& p, const CUtensorMap& k, const CUtensorMap& v, int ctas, cudaStream_t stream) {
    constexpr int smem = Layout<D, SPLIT>::kBytes;
    static_assert(smem + sizeof(Shared<SPLIT>) <= 227 * 1024, "shared memory");
    static thread_local int ready_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (ready_device != dev) {
        e = cudaFuncSetAttribute(attention_tc_kernel<D, SPLIT, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready_device = dev;
    }
    PdlLaunch l(dim3(ctas), dim3(kTcThreads), smem, stream);
    return cudaLaunchKernelEx(&l.cfg, attention_tc_kernel<D, SPLIT, CAP>, k, v, p);
}

template <int D>
cudaError_t launch_d(const Params& p, bool split, const CUtensorMap& k, const CUtensorMap& v, int ctas,
                     cudaStream_t stream) {
    const bool cap = p.map.cap != 0.f;
    if (split) return cap ? launch<D, true, true>(p, k, v, ctas, stream) : launch<D, true, false>(p, k, v, ctas, stream);
    return cap ? launch<D, false, true>(p, k, v, ctas, stream) : launch<D, false, false>(p, k, v, ctas, stream);
}

int row_tile_of(int64_t rows) { return rows <= 128 ? 128 : 256; }

// Tensor maps of recent pools, per host thread: they depend on the pool's
// address and shape only.
struct MapSlot {
    int dev = -1;
    const void *k = nullptr, *v = nullptr;
    int64_t page_stride = 0;
    int num_pages = 0, kv_heads = 0, page_shift = 0, head_dim = 0;
    CUtensorMap kmap, vmap;
};

cudaError_t pool_maps(const CacheView& c, const MapSlot** out) {
    static thread_local MapSlot slots[64];
    static thread_local int next = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    for (const MapSlot& s : slots)
        if (s.dev == dev && s.k == c.k && s.v == c.v && s.page_stride == c.page_stride && s.num_pages == c.num_pages &&
            s.kv_heads == c.kv_heads && s.page_shift == c.page_shift && s.head_dim == c.head_dim) {
            *out = &s;
            return cudaSuccess;
        }
    MapSlot& s = slots[next];
    s.dev = -1;
    if ((e = encode_kv_map(&s.kmap, c.k, c)) != cudaSuccess || (e = encode_kv_map(&s.vmap, c.v, c)) != cudaSuccess)
        return e;
    s.k = c.k;
    s.v = c.v;
    s.page_stride = c.page_stride;
    s.num_pages = c.num_pages;
    s.kv_heads = c.kv_heads;
    s.page_shift = c.page_shift;
    s.head_dim = c.head_dim;
    s.dev = dev;
    next = (next + 1) % 64;
    *out = &s;
    return cudaSuccess;
}

}  // namespace

size_t tc_workspace_bytes(int64_t rows, int d, int num_sms) { return parts_bytes(num_sms, row_tile_of(rows), d); }

cudaError_t launch_tc(const Params& in, int64_t rows, int num_sms, cudaStream_t stream) {
    Params p = in;
    p.cut.row_shift = row_tile_of(rows) == 128 ? 7 : 8;
    p.cut.key_shift = 7;
    const MapSlot* maps = nullptr;
    cudaError_t e = pool_maps(p.cache, &maps);
    if (e != cudaSuccess) return e;
    const bool split = p.cut.row_shift == 7;
    e = p.cache.head_dim == 64 ? launch_d<64>(p, split, maps->kmap, maps->vmap, num_sms, stream)
                               : launch_d<128>(p, split, maps->kmap, maps->vmap, num_sms, stream);
    return e == cudaSuccess ? launch_join(p, false, num_sms, stream) : e;
}

}  // namespace attn
}  // namespace mxfp4
