// Products of microscaled activations with MXFP4 weights for any number of
// tokens:  y[t][n] = sum_k x[t][k] * w[n][k],  and with a gated epilogue
// h[t][j] = SiLU(y[t][j]) * y[t][inter + j], which comes out as MX codes again.
//
// Both operands go to the tensor cores as they are stored, with their block
// scales: kind::mxf8f6f4 for E4M3 activations (weights spread to a byte per
// code by the copy), kind::mxf4 for E2M1 ones (both packed, twice the depth per
// instruction). Sums are fp32 in TMEM; y is rounded once, h not at all before
// its codes.
//
// A tile is 128 tokens (a pair of CTAs: 256) x `width` weight rows (width: a
// multiple of 32 up to 256; for the gated form the first half are gate rows, the
// second the up rows of the same outputs, so a thread finds both of its token in
// one TMEM lane). A stage is 128 bytes of every row: 128 values of k, or 256 in
// E2M1. Where there are few tiles, the CTAs (or pairs) of a cluster take a part of
// k each and hand their sums on through distributed shared memory.
//
// What bounds a stage: its products (512 cycles at 128 x 256 per SM in E4M3, and no
// less than 119 each however narrow), and shared memory, where every byte is
// written once and read once at 128 bytes a cycle: 512 cycles for a pair's 256-wide
// tile, 768 for a lone CTA's. Measured in CUDA graphs (and as calls from Python one
// after another, warmer): 4,096 tokens x 7,168 x 2 x 18,432 gated 610 to 645 us (653;
// 3.4 to 3.5 PFLOP/s, under the power cap), 4,096 x 18,432 x 7,168 in E2M1 150 us
// (167; 7.2 and 6.5), 512 x 7,168 x 9,216 25.7 us (27), 61 x 7,168 x 129,280 92 to 94
// us (100; 5.5 TB/s), 16 x 7,168 x 7,168 12 to 13 us (13), of which the products take
// 4 and the rest is the call's beginning, the exchange of its sums and its end.
//
// One CTA per SM walks over tiles, warp-specialised:
//   0-7    epilogue: warp w reads the lanes (tokens) 32 (w % 4) .. of the
//          accumulator, 32-column chunks by turns with warp w ^ 4
//   8      copies codes (TMA) into a ring of stages
//   9      issues the scales' copies into TMEM and the products
//   10-15  scales: 128 tokens, and weight rows 0-127 and 128-255 of the tile,
//          two warps each. A lane holds rows l, l + 32, l + 64, l + 96 and writes
//          the word of 128 values of each as one 16-byte line, the layout that the
//          copy into TMEM wants; the words of the next stages are loaded ahead
// Two accumulators alternate, so the next tile's products run under the
// epilogue. Every wait is bounded (device_common.cuh).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <mutex>

#include "device_common.cuh"
#include "mx_common.cuh"
#include "mx_launch.h"
#include "step_common.cuh"
#include "tc_common.cuh"

namespace mxfp4 {
namespace mxp {
namespace {

constexpr int kEpilogueWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kScaleWarp = 10, kScaleWarps = 6;
constexpr int kThreads = 32 * (kScaleWarp + kScaleWarps);
constexpr int kRows = 128;                 // tokens of a tile
constexpr int kStageRow = 128;             // bytes of a row in a stage
constexpr int kMaxStages = 16;
constexpr int kGroupWords = 4;             // scale words (128 values each) of a row that are handled at a time
constexpr int kMaxGroupSlots = 6;
constexpr int kMaxColumnSlots = 4;         // of TMEM columns with scales
constexpr int kAhead = 2;                  // groups that a warp loads ahead
constexpr int kTmemCols = 512;             // all of them, so the allocation begins at column 0
constexpr int kTurnRow = 80;               // 32 outputs of a token in shared memory, and a gap (banks)
constexpr int kTurn = 32 * kTurnRow;       // a warp's
// Shared memory that is asked for at least. Every kernel here that takes TMEM has
// more than 64 KB, so none shares an SM with this one. CTAs of clusters that held
// the columns of two SMs crosswise, each waiting for its other half, would never end.
constexpr int kLeastShared = 192 * 1024;
constexpr int kImage = 512;                // scales of 128 rows and 128 values

// Columns for two accumulators (of 256 each they share some); the rest holds
// scales, those of two stages at a time.
__host__ __device__ constexpr int acc_cols(bool e2m1) { return e2m1 ? 416 : 432; }

struct Params {
    const uint8_t *xs, *ws;
    uint8_t *y, *ys;
    unsigned* status;
    int64_t t, n, k;
    int m_tiles, n_tiles, tiles, width;
    int stages;                            // of the whole k
    int ring, slots;                       // stages and groups of scales in shared memory
    int split;                             // CTAs (or pairs) of a cluster that share a tile, each a part of k
    int rows_a, rows_b;                    // rows of a copied box
    bool out_e2m1;
    int align;                             // bytes that every row of y begins at a multiple of (32, 16 or 2)
};

// Barriers, then the abort flag and the TMEM base.
constexpr int kNumBars = 2 * kMaxStages + 2 * kMaxGroupSlots + 4 + kMaxColumnSlots + 1;
struct Bars {
    uint32_t base;
    __device__ uint32_t full(int s) const { return base + 8 * s; }
    __device__ uint32_t empty(int s) const { return base + 8 * (kMaxStages + s); }
    __device__ uint32_t scales_full(int g) const { return base + 8 * (2 * kMaxStages + g); }
    __device__ uint32_t scales_empty(int g) const { return base + 8 * (2 * kMaxStages + kMaxGroupSlots + g); }
    __device__ uint32_t acc_full(int b) const { return base + 8 * (2 * kMaxStages + 2 * kMaxGroupSlots + b); }
    __device__ uint32_t acc_empty(int b) const { return base + 8 * (2 * kMaxStages + 2 * kMaxGroupSlots + 2 + b); }
    __device__ uint32_t columns_free(int s) const { return base + 8 * (2 * kMaxStages + 2 * kMaxGroupSlots + 4 + s); }
    __device__ uint32_t drain() const { return base + 8 * (kNumBars - 1); }
    __device__ uint32_t abort_flag() const { return base + 8 * kNumBars; }
    __device__ uint32_t tmem_base() const { return base + 8 * kNumBars + 8; }
    // All of them, by the lanes of a warp (one thread alone takes 0.6 us).
    __device__ void init(int lane, uint32_t scales, uint32_t epilogue) const {
        for (int i = lane; i < kNumBars; i += 32) {
            const int g = i - 2 * kMaxStages, b = g - 2 * kMaxGroupSlots;
            mbar_init(base + 8 * i, g >= 0 && g < kMaxGroupSlots ? scales : b == 2 || b == 3 ? epilogue : 1u);
        }
        fence_barrier_init();
    }
};
constexpr int kBarBytes = 1024;
static_assert(8 * kNumBars + 16 <= kBarBytes, "barriers, flag and TMEM base");

// Shared memory from a 1024-byte boundary: barriers, the ring (A then B of each
// stage), the scale images of `slots` groups ([128 rows][word] each), room to
// turn outputs round (if so wanted).
struct Plan {
    int a, stage, sets, group;  // bytes of a stage's tokens, and of it all; sets of 128 rows with scales; bytes of a group's images
    // A product reads 128 rows of tokens. Where there are fewer in all, the rows behind them are whatever lies there (of
    // this stage's weights and what follows): each row of the result depends on its own token only. So a stage takes no
    // more room than it has tokens, and the ring is deeper.
    __host__ __device__ Plan(int width, int cg, int rows_a) {
        a = rows_a * kStageRow;
        stage = a + width / cg * kStageRow;
        sets = 1 + (width + 127) / 128;
        group = sets * kGroupWords * kImage;
    }
    __host__ __device__ int groups_at(int ring) const { return ring * stage; }  // from the ring's begin
    __host__ __device__ int turn_at(int ring, int slots) const {
        const int end = groups_at(ring) + slots * group, read = (ring - 1) * stage + kRows * kStageRow;
        return end > read ? end : read;
    }
    __host__ __device__ int bytes(int ring, int slots, bool turn) const {
        return kBarBytes + turn_at(ring, slots) + (turn ? kEpilogueWarps * kTurn : 0) + 1024;
    }
};

// What a CTA (or pair) works on: tiles first, first + step, ..., of each the
// groups [group0, group0 + groups) of k, stages [stage0, stage0 + stages).
struct Unit {
    int first, step;
    int group0, groups, stage0, stages;
    int part;               // of the cluster's parts of k
    uint32_t rank, leader;  // place in the pair; the cluster's rank of its first CTA
};

struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, const WaitCtx& wc) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc));
}

// Arrives on an mbarrier of the pair's first CTA, which issues the products.
// Without release at cluster scope, which waits for every load that the SM has
// under way (2,000 cycles): no memory is handed from one CTA to the other here.
// Scales are read, and accumulators were, where the arriving warp wrote or read
// them, by tensor-core instructions that start after this arrival.
__device__ __forceinline__ void arrive_at_first(uint32_t bar, const Unit& u) {
    if (u.rank == 0)
        mbar_arrive(bar);
    else
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_to_rank(bar, u.leader)) : "memory");
}

// Tile -> its first token and its first output. Tokens run fastest, in groups
// of 16 tiles, so that a wave of tiles reads few weight rows and its tokens stay in L2.
template <int CG, bool SWIGLU>
__device__ __forceinline__ void place(const Params& p, int tile, int64_t& t0, int64_t& n0) {
    constexpr int kGroup = 16;
    const int group = tile / (kGroup * p.n_tiles), in = tile - group * kGroup * p.n_tiles;
    const int high = min(kGroup, p.m_tiles - group * kGroup);
    const int nt = in / high;
    t0 = static_cast<int64_t>(group * kGroup + in - nt * high) * (CG * kRows);
    n0 = static_cast<int64_t>(nt) * (SWIGLU ? p.width / 2 : p.width);
}

// ---------------------------------------------------------------- copies
template <int CG, bool E2M1, bool SWIGLU>
struct Copier {
    const Params& p;
    const Plan& plan;
    const Unit& u;
    const CUtensorMap *amap, *bmap;
    uint32_t base;
    const Bars& bars;
    int first;           // stages of the first tile that fill the ring
    int64_t t0, n0;

    __device__ __forceinline__ Copier(const Params& p_, const Plan& plan_, const Unit& u_, const CUtensorMap* a,
                                      const CUtensorMap* b, uint32_t base_, const Bars& bars_)
        : p(p_), plan(plan_), u(u_), amap(a), bmap(b), base(base_), bars(bars_) {
        first = u.first < p.tiles ? min(p.ring, u.stages) : 0;
        place<CG, SWIGLU>(p, u.first, t0, n0);
    }
    // A stage's bytes, of both CTAs of a pair, complete on the first one's barrier.
    __device__ __forceinline__ uint32_t full(int slot) const {
        return CG == 1 ? bars.full(slot) : map_to_rank(bars.full(slot), u.leader);
    }
    __device__ __forceinline__ void codes(uint32_t dst, const CUtensorMap* map, int k, int64_t y, uint32_t bar) const {
        if constexpr (CG == 1)
            tc::load_box_2d(dst, map, k * kStageRow, static_cast<int>(y), bar);
        else
            tc::load_box_2d_pair(dst, map, k * kStageRow, static_cast<int>(y), bar);
    }
    __device__ __forceinline__ void weight_box(uint32_t dst, int k, int64_t y, uint32_t bar) const {
        if constexpr (E2M1)
            codes(dst, bmap, k, y, bar);
        else if constexpr (CG == 1)
            tc::load_box_3d(dst, bmap, 0, static_cast<int>(y), k, bar);
        else
            tc::load_box_3d_pair(dst, bmap, 0, static_cast<int>(y), k, bar);
    }
    // Weight rows of this CTA: a pair's CTAs take a half of the tile each, which is the gate rows and the up rows in the
    // gated form.
    __device__ __forceinline__ void weights(int slot, int k) const {
        const uint32_t b = base + slot * plan.stage + plan.a, bar = full(slot);
        if (u.rank == 0)
            mbar_arrive_expect_tx(bars.full(slot),
                                  CG * p.rows_a * kStageRow + p.width * (E2M1 ? kStageRow : kStageRow / 2));
        weight_box(b, k, CG == 1 ? n0 : SWIGLU ? n0 + u.rank * p.n : n0 + u.rank * p.rows_b, bar);
        if constexpr (SWIGLU && CG == 1) weight_box(b + p.rows_b * kStageRow, k, p.n + n0, bar);
    }
    __device__ __forceinline__ void tokens(int slot, int k) const {
        codes(base + slot * plan.stage, amap, k, t0 + u.rank * kRows, full(slot));
    }
    // Test-only builds: the first cluster's first CTA never gets its first stage.
    __device__ __forceinline__ bool withheld(int j) const { return u.first == 0 && withhold_stage(static_cast<uint32_t>(j)); }
    // The previous kernel of the stream may still write tokens and weights: nothing is read before it has ended. (Weights
    // fetched ahead into L2, which is safe too, cost more than they brought: 16 tokens 14.5 us against 12.3 to 13.2.)
    __device__ __forceinline__ void run(const WaitCtx& wc) {
        pdl_wait_previous();
        for (int j = 0; j < first; ++j) {
            if (withheld(j)) continue;
            weights(j, u.stage0 + j);
            tokens(j, u.stage0 + j);
        }
        Ring r;
        int issued = 0;
        bool ok = true;
        for (int tile = u.first; tile < p.tiles && ok; tile += u.step) {
            place<CG, SWIGLU>(p, tile, t0, n0);
            for (int k = u.stage0; k < u.stage0 + u.stages; ++k) {
                if (issued >= first) {
                    if (!mbar_wait(bars.empty(r.slot), r.phase ^ 1u, wc)) {
                        ok = false;
                        break;
                    }
                    weights(r.slot, k);
                    tokens(r.slot, k);
                }
                ++issued;
                r.next(p.ring);
            }
        }
        if (!ok) drain(issued);
    }
    // Copies in flight land before the CTA may exit (bounded, whatever the abort flag says).
    __device__ __forceinline__ void drain(int issued) const {
        int never = 0;
        const WaitCtx own{p.status, &never};
        if (u.rank == 0) {
            for (int j = issued > p.ring ? issued - p.ring : 0; j < issued; ++j)
                mbar_wait(bars.full(j % p.ring), static_cast<uint32_t>((j / p.ring) & 1), own);
        } else {
            // Theirs complete on the other CTA's barrier, which cannot be waited for from here: a box lands within
            // microseconds.
            const uint64_t begin = global_timer_ns();
            while (global_timer_ns() - begin < 2000000ull) __nanosleep(1000);
        }
    }
};

// ---------------------------------------------------------------- scales
// Set 0: tokens, 1 and 2: weight rows. Warp `turn` (0, 1) of the set takes every second group.
template <int CG, bool SWIGLU>
struct Scales {
    const Params& p;
    const Plan& plan;
    const Unit& u;
    int set, lane;
    uint32_t ring;
    const Bars& bars;
    const uint8_t* array;
    bool wide;              // 16-byte loads
    const uint8_t* row[4];  // of the tile that is being loaded
    // Each warp has its next kAhead groups on their way in registers: a group of 512 values is multiplied in 0.3 us and
    // more, its loads from HBM take over 1 us, and getting it into place some 1,000 cycles.
    uint4 v[kAhead][4];
    int tile, g;            // the next group to load
    bool turned;            // the rows are not this tile's yet
    int64_t left;           // groups of this CTA from the next one on
    Ring r;

    __device__ __forceinline__ Scales(const Params& p_, const Plan& plan_, const Unit& u_, int set_, int turn, int lane_,
                                      uint32_t ring_, const Bars& bars_)
        : p(p_), plan(plan_), u(u_), set(set_), lane(lane_), ring(ring_), bars(bars_) {
        array = set == 0 ? p.xs : p.ws;
        wide = p.k % 512 == 0 && (reinterpret_cast<uintptr_t>(array) & 15) == 0;
        tile = u.first;
        g = u.group0;
        left = tile < p.tiles ? static_cast<int64_t>((p.tiles - tile + u.step - 1) / u.step) * u.groups : 0;
        if (turn) {
            --left;
            if (tile < p.tiles) skip();
            r.next(p.slots);
        }
        if (tile < p.tiles) rows_of();
        turned = false;
    }
    __device__ __forceinline__ void rows_of() {
        const int64_t pitch = p.k / 32;
        int64_t t0, n0;
        place<CG, SWIGLU>(p, tile, t0, n0);
        t0 += u.rank * kRows;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = 32 * q + lane + 128 * (set - 1);
            int64_t at;
            bool valid;
            if (set == 0) {
                at = t0 + 32 * q + lane;
                valid = at < p.t;
            } else if (!SWIGLU) {
                at = n0 + r;
                valid = r < p.width && at < p.n;
            } else {
                const bool up = r >= p.width / 2;
                at = n0 + r - (up ? p.width / 2 : 0);
                valid = r < p.width && at < p.n;
                at += up ? p.n : 0;
            }
            row[q] = valid ? array + at * pitch : nullptr;
        }
    }
    __device__ __forceinline__ void skip() {
        if (++g == u.group0 + u.groups) {
            g = u.group0;
            tile = u.step < p.tiles - tile ? tile + u.step : p.tiles;
            turned = true;
        }
    }
    __device__ __forceinline__ void load(uint4 (&to)[4]) {
        if (tile >= p.tiles) return;
        if (turned) rows_of();
        turned = false;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            to[q] = make_uint4(0u, 0u, 0u, 0u);  // rows that do not exist: their results go nowhere
            if (!row[q]) continue;
            // Through L2: another kernel may have written them just now.
            if (wide) {
                to[q] = __ldcg(reinterpret_cast<const uint4*>(row[q]) + g);
            } else {
                const uint32_t* s = reinterpret_cast<const uint32_t*>(row[q]) + kGroupWords * g;
                const int words = static_cast<int>(p.k / 128) - kGroupWords * g;
                to[q].x = __ldcg(s);
                if (words > 1) to[q].y = __ldcg(s + 1);
                if (words > 2) to[q].z = __ldcg(s + 2);
                if (words > 3) to[q].w = __ldcg(s + 3);
            }
        }
        skip();
        if (tile < p.tiles) skip();
    }
    // The first groups, when the previous kernel of the stream, which may write them, has ended.
    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) load(v[d]);
    }
    __device__ __forceinline__ void run(const WaitCtx& wc) {
        while (left > 0) {
#pragma unroll
            for (int d = 0; d < kAhead; ++d) {
                if (left <= 0) break;
                left -= 2;
                if (!wait_all(bars.scales_empty(r.slot), r.phase ^ 1u, wc)) return;
                const uint4(&w)[4] = v[d];
                const uint32_t at = ring + plan.groups_at(p.ring) + r.slot * plan.group + set * kGroupWords * kImage + lane * 16;
                sts128(at, w[0].x, w[1].x, w[2].x, w[3].x);
                sts128(at + kImage, w[0].y, w[1].y, w[2].y, w[3].y);
                sts128(at + 2 * kImage, w[0].z, w[1].z, w[2].z, w[3].z);
                sts128(at + 3 * kImage, w[0].w, w[1].w, w[2].w, w[3].w);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) arrive_at_first(bars.scales_full(r.slot), u);
                load(v[d]);
                r.next(p.slots);
                r.next(p.slots);
            }
        }
    }
};

// -------------------------------------------------------------- products
// The instructions of one CTA or of a pair.
template <int CG>
__device__ __forceinline__ void copy_scales_to_tmem(uint32_t taddr, uint64_t desc) {
    if constexpr (CG == 1)
        tc::copy_scales_to_tmem(taddr, desc);
    else
        tc::copy_scales_to_tmem_pair(taddr, desc);
}
template <int CG>
__device__ __forceinline__ void commit_to(uint32_t bar, const Unit& u) {
    if constexpr (CG == 1)
        tc::commit_to(bar);
    else
        tc::commit_to_pair(bar, static_cast<uint16_t>(3u << u.leader));
}
template <int CG>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         bool acc) {
    if constexpr (CG == 1)
        tc::mma_mxf8f6f4(d, a, b, idesc, sfa, sfb, acc);
    else
        tc::mma_mxf8f6f4_pair(d, a, b, idesc, sfa, sfb, acc);
}
template <int CG>
__device__ __forceinline__ void mma_e2m1(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         bool acc) {
    if constexpr (CG == 1)
        tc::mma_mxf4(d, a, b, idesc, sfa, sfb, acc);
    else
        tc::mma_mxf4_pair(d, a, b, idesc, sfa, sfb, acc);
}

template <int CG, bool E2M1>
__device__ bool issue_products(const Params& p, const Plan& plan, const Unit& u, uint32_t base, const Bars& bars,
                               const WaitCtx& wc) {
    // Two stages are waited for and issued together: a round of waiting and issuing costs some 300 cycles whatever is
    // issued, the products of a stage take 256 to 512.
    constexpr int W = E2M1 ? 2 : 1;       // scale words of a row in a stage
    constexpr int S = kGroupWords / W;    // stages of a group of scales
    constexpr int kAccCols = acc_cols(E2M1);
    // TMEM scale slots above the accumulators, 4 columns an image: of each word the tokens', then the weight rows' sets. A
    // slot is written again only after the products that read it are done.
    const int word_cols = 4 * plan.sets, slot_cols = 2 * W * word_cols;
    const int slots = min((kTmemCols - kAccCols) / slot_cols, kMaxColumnSlots);
    const bool shared_cols = 2 * p.width > kAccCols;
    const uint32_t idesc = tc::mma_idesc(E2M1 ? tc::kFmtMxf4E2M1 : tc::kFmtE4M3, E2M1 ? tc::kFmtMxf4E2M1 : tc::kFmtE2M1,
                                         CG * kRows, static_cast<uint32_t>(p.width), 0);
    // All lanes walk through the stages and one issues, so that the operands stay in uniform registers (one lane alone took
    // twice the time a product).
    const bool one = elect_one();
    Ring r, gr, tr;
    int rounds = 0, i = 0;
    for (int tile = u.first; tile < p.tiles; tile += u.step, ++i) {
        const int back = shared_cols ? 1 : 2;  // whose epilogue frees this accumulator
        if (i >= back && !wait_all(bars.acc_empty(i & 1), static_cast<uint32_t>((i - back) >> 1) & 1u, wc)) return false;
        tc::fence_after_sync();
        const uint32_t d = (i & 1) ? kAccCols - p.width : 0;
        for (int k = 0; k < u.stages; k += 2, ++rounds) {
            const int n = min(2, u.stages - k), in = k % S;
            Ring r1 = r;
            if (n == 2) r1.next(p.ring);
            const uint32_t fb = bars.full(r.slot), fb1 = bars.full(r1.slot);
            const uint32_t b2 = in == 0 ? bars.scales_full(gr.slot) : fb, p2 = in == 0 ? gr.phase : r.phase;
            const uint32_t b3 = rounds >= slots ? bars.columns_free(tr.slot) : fb, p3 = rounds >= slots ? tr.phase ^ 1u : r.phase;
            while (!__all_sync(0xffffffffu, mbar_test4(fb, r.phase, fb1, r1.phase, b2, p2, b3, p3)))
                if (!wait_all(b3, p3, wc) || !wait_all(b2, p2, wc) || !wait_all(fb, r.phase, wc) ||
                    !wait_all(fb1, r1.phase, wc))
                    return false;
            const uint32_t images = base + plan.groups_at(p.ring) + gr.slot * plan.group + in * W * kImage;
            const uint32_t sf = kAccCols + tr.slot * slot_cols;
            const uint64_t sd = tc::scale_image_desc(images);
            const bool last = k + n == u.stages, ends = in + 2 >= S || last;
            if (one) {
                // The images of both stages, in memory [set][word] (there are four words to a group, whatever k).
#pragma unroll
                for (int w = 0; w < 2 * W; ++w) {
                    copy_scales_to_tmem<CG>(sf + w * word_cols, sd + w * (kImage >> 4));
                    copy_scales_to_tmem<CG>(sf + w * word_cols + 4, sd + (kGroupWords + w) * (kImage >> 4));
                    if (plan.sets > 2) copy_scales_to_tmem<CG>(sf + w * word_cols + 8, sd + (2 * kGroupWords + w) * (kImage >> 4));
                }
                // They are free once they are in TMEM.
                if (ends) commit_to<CG>(bars.scales_empty(gr.slot), u);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (j == 1 && n == 1) break;
                const uint32_t a = base + (j ? r1.slot : r.slot) * plan.stage;
                const uint64_t ad = tc::operand_desc(a), bd = tc::operand_desc(a + plan.a);
                if (one) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const bool acc = k != 0 || j != 0 || c != 0;
                        const uint32_t sfa = sf + (j * W + (E2M1 ? c >> 1 : 0)) * word_cols;
                        if constexpr (E2M1)
                            mma_e2m1<CG>(d, ad + 2 * c, bd + 2 * c, idesc | ((c & 1) * 2u) << 4 | ((c & 1) * 2u) << 29, sfa,
                                         sfa + 4, acc);
                        else
                            mma_e4m3<CG>(d, ad + 2 * c, bd + 2 * c,
                                         idesc | static_cast<uint32_t>(c) << 4 | static_cast<uint32_t>(c) << 29, sfa, sfa + 4,
                                         acc);
                    }
                    commit_to<CG>(bars.empty(j ? r1.slot : r.slot), u);
                    if (j == n - 1) commit_to<CG>(bars.columns_free(tr.slot), u);
                    if (last && j == n - 1) commit_to<CG>(bars.acc_full(i & 1), u);
                }
            }
            __syncwarp();
            if (ends) gr.next(p.slots);
            tr.next(slots);
            r = r1;
            r.next(p.ring);
        }
    }
    return true;
}

// -------------------------------------------------------------- epilogue
__device__ __forceinline__ void load32(uint32_t taddr, float (&v)[32]) {
    uint32_t(&r)[32] = *reinterpret_cast<uint32_t(*)[32]>(v);
    tc::tmem_load<32>(taddr, r);
}

// 32 bytes, a whole sector, in one store.
__device__ __forceinline__ void store32(void* to, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// The warp's 32 tokens x 32 outputs, lane i's of token `row`, `count` of them
// wanted. Straight from the registers a store of the warp writes 32 bytes, whole
// sectors, of 32 rows (through shared memory, 64 bytes of 8 rows, it was no
// faster: 4,000 x 512 x 20,000 49 us against 47). Rows that begin at any even
// address do go through shared memory: a thread's own 2-byte stores would each
// touch a sector.
__device__ __forceinline__ void store_rows(const Params& p, uint32_t turn, int64_t row, int64_t col, const float (&v)[32]) {
    const int count = static_cast<int>(p.n - col < 32 ? p.n - col : 32), lane = threadIdx.x & 31;
    uint32_t w[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
        w[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (p.align >= 16) {
        if (row >= p.t) return;
        __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(p.y) + row * p.n + col;
        if (count < 32) {  // a multiple of 8
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (8 * q < count)
                    reinterpret_cast<uint4*>(y)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        } else if (p.align >= 32) {
            store32(y, *reinterpret_cast<const uint32_t(*)[8]>(w));
            store32(y + 16, *reinterpret_cast<const uint32_t(*)[8]>(w + 8));
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                reinterpret_cast<uint4*>(y)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) sts128(turn + lane * kTurnRow + 16 * q, w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    __syncwarp();
    const int64_t row0 = row - lane;
    const int rows = static_cast<int>(p.t - row0 < 32 ? p.t - row0 : 32);
    uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + row0 * p.n + col + lane;
    for (int r = 0; r < rows; ++r, y += p.n) {
        uint16_t h;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(turn + r * kTurnRow + 2 * lane) : "memory");
        if (lane < count) *y = h;
    }
    __syncwarp();
}

template <bool OUT_E2M1>
__device__ __forceinline__ void store_block(uint8_t* q, uint8_t* s, const float (&h)[32]) {
    const uint32_t b = mx::scale_byte<OUT_E2M1>(mx::largest<32>(h));
    uint32_t w[OUT_E2M1 ? 4 : 8];
    mx::encode<OUT_E2M1, 32>(h, b, w);
    if constexpr (OUT_E2M1)
        *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    else if (reinterpret_cast<uintptr_t>(q) % 32 == 0)
        store32(q, w);
    else
#pragma unroll
        for (int i = 0; i < 2; ++i)
            reinterpret_cast<uint4*>(q)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    *s = static_cast<uint8_t>(b);
}

// 32 sums of one token at output `col`, or 32 of both of its halves (gate a, up b).
template <bool SWIGLU>
__device__ __forceinline__ void finish(const Params& p, uint32_t turn, int64_t row, int64_t col, float (&a)[32],
                                       const float (&b)[32]) {
    if (col >= p.n || row - (threadIdx.x & 31) >= p.t) return;  // none of the warp's tokens
    if constexpr (SWIGLU) {
        if (row >= p.t) return;
        mx::swiglu<32>(a, b);
        const int64_t e = row * p.n + col;
        if (p.out_e2m1)
            store_block<true>(p.y + e / 2, p.ys + e / 32, a);
        else
            store_block<false>(p.y + e, p.ys + e / 32, a);
    } else {
        store_rows(p, turn, row, col, a);
    }
}

template <int CG, bool SWIGLU>
__device__ void epilogue(const Params& p, const Unit& u, int warp, int lane, uint32_t turn, const Bars& bars,
                         const WaitCtx& wc, int kAccCols) {
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const bool shared_cols = 2 * p.width > kAccCols;
    const int chunks = (SWIGLU ? p.width / 2 : p.width) / 32;
    // Chunks that hold columns of the other accumulator come first.
    const int early = shared_cols ? (2 * p.width - kAccCols + 31) / 32 : chunks;
    int i = 0;
    for (int tile = u.first; tile < p.tiles; tile += u.step, ++i) {
        int64_t t0, n0;
        place<CG, SWIGLU>(p, tile, t0, n0);
        t0 += u.rank * kRows;
        if (!wait_all(bars.acc_full(i & 1), static_cast<uint32_t>(i >> 1) & 1u, wc)) return;
        tc::fence_after_sync();
        const uint32_t acc = lanes + ((i & 1) ? kAccCols - p.width : 0);
        const int64_t row = t0 + quarter * 32 + lane;
        // The accumulator is given back as soon as what the next tile needs of it is in registers: by then no chunk of
        // this warp's before `early` is left. Two chunks at a time (one of both halves) keep loads and stores under way.
        bool held = true;
        auto give_back = [&](int next) {
            if (!held || next < early) return;
            held = false;
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive_at_first(bars.acc_empty((i & 1) ^ (shared_cols ? 1 : 0)), u);
        };
        const bool down = shared_cols && !(i & 1);
        give_back(half);
        for (int c = half; c < chunks; c += SWIGLU ? 2 : 4) {
            const int at = down ? chunks - 1 - c : c;
            float a[32], b[32];
            load32(acc + 32 * at, a);
            if constexpr (SWIGLU) {
                load32(acc + p.width / 2 + 32 * at, b);
                tc::tmem_wait_ld();
                give_back(c + 2);
                finish<SWIGLU>(p, turn, row, n0 + 32 * at, a, b);
            } else {
                const int then = down ? at - 2 : at + 2;
                const bool two = c + 2 < chunks;
                if (two) load32(acc + 32 * then, b);
                tc::tmem_wait_ld();
                give_back(c + 4);
                finish<SWIGLU>(p, turn, row, n0 + 32 * at, a, a);
                if (two) finish<SWIGLU>(p, turn, row, n0 + 32 * then, b, b);
            }
        }
        give_back(chunks);
    }
}

// The end of a tile whose k is split over a cluster: chunk c of the columns
// belongs to part c % split, whose CTA takes the others' sums of it into its
// ring (free by then) and adds them to its own in the parts' order, so results
// do not depend on who comes first.
//   box (chunk c / split, sender): [8 or 2 x 8 pieces of 4 fp32][128 tokens], so
//   that a warp's store is 512 bytes in a row (stores of 16 bytes 128 apart
//   took 3 us longer a tile)
template <bool SWIGLU>
struct Exchange {
    static constexpr int kHalves = SWIGLU ? 2 : 1;
    const Params& p;
    const Unit& u;
    uint32_t base;
    int cg, chunks;
    __device__ Exchange(const Params& p_, const Unit& u_, uint32_t base_, int cg_)
        : p(p_), u(u_), base(base_), cg(cg_), chunks((SWIGLU ? p_.width / 2 : p_.width) / 32) {}
    __device__ uint32_t box(int c, int sender, int h, int token) const {
        const int place = (c / p.split) * (p.split - 1) + sender - (sender > c % p.split ? 1 : 0);
        return base + (place * kHalves + h) * kRows * 128 + token * 16;
    }
    __device__ void send(int warp, int lane, int64_t t0) const {
        const int quarter = warp & 3, token = quarter * 32 + lane;
        if (t0 + quarter * 32 >= p.t) return;  // the whole warp has no token
        for (int c = warp >> 2; c < chunks; c += 2) {
            const int owner = c % p.split;
            if (owner == u.part) continue;
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                float v[32];
                load32((static_cast<uint32_t>(quarter * 32) << 16) + h * (p.width / 2) + 32 * c, v);
                tc::tmem_wait_ld();
                const uint32_t to = map_to_rank(box(c, u.part, h, token), static_cast<uint32_t>(owner * cg) + u.rank);
                if (t0 + token < p.t) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        st_cluster_f32x4(to + q * kRows * 16, v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
            }
        }
    }
    __device__ void add(float (&v)[32], int c, int h, int token) const {
        for (int s = 0; s < p.split; ++s) {
            if (s == u.part) continue;
            const uint32_t from = box(c, s, h, token);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint4 w = lds128(from + q * kRows * 16);
                v[4 * q] += __uint_as_float(w.x);
                v[4 * q + 1] += __uint_as_float(w.y);
                v[4 * q + 2] += __uint_as_float(w.z);
                v[4 * q + 3] += __uint_as_float(w.w);
            }
        }
    }
    __device__ void receive(int warp, int lane, uint32_t turn, int64_t t0, int64_t n0) const {
        const int quarter = warp & 3, token = quarter * 32 + lane;
        if (t0 + quarter * 32 >= p.t) return;
        for (int c = u.part + (warp >> 2) * p.split; c < chunks; c += 2 * p.split) {
            const uint32_t acc = (static_cast<uint32_t>(quarter * 32) << 16) + 32 * c;
            float a[32], b[32];
            load32(acc, a);
            if constexpr (SWIGLU) load32(acc + p.width / 2, b);
            tc::tmem_wait_ld();
            add(a, c, 0, token);
            if constexpr (SWIGLU) add(b, c, 1, token);
            finish<SWIGLU>(p, turn, t0 + token, n0 + 32 * c, a, b);
        }
    }
};

// ---------------------------------------------------------------- kernel
template <int CG, bool E2M1, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    mx_product_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                      const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const Bars bars{(raw + 1023u) & ~1023u};
    const uint32_t base = bars.base + kBarBytes;  // of the ring
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + (bars.abort_flag() - raw));
    const WaitCtx wc{p.status, abort_flag};
    const Plan plan(p.width, CG, p.rows_a);
    // What takes long is begun first: TMEM by the issuing warp, barriers by the copying one.
    if (warp == kMmaWarp) {
        if constexpr (CG == 1) {
            tc::tmem_alloc(bars.tmem_base(), kTmemCols);
            tc::tmem_relinquish();
        } else {
            tc::tmem_alloc_pair(bars.tmem_base(), kTmemCols);
            tc::tmem_relinquish_pair();
        }
    }
    const bool alone = CG == 1 && p.split == 1;
    if (warp == kCopyWarp) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(&bmap) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(&amap) : "memory");
            *abort_flag = 0;
        }
        bars.init(lane, static_cast<uint32_t>(CG * plan.sets), CG * kEpilogueWarps);
        __syncwarp();
        // It goes on to the first copies while the others wait for TMEM.
        if (alone)
            asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
        else
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    Unit u;
    {
        constexpr int kGroupStages = kGroupWords / (E2M1 ? 2 : 1);
        const uint32_t in = blockIdx.x;  // a cluster is a row of the grid
        const int groups = (p.stages + kGroupStages - 1) / kGroupStages;
        u.first = blockIdx.y;
        u.step = gridDim.y;
        u.part = static_cast<int>(in) / CG;
        u.rank = in % CG;
        u.leader = in - u.rank;
        u.group0 = groups * u.part / p.split;
        u.groups = groups * (u.part + 1) / p.split - u.group0;
        u.stage0 = u.group0 * kGroupStages;
        u.stages = min(u.groups * kGroupStages, p.stages - u.stage0);
    }
    auto ready = [&] {
        tc::fence_before_sync();
        if (alone)
            asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
        else
            cluster_sync_all();
        tc::fence_after_sync();
    };
    // Every role waits for the previous kernel of the stream before its first bounded wait: that one may take long.
    bool summed = true;
    if (warp < kEpilogueWarps) {
        ready();
        pdl_wait_previous();  // the previous kernel may still use what y is written over
        const uint32_t turn = base + plan.turn_at(p.ring, p.slots) + warp * kTurn;
        if (p.split == 1)
            epilogue<CG, SWIGLU>(p, u, warp, lane, turn, bars, wc, acc_cols(E2M1));
        else
            summed = wait_all(bars.acc_full(0), 0, wc);  // a cluster has one tile
    } else if (warp == kCopyWarp) {
        Copier<CG, E2M1, SWIGLU> copier(p, plan, u, &amap, &bmap, base, bars);
        if (!alone) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (lane == 0) copier.run(wc);
    } else if (warp == kMmaWarp) {
        ready();
        // The next kernel of the stream is let in once this one has its TMEM (the other way round it could take the columns
        // and then wait for this kernel) and the previous one has ended: other calls of the library read weights before they
        // wait, and what they wait for is only the kernel right ahead of them.
        pdl_wait_previous();
        pdl_launch_dependents();
        if (u.rank == 0 && !issue_products<CG, E2M1>(p, plan, u, base, bars, wc)) {
            // Products issued so far may still read shared memory and write TMEM: waited for, bounded.
            if (lane == 0) {
                commit_to<CG>(bars.drain(), u);
                int never = 0;
                const WaitCtx own{p.status, &never};
                mbar_wait(bars.drain(), 0, own);
            }
        }
    } else {
        const int set = (warp - kScaleWarp) % 3;
        if (set < plan.sets) {
            Scales<CG, SWIGLU> scales(p, plan, u, set, (warp - kScaleWarp) / 3, lane, base, bars);
            if (alone) {
                ready();
                pdl_wait_previous();
                scales.begin();
            } else {
                // The cluster's barrier would wait for loads under way.
                asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
                pdl_wait_previous();
                scales.begin();
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            }
            scales.run(wc);
        } else {
            ready();
        }
    }
    __syncwarp();
    if (p.split > 1) {
        const Exchange<SWIGLU> ex(p, u, base, CG);
        int64_t t0, n0;
        place<CG, SWIGLU>(p, u.first, t0, n0);
        t0 += u.rank * kRows;
        tc::fence_after_sync();
        cluster_sync_all();  // every part is summed: the rings are free
        if (warp < kEpilogueWarps && summed) ex.send(warp, lane, t0);
        __syncwarp();
        cluster_sync_all();
        if (warp < kEpilogueWarps && summed)
            ex.receive(warp, lane, base + plan.turn_at(p.ring, p.slots) + warp * kTurn, t0, n0);
        __syncwarp();
    }
    tc::fence_before_sync();
    // A CTA of a pair stays until the other's copies, arrivals and products on it are done.
    if constexpr (CG == 1)
        __syncthreads();
    else
        cluster_sync_all();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        if constexpr (CG == 1)
            tc::tmem_dealloc(0, kTmemCols);
        else
            tc::tmem_dealloc_pair(0, kTmemCols);
    }
}

// ------------------------------------------------------------------ host
template <int CG, bool E2M1, bool SWIGLU>
cudaError_t configure(int smem) {
    return cudaFuncSetAttribute(mx_product_kernel<CG, E2M1, SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int CG, bool E2M1, bool SWIGLU>
cudaError_t launch(const CUtensorMap& amap, const CUtensorMap& bmap, const Params& p, int smem, dim3 grid,
                   cudaStream_t stream) {
    PdlLaunch l(grid, dim3(kThreads), smem, stream);
    if (CG * p.split > 1) {
        cudaLaunchAttribute& cluster = l.attr[l.cfg.numAttrs++];
        cluster.id = cudaLaunchAttributeClusterDimension;
        cluster.val.clusterDim.x = CG * p.split;
        cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    }
    return cudaLaunchKernelEx(&l.cfg, mx_product_kernel<CG, E2M1, SWIGLU>, amap, bmap, p);
}

template <int CG>
cudaError_t launch_any(bool e2m1, bool swiglu, const CUtensorMap& amap, const CUtensorMap& bmap, const Params& p,
                       int smem, dim3 grid, cudaStream_t stream) {
    if (e2m1)
        return swiglu ? launch<CG, true, true>(amap, bmap, p, smem, grid, stream)
                      : launch<CG, true, false>(amap, bmap, p, smem, grid, stream);
    return swiglu ? launch<CG, false, true>(amap, bmap, p, smem, grid, stream)
                  : launch<CG, false, false>(amap, bmap, p, smem, grid, stream);
}

// What the choice of a tile needs to know of a device.
struct Device {
    bool ready;
    int max_smem;
    int clusters[9];  // of so many CTAs, one to an SM, that are resident at once
};

cudaError_t device_of(const Device** out, int num_sms, int max_smem) {
    static Device devices[64];
    static std::mutex mutex;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    Device& d = devices[dev];
    std::lock_guard<std::mutex> lock(mutex);
    if (!d.ready) {
        cudaError_t e = cudaSuccess;
        for (auto set : {configure<1, false, false>, configure<1, false, true>, configure<1, true, false>,
                         configure<1, true, true>, configure<2, false, false>, configure<2, false, true>,
                         configure<2, true, false>, configure<2, true, true>})
            if ((e = set(max_smem))) return e;
        d.max_smem = max_smem;
        d.clusters[1] = num_sms;
        for (int c = 2; c <= 8; ++c) {
            cudaLaunchConfig_t cfg{};
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = c;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.gridDim = dim3(c * num_sms);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = max_smem;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if ((e = cudaOccupancyMaxActiveClusters(&d.clusters[c], mx_product_kernel<1, false, false>, &cfg))) return e;
        }
        d.ready = true;
    }
    *out = &d;
    return cudaSuccess;
}

// A tile's shape and the CTAs that share its k.
struct Choice {
    int cg, width, split, ring, slots, smem;
    int inbox;  // bytes of the other parts' sums that a CTA takes into its ring
    float us;
};

// Rows of tokens in a stage.
int token_rows(int64_t t) { return t < kRows ? static_cast<int>((t + 7) / 8 * 8) : kRows; }

// Stages in the ring, and slots for the scales of as many and two groups more; false if not even two stages fit.
bool fit(Choice& c, int rows_a, bool e2m1, bool turn, int max_smem) {
    const Plan plan(c.width, c.cg, rows_a);
    auto slots_for = [&](int ring) {
        const int s = (ring * (e2m1 ? 2 : 1) + kGroupWords - 1) / kGroupWords + 2;
        return s < kMaxGroupSlots ? s : kMaxGroupSlots;
    };
    c.ring = 1;
    while (c.ring < kMaxStages && plan.bytes(c.ring + 1, slots_for(c.ring + 1), turn) <= max_smem) ++c.ring;
    c.slots = slots_for(c.ring);
    c.smem = plan.bytes(c.ring, c.slots, turn);
    if (c.smem < kLeastShared) c.smem = kLeastShared;
    return c.ring > 1 && c.smem <= max_smem;
}

// The tile with the least time by a model of what was measured on GB300 (in
// CUDA graphs, us):
//   a stage of a CTA   0.14 + 0.0008 width (width 64 0.22, 128 0.24, 192 0.27-0.33, 256 0.30-0.42: its copies and
//                      products share the bandwidth of shared memory, 128 bytes a cycle)
//   a stage of a pair  0.13 + 0.0007 width (128 0.19-0.24, 192 0.20-0.30, 256 0.24-0.38: each CTA reads half the
//                      weights), for twice the tokens
//   a launch           4.5 (a pair 5.5): first copies, last products, the stores
//   a shared tile      1.7 and 20 KB a us for the sums that a CTA hands on
// A part of k less per CTA only pays while every tile is on the GPU at once.
Choice choose(int64_t t, int64_t n, int64_t k, bool e2m1, bool swiglu, bool turn, const Device& d) {
    const int stages = static_cast<int>((k + (e2m1 ? 255 : 127)) / (e2m1 ? 256 : 128));
    const int groups = static_cast<int>((k / 128 + kGroupWords - 1) / kGroupWords);
    const int rows_a = token_rows(t);
    Choice best{};
    best.us = 1e30f;
    for (int cg = 1; cg <= (t > kRows && d.clusters[2] > 0 ? 2 : 1); ++cg) {
        for (int width = swiglu ? 64 : 32; width <= 256; width += swiglu ? 64 : 32) {
            const int outputs = swiglu ? width / 2 : width;
            const float stage = cg == 1 ? 0.14f + 0.0008f * width : 0.13f + 0.0007f * width;
            const int64_t tiles = ((t + kRows * cg - 1) / (kRows * cg)) * ((n + outputs - 1) / outputs);
            for (int split = 1; split * cg <= 8 && split <= groups; ++split) {
                if (split > 1 && tiles > d.clusters[cg * split]) break;
                Choice c{cg, width, split, 0, 0, 0, 0, 0.f};
                const int64_t waves = (tiles + d.clusters[cg] - 1) / d.clusters[cg];
                const int longest = (groups + split - 1) / split * (kGroupWords / (e2m1 ? 2 : 1));
                c.us = (split > 1 ? 1 : waves) * stage * (longest < stages ? longest : stages) + (cg == 1 ? 4.5f : 5.5f);
                if (split > 1) c.us += 1.7f + rows_a * width * 4.f * (split - 1) / split / 20e3f;
                if (c.us >= best.us || !fit(c, rows_a, e2m1, turn, d.max_smem)) continue;
                // The sums of the others have to fit the ring (chunks of 32 columns, of both halves where swiglu).
                c.inbox = (outputs / 32 + split - 1) / split * (split - 1) * kRows * 128 * (swiglu ? 2 : 1);
                if (c.inbox > c.ring * Plan(width, cg, rows_a).stage) continue;
                best = c;
            }
        }
    }
    return best;
}

// A choice and what the launch makes of it.
struct Cut {
    Choice c;                  // c.cg == 0: none fits
    int rows_a, rows_b;        // rows of a copied box
    int64_t m_tiles, n_tiles;
    int cluster, rows;         // of the grid: CTAs of a cluster, and clusters
};

Cut cut(int64_t t, int64_t n, int64_t k, bool e2m1, bool swiglu, bool turn, const Device& d) {
    Cut r{};
    const Choice c = r.c = choose(t, n, k, e2m1, swiglu, turn, d);
    if (!c.cg) return r;
    const int outputs = swiglu ? c.width / 2 : c.width, rows = kRows * c.cg;
    r.rows_a = token_rows(t);
    r.rows_b = swiglu || c.cg == 2 ? c.width / 2 : c.width;
    r.m_tiles = (t + rows - 1) / rows;
    r.n_tiles = (n + outputs - 1) / outputs;
    const int64_t tiles = r.m_tiles * r.n_tiles;
    if (tiles >= (int64_t(1) << 27)) return Cut{};
    r.cluster = c.cg * c.split;
    r.rows = static_cast<int>(c.split > 1 || tiles < d.clusters[c.cg] ? tiles : d.clusters[c.cg]);
    return r;
}

}  // namespace
}  // namespace mxp

// How a product would be cut (host only).
bool plan_mx_product(int64_t t, int64_t k, int64_t n, bool e2m1, bool swiglu, bool aligned, int max_smem,
                     const int32_t* clusters, mxfp4_mx_plan_t* out) {
    using namespace mxp;
    Device d{};
    d.max_smem = max_smem;
    for (int c = 1; c <= 8; ++c) d.clusters[c] = clusters[c];
    const Cut r = cut(t, n, k, e2m1, swiglu, !swiglu && !aligned, d);
    const Choice& c = r.c;
    if (!c.cg) return false;
    const Plan plan(c.width, c.cg, r.rows_a);
    *out = mxfp4_mx_plan_t{};
    out->pair = c.cg == 2;
    out->width = c.width;
    out->split = c.split;
    out->ctas = r.cluster * r.rows;
    out->ring_slots = c.ring;
    out->stage_bytes = plan.stage;
    out->token_rows = r.rows_a;
    out->scale_slots = c.slots;
    out->scale_bytes = plan.group;
    out->inbox_bytes = c.inbox;
    out->smem_bytes = c.smem;
    return true;
}

cudaError_t launch_mx_product(const MxProductArgs& a, int num_sms, int max_smem, cudaStream_t stream) {
    using namespace mxp;
    const Device* device = nullptr;
    if (cudaError_t e = device_of(&device, num_sms, max_smem)) return e;
    // The choice takes some 10 us of host time: the last sizes' are kept.
    struct Kept {
        int64_t t, n, k;
        const Device* device;
        int kind;
        Cut cut;
    };
    thread_local Kept kept[16];
    const uintptr_t rows_at = reinterpret_cast<uintptr_t>(a.y) | static_cast<uintptr_t>(2 * a.n);
    const int align = rows_at % 32 == 0 ? 32 : rows_at % 16 == 0 ? 16 : 2;
    const bool turn = !a.swiglu && align < 16;
    const int kind = (a.e2m1 ? 2 : 0) + (a.swiglu ? 1 : 0) + (turn ? 4 : 0);
    Kept& slot = kept[(a.t * 31 + a.n * 7 + a.k / 128 + kind) & 15];
    if (slot.device != device || slot.t != a.t || slot.n != a.n || slot.k != a.k || slot.kind != kind)
        slot = Kept{a.t, a.n, a.k, device, kind, cut(a.t, a.n, a.k, a.e2m1, a.swiglu, turn, *device)};
    const Choice& c = slot.cut.c;
    if (!c.cg) return cudaErrorInvalidValue;
    Params p{};
    p.xs = a.xs;
    p.ws = a.ws;
    p.y = static_cast<uint8_t*>(a.y);
    p.ys = a.ys;
    p.status = a.status;
    p.t = a.t;
    p.n = a.n;
    p.k = a.k;
    p.width = c.width;
    p.split = c.split;
    p.ring = c.ring;
    p.slots = c.slots;
    p.out_e2m1 = a.out_e2m1;
    p.align = align;
    p.stages = static_cast<int>((a.k + (a.e2m1 ? 255 : 127)) / (a.e2m1 ? 256 : 128));
    p.m_tiles = static_cast<int>(slot.cut.m_tiles);
    p.n_tiles = static_cast<int>(slot.cut.n_tiles);
    p.tiles = p.m_tiles * p.n_tiles;
    p.rows_a = slot.cut.rows_a;
    p.rows_b = slot.cut.rows_b;
    const int64_t w_rows = a.swiglu ? 2 * a.n : a.n;
    CUtensorMap amap, bmap;
    cudaError_t e = encode_code_map(&amap, a.xq, a.t, a.e2m1 ? a.k / 2 : a.k, p.rows_a);
    if (e == cudaSuccess)
        e = a.e2m1 ? encode_code_map(&bmap, a.wq, w_rows, a.k / 2, p.rows_b)
                   : encode_spread_map(&bmap, a.wq, w_rows, a.k, p.rows_b);
    if (e != cudaSuccess) return e;
    const dim3 grid(slot.cut.cluster, slot.cut.rows);
    return c.cg == 1 ? launch_any<1>(a.e2m1, a.swiglu, amap, bmap, p, c.smem, grid, stream)
                     : launch_any<2>(a.e2m1, a.swiglu, amap, bmap, p, c.smem, grid, stream);
}

}  // namespace mxfp4
