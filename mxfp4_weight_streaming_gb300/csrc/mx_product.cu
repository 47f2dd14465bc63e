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
// A tile is 128 tokens x `width` weight rows (width: a multiple of 32 up to
// 256; for the gated form the first half are gate rows, the second the up rows
// of the same outputs, so a thread finds both of its token in one TMEM lane).
// A stage is 128 bytes of every row: 128 values of k, or 256 in E2M1.
//
// One CTA per SM walks over tiles, warp-specialised:
//   0-7    epilogue: warp w reads the lanes (tokens) 32 (w % 4) .. of the
//          accumulator, 32-column chunks by turns with warp w ^ 4
//   8      copies codes (TMA) into a ring of stages
//   9      issues the scales' copies into TMEM and the products
//   10-12  scales: 128 tokens, and weight rows 0-127 and 128-255 of the tile.
//          A lane holds rows l, l + 32, l + 64, l + 96 and writes the word of
//          128 values of each as one 16-byte line, the layout that the copy
//          into TMEM wants; the words of the next stages are loaded ahead
// Two accumulators alternate, so the next tile's products run under the
// epilogue.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "mx_common.cuh"
#include "mx_launch.h"
#include "step_common.cuh"
#include "tc_common.cuh"

namespace mxfp4 {
namespace mxp {
namespace {

constexpr int kEpilogueWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kScaleWarp = 10, kScaleWarps = 3;
constexpr int kThreads = 32 * (kScaleWarp + kScaleWarps);
constexpr int kRows = 128;                 // tokens of a tile
constexpr int kStageRow = 128;             // bytes of a row in a stage
constexpr int kStageA = kRows * kStageRow;
constexpr int kMaxStages = 8;
constexpr int kTmemCols = 512;
constexpr int kAccCols = 432;              // two accumulators; one of 256 columns shares some with the other
constexpr int kImage = 512;                // scales of 128 rows and 128 values

struct Params {
    const uint8_t *xs, *ws;
    uint8_t *y, *ys;
    unsigned* status;
    int64_t t, n, k;
    int m_tiles, tiles, width, stages;     // stages: of the whole k
    int ring;                              // stages in shared memory
    int rows_a, rows_b;                    // rows of a copied box
    bool out_e2m1;
    bool wide;                             // 16-byte stores of y
};

struct Bars {
    uint32_t base;
    __device__ uint32_t full(int s) const { return base + 8 * s; }
    __device__ uint32_t scales(int s) const { return base + 8 * (kMaxStages + s); }
    __device__ uint32_t empty(int s) const { return base + 8 * (2 * kMaxStages + s); }
    __device__ uint32_t acc_full(int b) const { return base + 8 * (3 * kMaxStages + b); }
    __device__ uint32_t acc_empty(int b) const { return base + 8 * (3 * kMaxStages + 2 + b); }
    __device__ uint32_t drain() const { return base + 8 * (3 * kMaxStages + 4); }
};
constexpr int kNumBars = 3 * kMaxStages + 5;

// Shared memory from a 1024-byte boundary: the ring (A then B of each stage),
// the stages' scale images, barriers, abort flag, TMEM base.
struct Plan {
    int stage, images, words;  // bytes of a stage; scale images of a stage; words of a row in a stage
    __host__ __device__ Plan(int width, bool e2m1) {
        stage = kStageA + width * kStageRow;
        words = e2m1 ? 2 : 1;
        images = (1 + (width + 127) / 128) * words;
    }
    __host__ __device__ int bars_at(int ring) const { return ring * (stage + images * kImage); }
    __host__ __device__ int bytes(int ring) const { return bars_at(ring) + 8 * kNumBars + 16 + 1024; }
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

// Tile -> its first token and its first output. Tokens run fastest, in groups
// of 16 tiles, so that a wave of tiles reads few weight rows and its tokens stay in L2.
template <bool SWIGLU>
__device__ __forceinline__ void place(const Params& p, int tile, int64_t& t0, int64_t& n0) {
    constexpr int kGroup = 16;
    const int n_tiles = p.tiles / p.m_tiles;
    const int group = tile / (kGroup * n_tiles), in = tile - group * kGroup * n_tiles;
    const int high = min(kGroup, p.m_tiles - group * kGroup);
    const int nt = in / high;
    t0 = static_cast<int64_t>(group * kGroup + in - nt * high) * kRows;
    n0 = static_cast<int64_t>(nt) * (SWIGLU ? p.width / 2 : p.width);
}

// ---------------------------------------------------------------- copies
template <bool E2M1, bool SWIGLU>
__device__ void copy_codes(const Params& p, const Plan& plan, const CUtensorMap* amap, const CUtensorMap* bmap,
                           uint32_t base, const Bars& bars, const WaitCtx& wc) {
    const uint32_t bytes = p.rows_a * kStageRow + p.width * (E2M1 ? kStageRow : kStageRow / 2);
    Ring r;
    int issued = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < p.tiles && ok; tile += gridDim.x) {
        int64_t t0, n0;
        place<SWIGLU>(p, tile, t0, n0);
        for (int k = 0; k < p.stages; ++k) {
            if (!mbar_wait(bars.empty(r.slot), r.phase ^ 1u, wc)) {
                ok = false;
                break;
            }
            const uint32_t a = base + r.slot * plan.stage, b = a + kStageA, full = bars.full(r.slot);
            ++issued;
            if (withhold_stage(static_cast<uint32_t>(issued - 1))) {  // test-only builds
                r.next(p.ring);
                continue;
            }
            mbar_arrive_expect_tx(full, bytes);
            tc::load_box_2d(a, amap, k * kStageRow, static_cast<int>(t0), full);
            auto weights = [&](uint32_t dst, int64_t row) {
                if constexpr (E2M1)
                    tc::load_box_2d(dst, bmap, k * kStageRow, static_cast<int>(row), full);
                else
                    tc::load_box_3d(dst, bmap, 0, static_cast<int>(row), k, full);
            };
            weights(b, n0);
            if constexpr (SWIGLU) weights(b + p.rows_b * kStageRow, p.n + n0);
            r.next(p.ring);
        }
    }
    if (!ok) {
        // Copies in flight land before the CTA may exit (bounded, whatever the abort flag says).
        int never = 0;
        const WaitCtx own{p.status, &never};
        for (int j = issued > p.ring ? issued - p.ring : 0; j < issued; ++j)
            mbar_wait(bars.full(j % p.ring), static_cast<uint32_t>((j / p.ring) & 1), own);
    }
}

// ---------------------------------------------------------------- scales
// Warp `image` of the scale warps: image 0 tokens, 1 and 2 weight rows.
template <bool E2M1, bool SWIGLU>
__device__ void copy_scales(const Params& p, const Plan& plan, int image, int lane, uint32_t base, const Bars& bars,
                            const WaitCtx& wc) {
    constexpr int W = E2M1 ? 2 : 1;   // words of a row in a stage
    constexpr int S = 4 / W;          // stages of a group of 4 words
    const int64_t pitch = p.k / 32;
    const int words = static_cast<int>(p.k / 128);
    const uint8_t* array = image == 0 ? p.xs : p.ws;
    const bool wide = pitch % 16 == 0 && (reinterpret_cast<uintptr_t>(array) & 15) == 0;
    const int groups = (p.stages + S - 1) / S;

    const uint8_t* row[4];
    auto rows_of = [&](int tile) {
        int64_t t0, n0;
        place<SWIGLU>(p, tile, t0, n0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = 32 * q + lane + 128 * (image - 1);
            int64_t at;
            bool valid;
            if (image == 0) {
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
    };
    uint4 v[4];
    auto load = [&](int g) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = make_uint4(0u, 0u, 0u, 0u);  // rows that do not exist: their results go nowhere
            if (!row[q]) continue;
            // Through L2: another kernel may have written them just now.
            if (wide) {
                v[q] = __ldcg(reinterpret_cast<const uint4*>(row[q]) + g);
            } else {
                const uint32_t* s = reinterpret_cast<const uint32_t*>(row[q]) + 4 * g;
                if (4 * g < words) v[q].x = __ldcg(s);
                if (4 * g + 1 < words) v[q].y = __ldcg(s + 1);
                if (4 * g + 2 < words) v[q].z = __ldcg(s + 2);
                if (4 * g + 3 < words) v[q].w = __ldcg(s + 3);
            }
        }
    };
    Ring r;
    if (static_cast<int>(blockIdx.x) < p.tiles) {
        rows_of(blockIdx.x);
        load(0);
    }
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        for (int g = 0; g < groups; ++g) {
            uint4 now[4] = {v[0], v[1], v[2], v[3]};
            if (g + 1 < groups) {
                load(g + 1);
            } else if (static_cast<int>(gridDim.x) < p.tiles - tile) {
                rows_of(tile + gridDim.x);
                load(0);
            }
            const uint32_t* a = reinterpret_cast<const uint32_t*>(now);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (g * S + s >= p.stages) break;
                if (!wait_all(bars.empty(r.slot), r.phase ^ 1u, wc)) return;
                const uint32_t at = base + p.ring * plan.stage + (r.slot * plan.images + image * W) * kImage + lane * 16;
#pragma unroll
                for (int w = 0; w < W; ++w)
                    sts128(at + w * kImage, a[s * W + w], a[4 + s * W + w], a[8 + s * W + w], a[12 + s * W + w]);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.scales(r.slot));
                r.next(p.ring);
            }
        }
    }
}

// -------------------------------------------------------------- products
template <bool E2M1>
__device__ bool issue_products(const Params& p, const Plan& plan, uint32_t base, uint32_t tbase, const Bars& bars,
                               const WaitCtx& wc) {
    // TMEM scale slots above the accumulators, 4 columns an image. A slot is
    // written again only after the products that read it are done.
    const int slots = (kTmemCols - kAccCols) / (4 * plan.images);
    const bool shared_cols = 2 * p.width > kAccCols;
    const int sfb_col = 4 * plan.words;
    const uint32_t idesc = tc::mma_idesc(E2M1 ? tc::kFmtMxf4E2M1 : tc::kFmtE4M3, E2M1 ? tc::kFmtMxf4E2M1 : tc::kFmtE2M1,
                                         kRows, static_cast<uint32_t>(p.width), 0);
    const bool one = elect_one();
    Ring r, behind;  // behind: the stage `slots` before
    int it = 0, tslot = 0, i = 0;
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, ++i) {
        const int back = shared_cols ? 1 : 2;  // whose epilogue frees this accumulator
        if (i >= back && !wait_all(bars.acc_empty(i & 1), static_cast<uint32_t>((i - back) >> 1) & 1u, wc)) return false;
        const uint32_t d = tbase + ((i & 1) ? kAccCols - p.width : 0);
        for (int k = 0; k < p.stages; ++k, ++it) {
            if (slots < p.ring && it >= slots) {
                if (!wait_all(bars.empty(behind.slot), behind.phase, wc)) return false;
                behind.next(p.ring);
            }
            if (!wait_all(bars.scales(r.slot), r.phase, wc)) return false;
            if (!wait_all(bars.full(r.slot), r.phase, wc)) return false;
            tc::fence_after_sync();
            const uint32_t a = base + r.slot * plan.stage;
            const uint32_t image = base + p.ring * plan.stage + r.slot * plan.images * kImage;
            const uint32_t sf = tbase + kAccCols + tslot * 4 * plan.images;
            const uint64_t ad = tc::operand_desc(a), bd = tc::operand_desc(a + kStageA), sd = tc::scale_image_desc(image);
            if (one) {
                // Images in memory: of the tokens by word, then of each 128 weight rows by word. In TMEM the weight
                // rows' images of one word lie next to each other.
#pragma unroll
                for (int w = 0; w < (E2M1 ? 2 : 1); ++w) {
                    tc::copy_scales_to_tmem(sf + 4 * w, sd + w * (kImage >> 4));
                    for (int b = 0; b * 128 < p.width; ++b)
                        tc::copy_scales_to_tmem(sf + sfb_col + (w * ((p.width + 127) / 128) + b) * 4,
                                                sd + ((1 + b) * plan.words + w) * (kImage >> 4));
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const bool acc = k != 0 || c != 0;
                    if constexpr (E2M1) {
                        const uint32_t sfb = sf + sfb_col + (c >> 1) * ((p.width + 127) / 128) * 4;
                        tc::mma_mxf4(d, ad + 2 * c, bd + 2 * c, idesc | ((c & 1) * 2u) << 4 | ((c & 1) * 2u) << 29,
                                     sf + 4 * (c >> 1), sfb, acc);
                    } else {
                        tc::mma_mxf8f6f4(d, ad + 2 * c, bd + 2 * c,
                                         idesc | static_cast<uint32_t>(c) << 4 | static_cast<uint32_t>(c) << 29, sf,
                                         sf + sfb_col, acc);
                    }
                }
                tc::commit_to(bars.empty(r.slot));
                if (k == p.stages - 1) tc::commit_to(bars.acc_full(i & 1));
            }
            __syncwarp();
            if (++tslot == slots) tslot = 0;
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

// 32 outputs of one token, `count` of them wanted.
__device__ __forceinline__ void store_row(__nv_bfloat16* y, const float (&v)[32], int count, bool wide) {
    if (wide && count >= 32) {
        uint4* o = reinterpret_cast<uint4*>(y);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const Bf16x8 b = pack8(*reinterpret_cast<const float(*)[8]>(v + 8 * q));
            o[q] = *reinterpret_cast<const uint4*>(&b);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j < count) y[j] = __float2bfloat16_rn(v[j]);
}

template <bool OUT_E2M1>
__device__ __forceinline__ void store_block(uint8_t* q, uint8_t* s, const float (&h)[32]) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) top = max(top, mx::abs_bits(h[j]));
    const uint32_t b = mx::scale_byte<OUT_E2M1>(top);
    uint32_t w[OUT_E2M1 ? 4 : 8];
    mx::encode<OUT_E2M1, 32>(h, b, w);
#pragma unroll
    for (int i = 0; i < (OUT_E2M1 ? 1 : 2); ++i)
        reinterpret_cast<uint4*>(q)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    *s = static_cast<uint8_t>(b);
}

template <bool SWIGLU>
__device__ void epilogue(const Params& p, int warp, int lane, uint32_t tbase, const Bars& bars, const WaitCtx& wc) {
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const bool shared_cols = 2 * p.width > kAccCols;
    const int chunks = (SWIGLU ? p.width / 2 : p.width) / 32;
    // Chunks that hold columns of the other accumulator come first.
    const int early = shared_cols ? (2 * p.width - kAccCols + 31) / 32 : chunks;
    int i = 0;
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, ++i) {
        int64_t t0, n0;
        place<SWIGLU>(p, tile, t0, n0);
        if (!wait_all(bars.acc_full(i & 1), static_cast<uint32_t>(i >> 1) & 1u, wc)) return;
        tc::fence_after_sync();
        const uint32_t acc = tbase + lanes + ((i & 1) ? kAccCols - p.width : 0);
        const int64_t row = t0 + quarter * 32 + lane;
        for (int c = 0; c <= chunks; ++c) {
            if (c == early || (c == chunks && early > chunks)) {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.acc_empty((i & 1) ^ (shared_cols ? 1 : 0)));
            }
            if (c == chunks) break;
            if ((c & 1) != half) continue;
            const int at = (i & 1) || !shared_cols ? c : chunks - 1 - c;
            const int64_t col = n0 + 32 * at;
            if constexpr (SWIGLU) {
                float a[32], b[32];
                load32(acc + 32 * at, a);
                load32(acc + p.width / 2 + 32 * at, b);
                tc::tmem_wait_ld();
                if (row < p.t && col < p.n) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) a[j] = mx::swiglu(a[j], b[j]);
                    const int64_t e = row * p.n + col;
                    if (p.out_e2m1)
                        store_block<true>(p.y + e / 2, p.ys + e / 32, a);
                    else
                        store_block<false>(p.y + e, p.ys + e / 32, a);
                }
            } else {
                float v[32];
                load32(acc + 32 * at, v);
                tc::tmem_wait_ld();
                if (row < p.t && col < p.n)
                    store_row(reinterpret_cast<__nv_bfloat16*>(p.y) + row * p.n + col, v,
                              static_cast<int>(p.n - col < 32 ? p.n - col : 32), p.wide);
            }
        }
    }
}

// ---------------------------------------------------------------- kernel
template <bool E2M1, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    mx_product_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const Plan plan(p.width, E2M1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Bars bars{base + plan.bars_at(p.ring)};
    const uint32_t flag = bars.base + 8 * kNumBars, tslot = flag + 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + (flag - raw));
    const WaitCtx wc{p.status, abort_flag};
    pdl_launch_dependents();
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tslot, kTmemCols);
        tc::tmem_relinquish();
    }
    if (warp == kCopyWarp && lane == 0) {
        for (int s = 0; s < p.ring; ++s) {
            mbar_init(bars.full(s), 1);
            mbar_init(bars.scales(s), static_cast<uint32_t>(plan.images / plan.words));
            mbar_init(bars.empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bars.acc_full(b), 1);
            mbar_init(bars.acc_empty(b), kEpilogueWarps);
        }
        mbar_init(bars.drain(), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = lds_u32_volatile(tslot);
    // Codes and scales may come from the previous kernel of the stream, and it may still read y.
    pdl_wait_previous();
    if (warp < kEpilogueWarps) {
        epilogue<SWIGLU>(p, warp, lane, tbase, bars, wc);
    } else if (warp == kCopyWarp) {
        if (lane == 0) copy_codes<E2M1, SWIGLU>(p, plan, &amap, &bmap, base, bars, wc);
    } else if (warp == kMmaWarp) {
        if (!issue_products<E2M1>(p, plan, base, tbase, bars, wc)) {
            // Products issued so far may still read shared memory and write TMEM: waited for, bounded.
            if (lane == 0) {
                tc::commit_to(bars.drain());
                int never = 0;
                const WaitCtx own{p.status, &never};
                mbar_wait(bars.drain(), 0, own);
            }
        }
    } else if ((warp - kScaleWarp) * plan.words < plan.images) {
        copy_scales<E2M1, SWIGLU>(p, plan, warp - kScaleWarp, lane, base, bars, wc);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, kTmemCols);
    }
}

template <bool E2M1, bool SWIGLU>
cudaError_t launch(const CUtensorMap& amap, const CUtensorMap& bmap, const Params& p, int smem, int grid,
                   cudaStream_t stream) {
    static int configured[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || configured[dev] < smem) {
        const cudaError_t e = cudaFuncSetAttribute(mx_product_kernel<E2M1, SWIGLU>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = smem;
    }
    PdlLaunch l(dim3(grid), dim3(kThreads), smem, stream);
    return cudaLaunchKernelEx(&l.cfg, mx_product_kernel<E2M1, SWIGLU>, amap, bmap, p);
}

}  // namespace
}  // namespace mxp

cudaError_t launch_mx_product(const MxProductArgs& a, int num_sms, int max_smem, cudaStream_t stream) {
    using namespace mxp;
    const int width = 256;
    const int outputs = a.swiglu ? width / 2 : width;
    Params p{};
    p.xs = a.xs;
    p.ws = a.ws;
    p.y = static_cast<uint8_t*>(a.y);
    p.ys = a.ys;
    p.status = a.status;
    p.t = a.t;
    p.n = a.n;
    p.k = a.k;
    p.width = width;
    p.out_e2m1 = a.out_e2m1;
    p.wide = a.n % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
    p.stages = static_cast<int>((a.k + (a.e2m1 ? 255 : 127)) / (a.e2m1 ? 256 : 128));
    const int64_t m_tiles = (a.t + kRows - 1) / kRows, n_tiles = (a.n + outputs - 1) / outputs;
    if (m_tiles * n_tiles >= (int64_t(1) << 31) - num_sms) return cudaErrorInvalidValue;
    p.m_tiles = static_cast<int>(m_tiles);
    p.tiles = static_cast<int>(m_tiles * n_tiles);
    p.rows_a = a.t < kRows ? static_cast<int>((a.t + 7) / 8 * 8) : kRows;
    p.rows_b = outputs;
    const Plan plan(width, a.e2m1);
    p.ring = 1;
    while (p.ring < kMaxStages && plan.bytes(p.ring + 1) <= max_smem) ++p.ring;
    const int64_t w_rows = a.swiglu ? 2 * a.n : a.n;
    CUtensorMap amap, bmap;
    cudaError_t e = encode_code_map(&amap, a.xq, a.t, a.e2m1 ? a.k / 2 : a.k, p.rows_a);
    if (e == cudaSuccess)
        e = a.e2m1 ? encode_code_map(&bmap, a.wq, w_rows, a.k / 2, p.rows_b)
                   : encode_spread_map(&bmap, a.wq, w_rows, a.k, p.rows_b);
    if (e != cudaSuccess) return e;
    const int grid = p.tiles < num_sms ? p.tiles : num_sms;
    const int smem = plan.bytes(p.ring);
    if (a.e2m1)
        return a.swiglu ? launch<true, true>(amap, bmap, p, smem, grid, stream)
                        : launch<true, false>(amap, bmap, p, smem, grid, stream);
    return a.swiglu ? launch<false, true>(amap, bmap, p, smem, grid, stream)
                    : launch<false, false>(amap, bmap, p, smem, grid, stream);
}

}  // namespace mxfp4
