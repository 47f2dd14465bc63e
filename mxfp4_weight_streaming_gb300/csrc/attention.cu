// Attention of a step's new tokens over the paged cache, for few rows per KV
// head (decode and verify): every K and V row is read once and serves all
// rows of its KV head.
//
// A CTA has 4 warps that never wait for one another inside an item: of each
// 64-key tile a warp takes 16 keys, which lie in one page. It keeps its own
// ring of K and V rows in shared memory (cp.async, zero-filled where a key is
// beyond the sequence, so stale or NaN rows there never meet a product), its
// own running maximum and sum, and its own output accumulators; the four are
// joined once per item. Scores and outputs are mma.sync m16n8k16 with fp32
// accumulation: at up to 32 rows the products take less time than the bytes.
//
// bf16 cache: bf16 products, probabilities rounded to bf16 (a product takes
// both operands in one type; attention_tc.cu has the errors). E4M3 cache: the
// rows become f16 in registers (exact), q is scaled per row by a power of
// two into f16's range and probabilities are f16. Sums, maxima and
// accumulators are fp32.
#include <cuda_fp16.h>

#include "attention_common.cuh"
#include "step_launch.h"

namespace mxfp4 {
namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 16;                // keys per warp and step
constexpr int kKeyTile = kKeys * kWarps;  // keys per CTA and step
constexpr int kKeyShift = 6;
static_assert(kKeyTile == 1 << kKeyShift);
// CTAs per SM, and the ring of a warp. The kernel is bound by the latency of
// its chains (load, score, maximum, product): with 16 rows and K rows of up to
// 128 bytes registers and rings leave room for three CTAs (64 requests of
// 6,000 tokens, E4M3, D = 128: 173 us with two, 142 with three, 200 with four,
// whose rings are too short).
__host__ __device__ constexpr bool three_ctas(int d, bool e4m3, int mt) { return mt == 1 && d * (e4m3 ? 1 : 2) <= 128; }
__host__ __device__ constexpr int ctas_per_sm(int d, bool e4m3, int mt) { return three_ctas(d, e4m3, mt) ? 3 : 2; }
__host__ __device__ constexpr int ring_bytes(int d, bool e4m3, int mt) { return three_ctas(d, e4m3, mt) ? 16384 : 24576; }
// A running maximum is raised only when a score exceeds it by more than this
// (log2): probabilities stay below 2^8, and the accumulators are seldom
// rescaled.
constexpr float kSlack = 8.f;

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                                  uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two E4M3 bytes (bits 0-15 or 16-31 of w) -> f16x2, exact.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async16_all(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Shared-memory address of 16-byte chunk c of row r: chunks are XORed with
// the row so that 8 rows of one column of chunks cover all banks.
template <int CH>
__device__ __forceinline__ int swizzle(int r) {
    return CH >= 8 ? (r & 7) : ((r >> 1) & (CH - 1));
}
template <int RB>
__device__ __forceinline__ uint32_t at(uint32_t base, int r, int c) {
    return base + r * RB + ((c ^ swizzle<RB / 16>(r)) << 4);
}

// Whether a 16-byte chunk of a V row holds an infinity or a NaN.
template <bool E4M3>
__device__ __forceinline__ bool chunk_not_finite(uint4 w) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (E4M3) bad |= __vcmpeq4(x[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        else bad |= __vcmpeq2(x[i] & 0x7f807f80u, 0x7f807f80u);
    }
    return bad != 0;
}

// Element d of V row r in a stage.
template <int RB, bool E4M3>
__device__ __forceinline__ float v_element(uint32_t vst, int r, int d) {
    const uint32_t byte = d * (E4M3 ? 1 : 2), a = at<RB>(vst, r, byte >> 4) + (byte & 15);
    if constexpr (E4M3) {
        __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(lds_u8(a)), __NV_E4M3);
        return __half2float(__half(h));
    } else {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    }
}

// PLACED: windows count from Params::positions (a variant of its own: in the
// other the look-up costs registers, 64 requests x 4 tokens, E4M3, 221 -> 269 us).
template <int D, bool E4M3, int MT, bool PLACED>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, E4M3, MT)) attention_rows_kernel(Params p) {
    constexpr int R = 16 * MT;                 // rows of a row tile
    constexpr int RB = D * (E4M3 ? 1 : 2);     // bytes of a K or V row
    constexpr int CH = RB / 16;
    constexpr int STAGE = 2 * kKeys * RB;      // K rows, then V rows
    constexpr int RING = ring_bytes(D, E4M3, MT);
    constexpr int STAGES = RING / STAGE < 8 ? RING / STAGE : 8;
    constexpr int KK = D / 16;
    static_assert(STAGES >= 3 && R * D * 4 <= STAGES * STAGE, "ring too small for the join");

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_before[kGroups + 1];
    __shared__ float s_m[kWarps][R], s_l[kWarps][R];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * (STAGES * STAGE);
    // A lane copies chunk lane % CH of rows lane / CH, + 32 / CH, ...: the row's
    // share of the address and of the XOR split into a lane's and a step's part.
    const uint32_t lane_at_row = (lane / CH) * RB;
    const int lane_chunk = (lane % CH) ^ swizzle<CH>(lane / CH);
    float* const join = reinterpret_cast<float*>(smem);  // [warp][R][D] over the rings
    constexpr int kJoinStride = STAGES * STAGE / 4;
    const CacheView& cv = p.cache;
    const Cut& cut = p.cut;
    const int page_mask = (1 << cv.page_shift) - 1;
    const Parts parts = parts_in(p.ws, gridDim.x, R, D);

    pdl_wait_previous();
    const int64_t total = count_units<kThreads>(cut, p.batch, threadIdx.x, s_before);
    const int64_t share = share_of(cut, total, gridDim.x);
    int64_t unit = share * blockIdx.x;
    const int64_t unit_end = min(unit + share, total);
    if (threadIdx.x == 0) parts.split[blockIdx.x].parts = 0;

    while (unit < unit_end) {
        const Item it = locate(cut, p.batch, s_before, unit);
        const int steps = static_cast<int>(min(unit_end - unit, static_cast<int64_t>(it.tiles - it.tile)));
        const int rows = min(R, it.n * cut.group - it.rt * R);
        const int start = it.seq - it.n;  // cache index of the first new token
        // First key of this warp's step 0.
        const int key0 = (it.begin / kKeyTile + it.tile) * kKeyTile + warp * kKeys;
        const int64_t head_off = static_cast<int64_t>(it.head) << cv.page_shift;

        auto load_page = [&](int step) {
            const int key = key0 + step * kKeyTile;
            return (step < steps && key < it.end) ? page_of(p.batch, it.b, key, cv.page_shift, cv.num_pages) : -1;
        };
        auto issue = [&](int step, int page) {
            if (step < steps) {
                const int key = key0 + step * kKeyTile;
                const uint32_t dst = ring + (step % STAGES) * STAGE;
                const int64_t off = (page < 0 ? 0 : page) * cv.page_stride + (head_off + (key & page_mask)) * D;
                const char* kp = static_cast<const char*>(cv.k) + off * (E4M3 ? 1 : 2) + lane * 16;
                const char* vp = static_cast<const char*>(cv.v) + off * (E4M3 ? 1 : 2) + lane * 16;
                // The rows of 16 keys are contiguous: copy i takes 512 bytes on.
                const bool all = page >= 0 && key >= it.begin && key + kKeys <= it.end;
                if (all) {
#pragma unroll
                    for (int i = 0; i < kKeys * CH / 32; ++i) {
                        const uint32_t to = dst + lane_at_row + i * 512 + ((lane_chunk ^ swizzle<CH>(i * (32 / CH))) << 4);
                        cp_async16_all(to, kp + i * 512);
                        cp_async16_all(to + kKeys * RB, vp + i * 512);
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < kKeys * CH / 32; ++i) {
                        const int r = i * (32 / CH) + lane / CH;
                        const bool valid = page >= 0 && key + r >= it.begin && key + r < it.end;
                        const uint32_t to = dst + lane_at_row + i * 512 + ((lane_chunk ^ swizzle<CH>(i * (32 / CH))) << 4);
                        cp_async16(to, valid ? kp + i * 512 : static_cast<const char*>(cv.k), valid);
                        cp_async16(to + kKeys * RB, valid ? vp + i * 512 : static_cast<const char*>(cv.v), valid);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        // Pages run one step ahead of the copies that need them.
        int page = load_page(0);
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            const int next = load_page(s + 1);
            issue(s, page);
            page = next;
        }

        // q as A operands, and of each of this thread's rows its token and
        // score factor.
        uint32_t qf[MT][KK][4];
        float q_mul[MT][2];
        int tok[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = mt * 16 + h * 8 + g;
                const bool in = r < rows;
                const int row = it.rt * R + (in ? r : 0);
                const int i = cut.by_group.div(row);
                tok[mt][h] = in ? i : -1;
                const __nv_bfloat16* src =
                    p.q + (it.first + i) * p.q_stride + (it.head * cut.group + row - i * cut.group) * D;
                if constexpr (!E4M3) {
                    q_mul[mt][h] = 1.f;
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        qf[mt][kk][h] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 2 * t) : 0u;
                        qf[mt][kk][h + 2] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8 + 2 * t) : 0u;
                    }
                } else {
                    // Thread t of a row holds elements 4t .. 4t + 3 of each
                    // 16 (the order the E4M3 rows of K come in).
                    uint2 w[KK];
                    float top = 0.f;
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        w[kk] = in ? *reinterpret_cast<const uint2*>(src + kk * 16 + 4 * t) : make_uint2(0, 0);
                        const __nv_bfloat162* f = reinterpret_cast<const __nv_bfloat162*>(&w[kk]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float2 v = __bfloat1622float2(f[j]);
                            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                        }
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // 2^-e with the row's largest magnitude in [2^e, 2^(e+1)),
                    // kept within the normal numbers.
                    const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -120), 120);
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    q_mul[mt][h] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const __nv_bfloat162* f = reinterpret_cast<const __nv_bfloat162*>(&w[kk]);
                        const float2 a = __bfloat1622float2(f[0]), b = __bfloat1622float2(f[1]);
                        qf[mt][kk][h] = pack_f16(a.x * down, a.y * down);
                        qf[mt][kk][h + 2] = pack_f16(b.x * down, b.y * down);
                    }
                }
            }
        if constexpr (E4M3) {
            const float ks = cv.k_scale ? cv.k_scale[it.head] : 1.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) q_mul[mt][0] *= ks, q_mul[mt][1] *= ks;
        }

        float o[MT][KK * 2][4];
        float m[MT][2], l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int n = 0; n < KK * 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[mt][n][j] = 0.f;
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.f;
        }
        // Keys below `open` are visible to every row (without a window).
        const int open = cut.tree ? start : start + cut.by_group.div(it.rt * R) + 1;

#pragma unroll 1
        for (int step = 0; step < steps; ++step) {
            {
                const int next = load_page(step + STAGES);
                __syncwarp();
                issue(step + STAGES - 1, page);
                page = next;
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
            __syncwarp();
            const uint32_t kst = ring + (step % STAGES) * STAGE, vst = kst + kKeys * RB;
            const int key = key0 + step * kKeyTile;

            float s[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[mt][n][j] = 0.f;
            if constexpr (!E4M3) {
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    uint32_t b[4];
                    ldmatrix_x4(at<RB>(kst, (lane >> 4) * 8 + (lane & 7), 2 * kk + ((lane >> 3) & 1)), b[0], b[1],
                                b[2], b[3]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma<false>(s[mt][0], qf[mt][kk], b[0], b[1]);
                        mma<false>(s[mt][1], qf[mt][kk], b[2], b[3]);
                    }
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < KK; kk += 2) {
                    uint32_t b[4];
                    ldmatrix_x4(at<RB>(kst, ((lane >> 3) & 1) * 8 + (lane & 7), kk + (lane >> 4)), b[0], b[1], b[2],
                                b[3]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t b00 = e4m3_lo(b[2 * x]), b01 = e4m3_hi(b[2 * x]);
                        const uint32_t b10 = e4m3_lo(b[2 * x + 1]), b11 = e4m3_hi(b[2 * x + 1]);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            mma<true>(s[mt][0], qf[mt][kk + x], b00, b01);
                            mma<true>(s[mt][1], qf[mt][kk + x], b10, b11);
                        }
                    }
                }
            }

            // Scores to the log2 domain, masked where the row does not see the key.
            const bool edge = key + kKeys > min(open, it.end) || cut.window != 0 || key < it.begin;
            bool raise = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    int pos = start + tok[mt][h];
                    unsigned long long word = 0;
                    if (edge && cut.tree && tok[mt][h] >= 0) {
                        word = p.tree_mask[it.first + tok[mt][h]];
                        if constexpr (PLACED) pos = window_from(p.positions + it.first + tok[mt][h], start, it.seq, cut.window);
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float& x = s[mt][n][2 * h + j];
                            x = p.map(E4M3 ? x * q_mul[mt][h] : x);
                            if (edge) {
                                const int k = key + n * 8 + 2 * t + j;
                                bool see = k < it.end && k >= it.begin && tok[mt][h] >= 0;
                                if (cut.tree)
                                    see = see && (k < start || (k - start < 64 && (word >> (k - start) & 1)));
                                else
                                    see = see && k <= pos;
                                if (cut.window) see = see && k > pos - cut.window;
                                if (!see) x = -INFINITY;
                            }
                            top = fmaxf(top, x);
                        }
                    raise = raise || top > m[mt][h] + kSlack;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float top = fmaxf(fmaxf(s[mt][0][2 * h], s[mt][0][2 * h + 1]),
                                          fmaxf(s[mt][1][2 * h], s[mt][1][2 * h + 1]));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        top = fmaxf(top, m[mt][h]);
                        const float f = top == m[mt][h] ? 1.f : exp2_fast(m[mt][h] - top);
                        m[mt][h] = top;
                        l[mt][h] *= f;
#pragma unroll
                        for (int n = 0; n < KK * 2; ++n) {
                            o[mt][n][2 * h] *= f;
                            o[mt][n][2 * h + 1] *= f;
                        }
                    }
            }
            uint32_t pf[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float base = m[mt][h] == -INFINITY ? 0.f : m[mt][h];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float a = exp2_fast(s[mt][n][2 * h] - base), b = exp2_fast(s[mt][n][2 * h + 1] - base);
                        l[mt][h] += a + b;
                        pf[mt][2 * n + h] = E4M3 ? pack_f16(a, b) : pack_bf16(a, b);
                    }
                }

            // A key that some rows see and others do not may hold an infinity
            // or a NaN, and 0 * NaN is NaN: then the product is taken key by
            // key, without the rows that do not see it.
            if (edge) {
                bool bad = false;
#pragma unroll
                for (int i = 0; i < kKeys * CH / 32; ++i) {
                    const int idx = i * 32 + lane;
                    bad = bad || chunk_not_finite<E4M3>(lds128(at<RB>(vst, idx / CH, idx % CH)));
                }
                if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
                    for (int kx = 0; kx < kKeys; ++kx)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t both = kx < 8 ? pf[mt][h] : pf[mt][2 + h];
                                const uint32_t w = __shfl_sync(0xffffffffu, both, (lane & ~3) | ((kx & 7) >> 1));
                                const uint16_t bits = static_cast<uint16_t>(kx & 1 ? w >> 16 : w);
                                if ((bits & 0x7fff) == 0) continue;
                                const float f = E4M3 ? __half2float(__ushort_as_half(bits))
                                                     : __uint_as_float(static_cast<uint32_t>(bits) << 16);
#pragma unroll
                                for (int n = 0; n < KK * 2; ++n)
#pragma unroll
                                    for (int j = 0; j < 2; ++j) {
                                        const int d = E4M3 ? (n >> 1) * 16 + 4 * t + 2 * j + (n & 1) : n * 8 + 2 * t + j;
                                        o[mt][n][2 * h + j] += f * v_element<RB, E4M3>(vst, kx, d);
                                    }
                            }
                    continue;
                }
            }
            if constexpr (!E4M3) {
#pragma unroll
                for (int j = 0; j < KK; ++j) {
                    uint32_t b[4];
                    ldmatrix_x4_trans(at<RB>(vst, ((lane >> 3) & 1) * 8 + (lane & 7), 2 * j + (lane >> 4)), b[0], b[1],
                                      b[2], b[3]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma<false>(o[mt][2 * j], pf[mt], b[0], b[1]);
                        mma<false>(o[mt][2 * j + 1], pf[mt], b[2], b[3]);
                    }
                }
            } else {
                // A transposed 8x8 of byte pairs gives (key 2t, key 2t + 1) x
                // (element 2g, 2g + 1): even elements go to one column tile,
                // odd ones to the next.
#pragma unroll
                for (int j = 0; j < KK; j += 2) {
                    uint32_t b[4];
                    ldmatrix_x4_trans(at<RB>(vst, ((lane >> 3) & 1) * 8 + (lane & 7), j + (lane >> 4)), b[0], b[1],
                                      b[2], b[3]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t lo = prmt(b[2 * x], 0, 0x3120), hi = prmt(b[2 * x + 1], 0, 0x3120);
                        const uint32_t e0 = e4m3_lo(lo), e1 = e4m3_lo(hi), d0 = e4m3_hi(lo), d1 = e4m3_hi(hi);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            mma<true>(o[mt][2 * (j + x)], pf[mt], e0, e1);
                            mma<true>(o[mt][2 * (j + x) + 1], pf[mt], d0, d1);
                        }
                    }
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();

        // The warp's part, over its own ring.
        float* mine = join + warp * kJoinStride;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = mt * 16 + h * 8 + g;
                float sum = l[mt][h];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (t == 0) {
                    s_m[warp][r] = m[mt][h];
                    s_l[warp][r] = sum;
                }
                if constexpr (!E4M3) {
#pragma unroll
                    for (int n = 0; n < KK * 2; ++n)
                        *reinterpret_cast<float2*>(mine + r * D + n * 8 + 2 * t) =
                            make_float2(o[mt][n][2 * h], o[mt][n][2 * h + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < KK; ++j)
                        *reinterpret_cast<float4*>(mine + r * D + j * 16 + 4 * t) =
                            make_float4(o[mt][2 * j][2 * h], o[mt][2 * j + 1][2 * h], o[mt][2 * j][2 * h + 1],
                                        o[mt][2 * j + 1][2 * h + 1]);
                }
            }
        __syncthreads();

        const bool whole = it.tile == 0 && steps == it.tiles;
        const int slot = 2 * blockIdx.x + (it.tile == 0);
        if (!whole && it.tile == 0 && threadIdx.x == 0) {
            const int64_t last = unit + it.tiles - 1;
            parts.split[blockIdx.x] =
                Split{static_cast<int>(last / share) - static_cast<int>(blockIdx.x) + 1, it.rt * R, rows, it.first, it.head};
        }
        const float vs = E4M3 && cv.v_scale ? cv.v_scale[it.head] : 1.f;
        for (int v = threadIdx.x; v < rows * (D / 4); v += kThreads) {
            const int r = v / (D / 4), d = (v % (D / 4)) * 4;
            float top = s_m[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
            const float base = top == -INFINITY ? 0.f : top;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = s_m[w][r] == top ? 1.f : exp2_fast(s_m[w][r] - base);
                const float4 x = *reinterpret_cast<const float4*>(join + w * kJoinStride + r * D + d);
                sum += f * s_l[w][r];
                acc.x += f * x.x;
                acc.y += f * x.y;
                acc.z += f * x.z;
                acc.w += f * x.w;
            }
            if (whole) {
                const int row = it.rt * R + r, i = cut.by_group.div(row);
                const int64_t to = static_cast<int64_t>(it.first + i) * p.q_heads + it.head * cut.group + row -
                                   i * cut.group;
                const float f = sum == 0.f ? 0.f : vs / sum;
                uint2 w;
                w.x = pack_bf16(acc.x * f, acc.y * f);
                w.y = pack_bf16(acc.z * f, acc.w * f);
                *reinterpret_cast<uint2*>(p.out + to * D + d) = w;
                if (p.lse && d == 0) p.lse[to] = sum == 0.f ? -INFINITY : (top + log2f(sum)) / kLog2e;
            } else {
                *reinterpret_cast<float4*>(parts.o + (static_cast<int64_t>(slot) * R + r) * D + d) = acc;
                if (d == 0) parts.ml[slot * R + r] = make_float2(top, sum);
            }
        }
        __syncthreads();
        unit += steps;
    }
    pdl_launch_dependents();
}

// Joins the parts of items that several CTAs shared: block (c, y, z) takes
// rows and elements of the item that begins in CTA c, a thread 4 elements of a
// row. Neighbouring threads are neighbours in the order of the parts: elements
// of a row, or (parts of attention_tc.cu) rows. Loads of 8 parts are in flight
// at a time: the join is all latency.
constexpr int kJoinThreads = 256;
constexpr int kJoinBatch = 8;
template <int D, bool E4M3, bool FROM_TC>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(Params p, int ctas) {
    const Cut& cut = p.cut;
    const int R = 1 << cut.row_shift;
    pdl_wait_previous();
    pdl_launch_dependents();
    const Parts parts = parts_in(p.ws, ctas, R, D);
    const Split sp = parts.split[blockIdx.x];
    if (sp.parts == 0) return;
    const int t = threadIdx.x;
    const int r = FROM_TC ? blockIdx.y * 32 + t % 32 : blockIdx.y * (4 * kJoinThreads / D) + t / (D / 4);
    if (r >= sp.rows) return;
    for (int d4 = FROM_TC ? blockIdx.z * 8 + t / 32 : t % (D / 4); d4 < D / 4; d4 += FROM_TC ? 8 * gridDim.z : D / 4) {
        auto slot = [&](int i) { return i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i); };
        // A running join: what came before is scaled down where a batch's maximum is larger.
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f, top = -INFINITY;
        for (int x0 = 0; x0 < sp.parts; x0 += kJoinBatch) {
            float2 ml[kJoinBatch];
            float4 o[kJoinBatch];
            float here = top;
#pragma unroll
            for (int x = 0; x < kJoinBatch; ++x) {
                ml[x] = make_float2(-INFINITY, 0.f);
                if (x0 + x >= sp.parts) continue;
                const int sl = slot(x0 + x);
                ml[x] = parts.ml[sl * R + r];
                o[x] = reinterpret_cast<const float4*>(
                    parts.o)[static_cast<int64_t>(sl) * R * (D / 4) + (FROM_TC ? d4 * R + r : r * (D / 4) + d4)];
            }
#pragma unroll
            for (int x = 0; x < kJoinBatch; ++x) here = fmaxf(here, ml[x].x);
            const float base = here == -INFINITY ? 0.f : here;
            const float old = top == here ? 1.f : exp2_fast(top - base);
            acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
            sum *= old;
            top = here;
#pragma unroll
            for (int x = 0; x < kJoinBatch; ++x) {
                if (x0 + x >= sp.parts) break;
                const float f = ml[x].x == here ? 1.f : exp2_fast(ml[x].x - base);
                sum += f * ml[x].y;
                acc.x += f * o[x].x;
                acc.y += f * o[x].y;
                acc.z += f * o[x].z;
                acc.w += f * o[x].w;
            }
        }
        const int row = sp.row0 + r, tok = cut.by_group.div(row);
        const int64_t to = static_cast<int64_t>(sp.first + tok) * p.q_heads + sp.head * cut.group + row - tok * cut.group;
        const float vs = E4M3 && p.cache.v_scale ? p.cache.v_scale[sp.head] : 1.f;
        const float f = sum == 0.f ? 0.f : vs / sum;
        *reinterpret_cast<uint2*>(p.out + to * D + 4 * d4) =
            make_uint2(pack_bf16(acc.x * f, acc.y * f), pack_bf16(acc.z * f, acc.w * f));
        if (p.lse && d4 == 0) p.lse[to] = sum == 0.f ? -INFINITY : (top + log2f(sum)) / kLog2e;
    }
}

template <int D, bool E4M3, int MT, bool PLACED>
cudaError_t launch(const Params& p, int ctas, cudaStream_t stream) {
    constexpr int smem = kWarps * ring_bytes(D, E4M3, MT);
    static thread_local int ready_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (ready_device != dev) {
        e = cudaFuncSetAttribute(attention_rows_kernel<D, E4M3, MT, PLACED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready_device = dev;
    }
    PdlLaunch l(dim3(ctas), dim3(kThreads), smem, stream);
    e = cudaLaunchKernelEx(&l.cfg, attention_rows_kernel<D, E4M3, MT, PLACED>, p);
    return e == cudaSuccess ? launch_join(p, E4M3, false, ctas, stream) : e;
}

template <int D, bool PLACED>
cudaError_t launch_d(const Params& p, bool e4m3, int mt, int ctas, cudaStream_t stream) {
    if (!e4m3) return launch<D, false, 1, PLACED>(p, ctas, stream);  // more than 16 rows: attention_tc.cu
    return mt == 1 ? launch<D, true, 1, PLACED>(p, ctas, stream) : launch<D, true, 2, PLACED>(p, ctas, stream);
}

// The tensor-core kernel where the rows of a KV head fill enough of its
// 128-row tiles (us, this kernel / attention_tc.cu). bf16, groups of 7, D = 128,
// 64 requests of 4,090 tokens: 7 rows 173 / 185, 14 rows 175 / 187; 28 rows over
// one request of 131,069 tokens 130 / 99. E4M3, where the bytes have to pass
// through converting warps: 14 rows 102 / 225; 28 rows 216 / 228, 8 requests of
// 2,000 34 / 36, 16 of 1,000 (21 rows) 34 / 37, but one of 131,069 116 / 102;
// D = 64, 20 rows: 64 x 4,090 150 / 138, 8 x 2,000 22 / 23, one of 131,069 82 / 73.
bool use_tc(int64_t rows, bool e4m3) { return rows > (e4m3 ? 32 : 16); }

template <int D, bool E4M3>
cudaError_t launch_join_d(const PdlLaunch& j, const Params& p, bool from_tc, int ctas) {
    return from_tc ? cudaLaunchKernelEx(&j.cfg, attention_join_kernel<D, E4M3, true>, p, ctas)
                   : cudaLaunchKernelEx(&j.cfg, attention_join_kernel<D, E4M3, false>, p, ctas);
}

}  // namespace

cudaError_t launch_join(const Params& p, bool e4m3, bool from_tc, int ctas, cudaStream_t stream) {
    const int rows = 1 << p.cut.row_shift, d = p.cache.head_dim, per = 4 * kJoinThreads / d;
    // With 256 rows an item's blocks are many as it is.
    const dim3 grid = from_tc ? dim3(ctas, rows / 32, rows == 128 ? d / 32 : 1) : dim3(ctas, (rows + per - 1) / per, 1);
    PdlLaunch j(grid, dim3(kJoinThreads), 0, stream);
    if (p.cache.head_dim == 64)
        return e4m3 ? launch_join_d<64, true>(j, p, from_tc, ctas) : launch_join_d<64, false>(j, p, from_tc, ctas);
    return e4m3 ? launch_join_d<128, true>(j, p, from_tc, ctas) : launch_join_d<128, false>(j, p, from_tc, ctas);
}

}  // namespace attn

size_t attention_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q, bool e4m3, int num_sms) {
    const int64_t rows = static_cast<int64_t>(max_q) * (q_heads / kv_heads);
    if (attn::use_tc(rows, e4m3)) return attn::tc_workspace_bytes(rows, head_dim, num_sms);
    const int mt = rows <= 16 ? 1 : 2;
    return attn::parts_bytes(attn::ctas_per_sm(head_dim, e4m3, mt) * num_sms, 16 * mt, head_dim);
}

cudaError_t launch_attention(const AttentionArgs& a, const CacheView& cache, const BatchView& batch, int num_sms,
                             cudaStream_t stream) {
    attn::Params p{};
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.q_stride = a.q_stride;
    p.tree_mask = a.tree_mask;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.ws = a.workspace;
    p.status = a.status;
    p.q_heads = a.q_heads;
    p.cut.group = a.q_heads / cache.kv_heads;
    p.cut.by_group = attn::divisor(p.cut.group);
    p.cut.kv_heads = cache.kv_heads;
    p.cut.window = a.window;
    p.cut.tree = a.tree_mask != nullptr;
    p.cut.placed = a.positions && a.window;
    p.positions = p.cut.placed ? a.positions : nullptr;
    p.cut.min_share = 1;
    p.cache = cache;
    p.batch = batch;
    const int64_t rows = static_cast<int64_t>(a.max_q) * p.cut.group;
    if (attn::use_tc(rows, a.e4m3)) {
        p.negate = a.scale < 0.f;
        // Masked scores are -inf and are multiplied by `mul`: it may not be 0.
        p.map = attn::score_map(fmaxf(fabsf(a.scale), 1e-36f), a.softcap);
        return attn::launch_tc(p, a.e4m3, rows, a.max_seq, num_sms, stream);
    }
    p.map = attn::score_map(a.scale, a.softcap);
    const int mt = rows <= 16 ? 1 : 2;
    p.cut.row_shift = mt == 1 ? 4 : 5;
    p.cut.key_shift = attn::kKeyShift;
    const int ctas = attn::ctas_for(p, rows, a.max_seq, attn::ctas_per_sm(cache.head_dim, a.e4m3, mt) * num_sms);
    if (p.cut.placed)
        return cache.head_dim == 64 ? attn::launch_d<64, true>(p, a.e4m3, mt, ctas, stream)
                                    : attn::launch_d<128, true>(p, a.e4m3, mt, ctas, stream);
    return cache.head_dim == 64 ? attn::launch_d<64, false>(p, a.e4m3, mt, ctas, stream)
                                : attn::launch_d<128, false>(p, a.e4m3, mt, ctas, stream);
}

}  // namespace mxfp4
