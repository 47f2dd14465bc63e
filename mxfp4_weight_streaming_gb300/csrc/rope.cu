// Rotary positions of a step's new tokens, with the write of their K and V
// rows into the paged cache.
//
// The angle of pair j at position p is p * inv_freq[j]; the pair is the
// elements (2j, 2j + 1) (interleaved) or (j, j + R/2) (halves) of the first
// R of a head's D elements, and becomes
//   (a cos - b sin, a sin + b cos) * factor.
// p * inv_freq reaches 1e5 and more, where an fp32 product is off by up to
// 2^-8 of a radian: the turns p * inv_freq / 2 pi are taken as a sum of two
// fp32 numbers (products with their rounding errors, by fma) and reduced to
// [-1/2, 1/2] before the sine and cosine. One pair's angle serves all heads.
//
// 2,024 tokens of 72 heads of 128 (70 MB, E4M3 cache) take 16.4 us, 63 % of the
// copy rate: what bounds it is the chain of look-ups per token (request,
// lengths, page), four blocks per SM deep, and the divisions by the scales
// (1 us). 4 tokens take 3 us.
#include "step_launch.h"

#include "step_common.cuh"

namespace mxfp4 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxRotary = 256;

struct RopeParams {
    const __nv_bfloat16* qkv;
    int64_t qkv_stride;
    const int* positions;
    const float* inv_freq;
    __nv_bfloat16* q_out;
    int q_heads, rotary;
    float factor;
    CacheView cache;
    BatchView batch;
};

// The request of a token: the last b with q_start[b] <= token.
__device__ __forceinline__ int request_of(const BatchView& bt, int token) {
    int lo = 0, hi = bt.batch;  // q_start[lo] <= token < q_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (load_word(bt.q_start + mid) <= token) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Turns of position pos at frequency f, less whole turns: 1/(2 pi) and the
// products carry their low parts. The low parts' own fp32 rounding grows with
// the position: off by 2^-22 + |pos| f 2^-47 of a turn at most (against 64-bit
// results at most 2^-24 up to 2^17, 2^-23.3 at 2^24, 2^-17.5 at 2^31).
__device__ __forceinline__ float turns_of(int pos, float f) {
    constexpr float kInv2Pi = 0.15915494f, kInv2PiLow = 6.4206383e-9f;  // 1/(2 pi) = 0.159154943091895335...
    const float hi = f * kInv2Pi;
    const float lo = fmaf(f, kInv2Pi, -hi) + f * kInv2PiLow;
    float frac = 0.f;
    // Both parts of the position are exact in fp32.
    const float part[2] = {static_cast<float>(pos & ~0xfff), static_cast<float>(pos & 0xfff)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float prod = part[i] * hi;
        frac += (prod - rintf(prod)) + (fmaf(part[i], hi, -prod) + part[i] * lo);
    }
    return frac - rintf(frac);
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = a * c - b * s;
    b = a * s + b * c;
    a = x;
}

// One block per token. A thread takes 8 consecutive elements of one head at a
// time; all its loads are under way before the token's request, page and
// angles are looked up. The partners of 8 elements are another lane's 8 (a
// head's vectors lie in one warp), or, where R/2 is no multiple of 8, loaded.
template <bool E4M3, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_append_kernel(RopeParams p) {
    constexpr int kBatch = 5;  // vectors per thread at a time: 80 heads of 128 in one go
    __shared__ __align__(16) float s_cos[kMaxRotary / 2], s_sin[kMaxRotary / 2];
    const int token = blockIdx.x;
    const CacheView& cv = p.cache;
    const int D = cv.head_dim, vshift = D == 128 ? 4 : 3;  // vectors of a head: 1 << vshift
    const int heads = p.q_heads + 2 * cv.kv_heads, total = heads << vshift;
    const int half = p.rotary / 2, hv = half / 8;
    const bool by_lane = half % 8 == 0;
    const int lane = threadIdx.x & 31;
    pdl_wait_previous();
    pdl_launch_dependents();
    const __nv_bfloat16* row = p.qkv + token * p.qkv_stride;
    uint4 w[kBatch];
    auto load = [&](int v0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int v = v0 + k * kRopeThreads + threadIdx.x;
            w[k] = v < total ? *reinterpret_cast<const uint4*>(row + 8 * v) : make_uint4(0, 0, 0, 0);
        }
    };
    load(0);
    const int b = request_of(p.batch, token);
    int first, n, seq;
    request_extent(p.batch, b, first, n, seq);
    const int i = token - first;
    if (i < 0 || i >= n) return;  // a row of q that belongs to no request
    const int at = seq - n + i;
    const int page = at >= 0 ? page_of(p.batch, b, at, cv.page_shift, cv.num_pages) : -1;
    const int pos = p.positions ? p.positions[token] : at;
    for (int j = threadIdx.x; j < half; j += kRopeThreads) {
        float s, c;
        sincospif(2.f * turns_of(pos, p.inv_freq[j]), &s, &c);
        s_cos[j] = c * p.factor;
        s_sin[j] = s * p.factor;
    }
    __syncthreads();

    const int slot = at & ((1 << cv.page_shift) - 1);
    for (int v0 = 0; v0 < total; v0 += kBatch * kRopeThreads) {
        if (v0) load(v0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int v = v0 + k * kRopeThreads + threadIdx.x;
            const int head = v >> vshift, vec = v & ((1 << vshift) - 1), d0 = vec * 8;
            uint4 z;
            if (!INTERLEAVED && by_lane) {
                const int from = vec < hv ? lane + hv : lane - hv;
                z.x = __shfl_sync(0xffffffffu, w[k].x, from);
                z.y = __shfl_sync(0xffffffffu, w[k].y, from);
                z.z = __shfl_sync(0xffffffffu, w[k].z, from);
                z.w = __shfl_sync(0xffffffffu, w[k].w, from);
            }
            if (v >= total) continue;
            const bool is_q = head < p.q_heads, is_v = head >= p.q_heads + cv.kv_heads;
            const bool turns = !is_v && d0 < p.rotary;
            float o[8];
            if (turns || E4M3) unpack8(*reinterpret_cast<const Bf16x8*>(&w[k]), o);
            if (turns && (INTERLEAVED ? d0 + 8 <= p.rotary : by_lane)) {
                // 4 neighbouring pairs' angles, or 8 in the half's order.
                const bool low = vec < hv;
                const int t0 = INTERLEAVED ? d0 / 2 : low ? d0 : d0 - half;
                const float4 *c4 = reinterpret_cast<const float4*>(s_cos + t0),
                             *s4 = reinterpret_cast<const float4*>(s_sin + t0);
                if (INTERLEAVED) {
                    const float4 c = c4[0], s = s4[0];
                    turn(o[0], o[1], c.x, s.x);
                    turn(o[2], o[3], c.y, s.y);
                    turn(o[4], o[5], c.z, s.z);
                    turn(o[6], o[7], c.w, s.w);
                } else {
                    float y[8];
                    unpack8(*reinterpret_cast<const Bf16x8*>(&z), y);
                    const float4 ca = c4[0], cb = c4[1], sa = s4[0], sb = s4[1];
                    const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
                    const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
                    const float sign = low ? -1.f : 1.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = fmaf(o[j], c[j], sign * y[j] * s[j]);
                }
            } else if (turns) {  // a rotary dimension that ends inside 8 elements, or whose half does
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int d = d0 + j;
                    if (d >= p.rotary) continue;
                    const bool low = INTERLEAVED ? !(d & 1) : d < half;
                    const int t = INTERLEAVED ? d >> 1 : low ? d : d - half;
                    const int step = INTERLEAVED ? 1 : half;
                    const float y = __bfloat162float(row[head * D + (low ? d + step : d - step)]);
                    o[j] = o[j] * s_cos[t] + (low ? -y : y) * s_sin[t];
                }
            }
            if (is_q) {
                uint4* to = reinterpret_cast<uint4*>(p.q_out) + static_cast<int64_t>(token) * (p.q_heads << vshift) + v;
                if (turns) *reinterpret_cast<Bf16x8*>(to) = pack8(o);
                else *to = w[k];
                continue;
            }
            if (page < 0) continue;
            const int kh = head - p.q_heads - (is_v ? cv.kv_heads : 0);
            const int64_t to = page * cv.page_stride + ((kh << cv.page_shift) + slot) * D + d0;
            if constexpr (E4M3) {
                const float* sc = is_v ? cv.v_scale : cv.k_scale;
                // A division each: a product with 1 / scale lands on the other side
                // of a middle between two codes now and then, and scales of the
                // form largest / 448 put many quotients there.
                const float scale = sc ? sc[kh] : 1.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = __fdiv_rn(o[j], scale);
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? cv.v : cv.k) + to) = pack8_e4m3(o);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? cv.v : cv.k) + to);
                if (turns) *reinterpret_cast<Bf16x8*>(dst) = pack8(o);
                else *dst = w[k];
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, const CacheView& cache, const BatchView& batch,
                               cudaStream_t stream) {
    RopeParams p{};
    p.qkv = static_cast<const __nv_bfloat16*>(a.qkv);
    p.qkv_stride = a.qkv_stride;
    p.positions = a.positions;
    p.inv_freq = a.inv_freq;
    p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
    p.q_heads = a.q_heads;
    p.rotary = a.rotary_dim;
    p.factor = a.factor;
    p.cache = cache;
    p.batch = batch;
    PdlLaunch l(dim3(batch.tokens, 1), dim3(kRopeThreads), 0, stream);
    if (a.interleaved)
        return a.e4m3 ? cudaLaunchKernelEx(&l.cfg, rope_append_kernel<true, true>, p)
                      : cudaLaunchKernelEx(&l.cfg, rope_append_kernel<false, true>, p);
    return a.e4m3 ? cudaLaunchKernelEx(&l.cfg, rope_append_kernel<true, false>, p)
                  : cudaLaunchKernelEx(&l.cfg, rope_append_kernel<false, false>, p);
}

}  // namespace mxfp4
