// Rotary positions of a step's new tokens, with the write of their K and V
// rows into the paged cache.
//
// The angle of pair j at position p is p * inv_freq[j]; the pair is the
// elements (2j, 2j + 1) (interleaved) or (j, j + R/2) (halves) of the first
// R of a head's D elements, and becomes
//   (a cos - b sin, a sin + b cos) * factor.
// p * inv_freq reaches 1e5 and more, where an fp32 product is off by up to
// 2^-8 of a radian: the product and its reduction to [-1/2, 1/2] turns are
// taken in fp64 (one per pair and token, shared by all heads), the sine and
// cosine in fp32.
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
    int q_heads, rotary, interleaved;
    float factor;
    CacheView cache;
    BatchView batch;
};

// The request of a token: the last b with q_start[b] <= token.
__device__ __forceinline__ int request_of(const BatchView& bt, int token) {
    int lo = 0, hi = bt.batch;  // q_start[lo] <= token < q_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(bt.q_start + mid) <= token) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One block per (token, share of its heads); a thread takes 8 consecutive
// elements of one head at a time.
template <bool E4M3>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(RopeParams p) {
    __shared__ float s_cos[kMaxRotary / 2], s_sin[kMaxRotary / 2];
    const int token = blockIdx.x;
    const CacheView& cv = p.cache;
    pdl_wait_previous();
    pdl_launch_dependents();
    const int b = request_of(p.batch, token);
    int first, n, seq;
    request_extent(p.batch, b, first, n, seq);
    const int i = token - first;
    if (i < 0 || i >= n) return;  // a row of q that belongs to no request
    const int at = seq - n + i;
    const int pos = p.positions ? p.positions[token] : at;
    const int half = p.rotary / 2;
    for (int j = threadIdx.x; j < half; j += kRopeThreads) {
        const double turns = static_cast<double>(pos) * static_cast<double>(p.inv_freq[j]) * 0.15915494309189535;
        const float frac = static_cast<float>(turns - rint(turns));
        float s, c;
        sincospif(2.f * frac, &s, &c);
        s_cos[j] = c * p.factor;
        s_sin[j] = s * p.factor;
    }
    const int page = at >= 0 ? page_of(p.batch, b, at, cv.page_shift, cv.num_pages) : -1;
    __syncthreads();

    const int D = cv.head_dim, vecs = D / 8;
    const int heads = p.q_heads + 2 * cv.kv_heads;
    const __nv_bfloat16* row = p.qkv + token * p.qkv_stride;
    const int slot = at & ((1 << cv.page_shift) - 1);
    const int total = heads * vecs;
    for (int v = blockIdx.y * kRopeThreads + threadIdx.x; v < total; v += gridDim.y * kRopeThreads) {
        const int head = v / vecs, d0 = (v % vecs) * 8;
        const __nv_bfloat16* src = row + head * D;
        float x[8], o[8];
        unpack8(*reinterpret_cast<const Bf16x8*>(src + d0), x);
        if (head >= p.q_heads + cv.kv_heads || d0 >= p.rotary) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = x[j];
        } else if (p.interleaved) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const int k = (d0 + j) / 2;
                const bool in = d0 + j < p.rotary;
                const float c = in ? s_cos[k] : 1.f, s = in ? s_sin[k] : 0.f;
                o[j] = x[j] * c - x[j + 1] * s;
                o[j + 1] = x[j] * s + x[j + 1] * c;
            }
        } else {
            float y[8];
            // The partners: 8 consecutive elements R/2 away, 16-byte aligned
            // unless R/2 is no multiple of 8.
            const bool low = d0 < half;
            if (half % 8 == 0) {
                unpack8(*reinterpret_cast<const Bf16x8*>(src + (low ? d0 + half : d0 - half)), y);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int d = d0 + j;
                    y[j] = d < p.rotary ? __bfloat162float(src[d < half ? d + half : d - half]) : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int d = d0 + j;
                const bool in = d < p.rotary, lo = d < half;
                const int k = lo ? d : d - half;
                const float c = in ? s_cos[k] : 1.f, s = in ? s_sin[k] : 0.f;
                o[j] = lo ? x[j] * c - y[j] * s : x[j] * c + y[j] * s;
            }
        }
        if (head < p.q_heads) {
            *reinterpret_cast<Bf16x8*>(p.q_out + (static_cast<int64_t>(token) * p.q_heads + head) * D + d0) = pack8(o);
            continue;
        }
        if (page < 0) continue;
        const bool is_v = head >= p.q_heads + cv.kv_heads;
        const int kh = head - p.q_heads - (is_v ? cv.kv_heads : 0);
        const int64_t to = page * cv.page_stride + ((static_cast<int64_t>(kh) << cv.page_shift) + slot) * D + d0;
        if constexpr (E4M3) {
            const float* sc = is_v ? cv.v_scale : cv.k_scale;
            const float scale = sc ? sc[kh] : 1.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = o[j] / scale;
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? cv.v : cv.k) + to) = pack8_e4m3(o);
        } else {
            *reinterpret_cast<Bf16x8*>(static_cast<__nv_bfloat16*>(is_v ? cv.v : cv.k) + to) = pack8(o);
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
    p.interleaved = a.interleaved;
    p.factor = a.factor;
    p.cache = cache;
    p.batch = batch;
    PdlLaunch l(dim3(batch.tokens, 1), dim3(kRopeThreads), 0, stream);
    return a.e4m3 ? cudaLaunchKernelEx(&l.cfg, rope_append_kernel<true>, p)
                  : cudaLaunchKernelEx(&l.cfg, rope_append_kernel<false>, p);
}

}  // namespace mxfp4
