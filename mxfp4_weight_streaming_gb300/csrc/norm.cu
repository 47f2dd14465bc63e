// Norms between two blocks, fused with the block's gate and the residual
// sum: per token
//   u = x, or N(x) * post_weight (+ post_bias);  u *= gate
//   r = residual + scale * u
//   y = N(r) * weight (+ bias)
// with N(z) = z / sqrt(mean(z^2) + eps), or the same of z - mean(z).
//
// A block takes rows blockIdx.x, + gridDim.x, ...; a row stays in registers
// between the two norms, so x, residual (and a gate per token) are read once
// and r and y written once, and the next row's loads are in flight meanwhile.
// Everything is fp32 until the one rounding of each output; y is the norm of
// the unrounded r.
//
// y may leave as microscaled codes (mx_common.cuh) instead: 4,096 tokens of 7,168
// with post norm and a gate per token, 265 MB, take 50 us, 77 % of the copy rate.
//
// Bound by HBM: 4,096 tokens of 7,168 with a gate per token, 294 MB, take 51
// us, 84 % of the copy rate (82 us with a block per row and no loads ahead);
// 4 tokens take 3.1 us, a launch.
#include "step_launch.h"

#include "mx_common.cuh"
#include "step_common.cuh"

namespace mxfp4 {
namespace {

struct NormParams {
    const __nv_bfloat16 *x, *residual, *post_weight, *post_bias, *gate, *weight, *bias;
    __nv_bfloat16 *y, *r_out;
    uint8_t *yq, *ys;     // y as codes and scales in its place
    int64_t gate_stride;  // elements between tokens; 0: one gate row for all
    int n, tokens;
    float scale, eps, weight_offset;
};

// Sum over the block, the same order on every call. `slot` alternates
// between calls of one kernel so that one barrier each is enough.
template <int WARPS>
__device__ __forceinline__ float block_sum(float v, float (*part)[32], int slot) {
    v = warp_sum(v);
    if constexpr (WARPS == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) part[slot][warp] = v;
    __syncthreads();
    v = lane < WARPS ? part[slot][lane] : 0.f;
    return warp_sum(v);
}

// CH chunks of 8 values per thread, as they come from memory. VEC: 16-byte
// accesses (n % 8 == 0 and 16-byte rows); otherwise one value at a time.
template <int THREADS, int CH, bool VEC>
struct Row {
    Bf16x8 v[CH];
    __device__ static int at(int c, int j) {
        return VEC ? (c * THREADS + static_cast<int>(threadIdx.x)) * 8 + j
                   : (c * 8 + j) * THREADS + static_cast<int>(threadIdx.x);
    }
    __device__ static Bf16x8 load_chunk(const __nv_bfloat16* p, int n, int c) {
        Bf16x8 w;
        if constexpr (VEC) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            const uint4 u = at(c, 0) < n ? *reinterpret_cast<const uint4*>(p + at(c, 0)) : z;
            w = *reinterpret_cast<const Bf16x8*>(&u);
        } else {
            __nv_bfloat16* e = reinterpret_cast<__nv_bfloat16*>(&w);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = at(c, j) < n ? p[at(c, j)] : __float2bfloat16_rn(0.f);
        }
        return w;
    }
    __device__ void load(const __nv_bfloat16* p, int n) {
#pragma unroll
        for (int c = 0; c < CH; ++c) v[c] = load_chunk(p, n, c);
    }
    __device__ static void store_chunk(__nv_bfloat16* p, int n, int c, const float (&f)[8]) {
        if constexpr (VEC) {
            if (at(c, 0) < n) *reinterpret_cast<Bf16x8*>(p + at(c, 0)) = pack8(f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at(c, j) < n) p[at(c, j)] = __float2bfloat16_rn(f[j]);
        }
    }
};

// How y leaves: bf16, or microscaled codes (VEC only).
enum { kBf16, kE4M3, kE2M1 };

// 8 values of y, at `at` of row t, as codes. Four neighbouring threads hold a
// block of 32 (n % 32 == 0, so none straddles the row's end).
template <bool E2M1>
__device__ __forceinline__ void store_codes(const NormParams& p, int64_t row, int at, const float (&v)[8]) {
    uint32_t top = mx::largest<8>(v);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t s = mx::scale_byte<E2M1>(top);
    uint32_t w[E2M1 ? 1 : 2];
    mx::encode<E2M1, 8>(v, s, w);
    if (at >= p.n) return;
    const int64_t e = row + at;
    if constexpr (E2M1)
        *reinterpret_cast<uint32_t*>(p.yq + e / 2) = w[0];
    else
        *reinterpret_cast<uint2*>(p.yq + e) = make_uint2(w[0], w[1]);
    if ((threadIdx.x & 3) == 0) p.ys[e / 32] = static_cast<uint8_t>(s);
}

template <int THREADS, int CH, bool VEC, bool LAYER, int OUT>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) residual_norm_kernel(NormParams p) {
    using R = Row<THREADS, CH, VEC>;
    constexpr int WARPS = THREADS / 32;
    __shared__ float part[4][32];
    const int n = p.n;
    const float inv_n = 1.f / n;

    // Factor of the norm of z; LAYER: z becomes z - mean first (padding stays 0).
    auto centre_and_factor = [&](float (&z)[CH][8], int slot) {
        if constexpr (LAYER) {
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) s += z[c][j];
            const float mean = block_sum<WARPS>(s, part, slot) * inv_n;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) z[c][j] = R::at(c, j) < n ? z[c][j] - mean : 0.f;
        }
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += z[c][j] * z[c][j];
        return rsqrtf(block_sum<WARPS>(s, part, slot + 1) * inv_n + p.eps);
    };

    pdl_wait_previous();
    pdl_launch_dependents();
    R x, res, gate;
    auto load_row = [&](int t) {
        const int64_t row = static_cast<int64_t>(t) * n;
        x.load(p.x + row, n);
        res.load(p.residual + row, n);
        if (p.gate_stride) gate.load(p.gate + t * p.gate_stride, n);
    };
    int t = blockIdx.x;
    load_row(t);
    while (true) {
        float u[CH][8], r[CH][8];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            unpack8(x.v[c], u[c]);
            unpack8(res.v[c], r[c]);
        }
        if (p.post_weight) {
            const float f = centre_and_factor(u, 0);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float w[8];
                unpack8(R::load_chunk(p.post_weight, n, c), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[c][j] = u[c][j] * f * (w[j] + p.weight_offset);
                if (p.post_bias) {
                    unpack8(R::load_chunk(p.post_bias, n, c), w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[c][j] += w[j];
                }
            }
        }
        const int64_t row = static_cast<int64_t>(t) * n;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (p.gate) {
                float w[8];
                unpack8(p.gate_stride ? gate.v[c] : R::load_chunk(p.gate, n, c), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[c][j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[c][j] = fmaf(p.scale, u[c][j], r[c][j]);
        }
        // Compared as a distance: t + gridDim.x may pass 2^31.
        const bool more = static_cast<int>(gridDim.x) < p.tokens - t;
        const int next = more ? t + static_cast<int>(gridDim.x) : t;
        if (more) load_row(next);
#pragma unroll
        for (int c = 0; c < CH; ++c) R::store_chunk(p.r_out + row, n, c, r[c]);
        const float f = centre_and_factor(r, 2);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float w[8];
            unpack8(R::load_chunk(p.weight, n, c), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[c][j] = r[c][j] * f * (w[j] + p.weight_offset);
            if (p.bias) {
                unpack8(R::load_chunk(p.bias, n, c), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[c][j] += w[j];
            }
            if constexpr (OUT == kBf16)
                R::store_chunk(p.y + row, n, c, r[c]);
            else
                store_codes<OUT == kE2M1>(p, row, R::at(c, 0), r[c]);
        }
        if (!more) break;
        t = next;
        __syncthreads();  // the sums' slots are free again
    }
}

// Blocks for `per_sm` of them on each SM, or a row each if there are fewer.
template <int THREADS, int CH>
cudaError_t launch(const NormParams& p, int per_sm, int num_sms, bool vec, bool layer, int out, cudaStream_t stream) {
    const int blocks = p.tokens < per_sm * num_sms ? p.tokens : per_sm * num_sms;
    PdlLaunch l(dim3(blocks), dim3(THREADS), 0, stream);
    auto go = [&](auto kernel) { return cudaLaunchKernelEx(&l.cfg, kernel, p); };
    if (p.yq && out == kE2M1)
        return layer ? go(residual_norm_kernel<THREADS, CH, true, true, kE2M1>)
                     : go(residual_norm_kernel<THREADS, CH, true, false, kE2M1>);
    if (p.yq)
        return layer ? go(residual_norm_kernel<THREADS, CH, true, true, kE4M3>)
                     : go(residual_norm_kernel<THREADS, CH, true, false, kE4M3>);
    if (vec)
        return layer ? go(residual_norm_kernel<THREADS, CH, true, true, kBf16>)
                     : go(residual_norm_kernel<THREADS, CH, true, false, kBf16>);
    return layer ? go(residual_norm_kernel<THREADS, CH, false, true, kBf16>)
                 : go(residual_norm_kernel<THREADS, CH, false, false, kBf16>);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs& a, int num_sms, cudaStream_t stream) {
    NormParams p{};
    p.x = static_cast<const __nv_bfloat16*>(a.x);
    p.residual = static_cast<const __nv_bfloat16*>(a.residual);
    p.post_weight = static_cast<const __nv_bfloat16*>(a.post_weight);
    p.post_bias = static_cast<const __nv_bfloat16*>(a.post_bias);
    p.gate = static_cast<const __nv_bfloat16*>(a.gate);
    p.weight = static_cast<const __nv_bfloat16*>(a.weight);
    p.bias = static_cast<const __nv_bfloat16*>(a.bias);
    const int out = !a.ys ? kBf16 : a.e2m1 ? kE2M1 : kE4M3;
    p.y = a.ys ? nullptr : static_cast<__nv_bfloat16*>(a.y);
    p.yq = a.ys ? static_cast<uint8_t*>(a.y) : nullptr;
    p.ys = a.ys;
    p.r_out = static_cast<__nv_bfloat16*>(a.r_out);
    p.gate_stride = a.gate_stride;
    p.n = static_cast<int>(a.n);
    p.scale = a.scale;
    p.eps = a.eps;
    p.weight_offset = a.weight_offset;
    const void* ptrs[] = {a.x, a.residual, a.post_weight, a.post_bias, a.gate, a.weight, a.bias, a.y, a.r_out};
    bool vec = a.n % 8 == 0 && a.gate_stride % 8 == 0;
    for (const void* q : ptrs) vec = vec && reinterpret_cast<uintptr_t>(q) % 16 == 0;
    p.tokens = static_cast<int>(a.tokens);
    const int chunks = static_cast<int>((a.n + 7) / 8);  // 8-value chunks of a row
    // Blocks per SM: as many as the registers of 1,024 threads allow at once, so
    // that every block has rows to the end (us; rms, post weight, no gate):
    // 32,768 rows of 1,024: 8 blocks 49.5, 4 68, 12 57; 16,384 of 2,048: 4 52, 6
    // 60; 8,192 of 4,096: 4 46, 2 56, 3 57; 4,096 of 7,168: 2 46, 1 57. Beyond
    // 16,384 columns a row's values spill: 2,048 rows of 18,432 take 193 us, 23 %
    // of the copy rate.
    if (chunks <= 128) return launch<128, 1>(p, 8, num_sms, vec, a.layer, out, stream);
    if (chunks <= 256) return launch<256, 1>(p, 4, num_sms, vec, a.layer, out, stream);
    if (chunks <= 512) return launch<256, 2>(p, 4, num_sms, vec, a.layer, out, stream);
    if (chunks <= 1024) return launch<512, 2>(p, 2, num_sms, vec, a.layer, out, stream);
    if (chunks <= 2048) return launch<1024, 2>(p, 1, num_sms, vec, a.layer, out, stream);
    return launch<1024, 4>(p, 1, num_sms, vec, a.layer, out, stream);
}

}  // namespace mxfp4
