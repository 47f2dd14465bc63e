// Microscaled (MX) activations: blocks of 32 values along a row share one E8M0
// scale 2^(s-127); elements are E4M3 or E2M1 (two codes a byte, the even index
// in the low nibble). What the kernels that make such blocks share.
//
// A block's scale is the smallest power of two that keeps every element within
// its type: with m = max|z|, the least e >= -127 with m <= 448 * 2^e (6 * 2^e).
// (The weights' packer takes floor(log2 m) - 2 and lets values saturate, up to
// 25 % off; an activation's largest values carry most of a product.) Element =
// nearest (ties to even) of z / 2^e. A block with a NaN or an infinity has scale
// NaN (255), which makes every product that it takes part in NaN.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"

namespace mxfp4 {
namespace mx {

constexpr uint32_t kNanScale = 255;

// Scale byte of a block by the bits of its largest magnitude. 448 = 1.75 * 2^8
// and 6 = 1.5 * 2^2, so the fraction decides between two exponents.
template <bool E2M1>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return kNanScale;
    const int e = static_cast<int>(amax_bits >> 23) - (E2M1 ? 2 : 8) +
                  ((amax_bits & 0x7fffffu) > (E2M1 ? 0x400000u : 0x600000u));
    return static_cast<uint32_t>(max(e, 0));
}

// 2^(127 - s): what a block's values are multiplied with (exact).
__device__ __forceinline__ float inverse_scale(uint32_t s) { return exp2_int(127 - static_cast<int>(s)); }

// Bits of the largest magnitude of N values (an even number); of a NaN's if there
// is one. Three-way maxima: half an instruction a value.
template <int N>
__device__ __forceinline__ uint32_t largest(const float* v) {
    float m = fabsf(v[0]);
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(v[1])));
#pragma unroll
    for (int i = 2; i < N; i += 2)
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(v[i])), "f"(fabsf(v[i + 1])));
    return __float_as_uint(m);
}

// N values, already in units of their scale, as N / 4 words of E4M3 or N / 8 of E2M1.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// N values of one block (its scale byte s) as codes. Under a NaN scale E4M3
// codes are NaN too; E2M1 has none.
template <bool E2M1, int N>
__device__ __forceinline__ void encode(const float* v, uint32_t s, uint32_t (&out)[E2M1 ? N / 8 : N / 4]) {
    const float f = inverse_scale(s);
    const uint64_t f2 = f32x2_pack(f, f);
    float z[N];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 w = f32x2_unpack(f32x2_mul(f32x2_pack(v[i], v[i + 1]), f2));
        z[i] = w.x;
        z[i + 1] = w.y;
    }
    if constexpr (E2M1) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) out[i] = s == kNanScale ? 0u : e2m1x8(z + 8 * i);
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            out[i] = s == kNanScale ? 0x7f7f7f7fu : e4m3x4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
    }
}

// SiLU(z) * up = z / (1 + 2^(-z log2 e)) * up in fp32, of two values.
__device__ __forceinline__ float2 gated(float z0, float z1, float up0, float up1) {
    const uint64_t minus_log2e = f32x2_pack(-1.44269504f, -1.44269504f), one = f32x2_pack(1.f, 1.f);
    const uint64_t a = f32x2_pack(z0, z1);
    float2 e = f32x2_unpack(f32x2_mul(a, minus_log2e));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    float2 d = f32x2_unpack(f32x2_fma(f32x2_pack(e.x, e.y), one, one));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d.y));
    return f32x2_unpack(f32x2_mul(f32x2_mul(a, f32x2_pack(d.x, d.y)), f32x2_pack(up0, up1)));
}

// Below this gate the power comes near the end of fp32's range and its reciprocal is
// lost, though up may be large enough for the product to count. There the 1 beside
// the power does not, and the product is (z e^(z/2)) (up e^(z/2)), no part of which
// leaves the range before the whole does.
constexpr float kFarGate = -87.f;
__device__ __forceinline__ float far_gated(float z, float up) {
    float half;
    asm("ex2.approx.f32 %0, %1;" : "=f"(half) : "f"(z * 0.72134752f));
    return (z * half) * (up * half);
}

__device__ __forceinline__ float gated_any(float z, float up) {
    return z < kFarGate ? far_gated(z, up) : gated(z, z, up, up).x;
}

// z[i] = SiLU(z[i]) * up[i], of gates that are not below kFarGate.
template <int N>
__device__ __forceinline__ void swiglu_near(float* z, const float* up) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 h = gated(z[i], z[i + 1], up[i], up[i + 1]);
        z[i] = h.x;
        z[i + 1] = h.y;
    }
}

// The same of any gates; each value comes out the same whatever stands beside it.
template <int N>
__device__ __forceinline__ void swiglu(float* z, const float* up) {
    float low = fminf(z[0], z[1]);
#pragma unroll
    for (int i = 2; i < N; i += 2) asm("min.f32 %0, %0, %1, %2;" : "+f"(low) : "f"(z[i]), "f"(z[i + 1]));
    if (!(low < kFarGate)) return swiglu_near<N>(z, up);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 h = gated(z[i], z[i + 1], up[i], up[i + 1]);
        z[i] = z[i] < kFarGate ? far_gated(z[i], up[i]) : h.x;
        z[i + 1] = z[i + 1] < kFarGate ? far_gated(z[i + 1], up[i + 1]) : h.y;
    }
}

}  // namespace mx
}  // namespace mxfp4
