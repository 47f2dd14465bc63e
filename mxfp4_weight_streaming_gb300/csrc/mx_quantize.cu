// Activations as microscaled codes: z = x, or SiLU(gate) * up of rows
// [gate | up], in fp32, then blocks of 32 (mx_common.cuh).
//
// A thread takes 16 values, half a block, at one place of the row and walks
// down the rows; the block's maximum is one shuffle between neighbours. Loads of
// one thread wait while it computes, so an SM holds as many threads as it can
// (32 registers each; with four rows' loads ahead in a thread and half as many
// threads, 2,048 gated rows of 18,432 took 47 us). Bound by HBM: 16,384 rows of
// 7,168 take 55 us, 95 % of the copy rate; gated ones by waiting for their loads:
// 2,048 of 18,432 35 us, 79 % (34 without the way for gates below -87, which
// costs registers), 33 as E2M1.
//
// The next kernel of the stream is not let in early: it may take these codes
// as weights, and mxfp4_linear and others read weights before they wait for the
// kernels ahead of them.
#include <type_traits>

#include "mx_common.cuh"
#include "mx_launch.h"
#include "step_common.cuh"

namespace mxfp4 {
namespace {

struct QuantizeParams {
    const __nv_bfloat16* x;
    int64_t x_stride, t;
    uint8_t *xq, *xs;
    int halves;  // of a row: k / 16
    int rows;    // that a block takes side by side (short ones)
};

struct alignas(16) Half {  // 16 bf16 values
    Bf16x8 v[2];
};

// In one load where rows begin at multiples of 32 bytes: two of 16 bytes each
// take twice the cycles of the load unit, 81 % of which a gated call then used.
template <bool WIDE>
__device__ __forceinline__ Half load_half(const __nv_bfloat16* p) {
    Half h;
    if constexpr (WIDE) {
        uint32_t(&w)[8] = *reinterpret_cast<uint32_t(*)[8]>(&h);
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        h.v[0] = *reinterpret_cast<const Bf16x8*>(p);
        h.v[1] = *reinterpret_cast<const Bf16x8*>(p + 8);
    }
    return h;
}

// Whether one of 16 gates is below kFarGate (or a NaN with its sign set). As unsigned
// halfwords negative numbers are above the others, and the larger the lower.
__device__ __forceinline__ bool far_gates(const Half& h) {
    constexpr uint32_t kFar = 0xc2ae;  // bf16 of -87
    static_assert(mx::kFarGate == -87.f, "its bits");
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&h);
    uint32_t m = __vimax3_u16x2(w[0], w[1], w[2]);
    m = __vimax3_u16x2(m, w[3], w[4]);
    m = __vimax3_u16x2(m, w[5], w[6]);
    m = __vmaxu2(m, w[7]);
    return (m >> 16) > kFar || (m & 0xffffu) > kFar;
}

__device__ __forceinline__ float load_one(const __nv_bfloat16* p) {
    uint16_t h;
    asm volatile("ld.global.b16 %0, [%1];" : "=h"(h) : "l"(p));
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
}

// SHORT: rows of at most 2,048 values, several side by side in a block (1,000,000
// rows of 32 take 16 us, with a block a row 497). Longer ones do without the
// division: 2,048 gated rows of 18,432 34 us against 39 (both without the way for
// gates below -87).
template <bool SWIGLU, bool E2M1, bool WIDE, bool SHORT>
__global__ void __launch_bounds__(256, 8) mx_quantize_kernel(QuantizeParams p) {
    // This thread's place in a row, and its row among those side by side. Halves are even, so that a block's two threads are
    // neighbours of one warp and have both work or none; whole warps take part in the shuffles.
    const int tid = static_cast<int>(threadIdx.x), rows = SHORT ? p.rows : 1;
    const int beside = SHORT ? tid / p.halves : 0;
    const int i = SHORT ? tid - beside * p.halves : static_cast<int>(blockIdx.x * blockDim.x) + tid;
    const bool mine = i < p.halves && beside < rows;
    const int64_t k = static_cast<int64_t>(p.halves) * 16, begin = mine ? static_cast<int64_t>(i) * 16 : 0;
    pdl_wait_previous();
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * rows; row0 < p.t; row0 += static_cast<int64_t>(gridDim.y) * rows) {
        const bool live = mine && (!SHORT || row0 + beside < p.t);
        const int64_t row = SHORT && live ? row0 + beside : row0, at = begin;
        const __nv_bfloat16* src = p.x + row * p.x_stride + at;
        const Half a = load_half<WIDE>(src);
        float z[16];
        unpack8(a.v[0], *reinterpret_cast<float(*)[8]>(z));
        unpack8(a.v[1], *reinterpret_cast<float(*)[8]>(z + 8));
        if constexpr (SWIGLU) {
            const Half b = load_half<WIDE>(src + k);
            float up[16];
            unpack8(b.v[0], *reinterpret_cast<float(*)[8]>(up));
            unpack8(b.v[1], *reinterpret_cast<float(*)[8]>(up + 8));
            mx::swiglu_near<16>(z, up);
            // All over again, from memory: kept, the gates and up values would not fit the 32 registers.
            if (far_gates(a)) {
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = mx::gated_any(load_one(src + j), load_one(src + k + j));
            }
        }
        uint32_t top = mx::largest<16>(z);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const uint32_t s = mx::scale_byte<E2M1>(top);
        uint32_t w[E2M1 ? 2 : 4];
        mx::encode<E2M1, 16>(z, s, w);
        if (!live) continue;
        const int64_t e = row * k + at;
        if constexpr (E2M1)
            *reinterpret_cast<uint2*>(p.xq + e / 2) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4*>(p.xq + e) = make_uint4(w[0], w[1], w[2], w[3]);
        if ((i & 1) == 0) p.xs[e / 32] = static_cast<uint8_t>(s);
    }
    __threadfence();  // what a next kernel that begins when the last block ends may read at once
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantizeArgs& a, int num_sms, cudaStream_t stream) {
    QuantizeParams p{};
    p.x = static_cast<const __nv_bfloat16*>(a.x);
    p.x_stride = a.x_stride;
    p.t = a.t;
    p.xq = static_cast<uint8_t*>(a.xq);
    p.xs = a.xs;
    p.halves = static_cast<int>(a.k / 16);
    // Blocks of at most 256 threads that cover the row evenly, in whole warps.
    const int across = (p.halves + 255) / 256;
    p.rows = p.halves <= 128 ? 256 / p.halves : 1;  // rows of up to 2,048 values side by side
    const int threads = ((p.halves * p.rows + across - 1) / across + 31) / 32 * 32;
    int64_t down = (static_cast<int64_t>(num_sms) * 8 + across - 1) / across;
    if (down > (a.t + p.rows - 1) / p.rows) down = (a.t + p.rows - 1) / p.rows;
    if (down > 65535) down = 65535;
    PdlLaunch l(dim3(across, static_cast<unsigned>(down)), dim3(threads), 0, stream);
    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 32 == 0 && a.x_stride % 16 == 0;  // k is a multiple of 32
    auto go = [&](auto kernel) { return cudaLaunchKernelEx(&l.cfg, kernel, p); };
    auto pick = [&](auto swiglu, auto e2m1) {
        constexpr bool S = decltype(swiglu)::value, E = decltype(e2m1)::value;
        if (p.rows > 1) return wide ? go(mx_quantize_kernel<S, E, true, true>) : go(mx_quantize_kernel<S, E, false, true>);
        return wide ? go(mx_quantize_kernel<S, E, true, false>) : go(mx_quantize_kernel<S, E, false, false>);
    };
    if (a.swiglu) return a.e2m1 ? pick(std::true_type{}, std::true_type{}) : pick(std::true_type{}, std::false_type{});
    return a.e2m1 ? pick(std::false_type{}, std::true_type{}) : pick(std::false_type{}, std::false_type{});
}

}  // namespace mxfp4
