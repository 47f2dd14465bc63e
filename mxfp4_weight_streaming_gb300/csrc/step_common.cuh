// What the kernels of the step's attention side (norms, rotary positions,
// attention, cache pages) share: views of the paged cache and of the step's
// batch, 16-byte vectors of bf16, and block-wide sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"
#include "mxfp4.h"

namespace mxfp4 {

// Device facts that the host side of a launch needs (see capi.cu).
struct DeviceCaps {
    int num_sms;
    int max_smem;
    unsigned* status;
};
int device_caps(DeviceCaps* out);

// The cache of one layer, as kernels take it. Offsets are 64-bit: a pool may
// hold far more than 2^31 elements.
struct CacheView {
    void* k;
    void* v;
    const float* k_scale;  // null: 1
    const float* v_scale;
    int64_t page_stride;   // elements
    int num_pages;
    int kv_heads;
    int page_shift;        // page size = 1 << page_shift tokens
    int head_dim;
};

// The step's new tokens and their sequences.
struct BatchView {
    const int* q_start;      // [batch + 1]
    const int* seq_lens;     // [batch], with the new tokens
    const int* block_table;  // [batch][table_stride]
    int64_t table_stride;
    int table_width;
    int room;                // tokens that a row of the table has pages for
    int batch;
    int tokens;
};

// A word of an array that an earlier kernel of the stream may have written: a
// kernel can be resident before that one has ended (programmatic dependent
// launch), which the read-only path does not allow for. Volatile: never ahead
// of pdl_wait_previous(); without a memory clobber, so that several are under
// way at once (loads kept in order with shared stores made a call 6 us longer).
__device__ __forceinline__ int load_word(const int* p) {
    int v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// Request b's rows of q [first, first + n) and its cache length, clamped to
// what the arrays and the table can hold, so a wrong length on the device
// never leads outside a buffer.
__device__ __forceinline__ void request_extent(const BatchView& bt, int b, int& first, int& n, int& seq) {
    const int a = load_word(bt.q_start + b), z = load_word(bt.q_start + b + 1), len = load_word(bt.seq_lens + b);
    const int lo = min(max(a, 0), bt.tokens);
    const int hi = min(max(z, lo), bt.tokens);
    first = lo;
    n = hi - lo;
    seq = min(max(len, 0), bt.room);
}

// Page of cache index `at` (< table_width << page_shift), or -1 when the
// table's entry lies outside the pool.
__device__ __forceinline__ int page_of(const BatchView& bt, int b, int at, int page_shift, int num_pages) {
    const int p = load_word(bt.block_table + b * bt.table_stride + (at >> page_shift));
    return (p >= 0 && p < num_pages) ? p : -1;
}

struct alignas(16) Bf16x8 {
    __nv_bfloat162 v[4];
};

__device__ __forceinline__ void unpack8(const Bf16x8& p, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(p.v[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

__device__ __forceinline__ Bf16x8 pack8(const float (&f)[8]) {
    Bf16x8 p;
#pragma unroll
    for (int i = 0; i < 4; ++i) p.v[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return p;
}

// Eight values as E4M3 (round to nearest even, saturating at 448).
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

inline int log2_exact(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return (1 << s) == v ? s : -1;
}

// A launch that may begin while the previous kernel of the stream drains
// (the kernel calls pdl_wait_previous before it touches memory).
struct PdlLaunch {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2]{};
    PdlLaunch(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
        cfg.gridDim = grid;
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};

}  // namespace mxfp4
