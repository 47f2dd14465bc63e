// Host interface of the kernels of a prompt chunk's way through MXFP4 weights
// (mx_quantize.cu, mx_product.cu; the norm is in norm.cu). Arguments are
// checked by mx_capi.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mxfp4.h"

namespace mxfp4 {

struct MxQuantizeArgs {
    const void* x;     // bf16 rows, x_stride elements apart
    int64_t x_stride;
    int64_t t, k;      // k values a row (of 2 k in memory where swiglu)
    void* xq;
    uint8_t* xs;
    bool swiglu, e2m1;
};
cudaError_t launch_mx_quantize(const MxQuantizeArgs& a, int num_sms, cudaStream_t stream);

struct MxProductArgs {
    const void* xq;
    const uint8_t* xs;
    const uint8_t* wq;
    const uint8_t* ws;
    int64_t t, k;
    int64_t n;         // outputs: rows of the weights, or half of them where swiglu
    void* y;           // bf16 [t, n], or where swiglu codes
    uint8_t* ys;       // scales (swiglu)
    bool e2m1;         // activations
    bool swiglu, out_e2m1;
    unsigned* status;
};
cudaError_t launch_mx_product(const MxProductArgs& a, int num_sms, int max_smem, cudaStream_t stream);

// How the launch would cut a product, without a device: clusters[c] (1 to 8) of c CTAs, one to an SM, are resident at once.
bool plan_mx_product(int64_t t, int64_t k, int64_t n, bool e2m1, bool swiglu, bool aligned, int max_smem,
                     const int32_t* clusters, mxfp4_mx_plan_t* out);

// Tensor maps (capi.cu). Codes as bytes [rows, row_bytes] in boxes of 128 bytes x box_rows, 128-byte swizzle.
cudaError_t encode_code_map(CUtensorMap* map, const void* codes, int64_t rows, int64_t row_bytes, int box_rows);
// E2M1 codes [rows, k / 2] spread out to a byte each: boxes of 128 values x box_rows.
cudaError_t encode_spread_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t k, int box_rows);

}  // namespace mxfp4
