// C ABI of a prompt chunk's way through MXFP4 weights: argument checks, then
// the launches of mx_quantize.cu, mx_product.cu and norm.cu.
#include <initializer_list>

#include "mx_launch.h"
#include "step_common.cuh"
#include "step_launch.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launched(cudaError_t e) { return e == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA; }

bool known(int format) { return format == MXFP4_MX_E4M3 || format == MXFP4_MX_E2M1; }

constexpr int64_t kMost = int64_t(1) << 31;  // coordinates of a copy are ints
constexpr int64_t kMostK = int64_t(1) << 24; // a tile's sums over k stay far below the limit of a wait
constexpr int64_t kMostStride = int64_t(1) << 31;

// Memory of an operand. Outputs may not lie in the inputs: rows are read and
// written by different blocks in any order.
struct Range {
    const void* at;
    int64_t bytes;
    bool meets(const Range& o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(at), b = reinterpret_cast<uintptr_t>(o.at);
        return at && o.at && a < b + o.bytes && b < a + bytes;
    }
};

bool any_meet(std::initializer_list<Range> outputs, std::initializer_list<Range> inputs) {
    for (const Range& o : outputs) {
        for (const Range& i : inputs)
            if (o.meets(i)) return true;
        for (const Range& p : outputs)
            if (&p != &o && o.meets(p)) return true;
    }
    return false;
}

int64_t code_bytes(int64_t values, int format) { return format == MXFP4_MX_E2M1 ? values / 2 : values; }

// Of the sizes of a product.
int product_shape(int64_t t, int64_t k, int64_t n, bool swiglu) {
    if (k % 128 || k > kMostK || t >= kMost - 256 || n >= (swiglu ? kMost / 2 : kMost) - 256 || (swiglu && n % 32))
        return MXFP4_ERR_SHAPE;
    return MXFP4_OK;
}

int product(const void* xq, const uint8_t* xs, int format, int64_t t, int64_t k, const uint8_t* wq, const uint8_t* ws,
            int64_t n, bool swiglu, int out_format, void* y, uint8_t* ys, void* stream) {
    if (!xq || !xs || !wq || !ws || !y || (swiglu && !ys) || t <= 0 || k <= 0 || n <= 0 || !known(format) ||
        !known(out_format))
        return MXFP4_ERR_INVALID_ARG;
    if (int rc = product_shape(t, k, n, swiglu)) return rc;
    if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(ws, 4) || !aligned(wq, format == MXFP4_MX_E4M3 ? 32 : 16) ||
        !aligned(y, swiglu ? 16 : 2))
        return MXFP4_ERR_ALIGN;
    const int64_t rows = swiglu ? 2 * n : n;
    const Range in[] = {{xq, code_bytes(t * k, format)}, {xs, t * k / 32}, {wq, rows * k / 2}, {ws, rows * k / 32}};
    if (any_meet({{y, swiglu ? code_bytes(t * n, out_format) : 2 * t * n}, {ys, t * n / 32}}, {in[0], in[1], in[2], in[3]}))
        return MXFP4_ERR_INVALID_ARG;
    mxfp4::DeviceCaps caps;
    if (int rc = mxfp4::device_caps(&caps)) return rc;
    mxfp4::MxProductArgs a{};
    a.xq = xq;
    a.xs = xs;
    a.wq = wq;
    a.ws = ws;
    a.t = t;
    a.k = k;
    a.n = n;
    a.y = y;
    a.ys = ys;
    a.e2m1 = format == MXFP4_MX_E2M1;
    a.swiglu = swiglu;
    a.out_e2m1 = out_format == MXFP4_MX_E2M1;
    a.status = caps.status;
    return launched(mxfp4::launch_mx_product(a, caps.num_sms, caps.max_smem, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int mxfp4_quantize_mx(const void* x, int64_t x_stride, int64_t t, int64_t k, int swiglu, int format, void* xq,
                      uint8_t* xs, void* stream) {
    if (!x || !xq || !xs || t <= 0 || k <= 0 || !known(format) || (x_stride && x_stride < (swiglu ? 2 : 1) * k))
        return MXFP4_ERR_INVALID_ARG;
    if (k % 32 || k >= kMost || t >= kMost || x_stride >= kMostStride) return MXFP4_ERR_SHAPE;
    if (!aligned(x, 16) || x_stride % 8 || !aligned(xq, 16)) return MXFP4_ERR_ALIGN;
    const int64_t width = (swiglu ? 2 : 1) * k, stride = x_stride ? x_stride : width;
    if (any_meet({{xq, code_bytes(t * k, format)}, {xs, t * k / 32}}, {{x, 2 * ((t - 1) * stride + width)}}))
        return MXFP4_ERR_INVALID_ARG;
    mxfp4::DeviceCaps caps;
    if (int rc = mxfp4::device_caps(&caps)) return rc;
    mxfp4::MxQuantizeArgs a{};
    a.x = x;
    a.x_stride = stride;
    a.t = t;
    a.k = k;
    a.xq = xq;
    a.xs = xs;
    a.swiglu = swiglu != 0;
    a.e2m1 = format == MXFP4_MX_E2M1;
    return launched(mxfp4::launch_mx_quantize(a, caps.num_sms, static_cast<cudaStream_t>(stream)));
}

int mxfp4_residual_norm_mx(const void* x, const void* residual, int64_t tokens, int64_t n, const void* post_weight,
                           const void* post_bias, const void* gate, int64_t gate_stride, float scale,
                           const void* weight, const void* bias, float weight_offset, float eps, int layer, int format,
                           void* yq, uint8_t* ys, void* r_out, void* stream) {
    if (!x || !residual || !weight || !yq || !ys || !r_out || tokens <= 0 || n <= 0 || (post_bias && !post_weight) ||
        gate_stride < 0 || (gate_stride && gate_stride < n) || !(eps >= 0.f) || !known(format))
        return MXFP4_ERR_INVALID_ARG;
    if (n > 32768 || n % 32 || tokens >= kMost || gate_stride >= kMostStride) return MXFP4_ERR_SHAPE;
    for (const void* p : {x, residual, post_weight, post_bias, gate, weight, bias, static_cast<const void*>(yq),
                          static_cast<const void*>(r_out)})
        if (!aligned(p, 16)) return MXFP4_ERR_ALIGN;
    if (gate_stride % 8) return MXFP4_ERR_ALIGN;
    const Range r{r_out, 2 * tokens * n}, codes{yq, code_bytes(tokens * n, format)}, scales{ys, tokens * n / 32};
    const int64_t gate_bytes = gate ? 2 * ((tokens - 1) * gate_stride + n) : 0;
    if (any_meet({codes, scales}, {r, {x, 2 * tokens * n}, {residual, 2 * tokens * n}, {gate, gate_bytes}, {weight, 2 * n},
                                   {bias, 2 * n}, {post_weight, 2 * n}, {post_bias, 2 * n}}) ||
        any_meet({r}, {{gate, gate_bytes}, {weight, 2 * n}, {bias, 2 * n}, {post_weight, 2 * n}, {post_bias, 2 * n}}))
        return MXFP4_ERR_INVALID_ARG;
    // r may be x or the residual as they lie: a row is read before it is written. Shifted, it would be another's row.
    for (const void* p : {x, residual})
        if (p != r_out && r.meets({p, 2 * tokens * n})) return MXFP4_ERR_INVALID_ARG;
    mxfp4::DeviceCaps caps;
    if (int rc = mxfp4::device_caps(&caps)) return rc;
    mxfp4::ResidualNormArgs a{};
    a.x = x;
    a.residual = residual;
    a.post_weight = post_weight;
    a.post_bias = post_bias;
    a.gate = gate;
    a.weight = weight;
    a.bias = bias;
    a.y = yq;
    a.ys = ys;
    a.r_out = r_out;
    a.tokens = tokens;
    a.n = n;
    a.gate_stride = gate_stride;
    a.scale = scale;
    a.eps = eps;
    a.weight_offset = weight_offset;
    a.layer = layer != 0;
    a.e2m1 = format == MXFP4_MX_E2M1;
    return launched(mxfp4::launch_residual_norm(a, caps.num_sms, static_cast<cudaStream_t>(stream)));
}

int mxfp4_linear_mx(const void* xq, const uint8_t* xs, int format, int64_t t, int64_t k, const uint8_t* wq,
                    const uint8_t* ws, int64_t n, void* y, void* stream) {
    return product(xq, xs, format, t, k, wq, ws, n, false, MXFP4_MX_E4M3, y, nullptr, stream);
}

int mxfp4_linear_mx_plan(int64_t t, int64_t k, int64_t n, int format, int swiglu, int aligned_rows, int max_smem,
                         const int32_t* clusters, mxfp4_mx_plan_t* out) {
    // Of 2 to 8 CTAs with most of an SM's shared memory each, as a GB300 holds them at once.
    static const int32_t kGb300[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
    if (t <= 0 || k <= 0 || n <= 0 || !known(format) || max_smem <= 0 || !out) return MXFP4_ERR_INVALID_ARG;
    if (!clusters) clusters = kGb300;
    for (int c = 1; c <= 8; ++c)
        if (clusters[c] < (c == 1 ? 1 : 0)) return MXFP4_ERR_INVALID_ARG;
    if (int rc = product_shape(t, k, n, swiglu != 0)) return rc;
    return mxfp4::plan_mx_product(t, k, n, format == MXFP4_MX_E2M1, swiglu != 0, aligned_rows != 0, max_smem, clusters, out)
               ? MXFP4_OK
               : MXFP4_ERR_SHAPE;
}

int mxfp4_swiglu_mx(const void* xq, const uint8_t* xs, int format, int64_t t, int64_t k, const uint8_t* w1q,
                    const uint8_t* w1s, int64_t inter, int out_format, void* hq, uint8_t* hs, void* stream) {
    return product(xq, xs, format, t, k, w1q, w1s, inter, true, out_format, hq, hs, stream);
}

}  // extern "C"
