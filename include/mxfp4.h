/*
 * mxfp4.h -- C ABI of the GB300 (sm_103a) MXFP4 weight-streaming library.
 *
 * The decode / speculative-verify step reads every weight it needs from HBM
 * once and applies it to the handful of tokens in the step ("Zyphra
 * Inference Wave 2", section "Speculative decoding"; AMD "megakernel-intro",
 * section "3. Low-Precision Data Types"). Weights are MXFP4: blocks of 32
 * E2M1 values (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign bit) that
 * share one E8M0 power-of-two scale, 4.25 bits per value ("Zyphra Inference
 * Wave 2", section "Quantization"). Activations are bf16 and outputs bf16
 * with fp32 accumulation (the a16w4 kernel of "Zyphra Inference Wave 2",
 * section "Kernel Results").
 *
 * Packed layout (shared by every entry point):
 *   wq  uint8 [rows, K/2]   byte j of a row holds the code of column 2j in
 *                           its low nibble and of column 2j+1 in its high
 *                           nibble; code bit 3 is the sign.
 *   ws  uint8 [rows, K/32]  E8M0 byte s of each 32-column block: 2^(s-127).
 *
 * Conventions for every call:
 *   - All pointers are device memory owned by the caller. The library
 *     allocates nothing; the MoE and FFN scratch comes from the caller's
 *     workspace. Exception: mxfp4_moe_noalloc keeps its scratch in one
 *     fixed array of the library (see there).
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream). Calls
 *     only enqueue work and return; results are ready when the stream is.
 *   - Argument errors are returned before anything is launched. A failed
 *     launch returns MXFP4_ERR_CUDA.
 *   - Kernels never spin unboundedly: every wait gives up after about two
 *     seconds, sets a per-device status word and lets the kernel exit.
 *     mxfp4_last_device_status() reports (and clears) that word.
 *   - Identical inputs give bit-identical outputs (no floating-point
 *     atomics); calls are stateless and thread-safe apart from the
 *     caller's own buffers. Exception: calls of mxfp4_moe_noalloc that
 *     overlap on the GPU (unordered streams, or threads) race on its
 *     shared scratch array.
 *   - mxfp4_linear, mxfp4_ffn and mxfp4_moe (and their forms) read weights and
 *     their scales before earlier kernels of the stream have ended. What
 *     mxfp4_quantize and mxfp4_quantize_mx write is complete by then: they let
 *     no other kernel begin before their stores are performed. So is what a
 *     copy brings. Weights that any other kernel writes (one of another
 *     library; mxfp4_residual_norm_mx and mxfp4_swiglu_mx, whose E2M1 codes are
 *     activations) have to be complete before such a call, however many calls
 *     lie between: by a wait on the host, by an event of another stream, or by
 *     a copy or memset in this one. mxfp4_linear_mx and mxfp4_swiglu_mx read
 *     nothing ahead and take weights from anything.
 *   - The first call on a device looks up per-device addresses (the status
 *     word, the mxfp4_moe_noalloc scratch) and keeps them for the life of
 *     the process. After cudaDeviceReset, or anything else that replaces
 *     the device's primary context, unload and reload the library.
 *   - There is no CPU path: without a GB300-class GPU every compute call
 *     returns MXFP4_ERR_CUDA.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include <stddef.h>
#include <stdint.h>

/* The library is built with hidden visibility; only these declarations are
 * exported, so two builds loaded into one process never share a symbol. */
#if defined(__GNUC__)
#pragma GCC visibility push(default)
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MXFP4_OK = 0,
    MXFP4_ERR_INVALID_ARG = 1, /* null pointer, negative or zero size     */
    MXFP4_ERR_SHAPE = 2,       /* a size the kernels do not support       */
    MXFP4_ERR_ALIGN = 3,       /* a pointer is not aligned as documented  */
    MXFP4_ERR_WORKSPACE = 4,   /* workspace missing or too small          */
    MXFP4_ERR_CUDA = 5,        /* CUDA runtime or launch failure          */
    MXFP4_ERR_TIMEOUT = 6      /* a device-side bounded wait expired      */
} mxfp4_status;

/* Human-readable name of a status code (static string, never NULL). */
const char* mxfp4_strerror(int status);

/*
 * MXFP4 packer ("Zyphra Inference Wave 2", section "Quantization"; the OCP
 * MX rule for the shared scale). For every 32-value block of a row:
 * amax = max |w|, s = clamp(floor(log2 amax) - 2 + 127, 0, 254) (0 for an
 * all-zero block), each value w * 2^(127-s) rounded to the nearest E2M1
 * point with ties to even and saturation at 6, keeping its sign bit.
 *   w   device float32 [n, k], row-major, 16-byte aligned, finite values
 *   n   rows (>= 1);  k  columns (>= 32, k % 32 == 0)
 *   wq  device uint8 [n, k/2], 16-byte aligned (output)
 *   ws  device uint8 [n, k/32] (output)
 * Bit-exact with the oracle. NaN/Inf inputs are not supported (their codes
 * are unspecified).
 */
int mxfp4_quantize(const float* w, int64_t n, int64_t k, uint8_t* wq, uint8_t* ws, void* stream);

/*
 * Weight-streaming linear layer, dense and LM-head shapes ("Zyphra
 * Inference Wave 2", section "Speculative decoding": one target token plus
 * drafts, or one token per concurrent request, per step):
 *   y[t][j] = bf16( sum_k x[t][k] * w[j][k] ),  w = dequantized (wq, ws)
 *   x   device bf16 [t, k], row-major, 16-byte aligned
 *   t   tokens, 1 <= t <= 32
 *   k   reduction length, k % 32 == 0, k >= 32
 *   wq  device uint8 [n, k/2], 16-byte aligned;  ws device uint8 [n, k/32],
 *       16-byte aligned
 *   n   output features (>= 1, < 2^31)
 *   y   device bf16 [t, n], row-major, 2-byte aligned (output)
 * Accumulation is fp32 (tensor-core fp32 accumulate); the summation order
 * is the kernel's. Three kernels serve the call (mxfp4_linear_plan says
 * which):
 *   - k % 512 == 0 and t <= 8, or 9 <= t <= 16 where each CTA's tiles of
 *     128 rows fit one accumulator batch (dense widths; not the LM head):
 *     the packed-E2M1 tensor-core kernel
 *     (tcgen05.mma kind::mxf4: the weight codes go from HBM to the tensor
 *     cores as stored, two per byte, with their E8M0 scales). Its other
 *     operand is E2M1 too, so each bf16 activation is written as eight
 *     E2M1 digit pieces: with E = floor(log2) of the largest magnitude of
 *     its (token, 32 values) block (at least -112), X = round(|x| 2^(15-E))
 *     has eight 2-bit digits D_p (most significant first) and
 *     x = sign * sum_p (D_p / 2) 2^(E - 2p). Exact for every value within
 *     2^8 of its block's largest magnitude; smaller ones keep an absolute
 *     error of at most 2^(E-16) (for blocks whose largest magnitude is
 *     below 2^-112, at most 2^-128: the lowest piece scale is 2^-127).
 *   - k % 512 != 0, or t >= 9 with wq not 32-byte aligned: the streaming
 *     engine (E2M1 -> f16 in registers, mma.sync, fp32 block scaling).
 *   - otherwise (9 <= t <= 32): the E4M3-split tensor-core kernel
 *     (tcgen05.mma kind::mxf8f6f4: the E2M1 codes and E8M0 scales go to
 *     the tensor cores as stored). Its other operand is 8-bit, so each bf16
 *     activation is split into two E4M3 pieces under one power-of-two scale
 *     per (token, 32 values) -- the pages' production format pairs MXFP4
 *     weights with MXFP8 activations ("Zyphra Inference Wave 2", section
 *     "Quantization"; AMD "megakernel-intro", section "3. Low-Precision
 *     Data Types"). The split is exact for values within 2^9 of their
 *     block's largest magnitude; smaller ones keep an absolute error below
 *     2^-17 of that maximum, far inside the tolerance's RSS term.
 * Returns MXFP4_ERR_SHAPE when no shared-memory plan fits. The binding
 * limit is k: a row group's scale bytes for all of k (k/2 bytes) stay on
 * chip next to the staging buffers. Every t <= 32 and n plans for
 * k <= 262144 on GB300.
 */
int mxfp4_linear(const void* x, int64_t t, int64_t k, const uint8_t* wq, const uint8_t* ws, int64_t n,
                 void* y, void* stream);

/*
 * How mxfp4_linear cuts the weight stream for one shape (the plan it would
 * launch). The pages have no counterpart to this entry point: it reports
 * the kernel's choices, which set its speed, and lets them be checked
 * without a GPU.
 *   t, k, n    as for mxfp4_linear (same argument checks)
 *   num_sms    streaming multiprocessors of the device
 *              (cudaDevAttrMultiProcessorCount; 152 on GB300)
 *   max_smem   opt-in shared memory per block in bytes
 *              (cudaDevAttrMaxSharedMemoryPerBlockOptin)
 *   out        host struct, written on MXFP4_OK (caller-owned)
 * Host only: no CUDA call, no device needed. Returns MXFP4_ERR_SHAPE when
 * mxfp4_linear would (no plan fits max_smem). It takes wq to be 32-byte
 * aligned (a mode-3 shape whose wq is not runs the streaming engine).
 */
typedef struct {
    int32_t mode;        /* 0: whole K per CTA; 1: K walked in parts per CTA;
                            2: K split over a thread-block cluster (modes 0-2:
                            the streaming engine); 3: the block-scaled
                            tensor-core kernel with E4M3 activation pieces;
                            4: the packed-E2M1 tensor-core kernel (modes 3-4:
                            cluster 2 = K split in halves) */
    int32_t ctas;        /* CTAs launched (mode 2: an upper bound; the number
                            of co-resident clusters decides) */
    int32_t cluster;     /* CTAs per cluster (1 unless mode 2) */
    int32_t stage_steps; /* K steps of 256 values per weight-ring stage */
    int32_t chunk_steps; /* K steps a consumer warp takes at a time (mode 3:
                            a whole stage) */
    int32_t ring_slots;  /* stages in the weight ring */
    int32_t part_steps;  /* mode 1: K steps per part; else 0 */
    int32_t batch_units; /* mode 1: row groups of 16 rows per batch; mode 3:
                            128-row tiles per CTA at most; mode 4: tiles of
                            at most 128 rows per group; else 0 */
    int32_t smem_bytes;  /* dynamic shared memory per CTA */
    int32_t group_rows;  /* mode 4: output rows per CTA (or per cluster), a
                            multiple of 8; else 0 */
} mxfp4_linear_plan_t;
int mxfp4_linear_plan(int64_t t, int64_t k, int64_t n, int num_sms, int max_smem, mxfp4_linear_plan_t* out);

/*
 * Bytes of device workspace mxfp4_moe needs for t tokens, e experts,
 * top_k experts per token, hidden size `hidden` and expert width `inter`.
 */
size_t mxfp4_moe_workspace_size(int64_t t, int64_t e, int top_k, int64_t hidden, int64_t inter);

/*
 * Grouped top-k mixture-of-experts layer with fused SwiGLU ("Zyphra
 * Inference Wave 2", sections "Kernel Results" and "Quantization": at low
 * concurrency a step reads only the routed experts' weights; each expert
 * receives a few token rows). For each token t:
 *   ids = the top_k largest router logits (descending, ties to the smaller
 *         expert index), g = softmax over those top_k logits;
 *   for each selected expert e: a = W1_e[0:inter] x_t (gate rows),
 *         b = W1_e[inter:2*inter] x_t (up rows), h = SiLU(a) * b (fp32),
 *         o = W2_e h;
 *   y[t] = bf16( sum over the selected experts in selection order of g*o ).
 * Only experts that some token selects have their weights read.
 *   x              device bf16 [t, hidden], 16-byte aligned
 *   t              tokens, 1 <= t <= 256
 *   hidden, inter  multiples of 32 (hidden >= 32, inter >= 32)
 *   router_logits  device float32 [t, e]
 *   e              experts, top_k <= e <= 1024;  1 <= top_k <= 16
 *   w1q, w1s       device uint8 [e, 2*inter, hidden/2], [e, 2*inter, hidden/32]
 *                  (rows 0..inter-1 gate, inter..2*inter-1 up), 16-byte aligned
 *   w2q, w2s       device uint8 [e, hidden, inter/2], [e, hidden, inter/32],
 *                  16-byte aligned
 *   y              device bf16 [t, hidden] (output)
 *   topk_ids       optional device int32 [t, top_k] output (NULL = skip)
 *   topk_w         optional device float32 [t, top_k] output (NULL = skip)
 *   workspace      device scratch of at least mxfp4_moe_workspace_size()
 *                  bytes, 256-byte aligned; its contents on entry do not
 *                  matter and are overwritten.
 * Routing indices are exact (bit-identical to the oracle); gate weights
 * are fp32.
 */
int mxfp4_moe(const void* x, int64_t t, int64_t hidden, const float* router_logits, int64_t e, int top_k,
              const uint8_t* w1q, const uint8_t* w1s, const uint8_t* w2q, const uint8_t* w2s, int64_t inter,
              void* y, int32_t* topk_ids, float* topk_w, void* workspace, size_t workspace_bytes,
              void* stream);

/*
 * Bytes of device workspace mxfp4_moe_shared needs (arguments as there).
 */
size_t mxfp4_moe_shared_workspace_size(int64_t t, int64_t e, int top_k, int n_shared, int64_t hidden,
                                       int64_t inter);

/*
 * mxfp4_moe with shared experts ("Zyphra Inference Wave 2", section
 * "Quantization": a decode token uses its top-k routed experts plus the
 * layer's shared experts, e.g. 8 routed and 1 shared of 257, all MXFP4).
 * The weight arrays hold e + n_shared experts: 0..e-1 routed (selected by
 * the e router logits, exactly as in mxfp4_moe), e..e+n_shared-1 shared.
 * Every token applies every shared expert, after its routed ones, with
 * weight 1:
 *   y[t] = bf16( sum_j g_j * o_{ids_j} + sum_s o_{e+s} )   (in that order).
 * The page prints no weight for a shared expert; 1 is the plain reading.
 *   n_shared       0 <= n_shared <= 16, e + n_shared <= 1024 (0 gives
 *                  mxfp4_moe's result)
 *   w1q .. w2s     as for mxfp4_moe with e + n_shared experts
 *   topk_ids, topk_w  the routed selection only, [t, top_k]
 *   workspace      at least mxfp4_moe_shared_workspace_size() bytes
 * Every other argument, limit and error is as for mxfp4_moe.
 */
int mxfp4_moe_shared(const void* x, int64_t t, int64_t hidden, const float* router_logits, int64_t e, int top_k,
                     int n_shared, const uint8_t* w1q, const uint8_t* w1s, const uint8_t* w2q, const uint8_t* w2s,
                     int64_t inter, void* y, int32_t* topk_ids, float* topk_w, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace mxfp4_ffn needs for t tokens (hidden unused).
 */
size_t mxfp4_ffn_workspace_size(int64_t t, int64_t hidden, int64_t inter);

/*
 * Dense FFN chain, up -> SwiGLU -> down (lithosai "Low-Latency Inference on
 * AMD MI355X" and AMD "megakernel-intro", section "1. Megakernels": a
 * layer's stages back to back, the next stage's weights preloaded while the
 * previous one runs). The arithmetic is one SwiGLU expert of mxfp4_moe
 * applied to every token with weight 1. For each token t:
 *   a = W1[0:inter] x_t (gate rows), b = W1[inter:2*inter] x_t (up rows),
 *   h = SiLU(a) * b (fp32), y[t] = bf16( W2 h ).
 * Two forms, chosen by shape:
 *   t <= 4 with hidden and inter multiples of 512: two launches of the
 *     packed-E2M1 tensor-core kernel on the stream. The first writes a | b
 *     in fp32 to the workspace; the second computes h = SiLU(a) * b in fp32
 *     while it converts its activations (digit pieces of h: each element
 *     within 2^(E-16) of its value, E its 32-block's largest exponent), and
 *     starts streaming W2 before the first has finished (programmatic
 *     dependent launch: it waits only where it reads a | b).
 *   otherwise: ONE persistent cooperative launch (h in the workspace),
 *     preceded by a 4-byte memset of the workspace.
 *   x              device bf16 [t, hidden], 16-byte aligned; 1 <= t <= 8
 *   hidden, inter  multiples of 32, at most 2^20 (MXFP4_ERR_SHAPE also when
 *                  the staged activations of one phase do not fit on chip)
 *   w1q, w1s       device uint8 [2*inter, hidden/2], [2*inter, hidden/32]
 *                  (gate rows first), 16-byte aligned
 *   w2q, w2s       device uint8 [hidden, inter/2], [hidden, inter/32],
 *                  16-byte aligned
 *   y              device bf16 [t, hidden] (output)
 *   workspace      device scratch of at least mxfp4_ffn_workspace_size()
 *                  bytes, 256-byte aligned; contents on entry do not matter.
 * The cooperative form's CTAs wait (bounded) for the gate/up results of all
 * the others, so the whole grid must be resident. A call that shares the
 * GPU with other work that holds SMs may therefore end in MXFP4_ERR_TIMEOUT
 * (reported as for every call) instead of a result.
 */
int mxfp4_ffn(const void* x, int64_t t, int64_t hidden, const uint8_t* w1q, const uint8_t* w1s, const uint8_t* w2q,
              const uint8_t* w2s, int64_t inter, void* y, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Capacity in bytes of the scratch array built into the library for
 * mxfp4_moe_noalloc (held on every GPU that loads the library).
 */
#define MXFP4_MOE_NOALLOC_SCRATCH_BYTES ((size_t)12 << 20)

/*
 * mxfp4_moe without a workspace argument, for callers that cannot allocate
 * device memory where they run the layer: plugins whose host framework's
 * memory pool owns the device memory, serving loops that forbid allocation
 * after warm-up, and latency-bound loops that cannot take cudaMalloc's
 * implicit synchronisation. The pages have no counterpart to this entry
 * point.
 *   Arguments, layouts and results are those of mxfp4_moe, minus
 *   `workspace` / `workspace_bytes`.
 *   Scratch: a fixed device array of MXFP4_MOE_NOALLOC_SCRATCH_BYTES (12 MiB)
 *   inside the library. Problems needing more (mxfp4_moe_workspace_size)
 *   return MXFP4_ERR_WORKSPACE before any launch.
 *   The first call on a device looks up the array's device address; make
 *   it before any stream capture. Calls share the array: calls that overlap
 *   on the GPU race. Nothing is allocated or freed.
 */
int mxfp4_moe_noalloc(const void* x, int64_t t, int64_t hidden, const float* router_logits, int64_t e, int top_k,
                      const uint8_t* w1q, const uint8_t* w1s, const uint8_t* w2q, const uint8_t* w2s, int64_t inter,
                      void* y, int32_t* topk_ids, float* topk_w, void* stream);

/*
 * ------------------------------------------------------------------------
 * The attention side of a step: norms around a block, rotary positions with
 * the write into the KV cache, attention of the step's new tokens over the
 * cache, and the cache's pages between steps. They sit next to the weight
 * calls above: their bf16 inputs and outputs are mxfp4_linear's outputs and
 * inputs. No call synchronises, and every length and page number is read on
 * the device, so a step can be captured once in a CUDA graph and replayed
 * while the lengths change. (mxfp4_cache_update writes the new table and
 * lengths beside the old ones: a captured step copies them to where its other
 * calls read them.)
 *
 * Paged KV cache. K and V each live in a pool of pages of page_size tokens;
 * a page holds [kv_heads][page_size][head_dim] elements, dense, and pages
 * lie page_stride elements apart. The block table gives the pages of each
 * sequence in order; an entry outside [0, num_pages) stands for no page:
 * nothing is written there, and it reads as rows of zeros.
 */
typedef enum {
    MXFP4_KV_BF16 = 0,
    MXFP4_KV_E4M3 = 1 /* element * scale of its KV head */
} mxfp4_kv_dtype;

typedef struct {
    void* k;              /* device, 16-byte aligned; layer 0's pool */
    void* v;              /* device, 16-byte aligned */
    const float* k_scale; /* device float32 [kv_heads], E4M3 only; NULL = 1 */
    const float* v_scale; /* the same for V */
    int64_t page_stride;  /* elements between pages; 0 = kv_heads * page_size * head_dim */
    int64_t layer_stride; /* elements between layers' pools (mxfp4_cache_copy, _accept); 0 = num_pages * page_stride */
    int64_t num_pages;    /* pages of a layer's pool, < 2^24 */
    int32_t layers;       /* layers that mxfp4_cache_copy and _accept work on (1 .. 1024) */
    int32_t kv_heads;     /* 1 .. 1024 */
    int32_t page_size;    /* tokens: a power of two, 16 .. 1024 */
    int32_t head_dim;     /* 64 or 128 */
    int32_t dtype;        /* mxfp4_kv_dtype */
    int32_t reserved;     /* 0 */
} mxfp4_kv_cache_t;

/*
 * The new tokens of a step. Request b brings rows q_start[b] .. q_start[b+1]-1
 * of the step's token arrays (none is allowed); they are the last tokens of
 * its sequence: new token i of n has cache index seq_lens[b] - n + i.
 * Lengths beyond the block table's room are cut to it.
 */
typedef struct {
    const int32_t* q_start;     /* device int32 [batch + 1], ascending from 0 to at most tokens */
    const int32_t* seq_lens;    /* device int32 [batch]: tokens in the cache, the new ones included */
    const int32_t* block_table; /* device int32 [batch][table_width], rows table_stride apart */
    int64_t table_stride;       /* entries; 0 = table_width */
    int32_t table_width;
    int32_t batch;              /* requests, 1 .. 1024 */
    int32_t tokens;             /* rows of the step's token arrays */
    int32_t max_q;              /* most new tokens of a request (sizes the kernels; longer ones stay right) */
    int32_t max_seq;            /* most tokens of a sequence (the same) */
    int32_t reserved;           /* 0 */
} mxfp4_kv_batch_t;

/*
 * Norms between two blocks, with the block's gate and the residual sum. Per
 * token, in fp32, each output rounded once:
 *   u = x, or N(x) * (post_weight + weight_offset) + post_bias
 *   u = u * gate
 *   r = residual + scale * u
 *   y = N(r) * (weight + weight_offset) + bias       (of the unrounded r)
 * N(z) = z / sqrt(mean(z^2) + eps); layer != 0: the same of z - mean(z).
 *   x, residual, y, r_out   device bf16 [tokens, n]; r_out may be residual
 *                  and y may be x (each row is read before it is written)
 *   post_weight    device bf16 [n], or NULL for no norm of x
 *   post_bias      device bf16 [n] or NULL (needs post_weight)
 *   gate           device bf16, rows gate_stride elements apart (0: one row
 *                  for every token; otherwise >= n), or NULL
 *   weight         device bf16 [n];  bias device bf16 [n] or NULL
 *   n              1 .. 32768; every pointer 2-byte aligned (16 bytes, with
 *                  n and gate_stride multiples of 8, takes the wide loads)
 */
int mxfp4_residual_norm(const void* x, const void* residual, int64_t tokens, int64_t n, const void* post_weight,
                        const void* post_bias, const void* gate, int64_t gate_stride, float scale,
                        const void* weight, const void* bias, float weight_offset, float eps, int layer, void* y,
                        void* r_out, void* stream);

/*
 * Rotary positions of a step's new tokens, and the write of their K and V
 * into the cache (of the layer `cache` names). The first rotary_dim elements
 * of each q and k head turn in pairs by position * inv_freq[j]: pair j is
 * the elements (2j, 2j+1) (interleaved != 0) or (j, j + rotary_dim/2):
 *   (a, b) -> (a cos - b sin, a sin + b cos) * factor
 * The rest of the head, and V, pass unchanged. Angles are reduced as sums of
 * two fp32 numbers, so long positions keep their accuracy: off by 2^-22 +
 * |position| * inv_freq * 2^-47 of a turn at most. Stretching a model to longer
 * contexts is a matter of inv_freq and factor.
 *   qkv          device bf16, rows of (q_heads + 2 kv_heads) * head_dim (q,
 *                then k, then v) qkv_stride elements apart, 16-byte aligned,
 *                qkv_stride % 8 == 0
 *   positions    device int32 [tokens], or NULL: the cache index
 *   inv_freq     device float32 [rotary_dim / 2]
 *   rotary_dim   even, 0 .. head_dim (0: nothing turns, inv_freq may be NULL)
 *   q_out        device bf16 [tokens, q_heads, head_dim], 16-byte aligned
 * E4M3 caches store value / scale, the fp32 quotient rounded to nearest even
 * and saturating at 448. Rows of qkv beyond q_start[batch] are left out.
 */
int mxfp4_rope_append(const void* qkv, int64_t qkv_stride, int q_heads, const int32_t* positions,
                      const float* inv_freq, int rotary_dim, int interleaved, float factor,
                      const mxfp4_kv_cache_t* cache, const mxfp4_kv_batch_t* batch, void* q_out, void* stream);

/*
 * Attention of a step's new tokens over the paged cache, their own K and V
 * already in it. q_heads / kv_heads query heads in a row share a KV head.
 *   s_j = scale * q . k_j, or softcap * tanh(scale * q . k_j / softcap)
 *   o = sum_j softmax(s)_j v_j   over the visible keys j
 * A query at cache index c sees j <= c; with a window, j > c - window too.
 * tree_mask replaces j <= c among the new tokens of a request: bit j of a
 * query's word says that it sees new token j (a draft tree's ancestors and
 * itself); what lies before the new tokens stays visible. A window counts
 * cache indices, for drafts of a tree too: a draft at index i and depth d < i
 * loses the i - d oldest keys that decoding it alone would see.
 * mxfp4_attention_at counts from the drafts' positions. A query that sees
 * nothing gives 0 (lse -inf). What is not visible has no part in a result,
 * whatever it holds (NaN and infinities included).
 *   q          device bf16, rows of q_heads * head_dim, q_stride elements
 *              apart, 16-byte aligned, q_stride % 8 == 0
 *   q_heads    a multiple of kv_heads, at most 128 * kv_heads; tokens *
 *              q_heads / kv_heads at most 2^31 - 256
 *   softcap    0: none;  window 0: none
 *   tree_mask  device uint64 [tokens] or NULL; max_q <= 64
 *   out        device bf16 [tokens, q_heads, head_dim], 16-byte aligned;
 *              rows of no request are not written
 *   lse        device float32 [tokens, q_heads] or NULL: log sum_j exp(s_j)
 *   workspace  device, at least mxfp4_attention_workspace_size() bytes,
 *              256-byte aligned, contents on entry do not matter
 * Scores, maxima, sums and outputs accumulate in fp32; the probabilities of
 * a product with V are rounded to bf16 (E4M3 caches: to f16).
 */
size_t mxfp4_attention_workspace_size(int q_heads, const mxfp4_kv_cache_t* cache, const mxfp4_kv_batch_t* batch);
int mxfp4_attention(const void* q, int64_t q_stride, int q_heads, const mxfp4_kv_cache_t* cache,
                    const mxfp4_kv_batch_t* batch, float scale, float softcap, int window,
                    const uint64_t* tree_mask, void* out, float* lse, void* workspace, size_t workspace_bytes,
                    void* stream);

/*
 * The same with the drafts' positions, as mxfp4_rope_append takes them: a
 * window leaves out what lies before the new tokens at cache index
 * <= position - window. Which of the new tokens a query sees is the
 * tree_mask's alone (one that the window has left is not in it).
 *   positions  device int32 [tokens], each cut to the cache indices of its
 *              request's new tokens (first new token + depth in the tree lies
 *              among them); needs tree_mask; NULL = mxfp4_attention
 */
int mxfp4_attention_at(const void* q, int64_t q_stride, int q_heads, const mxfp4_kv_cache_t* cache,
                       const mxfp4_kv_batch_t* batch, float scale, float softcap, int window,
                       const uint64_t* tree_mask, const int32_t* positions, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * The cache's pages from one step to the next, in one call: fork, reorder,
 * cut back, extend and free. New sequence i continues old sequence
 * parent[i] (or begins empty: parent[i] outside [0, old_sequences)), cut to
 * its first keep[i] tokens (keep NULL: all), and gets room for grow[i] more:
 *   - pages that hold kept tokens are shared, as often as they are wanted;
 *   - a partly filled page that will grow is copied first, unless every new
 *     sequence that holds the page will write to it and this is the first of them;
 *   - new pages are the lowest-numbered ones that no new sequence holds,
 *     dealt in sequence order (a copy's first). Old sequences that nobody
 *     continues are thereby freed.
 * Where the pool runs short, later sequences get less: lens_out says what
 * each can hold (without its copy a sequence gets no growth at all).
 *   table       device int32 [old_sequences][table_width], rows table_stride
 *               (0 = table_width) apart;  seq_lens device int32 [old_sequences]
 *   parent, keep, grow   device int32 [sequences] (1 .. 65536)
 *   table_out   device int32 [sequences][table_width], not `table`; entries
 *               past a sequence's pages are -1
 *   lens_out    device int32 [sequences]: kept + grown tokens
 *   copies      device int32 [sequences][3]: source page, target page and
 *               rows of a page to copy (mxfp4_cache_copy), or -1, -1, 0
 *   info        device int32 [2]: pages left free; pages asked for in vain
 *               (2^31 - 1 at most)
 *   workspace   at least mxfp4_cache_workspace_size() bytes, 256-byte
 *               aligned, contents on entry do not matter
 */
size_t mxfp4_cache_workspace_size(int64_t sequences, int64_t num_pages);
int mxfp4_cache_update(const int32_t* table, int64_t table_stride, int table_width, const int32_t* seq_lens,
                       int old_sequences, const int32_t* parent, const int32_t* keep, const int32_t* grow,
                       int sequences, int64_t num_pages, int page_size, int32_t* table_out, int32_t* lens_out,
                       int32_t* copies, int32_t* info, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Copies the first rows of pages that mxfp4_cache_update lists, K and V, in
 * every layer of the cache.   copies  device int32 [sequences][3]
 */
int mxfp4_cache_copy(const mxfp4_kv_cache_t* cache, const int32_t* copies, int sequences, void* stream);

/*
 * After a verify step: moves the K and V rows of the accepted draft path to
 * the front of each request's new tokens, in every layer. Row i of the new
 * tokens becomes row path[b][i] for i < n_accept[b]; entries outside the new
 * tokens, or of tokens that lie before the sequence, move nothing.
 *   path       device int32 [batch][path_len], path_len 1 .. 64
 *   n_accept   device int32 [batch], cut to [0, new tokens] and to path_len
 *   lens_out   device int32 [batch], not seq_lens: seq_lens - new tokens +
 *              n_accept, not below 0
 */
int mxfp4_cache_accept(const mxfp4_kv_cache_t* cache, const mxfp4_kv_batch_t* batch, const int32_t* path,
                       int path_len, const int32_t* n_accept, int32_t* lens_out, void* stream);

/*
 * ------------------------------------------------------------------------
 * Many tokens at once (the chunks of a prompt, large batches): activations as
 * microscaled (MX) codes, and their products with MXFP4 weights on the tensor
 * cores. A block's chain is norm -> codes -> product -> codes -> product.
 *
 * MX codes of rows of k values (k % 32 == 0): each 32 consecutive values of a
 * row share one E8M0 byte s, a value is its element times 2^(s-127).
 *   codes   E4M3: uint8 [t, k];  E2M1: uint8 [t, k/2], the even index in the
 *           low nibble (as in the weights)
 *   scales  uint8 [t, k/32]
 * The scale is the smallest power of two, 2^-127 at least, that keeps every
 * element of the block within its type (448 or 6): nothing saturates. Elements
 * are rounded to nearest, ties to even. A block that holds a NaN or an
 * infinity gets scale 255, NaN, and every output it takes part in is NaN.
 * (mxfp4_quantize's rule for weights is another: theirs may saturate.)
 * Outputs may not overlap inputs or each other (but r_out may be residual or x,
 * at the same address).
 */
typedef enum {
    MXFP4_MX_E4M3 = 0, /* 8 bits: 4 significant ones, 8.25 bits a value in all */
    MXFP4_MX_E2M1 = 1  /* 4 bits: 2 significant ones, 4.25 bits a value */
} mxfp4_mx_format;

/*
 * Rows of bf16 as MX codes; swiglu != 0: of z[j] = SiLU(x[j]) * x[k + j] (fp32).
 *   x       device bf16, t rows of k (swiglu: 2 k) values, x_stride elements
 *           apart (0: dense), 16-byte aligned, x_stride % 8 == 0
 *   xq, xs  device codes (16-byte aligned) and scales (outputs)
 */
int mxfp4_quantize_mx(const void* x, int64_t x_stride, int64_t t, int64_t k, int swiglu, int format, void* xq,
                      uint8_t* xs, void* stream);

/*
 * mxfp4_residual_norm with y as MX codes of the unrounded fp32 values.
 *   n       a multiple of 32, at most 32768; every pointer but ys 16-byte
 *           aligned, gate_stride % 8 == 0
 *   yq, ys  device codes and scales of y (outputs)
 * Every other argument is as there; r_out may be residual or x.
 */
int mxfp4_residual_norm_mx(const void* x, const void* residual, int64_t tokens, int64_t n, const void* post_weight,
                           const void* post_bias, const void* gate, int64_t gate_stride, float scale,
                           const void* weight, const void* bias, float weight_offset, float eps, int layer, int format,
                           void* yq, uint8_t* ys, void* r_out, void* stream);

/*
 * y[i][j] = bf16( sum_k x[i][k] * w[j][k] ) for any number of tokens.
 *   xq, xs  device MX codes (16-byte aligned) and scales (4-byte aligned) of x
 *           [t, k]; format: theirs
 *   k       a multiple of 128, at most 2^24
 *   wq, ws  device uint8 [n, k/2], [n, k/32], MXFP4 weights as for
 *           mxfp4_linear, wq 16-byte aligned (with E4M3 activations 32), ws 4;
 *           a scale byte of 255 is NaN
 *   y       device bf16 [t, n], 2-byte aligned (output; 16-byte aligned with
 *           n % 8 == 0 takes the wide stores)
 * Products of codes are exact, sums fp32 in the tensor cores' order. Activations
 * and weights may come from any earlier work of the stream, the call right before
 * included: nothing is read before it has ended.
 */
int mxfp4_linear_mx(const void* xq, const uint8_t* xs, int format, int64_t t, int64_t k, const uint8_t* wq,
                    const uint8_t* ws, int64_t n, void* y, void* stream);

/*
 * How mxfp4_linear_mx (swiglu != 0: mxfp4_swiglu_mx, n = inter) cuts a product:
 * what sets its speed, to be checked without a GPU (host only, no CUDA call).
 *   t, k, n, format  as there (same checks of the sizes)
 *   aligned_rows     whether rows of y begin at multiples of 16 bytes
 *   max_smem         opt-in shared memory per block in bytes (232448 on GB300)
 *   clusters         int32 [9]: of 1 .. 8 CTAs, one to an SM, so many clusters are
 *                    resident at once (entry 0 unused); NULL: as on GB300
 *   out              host struct, written on MXFP4_OK
 */
typedef struct {
    int32_t pair;        /* 1: a pair of CTAs takes 256 tokens, 0: one takes 128 */
    int32_t width;       /* weight rows of a tile (gate and up rows together) */
    int32_t split;       /* CTAs or pairs of a cluster that share a tile's k */
    int32_t ctas;        /* CTAs launched */
    int32_t ring_slots;  /* stages in shared memory: 128 bytes of codes of every row */
    int32_t stage_bytes;
    int32_t token_rows;  /* rows of tokens in a stage */
    int32_t scale_slots; /* groups of scales (512 values of k) in shared memory */
    int32_t scale_bytes; /* of a group */
    int32_t inbox_bytes; /* split > 1: of the others' sums, taken into the ring */
    int32_t smem_bytes;  /* dynamic shared memory per CTA */
} mxfp4_mx_plan_t;
int mxfp4_linear_mx_plan(int64_t t, int64_t k, int64_t n, int format, int swiglu, int aligned_rows, int max_smem,
                         const int32_t* clusters, mxfp4_mx_plan_t* out);

/*
 * The gated half of an FFN, from codes to codes:
 *   h[i][j] = SiLU( sum_k x[i][k] w1[j][k] ) * sum_k x[i][k] w1[inter + j][k]
 * in fp32, and its MX codes (out_format), with no intermediate in memory.
 *   w1q, w1s  device uint8 [2*inter, k/2], [2*inter, k/32] (gate rows first)
 *   inter     a multiple of 32
 *   hq, hs    device codes (16-byte aligned) and scales of h [t, inter]
 *             (outputs)
 * Every other argument is as for mxfp4_linear_mx.
 */
int mxfp4_swiglu_mx(const void* xq, const uint8_t* xs, int format, int64_t t, int64_t k, const uint8_t* w1q,
                    const uint8_t* w1s, int64_t inter, int out_format, void* hq, uint8_t* hs, void* stream);

/*
 * Synchronizes `stream`, then returns MXFP4_OK, MXFP4_ERR_TIMEOUT if some
 * kernel of this library on the current device gave up a bounded wait since
 * the last call, or MXFP4_ERR_CUDA if the stream reports an error. Clears
 * the device status word.
 */
int mxfp4_last_device_status(void* stream);

#ifdef __cplusplus
}
#endif

#if defined(__GNUC__)
#pragma GCC visibility pop
#endif

#endif /* MXFP4_H */
