/*
 * moe_ffn.h -- C ABI of the GB300 (sm_103a) batched routed-MoE FFN library.
 *
 * The layer (one call, moe_ffn_prefill) follows the SharpInference issue pages:
 *   router matvec over all N tokens, softmax + top-k (norm_topk_prob on/off)
 *   and shared-expert gate   -- "Carnice prefill toward llama.cpp 676 t/s"
 *                               (#388), breakdown table "router" row and
 *                               "Remaining levers" item 1;
 *   GPU-side expert bucketing into the expStart/expTokI/expTokK CSR
 *                             -- #388 "Remaining levers" item 1 ("Hard part");
 *   gather tokens per expert -> grouped expert GEMM -> scatter
 *                             -- "batched int8-MMQ trunk prefill gated off for
 *                               MoE" (#406), "The work" item 2; #388 lever 3;
 *   Q8_0 weights x Q8_1 activations (int8 block dot products)
 *                             -- #406 references (Q8_0 MMQ), "full-offload MoE
 *                               decode" (#408) lever 2 (Q8_1 / dp4a);
 *   weighted scatter-reduce in top-k slot order k = 0..na-1, then the shared
 *   expert row             -- issue #129, "Scope".
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers (CUDA global memory of the
 *     current device) unless a comment says otherwise.  Arrays are dense,
 *     row-major, C order.  The caller owns every buffer it passes; the library
 *     owns only what moe_weights_create allocates.
 *   - Calls are asynchronous on `stream`: they enqueue kernels and return.
 *     Only moe_weights_create/destroy and moe_workspace_status synchronise.
 *     No call on the hot path allocates memory or copies to/from the host.
 *   - Return value: MOE_OK (0) or a negative moe_status code for an error the
 *     host can see before launching (bad argument, unsupported shape, small
 *     workspace, launch failure).  Errors found by the kernels (an expert
 *     index out of range, a token that selects an expert twice, a malformed
 *     CSR, a device wait that timed out) are OR-ed into the status word at the
 *     start of the workspace; read them with moe_workspace_status.  A kernel
 *     that finds such an error writes a safe result (empty segments, zero
 *     rows) instead of reading out of bounds.
 *   - Shapes: D (hidden), F (routed expert intermediate) and Fs (shared
 *     expert intermediate) are multiples of 32 (the Q8 block).  The tensor-
 *     core path also needs D % 128 == 0, F % 64 == 0 and Fs % 64 == 0; other
 *     shapes run on the matvec path.  1 <= top_k <= min(E, 32), E <= 1024, N >= 1.
 *
 * Block formats
 *   Q8_0 (weights, GGUF): per 32 values one 34-byte block: fp16 scale d
 *     (little-endian) followed by 32 int8 quants q; value = d * q.
 *   Q8_1 (activations, produced on the device): per 32 values
 *     d = amax/127 (fp32), q = roundf(x * (1/d)) (int8), stored scale fp16(d).
 *     This library stores the quants as int8 and the stored scale widened to
 *     fp32 (exactly the fp16 value); the Q8_1 sum field d*sum(q) is only
 *     consumed by weight formats with an offset, so it is not produced.
 */
#ifndef MOE_FFN_H
#define MOE_FFN_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_FFN_ABI_VERSION 1

enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1,        /* null required pointer, N < 1, top_k > E, ... */
    MOE_ERR_UNSUPPORTED_SHAPE = -2,  /* D/F/Fs not a multiple of 32, E > 1024, sizes overflow */
    MOE_ERR_WORKSPACE_TOO_SMALL = -3,
    MOE_ERR_CUDA = -4,               /* a CUDA call or launch failed */
    MOE_ERR_DEVICE_TIMEOUT = -5,     /* a bounded device-side wait gave up */
    MOE_ERR_UNSUPPORTED_DEVICE = -6, /* not compute capability 10.3 */
    MOE_ERR_BAD_ROUTING = -7,        /* expert index out of range / selected twice */
    MOE_ERR_BAD_CSR = -8             /* CSR offsets or token indices out of range */
};

/* Device status word bits (moe_workspace_status returns the word; a nonzero
 * word maps to the first matching moe_status in this order). */
#define MOE_DEV_BAD_ROUTING 0x1u
#define MOE_DEV_BAD_CSR 0x2u
#define MOE_DEV_TIMEOUT 0x4u

/* Human-readable name of a moe_status code (static string, never NULL). */
const char *moe_status_string(int status);

/* MOE_FFN_ABI_VERSION of the loaded library. */
int moe_abi_version(void);

/* Path selection for moe_grouped_ffn_ex / moe_ffn_prefill_ex. */
enum moe_path {
    MOE_PATH_AUTO = 0,   /* tensor-core grouped GEMM for prefill batches, matvec for small N */
    MOE_PATH_MATVEC = 1, /* fused gather-matvec (dp4a int8 dots), any N */
    MOE_PATH_TENSOR = 2  /* tcgen05 grouped GEMM (needs the shapes above) */
};

/* ---------------------------------------------------------------------------
 * Expert weights.  moe_weights_create copies the caller's Q8_0 tensors into a
 * library-owned device copy laid out for the kernels (int8 quants and fp32
 * scales split apart; a second copy of the quants as exact fp16 integers in
 * 128-row tiles for the tensor cores).  It allocates device memory and
 * synchronises `stream`.  The caller's buffers may be freed afterwards.
 *   gate_q8_0, up_q8_0 : device, Q8_0 blocks [E][F][D/32]  (row f reduces over D)
 *   down_q8_0          : device, Q8_0 blocks [E][D][F/32]
 *   sh_gate, sh_up     : device, Q8_0 blocks [Fs][D/32], or NULL when Fs == 0
 *   sh_down            : device, Q8_0 blocks [D][Fs/32], or NULL when Fs == 0
 * Returns MOE_ERR_UNSUPPORTED_DEVICE on anything but compute capability 10.3.
 * ------------------------------------------------------------------------- */
typedef struct moe_weights_s *moe_weights_t;

int moe_weights_create(moe_weights_t *out, int E, int D, int F,
                       const void *gate_q8_0, const void *up_q8_0, const void *down_q8_0,
                       int Fs, const void *sh_gate_q8_0, const void *sh_up_q8_0,
                       const void *sh_down_q8_0, cudaStream_t stream);

/* Block format of the caller's expert weights. */
enum moe_weight_format {
    MOE_WFMT_Q8_0 = 0, /* GGUF Q8_0: 34-byte blocks of 32 (fp16 d, 32 int8) */
    MOE_WFMT_Q4_K = 1, /* GGUF Q4_K: 144-byte super-blocks of 256 (fp16 d, fp16 dmin, 12 bytes
                          of 6-bit sub-block scales sc_j and mins m_j, 128 bytes of 4-bit
                          quants q): value = d*sc_j*q - dmin*m_j ("Q8_0/Q4_K MMQ", #406
                          references).  Needs D, F, Fs multiples of 256. */
    MOE_WFMT_Q3_K = 2  /* GGUF Q3_K: 110-byte super-blocks of 256 (32 bytes of high bits, 64
                          bytes of 2-bit low parts, 12 bytes of sixteen 6-bit scales s_j + 32,
                          fp16 d): value = d*s_j*q, q in [-4, 3], one s_j per 16 values (the
                          routed experts' format on the Carnice prefill page, #388 "Key
                          references").  Needs D, F, Fs multiples of 256. */
};
/* moe_weights_create for either format: the same arrays, rows in `format`'s
 * blocks ([E][F][D/256] super-blocks for Q4_K gate/up, [E][D][F/256] down,
 * and likewise for the shared expert).  A Q4_K layer computes, per 32-wide
 * sub-block b, the exact int32 dot of the quants (0..15) with the Q8_1
 * activation codes and the code sum of the activation block:
 *   sum_b d_x[b] * (d*sc_b * isum_b - dmin*m_b * xsum_b).
 * A Q3_K layer folds the 16-wide sub-block scales into the integer codes at
 * load time: per 32-wide block b it stores c_i = -s_j*q_i (always in
 * [-128, 124], one int8) with the block scale -d, and computes
 *   sum_b d_x[b] * (-d) * (sum_i c_i * x_i) = sum_b d_x[b] * d * (s_2b*isum_2b + s_2b+1*isum_2b+1),
 * the same exact block integer as the format's own definition (the signs
 * cancel in every product).
 * MOE_ERR_UNSUPPORTED_SHAPE for shapes the format cannot hold; an unknown
 * format is MOE_ERR_INVALID_ARG. */
int moe_weights_create_ex(moe_weights_t *out, int format, int E, int D, int F,
                          const void *gate, const void *up, const void *down, int Fs,
                          const void *sh_gate, const void *sh_up, const void *sh_down,
                          cudaStream_t stream);
/* MOE_WFMT_* of a weights handle, or MOE_ERR_INVALID_ARG for NULL. */
int moe_weights_format(moe_weights_t w);
int moe_weights_destroy(moe_weights_t w);
/* Shape of a weights handle (any output pointer may be NULL; host pointers). */
int moe_weights_shape(moe_weights_t w, int *E, int *D, int *F, int *Fs);
/* Library-owned device bytes held by the handle. */
size_t moe_weights_device_bytes(moe_weights_t w);
/* 1 when the tensor-core path can run on these weights (shapes and build), else 0. */
int moe_weights_tensor_path(moe_weights_t w);

/* ---------------------------------------------------------------------------
 * Workspace: one caller-owned device buffer per concurrent call chain.  The
 * first 256 bytes hold the device status word (and the bucketing kernel's
 * grid-barrier words and the small-batch routing's arrival counter, all zero
 * between calls).  moe_workspace_init zeroes those 256 bytes
 * (asynchronously); moe_workspace_status synchronises the
 * stream, returns the status word (host int, MOE_DEV_* bits) and, when
 * clear != 0, zeroes it.  Two call chains must not share a workspace.
 * moe_ffn_workspace_size covers every entry point below for that shape.
 * ------------------------------------------------------------------------- */
size_t moe_ffn_workspace_size(int N, int D, int E, int F, int top_k, int Fs);
int moe_workspace_init(void *ws, size_t ws_bytes, cudaStream_t stream);
int moe_workspace_status(void *ws, int clear, cudaStream_t stream);
/* Map a status word to the moe_status code of its first error (MOE_OK if 0). */
int moe_status_from_word(int word);

/* ---------------------------------------------------------------------------
 * moe_router_topk -- router, softmax, top-k, shared gate, Q8_1 of x (#388
 * breakdown table "router" row: matvec + softmax + top-k + shexp-gate;
 * levers item 1: norm[N x embDim] x routerW[numExperts x embDim]).
 *   hidden     [N][D] fp32          routerW [E][D] fp32
 *   shexp_gate [D] fp32 or NULL     (shared-expert gate vector)
 *   topk_idx   [N][top_k] int32 out: experts by decreasing logit, ties to
 *              the lower index (slot 0 = largest)
 *   topk_w     [N][top_k] fp32 out: softmax over all E experts at the
 *              selected experts; divided by their sum when norm_topk_prob
 *   shexp_scale [N] fp32 out, sigmoid(hidden[t] . shexp_gate); NULL iff
 *              shexp_gate is NULL
 *   x_q [N][D] int8 out, x_d [N][D/32] fp32 out: Q8_1 of hidden
 *   logits_out [N][E] fp32 out or NULL (the router logits)
 *   ws: workspace (split-K partial logits).
 * ------------------------------------------------------------------------- */
int moe_router_topk(const float *hidden, const float *routerW, const float *shexp_gate,
                    int N, int D, int E, int top_k, int norm_topk_prob,
                    int32_t *topk_idx, float *topk_w, float *shexp_scale,
                    int8_t *x_q, float *x_d, float *logits_out,
                    void *ws, size_t ws_bytes, cudaStream_t stream);

/* moe_router_topk for callers that cannot allocate device memory (no
 * counterpart on the pages: it exists only for hosts whose device memory is
 * owned by another allocator, or that forbid cudaMalloc after start-up).  Same
 * arguments and results as moe_router_topk, without the workspace: the router's
 * split-K partial logits go to a 16 MiB array inside the library (2^22 floats,
 * held on every GPU that loads the library until exit).  The problem must fit:
 * nsplit * N * (E + 1) <= 2^22 floats, nsplit being the router's split-K factor:
 * 1 when N <= 8 and D % 4 == 0; otherwise, with tiles = ceil(N/64)*ceil(E/64)
 * and SMs the current device's multiprocessor count, the largest s that
 * divides D/32 with s <= min(ceil(4*SMs/tiles), D/depth), depth = 32 when
 * tiles <= 4 and 128 otherwise (so at most min(4*SMs, D/32)).  A problem that
 * does not fit returns MOE_ERR_WORKSPACE_TOO_SMALL and nothing runs.  The first call on a device looks the array's device address up
 * (cudaGetSymbolAddress, which may load the library's kernels onto that device)
 * and should therefore come before any stream capture.  All calls on a device
 * share the array, so calls that may overlap on the GPU race and must be
 * ordered by the caller.  Allocates nothing. */
int moe_router_topk_noalloc(const float *hidden, const float *routerW, const float *shexp_gate,
                            int N, int D, int E, int top_k, int norm_topk_prob,
                            int32_t *topk_idx, float *topk_w, float *shexp_scale,
                            int8_t *x_q, float *x_d, float *logits_out, cudaStream_t stream);

/* Softmax + top-k alone, from given logits [N][E] (same outputs as above).
 * Lets a caller check routing against logits computed elsewhere. */
int moe_topk_from_logits(const float *logits, int N, int E, int top_k, int norm_topk_prob,
                         int32_t *topk_idx, float *topk_w, cudaStream_t stream);

/* Q8_1 quantisation of n_blocks consecutive 32-value blocks: q [n_blocks*32]
 * int8, d [n_blocks] fp32 (the fp16 stored scale, widened).  The same rule
 * moe_router_topk applies to hidden. */
int moe_quantize_q8_1(const float *x, int64_t n_blocks, int8_t *q, float *d, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * moe_bucket -- expert bucketing into a CSR on the device (#388 levers item 1:
 * expStart/expTokI/expTokK).  A counting sort of the N*top_k (token, slot)
 * pairs by expert, stable in token order:
 *   expStart [E+1] int32 out: segment offsets, expStart[0] = 0,
 *            expStart[E] = N*top_k
 *   expTokI  [N*top_k] int32 out: token of each entry (ascending per segment)
 *   expTokK  [N*top_k] int32 out: top-k slot of that token for this expert
 * A bad index or a repeated expert within a token sets MOE_DEV_BAD_ROUTING
 * and leaves every segment empty.  One cooperative kernel: each CTA counts a
 * token range, a grid barrier, then every CTA scans the count table and
 * scatters its range (histogram, scan and scatter in one launch).
 * ws: 256-byte aligned, at least moe_bucket_workspace_size(N, top_k, E)
 * bytes (a moe_ffn_workspace_size workspace of the same N, E, top_k always
 * is), initialised once by moe_workspace_init; the barrier keeps its words at
 * zero between calls.  If the barrier times out (MOE_DEV_TIMEOUT) the outputs
 * are undefined; run moe_workspace_init before the next call.
 * ------------------------------------------------------------------------- */
size_t moe_bucket_workspace_size(int N, int top_k, int E);
int moe_bucket(const int32_t *topk_idx, int N, int top_k, int E,
               int32_t *expStart, int32_t *expTokI, int32_t *expTokK,
               void *ws, size_t ws_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * moe_grouped_ffn -- every routed expert over its CSR segment, plus the shared
 * expert over all tokens (#406 "The work" item 2: gather -> grouped GEMM ->
 * scatter; #129 intro: gate/up/down grouped by expert; #129 "Scope": the
 * optionally batched shared expert):
 *   for entry j of expert e (t = expTokI[j], s = expTokK[j]):
 *     h_j = Q8_1( SiLU(W_g[e] x_t) * (W_u[e] x_t) )      (x_t = Q8_1 row t)
 *     partials[t*top_k + s][0..D) = W_d[e] h_j            (fp32, unweighted)
 *   shared (when the weights have Fs > 0 and shared_out != NULL):
 *     shared_out[t][0..D) = shexp_scale[t] * W_sd Q8_1(SiLU(W_sg x_t) * (W_su x_t))
 *   x_q [N][D] int8, x_d [N][D/32] fp32: Q8_1 rows (moe_router_topk output)
 *   partials [N*top_k][D] fp32 out; shared_out [N][D] fp32 out or NULL.
 * Every dot product is a sum over 32-blocks of fp16(d_w)*d_x*isum with isum
 * the exact int32 dot of the block's quants.
 * ------------------------------------------------------------------------- */
int moe_grouped_ffn(moe_weights_t w, const int8_t *x_q, const float *x_d,
                    const int32_t *expStart, const int32_t *expTokI, const int32_t *expTokK,
                    int N, int top_k, const float *shexp_scale, float *partials, float *shared_out,
                    void *ws, size_t ws_bytes, cudaStream_t stream);

/* As moe_grouped_ffn with an explicit path (enum moe_path). */
int moe_grouped_ffn_ex(moe_weights_t w, const int8_t *x_q, const float *x_d,
                       const int32_t *expStart, const int32_t *expTokI, const int32_t *expTokK,
                       int N, int top_k, const float *shexp_scale, float *partials, float *shared_out,
                       int path, void *ws, size_t ws_bytes, cudaStream_t stream);

/* The two halves of moe_grouped_ffn, for checking each on its own.
 * moe_expert_gate_up writes the requantised activations of every entry in
 * segment order: h_q [N*top_k][F] int8, h_d [N*top_k][F/32] fp32.
 * moe_expert_down consumes them (from any source) and writes partials. */
int moe_expert_gate_up(moe_weights_t w, const int8_t *x_q, const float *x_d,
                       const int32_t *expStart, const int32_t *expTokI, int N, int top_k,
                       int8_t *h_q, float *h_d, int path, void *ws, size_t ws_bytes,
                       cudaStream_t stream);
int moe_expert_down(moe_weights_t w, const int8_t *h_q, const float *h_d,
                    const int32_t *expStart, const int32_t *expTokI, const int32_t *expTokK,
                    int N, int top_k, float *partials, int path, void *ws, size_t ws_bytes,
                    cudaStream_t stream);

/* Raw int32 block dot products of the gate/up GEMM for one 32-block `block`
 * of the reduction dimension: dots [N*top_k][2][F] int32, entry j in segment
 * order, [.][0][f] = isum(W_g[e][f], x_t), [.][1][f] = isum(W_u[e][f], x_t),
 * as computed inside the selected path's kernel.  The weight codes are the
 * stored ones: Q8_0 quants, Q4_K quants 0..15, and for Q3_K c_i = -s_j*q_i,
 * so a Q3_K dot is -(s_2b*isum_2b + s_2b+1*isum_2b+1). */
int moe_debug_gate_up_block_dots(moe_weights_t w, const int8_t *x_q, const float *x_d,
                                 const int32_t *expStart, const int32_t *expTokI, int N, int top_k,
                                 int block, int32_t *dots, int path, void *ws, size_t ws_bytes,
                                 cudaStream_t stream);

/* Raw int32 block dot products of the down GEMM for one 32-block `block` of
 * its reduction dimension (the intermediate size F), given requantised
 * activations h_q [N*top_k][F] int8 and h_d [N*top_k][F/32] fp32 in segment
 * order (as moe_expert_gate_up writes them): dots [N*top_k][D] int32, entry j
 * in segment order, [j][c] = isum(W_d[e][c], h_j) over block `block`, as
 * computed inside the selected path's kernel (stored weight codes, as for
 * moe_debug_gate_up_block_dots).  expTokK is needed because the tensor path's
 * plan (and its partial rows, written to the workspace) uses it.  Same errors
 * as moe_expert_down; block outside [0, F/32) is MOE_ERR_UNSUPPORTED_SHAPE. */
int moe_debug_down_block_dots(moe_weights_t w, const int8_t *h_q, const float *h_d,
                              const int32_t *expStart, const int32_t *expTokI, const int32_t *expTokK,
                              int N, int top_k, int block, int32_t *dots, int path, void *ws,
                              size_t ws_bytes, cudaStream_t stream);

/* Failure-detection check of the bucketing kernel's grid barrier: runs
 * moe_bucket with the barrier waiting for one more arrival than there are
 * CTAs, so it can never complete, and a wait limit of limit_ms (1..2000)
 * instead of the normal 1 s.  Every CTA gives up after the limit, sets
 * MOE_DEV_TIMEOUT in the workspace status word and returns without writing
 * the CSR; the context stays usable.  The barrier's words are left mid-count:
 * call moe_workspace_init before the workspace serves another call.  Needs a
 * batch large enough for more than one token range (otherwise there is no
 * barrier): MOE_ERR_UNSUPPORTED_SHAPE.  Same arguments as moe_bucket. */
int moe_debug_bucket_barrier_timeout(const int32_t *topk_idx, int N, int top_k, int E,
                                     int32_t *expStart, int32_t *expTokI, int32_t *expTokK,
                                     int limit_ms, void *ws, size_t ws_bytes, cudaStream_t stream);

/* Failure-detection check of the tensor path: runs the gate/up grouped GEMM with
 * its TMA producer told to issue nothing, so the MMA's first wait can never be
 * satisfied.  Every device wait is bounded; after limit_ms (1..2000) the kernel
 * gives up, sets MOE_DEV_TIMEOUT in the workspace status word, lets in-flight
 * work drain, frees its tensor memory and returns, leaving the context usable.
 * Returns the launch status; read the outcome with moe_workspace_status. */
int moe_debug_expert_wait_timeout(moe_weights_t w, const int8_t *x_q, const float *x_d,
                                  const int32_t *expStart, const int32_t *expTokI, int N, int top_k,
                                  int limit_ms, void *ws, size_t ws_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * moe_combine -- batched weighted scatter-reduce (#129 "Scope"), one launch
 * over N x D: for every token t and column c
 *   acc = +0.0f;
 *   for s = 0..top_k-1: acc = fmaf(topk_w[t][s], partials[t*top_k+s][c], acc);
 *   if (shared) acc = acc + shared[t][c];
 *   out[t][c] = acc;
 * in exactly this order and rounding (bit-reproducible).
 *   partials [N*top_k][D] fp32, topk_w [N][top_k] fp32, shared [N][D] or NULL,
 *   out [N][D] fp32 (may not alias the inputs).
 * ------------------------------------------------------------------------- */
int moe_combine(const float *partials, const float *topk_w, const float *shared,
                int N, int top_k, int D, float *out, cudaStream_t stream);
/* moe_combine followed by the residual add of the pages' per-layer combine,
 * (routed + shared) + resid ("Carnice prefill toward llama.cpp 676 t/s", #388,
 * "Dead ends"): after the shared row, acc = acc + residual[t][c] (one fp32
 * add), out[t][c] = acc.  residual [N][D] fp32, 16-byte aligned; it may be
 * `out` itself (an in-place residual update), otherwise it may not overlap
 * out.  residual == NULL is moe_combine. */
int moe_combine_residual(const float *partials, const float *topk_w, const float *shared,
                         const float *residual, int N, int top_k, int D, float *out,
                         cudaStream_t stream);
/* moe_combine_residual, then the next layer's input norm of every output row.
 * The pages feed the router a normalised activation ("Carnice prefill toward
 * llama.cpp 676 t/s", #388, "Remaining levers" item 1: norm[N x embDim] x
 * routerW) and chain the layers through this residual stream (item 2); the
 * norm is read as RMSNorm with a per-column weight:
 *   out[t][c]    = moe_combine_residual's value (bit for bit);
 *   normed[t][c] = (out[t][c] * r_t) * gamma[c],
 *   r_t          = 1 / sqrt(sum_c out[t][c]^2 / D + eps)   (fp32; the row sum in a
 *                  fixed order: each thread's columns, then a warp butterfly,
 *                  then the warps in order; 128 threads per row, or 512 when N
 *                  is below 8 times the SM count, so its grouping, and the last
 *                  bits of normed, depend on N).
 * residual [N][D] fp32, non-NULL (it may be `out`); gamma [D] fp32, device;
 * eps > 0 and finite; normed [N][D] fp32, overlapping neither out nor any
 * input; gamma and normed 16-byte aligned.  MOE_ERR_INVALID_ARG otherwise. */
int moe_combine_residual_rmsnorm(const float *partials, const float *topk_w, const float *shared,
                                 const float *residual, const float *gamma, float eps, int N,
                                 int top_k, int D, float *out, float *normed, cudaStream_t stream);
/* The same norm of rows x alone: normed[t][c] = (x[t][c] * r_t) * gamma[c],
 * r_t = 1 / sqrt(sum_c x[t][c]^2 / D + eps), summed as above (the input norm of
 * a stack's first layer).  x [N][D], gamma [D], normed [N][D] (not x): fp32,
 * device, 16-byte aligned; eps > 0 and finite. */
int moe_rmsnorm(const float *x, const float *gamma, float eps, int N, int D, float *normed,
                cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * moe_ffn_prefill -- the whole layer in one call (all of the above, on one
 * stream, with no host round trip): the pages' batched routed-MoE FFN over
 * N prompt tokens.
 *   hidden [N][D] fp32, routerW [E][D] fp32, shexp_gate [D] fp32 or NULL
 *   (NULL: no shared expert even if the weights carry one; non-NULL needs
 *   weights with Fs > 0), out [N][D] fp32 (the FFN output; no residual).
 * ------------------------------------------------------------------------- */
int moe_ffn_prefill(moe_weights_t w, const float *hidden, const float *routerW,
                    const float *shexp_gate, int N, int top_k, int norm_topk_prob, float *out,
                    void *ws, size_t ws_bytes, cudaStream_t stream);
int moe_ffn_prefill_ex(moe_weights_t w, const float *hidden, const float *routerW,
                       const float *shexp_gate, int N, int top_k, int norm_topk_prob, float *out,
                       int path, void *ws, size_t ws_bytes, cudaStream_t stream);
/* moe_ffn_prefill_ex whose combine also adds the residual row (moe_combine_residual):
 * out = residual + FFN(hidden).  residual [N][D] fp32, non-NULL, 16-byte aligned;
 * it may be `out` itself (the residual stream updated in place). */
int moe_ffn_prefill_residual(moe_weights_t w, const float *hidden, const float *routerW,
                             const float *shexp_gate, const float *residual, int N, int top_k,
                             int norm_topk_prob, float *out, int path, void *ws, size_t ws_bytes,
                             cudaStream_t stream);
/* moe_ffn_prefill_residual whose combine also writes the next layer's normalised
 * input (moe_combine_residual_rmsnorm): out = residual + FFN(hidden), normed =
 * RMSNorm(out) * gamma.  Arguments as there and as moe_combine_residual_rmsnorm;
 * normed may be `hidden` itself (the router has read it before the combine writes). */
int moe_ffn_prefill_residual_rmsnorm(moe_weights_t w, const float *hidden, const float *routerW,
                                     const float *shexp_gate, const float *residual,
                                     const float *gamma, float eps, int N, int top_k,
                                     int norm_topk_prob, float *out, float *normed, int path,
                                     void *ws, size_t ws_bytes, cudaStream_t stream);

/* moe_ffn_prefill_ex with hidden and out in HOST memory (the layer as a host
 * program calls it).  No staging copies: the router reads the hidden rows and
 * the combine writes the output rows in place over the host link (NVLink-C2C
 * on Grace-Blackwell), so that traffic overlaps the two kernels' own work.
 *   hidden_host [N][D] fp32, out_host [N][D] fp32: host memory the device can
 *   address -- pinned (cudaHostAlloc, cudaHostRegister) on any system, or any
 *   host allocation where the device reports pageable access through the host
 *   page tables.  Device (or managed) memory, or unreachable host memory:
 *   MOE_ERR_INVALID_ARG and nothing is launched.  out_host may not alias
 *   hidden_host.  routerW, shexp_gate, ws as for moe_ffn_prefill (device
 *   memory).  The call is asynchronous like the others: out_host holds the
 *   result once `stream` has reached the end of it. */
int moe_ffn_prefill_host(moe_weights_t w, const float *hidden_host, const float *routerW,
                         const float *shexp_gate, int N, int top_k, int norm_topk_prob,
                         float *out_host, int path, void *ws, size_t ws_bytes, cudaStream_t stream);
/* 1 when `p` is host memory the current device can address (what
 * moe_ffn_prefill_host accepts), 0 otherwise (device or managed memory,
 * NULL, or pageable memory on a system without host page-table access). */
int moe_host_memory_addressable(const void *p);
/* The host NUMA node closest to the current device (where the host buffers of
 * moe_ffn_prefill_host cross the fewest links: on a multi-socket host, memory
 * of another socket is reached through the inter-socket link as well), or -1
 * when the system reports no NUMA placement.  *node: host pointer.  Returns 0,
 * MOE_ERR_INVALID_ARG for NULL, MOE_ERR_CUDA if the query fails. */
int moe_device_host_numa_node(int *node);

/* A stack of routed-MoE FFN layers applied in place, one after another on
 * `stream`: for l = 0..n_layers-1, hidden <- hidden + FFN_l(hidden), each
 * layer exactly as moe_ffn_prefill_residual computes it with the residual
 * and output both `hidden` (so the results equal n_layers such calls bit for
 * bit).  Layer l uses weights w[l], routerW[l] and shexp_gate[l] (the array
 * itself may be NULL when no layer has a shared expert; entries may be NULL
 * per layer).  w, routerW and shexp_gate are HOST arrays of n_layers handles
 * / device pointers.  Every layer shares N, top_k, norm_topk_prob, path and
 * the workspace, which must be large enough for each layer's shapes (same D
 * in every layer).  From the second layer on, the router is launched so that
 * it may start while the previous layer's combine is still running
 * (cross-layer overlap, #388 "Remaining levers" 2): it first pulls its own
 * router weights into L2, then waits on the device for the previous layer's
 * output before reading it.  Errors as moe_ffn_prefill; nothing is launched
 * when an argument check fails. */
int moe_ffn_prefill_stack(const moe_weights_t *w, const float *const *routerW,
                          const float *const *shexp_gate, int n_layers, float *hidden, int N,
                          int top_k, int norm_topk_prob, int path, void *ws, size_t ws_bytes,
                          cudaStream_t stream);
/* moe_ffn_prefill_stack with an input norm before every layer (the pre-norm
 * chain the pages' router input implies, #388 "Remaining levers" items 1-2):
 *   normed = RMSNorm_0(hidden);  for l: hidden = hidden + FFN_l(normed),
 *   normed = RMSNorm_{l+1}(hidden) (fused into layer l's combine; after the last
 *   layer only when gamma[n_layers] is not NULL).
 * gamma: host array of n_layers + 1 device pointers to [D] fp32 weights (the
 * last may be NULL); normed [N][D] fp32 device (not hidden), holds the last
 * norm on return; eps > 0 and finite.  Every router after the first norm is
 * launched behind the kernel that writes its input.  Errors as
 * moe_ffn_prefill_stack. */
int moe_ffn_prefill_stack_rmsnorm(const moe_weights_t *w, const float *const *routerW,
                                  const float *const *shexp_gate, const float *const *gamma,
                                  float eps, int n_layers, float *hidden, float *normed, int N,
                                  int top_k, int norm_topk_prob, int path, void *ws,
                                  size_t ws_bytes, cudaStream_t stream);

/* moe_ffn_prefill_ex that also records seven caller-created CUDA events on
 * `stream` around its stages, for measuring each kernel in place:
 *   [0] start, [1] after the router (+softmax/top-k/Q8_1), [2] after bucketing
 *   (which on the tensor path also writes the GEMM plan), [3] after the gather
 *   (tensor path; nothing on the matvec path), [4] after gate/up, [5] after
 *   down (both incl. the shared expert), [6] after the combine.
 * stage_events: host array of 7 cudaEvent_t (created by the caller). */
int moe_ffn_prefill_timed(moe_weights_t w, const float *hidden, const float *routerW,
                          const float *shexp_gate, int N, int top_k, int norm_topk_prob, float *out,
                          int path, void *ws, size_t ws_bytes, cudaStream_t stream,
                          cudaEvent_t *stage_events);

/* ---------------------------------------------------------------------------
 * Token rows sorted by expert and back, for experts that run outside this
 * library between the router and the combine, in training as well: element
 * types fp32, fp16 and bf16, dropped entries, rows apart by any stride, and
 * the gradients.  Sums and weights are fp32, each result is rounded to the
 * element type once.
 *   dtype       enum moe_dtype of every tensor that is not stated otherwise
 *   1 <= D <= 2^24, N >= 1, 1 <= top_k <= min(E, 32), E <= 1024, N * top_k < 2^30,
 *   1 <= n_rows < 2^30 (MOE_ERR_UNSUPPORTED_SHAPE; MOE_ERR_INVALID_ARG for n_rows < 1)
 *   *_stride    elements from one row to the next (at most 2^30); an input's
 *               may be 0 (one row for all), an output's is at least D
 *   tokRow      [N][top_k] int32: the sorted row of each entry, or -1 for a
 *               dropped one
 * 16-byte accesses are used when pointers, strides and D allow, smaller ones
 * otherwise; the results are the same.
 * ws: status word and scratch, 256-byte aligned, moe_sort_workspace_size bytes
 * for moe_sort_tokens and 256 for the others, initialised once by
 * moe_workspace_init (any workspace of this library that is large enough: no
 * more than those bytes at its start are used, and arguments may lie behind them).
 * Outputs overlap no input and no other output (MOE_ERR_INVALID_ARG).  Column
 * slices of one buffer, rows equally far apart, do not.
 * ------------------------------------------------------------------------- */
enum moe_dtype { MOE_DTYPE_F32 = 0, MOE_DTYPE_F16 = 1, MOE_DTYPE_BF16 = 2 };

size_t moe_sort_workspace_size(int N, int top_k, int E);

/* moe_sort_tokens -- the CSR of moe_bucket with dropped entries, and the rows
 * in its order ("gather tokens per expert", #406 "The work" item 2):
 *   topk_idx [N][top_k] int32: an expert, or -1 for an entry that goes nowhere
 *            (padding, an expert held elsewhere).  Unlike moe_bucket a token
 *            may name an expert more than once.
 *   expStart [E+1] int32 out: segment offsets; expStart[E] = entries kept
 *   expTokI, expTokK [N*top_k] int32 out: token and slot of each sorted row,
 *            by expert, then token, then slot; -1 from expStart[E] on
 *   tokRow   [N][top_k] int32 out: the inverse, -1 where dropped
 *   rows     [N*top_k][D] out: rows[r] = x[expTokI[r]], bit for bit; rows from
 *            expStart[E] on are left as they were
 * Any other negative index, or one of E and above, sets MOE_DEV_BAD_ROUTING
 * and counts as dropped.  A copy inside the kernel that takes more than two
 * seconds sets MOE_DEV_TIMEOUT: rows are then incomplete. */
int moe_sort_tokens(const void *x, int64_t x_stride, int dtype, const int32_t *topk_idx, int N,
                    int top_k, int E, int D, int32_t *expStart, int32_t *expTokI, int32_t *expTokK,
                    int32_t *tokRow, void *rows, void *ws, size_t ws_bytes, cudaStream_t stream);

/* Failure-detection check of the sort's copies: runs moe_sort_tokens with every
 * copy in waiting for more bytes than it brings, so that no wait can end, and a
 * limit of limit_ms (1..2000) instead of the normal two seconds (the copies
 * waited for after the first timeout have that limit each again).  Sets
 * MOE_DEV_TIMEOUT; the CSR and tokRow are right, every row is left as it was,
 * and workspace and context stay usable.  Only where the rows go by bulk copies
 * (x, rows, x_stride and D multiples of 16 bytes): else MOE_ERR_UNSUPPORTED_SHAPE. */
int moe_debug_sort_wait_timeout(const void *x, int64_t x_stride, int dtype, const int32_t *topk_idx, int N,
                                int top_k, int E, int D, int32_t *expStart, int32_t *expTokI,
                                int32_t *expTokK, int32_t *tokRow, void *rows, int limit_ms, void *ws,
                                size_t ws_bytes, cudaStream_t stream);

/* Its gradient: d_x[t][c] = sum over the slots s of t, in slot order, of
 * d_rows[tokRow[t][s]][c] (dropped entries add nothing; a token without
 * entries gets zeros).  d_rows [n_rows][D], d_x [N][D].  An entry of tokRow
 * outside [-1, n_rows) sets MOE_DEV_BAD_CSR and counts as dropped, here and in
 * the two functions below. */
int moe_sort_tokens_grad(const void *d_rows, int64_t n_rows, int dtype, const int32_t *tokRow, int N,
                         int top_k, int D, void *d_x, int64_t d_x_stride, void *ws, size_t ws_bytes,
                         cudaStream_t stream);

/* moe_unsort_tokens -- sorted rows back to their tokens, weighted (the combine
 * of moe_combine for rows in CSR order and any element type):
 *   acc = +0; for s = 0..top_k-1: if tokRow[t][s] >= 0:
 *       acc = fmaf(topk_w[t][s], rows[tokRow[t][s]][c], acc);
 *   out[t][c] = acc.
 *   rows [n_rows][D], topk_w [N][top_k] fp32, out [N][D].  A dropped entry's
 *   weight is not used; a weight of zero still multiplies its row. */
int moe_unsort_tokens(const void *rows, int64_t n_rows, int dtype, const int32_t *tokRow,
                      const float *topk_w, int N, int top_k, int D, void *out, int64_t out_stride,
                      void *ws, size_t ws_bytes, cudaStream_t stream);

/* Its gradients, for d_out [N][D]:
 *   d_rows[tokRow[t][s]][c] = topk_w[t][s] * d_out[t][c]   (one rounding)
 *   d_topk_w[t][s] = sum_c d_out[t][c] * rows[tokRow[t][s]][c]  (fp32; 0 where dropped)
 * in one pass.  d_rows [n_rows][D]: rows that no entry names are left as they
 * were; two entries that name one row (moe_sort_tokens gives none) leave
 * either's value.  The dot's order is fixed for given N, top_k, D, type and
 * alignment. */
int moe_unsort_tokens_grad(const void *d_out, int64_t d_out_stride, const void *rows, int64_t n_rows,
                           int dtype, const int32_t *tokRow, const float *topk_w, int N, int top_k,
                           int D, void *d_rows, float *d_topk_w, void *ws, size_t ws_bytes,
                           cudaStream_t stream);

/* moe_topk_grad -- the gradient of the routing weights (moe_router_topk's and
 * moe_topk_from_logits' topk_w) to the router logits:
 *   norm_topk_prob == 0: p = softmax(logits[t]), v[e] = sum of d_topk_w[t][s] over the
 *       slots with topk_idx[t][s] == e:  d_logits[t][e] = p[e] * (v[e] - sum_j p[j] v[j])
 *   norm_topk_prob != 0: the same with the softmax taken over the selected experts
 *       alone, and d_logits 0 at the others.
 * logits, d_logits [N][E] fp32, topk_idx [N][top_k] int32, d_topk_w [N][top_k] fp32.
 * A slot of -1 counts as not selected; any other index outside [0, E) does too and
 * sets MOE_DEV_BAD_ROUTING.  A token whose softmax has no logit above -inf gets zeros.
 * The sums' order is fixed for given N, E, top_k and alignment. */
int moe_topk_grad(const float *logits, const int32_t *topk_idx, const float *d_topk_w, int N, int E,
                  int top_k, int norm_topk_prob, float *d_logits, void *ws, size_t ws_bytes,
                  cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Products with 4-bit weights and group scales, the activations unquantised
 * (the decode matvecs of #408 levers 1 and 2 for weights that come as codes,
 * scales and zero points, beside the K-quants above):
 *   W[e][r][k] = scales[e][r][k/group] * (q[e][r][k] - zeros[e][r][k/group])
 *   moe_w4_matvec: y[j][r] = sum_k W[e(j)][r][k] * x[j][k]
 * moe_w4_weights_create lays the caller's arrays out for the kernel in a
 * library-owned device copy (it allocates and synchronises `stream`; the
 * caller's buffers may be freed afterwards).
 *   q      [E][R][K/2] bytes: the code 0..15 of column 2b in the low, of 2b + 1
 *          in the high four bits of byte b
 *   scales [E][R][K/group] fp16 or bf16 (scale_dtype)
 *   zeros  [E][R][K/group] bytes, 0..15 (the low four bits count), or NULL: 8
 *   group  32, 64 or 128; K a multiple of it, at most 32768; 1 <= R <= 2^24; E <= 1024
 *   up_q, up_scales, up_zeros: NULL, or a second matrix of the same shape (up_zeros
 *          NULL iff zeros is): the handle then holds gate and up, and the product is
 *          y = SiLU(gate) * up, SiLU(z) = z / (1 + exp(-z)), in fp32 before the one
 *          rounding to y's type.
 * ------------------------------------------------------------------------- */
typedef struct moe_w4_weights_s *moe_w4_weights_t;

int moe_w4_weights_create(moe_w4_weights_t *out, int E, int R, int K, int group, int scale_dtype,
                          const uint8_t *q, const void *scales, const uint8_t *zeros,
                          const uint8_t *up_q, const void *up_scales, const uint8_t *up_zeros,
                          cudaStream_t stream);
int moe_w4_weights_destroy(moe_w4_weights_t w);
/* Shape of a handle; *pair is 1 when it holds gate and up (any output may be NULL; host pointers). */
int moe_w4_weights_shape(moe_w4_weights_t w, int *E, int *R, int *K, int *group, int *pair);
size_t moe_w4_weights_device_bytes(moe_w4_weights_t w);

/* y[j] = the handle's product of row x[j], for rows in CSR order (moe_sort_tokens).
 *   x [n_rows][K], y [n_rows][R] of `dtype`; n_rows, strides and overlaps as for moe_sort_tokens
 *   expStart [E+1] int32 device: rows expStart[e]..expStart[e+1]-1 are expert e's;
 *            rows from expStart[E] on are left as they were.  NULL (E == 1 only):
 *            every row is expert 0's.  Offsets that do not start at 0, decrease or
 *            pass n_rows set MOE_DEV_BAD_CSR and every row is left.
 * Codes less zero points are exact, and so are fp16 rows; bf16 rows are exact down to 2^-31 of their
 * largest magnitude (smaller values lose at most 2^-39 of it); of fp32 rows at most 2^-22 of each value, or
 * 2^-50 of the row's largest, is lost.  A group's products are summed by the tensor cores: 16 of them and the
 * sum so far at a time, in fp32, but each addend may be cut 23 bits below the largest of them where fp32
 * additions would round.  The groups' sums, times their scales, are added in fp32.  The weights' shape and the
 * type fix the order: a row's result does not depend on the rows beside it.  Sums leave fp32's range only where
 * the definition's own do, whatever the magnitudes of scales and rows.  An infinity or NaN stays in its row.
 * Made for few rows an expert (decode).  An expert's weights are read once for each pass of at most
 *   E > 1:  max(8, 2 ceil(n_rows / E)) of its rows (fp32: 4 in the place of 8), twice the mean, so that an expert
 *           with more of them costs a pass for each as many;
 *   E == 1: all rows (8 where R is so small that each 8 can have CTAs of their own; fp32: 4),
 * in both cases at most 32 rows (fp32: 16), and fewer where K is long.
 * MOE_ERR_UNSUPPORTED_SHAPE past 2^31 pairs of 16 weight rows and such a pass.
 *   ws: status word (256 bytes). */
int moe_w4_matvec(moe_w4_weights_t w, const void *x, int64_t x_stride, int dtype,
                  const int32_t *expStart, int n_rows, void *y, int64_t y_stride, void *ws,
                  size_t ws_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Norms of token rows with gradients (beside moe_rmsnorm), for training and for
 * rows of any element type:
 *   moe_layernorm:      y[t][c] = (x[t][c] - m_t) r_t gamma[c] (+ beta[c]),
 *       m_t = mean(x[t]), r_t = 1 / sqrt(mean((x[t] - m_t)^2) + eps)
 *   moe_layernorm_grad: with h = (x - m) r and g = gamma d_y, along each row
 *       d_x = r (g - mean(g) - h mean(g h)),
 *       d_gamma[c] = sum_t d_y[t][c] h[t][c],   d_beta[c] = sum_t d_y[t][c]
 *   moe_rmsnorm_grad:   of moe_rmsnorm, h = x r, r = 1 / sqrt(mean(x^2) + eps):
 *       d_x = r (g - h mean(g h)),   d_gamma[c] = sum_t d_y[t][c] h[t][c]
 * x, d_y [N][D], y, d_x [N][D] of `dtype`, rows apart by their strides as for
 * moe_sort_tokens (an input's may be 0: a gradient that is the same for all
 * rows); gamma, beta (NULL: 0), d_gamma, d_beta (NULL: not wanted) [D] fp32.
 * 1 <= D <= 32768, 1 <= N < 2^30 (MOE_ERR_UNSUPPORTED_SHAPE); eps > 0 and finite.
 * The gradients form m and r from x again: nothing is kept by the forward call.
 * Sums are fp32, in an order fixed for given N, D, type, alignment and device;
 * the variance is summed from the deviations.  Each result is rounded to its type once.
 * ws: moe_norm_workspace_size(N, D) bytes, as for moe_sort_tokens (the forward
 * call needs none).  Outputs overlap no input and no other output.
 * ------------------------------------------------------------------------- */
int moe_layernorm(const void *x, int64_t x_stride, int dtype, const float *gamma, const float *beta, float eps, int N,
                  int D, void *y, int64_t y_stride, cudaStream_t stream);
size_t moe_norm_workspace_size(int N, int D);
int moe_layernorm_grad(const void *d_y, int64_t d_y_stride, const void *x, int64_t x_stride, int dtype,
                       const float *gamma, float eps, int N, int D, void *d_x, int64_t d_x_stride, float *d_gamma,
                       float *d_beta, void *ws, size_t ws_bytes, cudaStream_t stream);
int moe_rmsnorm_grad(const void *d_y, int64_t d_y_stride, const void *x, int64_t x_stride, int dtype,
                     const float *gamma, float eps, int N, int D, void *d_x, int64_t d_x_stride, float *d_gamma,
                     void *ws, size_t ws_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * moe_matmul -- products of 16-bit rows with 16-bit matrices, one matrix or one
 * per expert over rows in CSR order (moe_sort_tokens), the epilogue in the same
 * pass:
 *   y[j][r] = act(sum_k w[e][r][k] x[j][k] + bias[e][r])
 *             (* (sum_k w_up[e][r][k] x[j][k] + bias_up[e][r]))  (+ residual[j][r])
 *   dtype       MOE_DTYPE_F16 or MOE_DTYPE_BF16, of x, w, w_up, residual and y
 *   x [n_rows][K], y [n_rows][R]; w, w_up (NULL: no second factor) [E][R][K]
 *   bias, bias_up [E][R] fp32 or NULL (bias_up only with w_up)
 *   act         enum moe_act; GELU is v Phi(v), Phi the normal distribution
 *   residual    [n_rows][R] or NULL; it may be y itself (same stride)
 *   expStart    [E+1] int32 device: rows expStart[e]..expStart[e+1]-1 are expert
 *               e's; rows from expStart[E] on are left as they were.  NULL (E == 1
 *               only): every row is expert 0's.  Offsets that do not start at 0,
 *               decrease or pass n_rows set MOE_DEV_BAD_CSR and every row is left.
 * K a multiple of 8, at most 2^24; x and w 16-byte aligned, x_stride a multiple of 8
 * and at least K; y and the residual may lie anywhere (16-byte accesses are used
 * where they fit).  1 <= E <= 1024, 1 <= R, E * R <= 2^31 - 256, 1 <= n_rows < 2^30
 * (MOE_ERR_UNSUPPORTED_SHAPE, as for few rows with more than 2^30 pieces of work).
 * Products are exact and summed in fp32 by the tensor cores (in an order that
 * depends on the sizes, not on the other rows' values); the epilogue is fp32,
 * SiLU within 2^-16 of its value, GELU within 2^-18 above -4 and 2^-15 below (values under
 * 2^-126 may be 0); one rounding to y's type.
 * Few rows (8 an expert, 32 in all; up to 32 of fewer experts where their matrices are
 * small) run on a kernel that reads each touched expert's weights once; more rows on
 * tensor-core tiles of 256 weight rows x up to 256 rows.  What a
 * row holds reaches its own result only, what an expert's weights hold its own rows.
 *   ws: status word (256 bytes); calls on several streams may share it. */
enum moe_act { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3 };

int moe_matmul(const void *x, int64_t x_stride, int dtype, const void *w, const void *w_up, const float *bias,
               const float *bias_up, int act, const void *residual, int64_t residual_stride, const int32_t *expStart,
               int E, int n_rows, int R, int K, void *y, int64_t y_stride, void *ws, size_t ws_bytes,
               cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * moe_ffn_decode -- the whole layer for a decode batch of at most 32 tokens, with
 * 16-bit expert weights as a program holds them (no handle), in one kernel:
 *   l = routerW x[t]; (e_s, w_s) = softmax over all E and top-k of l, as moe_router_topk;
 *   out[t] = sum_s w_s down[e_s] (SiLU(gate[e_s] x[t]) * (up[e_s] x[t]))
 *            (+ sigmoid(shexp_gate . x[t]) shared(x[t]))  (+ residual[t])
 *   dtype       MOE_DTYPE_F16 or MOE_DTYPE_BF16, of x, the expert weights, residual and out
 *   x [N][D], out [N][D], residual [N][D] or NULL (it may be out itself, same stride)
 *   routerW [E][D] fp32; gate, up [E][F][D], down [E][D][F]
 *   sh_gate, sh_up [Fs][D], sh_down [D][Fs]: the shared expert, NULL iff Fs == 0;
 *   shexp_gate [D] fp32, or NULL: the shared expert counts once
 * D, F and Fs multiples of 8, D <= 32768, F, Fs <= 65536; x, the weights, routerW and
 * shexp_gate 16-byte aligned, x_stride a multiple of 8 (or 0); 1 <= top_k <= min(E, 32),
 * E <= 1024, 1 <= N <= 32.
 * Sums are fp32; SiLU(gate) * up, with its weight, enters the second product with 16
 * significant bits (bf16), or within 2^-22 of itself or 2^-39 of the token's largest,
 * whichever is more (fp16); one rounding to out's type.  The order of the sums is fixed for
 * given sizes and device, so a token's row does not depend on the other tokens.
 * An expert whose logit is -inf is not chosen while others are left (and counts 0 then); a
 * NaN or +inf logit, no logit above -inf, or SiLU(gate) * up that is not finite makes its own
 * token's row NaN.  Weights that are not finite reach their experts' tokens only.
 * The kernel takes every SM (a cooperative launch with two grid barriers, each wait
 * limited to a second: MOE_DEV_TIMEOUT, after which out is undefined; when a barrier ran out,
 * every later call on the workspace sets MOE_DEV_TIMEOUT and leaves its out as it was, also
 * when the status has been cleared, until moe_workspace_init).
 *   ws: moe_decode_workspace_size bytes (of N tokens, or more), 256-byte aligned,
 *   initialised once by moe_workspace_init (its status block holds the barriers' 64-bit
 *   arrival count, which runs on from call to call); calls that may overlap, captured
 *   ones among them, must not share one.  A workspace stays on its device. */
size_t moe_decode_workspace_size(int N, int D, int E, int F, int top_k, int Fs);
int moe_ffn_decode(const void *x, int64_t x_stride, int dtype, const float *routerW, const float *shexp_gate,
                   const void *gate, const void *up, const void *down, const void *sh_gate, const void *sh_up,
                   const void *sh_down, const void *residual, int64_t residual_stride, int N, int D, int E, int F,
                   int Fs, int top_k, int norm_topk_prob, void *out, int64_t out_stride, void *ws, size_t ws_bytes,
                   cudaStream_t stream);

/* Failure-detection check of its first grid barrier: moe_ffn_decode with the barrier waiting for one more arrival
 * than there are CTAs, and a limit of limit_ms (1..1000).  Every CTA gives up, MOE_DEV_TIMEOUT is set, out is left as
 * it was and the context stays usable; later calls on the workspace are refused until moe_workspace_init. */
int moe_debug_decode_barrier_timeout(const void *x, int64_t x_stride, int dtype, const float *routerW, const void *gate,
                                     const void *up, const void *down, int N, int D, int E, int F, int top_k, void *out,
                                     int64_t out_stride, int limit_ms, void *ws, size_t ws_bytes, cudaStream_t stream);

/* Device pointers to the intermediates moe_ffn_prefill leaves in `ws`
 * (valid after it ran on that workspace with the same shape); any output
 * pointer may be NULL.  Host pointers to receive device addresses. */
int moe_workspace_views(void *ws, int N, int D, int E, int F, int top_k, int Fs,
                        int32_t **topk_idx, float **topk_w, float **shexp_scale,
                        int8_t **x_q, float **x_d, int32_t **expStart, int32_t **expTokI,
                        int32_t **expTokK, float **partials, float **shared_out);

#ifdef __cplusplus
}
#endif
#endif /* MOE_FFN_H */
