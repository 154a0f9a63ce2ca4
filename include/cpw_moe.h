/*
 * cpw_moe.h -- C ABI of the fused FP8 Mixture-of-Experts layer ("Mega-MoE") on one GPU.
 *
 * One call of moe_forward computes, for every token t,
 *     out[t] = bf16( sum_k  w[t,k] * Expert_{idx[t,k]}(x[t]) ),   idx == -1 skipped,
 * where Expert_e(x) = W_down[e] . requant_1x128( silu(W_gate[e] . x) * (W_up[e] . x) )
 * with FP8 e4m3 operands and fp32 block scales.  The steps follow the fused layer of the
 * source pages, on one GPU whose tokens are split into R logical source partitions:
 *   routing count + packed 64-bit slot claim      ("Mega-MoE 内核代码导读：从 Dispatch 到
 *                                                   WGMMA 的融合流水线" §4.1-4.2)
 *   [expert][source][slot] index table            (same page §4.3; Mega-MoE walkthrough,
 *                                                   part 2, kwkr.cn/news/1317662, §1.1)
 *   expert segments + round-robin min-peeling      (walkthrough part 2 §2.4-2.5)
 *   gather into the expert-major FP8 pool          (walkthrough part 2 §2.6)
 *   grouped FP8 GEMMs gate_up -> SwiGLU -> down    (first page §六, §八)
 *   weighted scatter through {source,token,topk}   ("DeepGEMM Mega MoE 对称内存（Symmetric
 *   metadata + top-k combine reduce                 Memory）深度分析" §8-§9)
 *   Output(T) = sum_k w_k Expert_k(T)              ("Dispatch/Combine: 博客理论 ↔ DeepEP 源码
 *                                                   ↔ DeepGEMM Mega MoE 三方对比分析" §1)
 *
 * Conventions for every call below:
 *   - All tensor pointers are DEVICE pointers unless the name says host; they are
 *     row-major, contiguous, and owned by the caller.  FP8 tensors are e4m3 bytes
 *     (OCP FP8 E4M3, largest finite 448).  FP8 row pointers must be 16-byte aligned.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *   - Every function returns a moe_status code.  Host-detectable problems are returned
 *     synchronously; problems found by the GPU (bad expert id, slot overflow, a wait
 *     that ran past its time limit) are recorded in a sticky per-handle word that
 *     moe_get_error returns; while it is set, forwards skip their work and `out` is
 *     undefined.
 *   - A handle serves one forward at a time: its workspace is shared by its calls.
 */
#ifndef CPW_MOE_H
#define CPW_MOE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_ctx *moe_handle_t;

enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,        /* bad size, null or misaligned pointer            */
    MOE_ERR_CUDA = 2,               /* a CUDA runtime/driver call failed               */
    MOE_ERR_CAPACITY = 3,           /* T above the reserved maximum                    */
    MOE_ERR_NO_WEIGHTS = 4,         /* forward before the weights (routed and shared) are loaded */
    MOE_ERR_UNSUPPORTED_DEVICE = 5, /* not an sm_103 GPU, or a shape this build lacks  */
    MOE_ERR_BAD_INDEX = 6,          /* device: an expert id outside [0,E) other than -1 */
    MOE_ERR_TIMEOUT = 7,            /* device: a bounded wait gave up                  */
    MOE_ERR_SLOT_OVERFLOW = 8,      /* device: > T/R rows of one source for one expert */
    MOE_ERR_NOT_RESERVED = 9,       /* forward before moe_reserve                      */
    MOE_ERR_BAD_SCALE = 10          /* block-scaled mode: a weight scale (at the forward) or
                                       an activation scale (device) is not a power of two;
                                       MXFP4 weights: a NaN scale byte (at load), or a forward
                                       forced to the fp32-scale kernel */
};

/* Create a layer for E experts, hidden size H, expert intermediate size I, top-k, and R
 * logical source partitions (the layer object the pages' Python API builds before its
 * forward: "DeepGEMM Mega MoE 对称内存（Symmetric Memory）深度分析" §10.1).  Requires
 * H % 128 == 0, I % 128 == 0, H <= 16384, I <= 16384, 1 <= topk <= 32, topk <= E <= 1024,
 * 1 <= R <= 64, E*R <= 16384, on the current device, which must be sm_103.  Allocates no
 * device memory.  *out receives the handle. */
int moe_create(int E, int H, int I, int topk, int R, moe_handle_t *out);

/* As moe_create, with n_shared shared experts besides the E routed ones ("DeepGEMM Mega MoE
 * 对称内存（Symmetric Memory）深度分析" §8.2: the combine buffer gets a plane after the top-k
 * ones when shared experts exist, and §10.1 passes their weights separately).  Every token
 * also goes through each shared expert (same H and I as the routed ones), whose output is
 * added to the token's top-k sum with weight 1.  The caller's topk_idx / topk_w stay
 * [T][topk] (routed only); the shared experts' weights come from moe_load_shared_weights.
 * Requires E + n_shared <= 1024, topk + n_shared <= 32, (E + n_shared)*R <= 16384;
 * n_shared = 0 is moe_create. */
int moe_create_shared(int E, int H, int I, int topk, int R, int n_shared, moe_handle_t *out);

/* Allocate the device workspace for up to max_tokens tokens per forward (the pages'
 * host pre-sizing: a larger batch is an error, not a reallocation).  May be called
 * again to grow; not while a forward is in flight. */
int moe_reserve(moe_handle_t h, int max_tokens);

/* Copy the expert weights into the handle (re-laid-out for the GEMMs; the caller keeps
 * ownership of its buffers, which may be freed after the stream has run the copies).
 *   w_gate_up  [E][2I][H] e4m3, rows 0..I-1 = gate, rows I..2I-1 = up
 *   sf_gate_up [E][2I/128][H/128] fp32, one scale per 128x128 block
 *   w_down     [E][H][I] e4m3
 *   sf_down    [E][H/128][I/128] fp32
 * The gate/up rows are interleaved in groups of 8 inside the handle
 * ("DeepGEMM Mega MoE 对称内存（Symmetric Memory）深度分析" §10.2). */
int moe_load_weights(moe_handle_t h, const uint8_t *w_gate_up, const float *sf_gate_up,
                     const uint8_t *w_down, const float *sf_down, void *stream);

/* Weights of the n_shared shared experts, layouts as moe_load_weights with n_shared in
 * place of E.  Required before a forward of a handle made with n_shared > 0;
 * MOE_ERR_INVALID_ARG on a handle without shared experts. */
int moe_load_shared_weights(moe_handle_t h, const uint8_t *w_gate_up, const float *sf_gate_up,
                            const uint8_t *w_down, const float *sf_down, void *stream);

/* Weight formats (moe_info.weight_format). */
enum moe_weight_format {
    MOE_WEIGHTS_FP8 = 0,    /* e4m3 with fp32 128x128 block scales (moe_load_weights)     */
    MOE_WEIGHTS_MXFP4 = 1   /* E2M1 with UE8M0 1x32 scales (moe_load_weights_mxfp4)       */
};

/* MXFP4 expert weights (FP8 activations x FP4 weights: the pages name an FP8 x FP4 variant
 * of the SM100 kernel, "DeepGEMM Mega MoE 对称内存（Symmetric Memory）深度分析" §11, without
 * its format; this is the OCP Microscaling MXFP4 block: 32 consecutive elements of a row
 * share one power-of-two scale).
 *   w_gate_up  [E][2I][H/2] bytes of packed E2M1 codes (element 2j in the low nibble of byte
 *              j, element 2j+1 in the high nibble), rows 0..I-1 = gate, I..2I-1 = up
 *   sf_gate_up [E][2I][H/32] UE8M0 bytes (scale 2^(b-127) of elements 32j..32j+31 of a row)
 *   w_down     [E][H][I/2] packed E2M1
 *   sf_down    [E][H][I/32] UE8M0
 * Weight pointers 16-byte aligned, scale pointers 4-byte aligned.  The forward then runs the
 * block-scaled UMMA with E2M1 weight operands; the activation scales (x_sf) must be powers of
 * two, and MOE_OPT_SCALE_MODE 0 makes moe_forward return MOE_ERR_BAD_SCALE.  A scale byte
 * 0xFF (NaN) makes this call return MOE_ERR_BAD_SCALE and leaves the weights unloaded.
 * Routed and shared weights must be loaded in one format: until they are, moe_forward
 * returns MOE_ERR_NO_WEIGHTS. */
int moe_load_weights_mxfp4(moe_handle_t h, const uint8_t *w_gate_up, const uint8_t *sf_gate_up,
                           const uint8_t *w_down, const uint8_t *sf_down, void *stream);

/* The n_shared shared experts' weights as MXFP4, layouts as moe_load_weights_mxfp4. */
int moe_load_shared_weights_mxfp4(moe_handle_t h, const uint8_t *w_gate_up, const uint8_t *sf_gate_up,
                                  const uint8_t *w_down, const uint8_t *sf_down, void *stream);

/* The layer on T tokens (0 <= T <= max_tokens, T % R == 0; source r owns tokens
 * [r*T/R, (r+1)*T/R)): Output(T) = sum_k w_k Expert_k(T) ("Dispatch/Combine: 博客理论 ↔
 * DeepEP 源码 ↔ DeepGEMM Mega MoE 三方对比分析" §1), by the fused call sequence of "DeepGEMM
 * Mega MoE 对称内存（Symmetric Memory）深度分析" §10.1.  Asynchronous on `stream`.
 *   x        [T][H] e4m3            x_sf [T][H/128] fp32 (1x128 activation scales)
 *   topk_idx [T][topk] int64, -1 = skip this slot
 *   topk_w   [T][topk] fp32 gate weights
 *   out      [T][H] bf16 bits, fully written (a token with no valid slot gets 0). */
int moe_forward(moe_handle_t h, int T, const uint8_t *x, const float *x_sf,
                const int64_t *topk_idx, const float *topk_w, uint16_t *out, void *stream);

/* moe_forward from HOST buffers (same shapes as above), all on `stream`, returning after
 * the stream has finished.  Inputs in pinned (page-locked, device-mapped) memory with
 * 16-byte aligned addresses are read in place by one staging kernel into the handle's
 * device staging buffers; others are copied there by cudaMemcpyAsync.  A pinned, 16-byte
 * aligned `host_out` is written in place by the kernel that completes the combine (with
 * power-of-two scales or MXFP4 weights the FFN kernel itself in the default combine mode, see
 * MOE_OPT_COMBINE_MODE); otherwise the result is
 * copied back from a staging buffer.  Pageable buffers work but are slower. */
int moe_forward_host(moe_handle_t h, int T, const uint8_t *host_x, const float *host_x_sf,
                     const int64_t *host_topk_idx, const float *host_topk_w,
                     uint16_t *host_out, void *stream);

/* As moe_forward_host, but returns once the work is enqueued: the host buffers must stay
 * valid and unchanged, and `host_out` is complete, once `stream` has been synchronized
 * (moe_get_error synchronizes it too).  Forwards enqueued on one stream run in order, so a
 * caller may enqueue the next batch before the previous one has finished. */
int moe_forward_host_async(moe_handle_t h, int T, const uint8_t *host_x, const float *host_x_sf,
                           const int64_t *host_topk_idx, const float *host_topk_w,
                           uint16_t *host_out, void *stream);

/* Wait for the handle's last stream, then return (and clear) the sticky device status in
 * *device_status (a moe_status value; MOE_OK if none).  The pages' kernel stops with an
 * assertion when a bounded wait runs out ("DeepGEMM Mega MoE 对称内存（Symmetric Memory）深度
 * 分析" §6.2); here the kernels record the failure and this call reports it.  Clearing also resets the
 * workspace counters so the next forward starts clean. */
int moe_get_error(moe_handle_t h, int *device_status);

/* Routing results of the last forward (host copies, after syncing its stream), i.e. the
 * per-expert counts, expert segments and pool metadata of "Mega-MoE walkthrough part 2"
 * (kwkr.cn/news/1317662) §2.4-2.6:
 *   counts [E] rows per expert, recv [E][R] rows per (expert, source),
 *   block_offset [E+1] first M-block of each expert in the pool (last = total blocks),
 *   meta [P][3] {source, token, topk slot} of every pool row (rows past an expert's
 *   count hold padding), *P = pool rows used = block_offset[E] * block_m,
 *   *block_m = rows per M-block.  Any output pointer may be NULL.  meta needs room for
 *   the pool rows of the last forward: (ceil(T*topk/block_m) + E) * block_m rows. */
int moe_debug_routing(moe_handle_t h, uint32_t *counts, uint32_t *recv, int32_t *block_offset,
                      uint32_t *meta, int *P, int *block_m);

/* Per-expert routed rows accumulated over every forward since the handle was created
 * (host copy, [E]). */
int moe_cumulative_expert_rows(moe_handle_t h, uint64_t *rows);

/* Host copy of an intermediate buffer of the last forward (for stage-by-stage tests):
 *   MOE_BUF_POOL_X   [P][H] e4m3 gathered rows      MOE_BUF_POOL_SF [H/128][P] fp32
 *   MOE_BUF_ACT      [P][I] e4m3 SwiGLU output      MOE_BUF_ACT_SF  [I/128][P] fp32
 *   MOE_BUF_COMBINE  [topk][T][H] bf16 weighted expert outputs
 *   MOE_BUF_TABLE    [E][R][max_tokens/R] int32 index table (token_in_source*topk + k)
 * where P is the reserved pool row capacity (moe_info).  `bytes` must equal the
 * buffer's size; returns MOE_ERR_INVALID_ARG otherwise. */
enum moe_buffer {
    MOE_BUF_POOL_X = 0, MOE_BUF_POOL_SF = 1, MOE_BUF_ACT = 2, MOE_BUF_ACT_SF = 3,
    MOE_BUF_COMBINE = 4, MOE_BUF_TABLE = 5
};
int moe_debug_buffer(moe_handle_t h, int which, void *host_dst, uint64_t bytes);

/* Sizes and launch shape of the handle. */
typedef struct moe_info {
    int E, H, I, topk, R;
    int max_tokens;       /* reserved tokens per forward                     */
    int pool_rows;        /* reserved pool row capacity P                    */
    int block_m;          /* rows per M-block (GEMM tile rows)               */
    int block_n;          /* GEMM tile columns                               */
    int num_sms;          /* persistent grid size                            */
    uint64_t workspace_bytes;
    uint64_t weight_bytes;
    int n_shared;         /* shared experts; E and topk above include them: shared expert s
                             is expert slot E - n_shared + s and combine plane
                             topk - n_shared + s (the debug buffers use these sizes) */
    int weight_format;    /* moe_weight_format of the routed weights last loaded          */
} moe_info;
int moe_get_info(moe_handle_t h, moe_info *info);

/* Options.  MOE_OPT_TIMEOUT_NS: time limit of every device-side wait (default 2e9 ns);
 * MOE_OPT_DEBUG_SKIP_BARRIER: when 1, one CTA of the routing kernel skips its arrival
 * at the grid barrier, so the others give up after the time limit and the forward
 * ends with MOE_ERR_TIMEOUT (failure-path test; never on in normal use);
 * MOE_OPT_FFN_MODE: how the expert FFN kernel covers its tiles: 0 = automatic (default) and
 * 1 = one CTA per 128-row tile, which are the same kernel; other values are refused;
 * MOE_OPT_SCALE_MODE: 0 = arbitrary fp32 block scales (the UMMA accumulates each 128-deep
 * K block in TMEM and the scales are applied on the CUDA cores); 1 = every scale (x_sf, both
 * weight scale tensors) is a power of two: the UMMA applies them itself as UE8M0 scale
 * factors and accumulates the whole K range in TMEM ("DeepGEMM Mega MoE 对称内存
 * （Symmetric Memory）深度分析" §8.1), and the SwiGLU requant uses the smallest power-of-two
 * scale >= max(amax, 1e-4)/448; 2 = automatic (default): mode 1 when every scale of the
 * loaded weights is a power of two (checked by moe_load_weights), else mode 0.  In mode 1
 * weights that are not all powers of two make moe_forward return MOE_ERR_BAD_SCALE; in
 * modes 1 and 2 an activation scale that is not, on the block-scaled path, is reported by
 * the device the same way (sticky);
 * MOE_OPT_COMBINE_MODE: where the top-k combine runs ("DeepGEMM Mega MoE 对称内存（Symmetric
 * Memory）深度分析" §9: the per-token fp32 reduce of the top-k expert outputs).  0 = a
 * separate kernel after the expert FFN kernel; 1 = inside the expert FFN kernel: a down tile's
 * scattered rows are counted per (token, 256-column n-tile), and the epilogue warps reduce every
 * (token, n-tile) whose routed rows are all scattered while other tiles are still being
 * computed (the forward is then two kernels, three with shared experts); 2 = automatic
 * (default): 1 when a host-buffer entry point writes the output into pinned host memory in
 * place and the block-scaled FFN kernel runs (power-of-two scales or MXFP4 weights: its rows
 * then cross to the host while the GEMMs still run), else 0 (with arbitrary fp32 scales the
 * reduce would lengthen the FFN kernel's critical epilogue more than it saves).  All modes
 * give the same output bits.  Other values are refused. */
enum moe_option {
    MOE_OPT_TIMEOUT_NS = 0,
    MOE_OPT_DEBUG_SKIP_BARRIER = 1,
    MOE_OPT_FFN_MODE = 2,
    MOE_OPT_SCALE_MODE = 3,
    MOE_OPT_COMBINE_MODE = 4
};
int moe_set_option(moe_handle_t h, int option, int64_t value);

/* Stage timing with CUDA events recorded on the forward's own stream.  enable = N > 0:
 * the 1st, (N+1)-th, (2N+1)-th ... moe_forward from now records an event before and after
 * each of its three kernels (dispatch; expert FFN = gate_up GEMM + SwiGLU + down GEMM +
 * weighted scatter; combine) — N > 1 samples the forwards, so the events (which serialise
 * the kernels they sit between) disturb only one step in N; enable = 0 stops.  With the
 * combine inside the FFN kernel the combine stage brackets no kernel (its time is ~0 and the
 * FFN stage includes the reduce).
 * moe_profile_read waits for the last stream, returns the summed milliseconds of each
 * stage over the recorded forwards in stage_ms[3] and their number in *calls, and starts
 * a new window.  At most 8192 forwards are recorded per window (later ones are counted in
 * *dropped, not timed). */
int moe_profile_enable(moe_handle_t h, int enable);
int moe_profile_read(moe_handle_t h, double *stage_ms, int *calls, int *dropped);

/* Routing without any device allocation, for callers that may not allocate GPU memory
 * themselves or through this library (code running under another framework's memory
 * pool or a fixed memory budget, real-time loops that must stay out of the allocator,
 * plug-ins whose host owns every allocation).  The pages have no counterpart: it is a
 * deployment convenience, not a step of the method.  It needs no handle and no weights.
 * It computes what moe_debug_routing reports after a forward: counts [E], recv [E][R],
 * block_offset [E+1] (M-blocks of 128 rows) and, for every received row, its pool row's
 * {source, token, topk slot} in meta [(ceil(T*topk/128) + E) * 128][3] (padding rows are
 * left untouched), plus *status (device int32: MOE_OK, MOE_ERR_BAD_INDEX or
 * MOE_ERR_SLOT_OVERFLOW; on an error the other outputs are left untouched).  All pointers
 * are device pointers owned by the caller; topk_idx is [T][topk] int64 with -1 = skip.
 * Scratch (slot counters and the index table) lives in one fixed array of about 4 MB per
 * GPU, kept until the process exits; sizes beyond it return MOE_ERR_CAPACITY: at most
 * E*R <= 4096, T*topk <= 131072 and E*T <= 1048576 (plus the moe_create limits on E, topk
 * and R, and T % R == 0).  The first call on a device looks up that array's device
 * address and should come before any stream capture; the address is kept until the process
 * exits, so the entry point must not be used on a device after that device was reset
 * (cudaDeviceReset).  Asynchronous on `stream`, which must belong to the current device
 * (MOE_ERR_INVALID_ARG otherwise); calls that overlap on the GPU share the scratch and race. */
int moe_route_noalloc(int T, int E, int topk, int R, const int64_t *topk_idx, uint32_t *counts,
                      uint32_t *recv, int32_t *block_offset, uint32_t *meta, int32_t *status,
                      void *stream);

/* ---------------------------------------------------------------------------------------
 * Operators around the expert layer, for training a block and for feeding the layer above:
 * layer and RMS norm, routers with their gradients, rows into and out of expert order, products
 * with one weight per expert over ragged groups of rows, the experts' activation and 8-bit checkpoints.  They need no handle; the caller owns
 * every buffer, workspaces included (the *_workspace calls say how many bytes).  All are
 * asynchronous on `stream`, which belongs to the current device, an sm_103 GPU
 * (MOE_ERR_UNSUPPORTED_DEVICE otherwise), allocate nothing, and may be captured into a graph.
 * The source pages have no counterpart of them.
 *
 * Pointers are device pointers aligned to their element type unless a call asks for more; a row
 * stride (ld...) counts elements and is at least the row's length; other tensors are contiguous.
 * Results and workspaces share no memory with the inputs (an accumulating dw is its own).
 * T, M, T*topk and the rows' H are at most 2^30.
 * Calls with T == 0 (or M == 0) do nothing but write the results that an empty batch has (zero
 * gradients of weights, zero offsets). */

/* Element types. */
enum moe_dtype { MOE_F32 = 0, MOE_BF16 = 1, MOE_F16 = 2 };

/* Layer norm of each of T rows: y = (x - mean) * rstd * weight + bias with the biased variance
 * and rstd = 1 / sqrt(var + eps); statistics in fp32, y [T][H] of x's type.  weight and bias
 * [H] are of w_dtype (x's type or MOE_F32), either may be NULL; mean and rstd [T] fp32 (NULL:
 * not written) are what the backward call reads.  1 <= H <= 16384. */
int moe_layer_norm(int T, int H, const void *x, int64_t ldx, int dtype, const void *weight, const void *bias,
                   int w_dtype, float eps, void *y, float *mean, float *rstd, void *stream);

/* Layer norm written as the FP8 rows and 1x128 scales that moe_forward reads: q [T][H] e4m3,
 * sf [T][H/128] = max(amax, 1e-4) / 448 of each group of 128, or with pow2_scales = 1 the
 * smallest power of two at or above it (what the block-scaled kernel needs).  Codes are y times the scale's reciprocal: beside scales that
 * are no powers of two they may be one step off the quotient's.  H % 128 == 0;
 * x, weight, bias and q 16-byte aligned, rows of x too. */
int moe_layer_norm_fp8(int T, int H, const void *x, int64_t ldx, int dtype, const void *weight, const void *bias,
                       int w_dtype, float eps, int pow2_scales, uint8_t *q, float *sf, void *stream);

/* Gradients of moe_layer_norm: dx [T][H] of x's type, and the sums over the rows dweight and
 * dbias [H] of w_dtype (either may be NULL).  weight may be NULL (all ones).  Sums in fp32, in a
 * fixed order on one kind of GPU: equal inputs give equal bits.  The workspace is needed when
 * dweight or dbias is asked for (16-byte aligned). */
int moe_layer_norm_backward_workspace(int T, int H, uint64_t *bytes);
int moe_layer_norm_backward(int T, int H, const void *dy, int64_t lddy, const void *x, int64_t ldx, int dtype,
                            const void *weight, int w_dtype, const float *mean, const float *rstd, void *dx,
                            void *dweight, void *dbias, void *workspace, uint64_t workspace_bytes, void *stream);

/* The router: the topk largest logits of each token ([T][E], rows ld apart), in descending order,
 * ties to the lowest expert, and their gate weights: the softmax over the chosen experts
 * (renormalize = 1) or over all of them (0).  topk_idx and topk_w [T][topk] are moe_forward's.  A logit
 * of -inf is never chosen: a token with fewer others gets idx -1 and weight 0 in the slots left
 * over.  A NaN counts as the largest value and makes the token's weights NaN.  token_mask [T]
 * (bytes; NULL: all ones) is 0 for a token that is not routed: idx -1 and weight 0 throughout,
 * whatever its logits hold.  E <= 1024, topk <= 32, topk <= E. */
int moe_route_topk(int T, int E, int topk, const void *logits, int64_t ld, int dtype, const uint8_t *token_mask,
                   int renormalize, int64_t *topk_idx, float *topk_w, void *stream);

/* Gradient of the logits ([T][E], of `dtype`) from that of the gate weights, dw [T][topk] fp32, with the
 * indices and weights that the forward call gave.  The choice itself is constant.  logits is
 * read only with renormalize = 0 (may be NULL with 1).  dw in a slot of index -1 is not read. */
int moe_route_topk_backward(int T, int E, int topk, const float *dw, const int64_t *topk_idx, const float *topk_w,
                            const void *logits, int64_t ld, int dtype, int renormalize, void *dlogits, void *stream);

/* Expert-major order of the T*topk slots: by expert, then token, then slot.  offsets [E+1] (expert
 * e has rows offsets[e] .. offsets[e+1]) and rows [T][topk], the row of each slot or -1 for a
 * skipped one.  *status (device int32) is MOE_OK, or MOE_ERR_BAD_INDEX if an id is neither -1
 * nor in [0, E); such a slot is skipped.  E <= 1024, topk <= 32. */
int moe_expert_order_workspace(int T, int topk, int E, uint64_t *bytes);
int moe_expert_order(int T, int topk, int E, const int64_t *topk_idx, int32_t *offsets, int32_t *rows,
                     int32_t *status, void *workspace, uint64_t workspace_bytes, void *stream);

/* out[rows[t][j]] = x[t] for every slot with a row in [0, M); the rows of out [M][H] from
 * offsets[E] on are zeroed.  rows and offsets are an order as moe_expert_order gives it: every row
 * before offsets[E] has its slot (one that had none would keep what out held), none from there on has.  Its gradient is moe_combine_rows with w = NULL. */
int moe_gather_rows(int T, int topk, int H, int E, int64_t M, const void *x, int64_t ldx, int dtype,
                    const int32_t *rows, const int32_t *offsets, void *out, void *stream);

/* out[t] = sum over j of w[t][j] * y[rows[t][j]], in fp32 with j ascending, rounded once to y's
 * type; slots without a row in [0, M) are left out (their w and y are not read).  w = NULL: ones. */
int moe_combine_rows(int T, int topk, int H, int64_t M, const void *y, int dtype, const int32_t *rows, const float *w,
                     void *out, void *stream);

/* Gradients of moe_combine_rows: dy[rows[t][j]] = w[t][j] * dout[t] (rows of dy [M][H] from offsets[E]
 * on are zeroed; rows and offsets as in moe_gather_rows) and dw[t][j] = <dout[t], y[rows[t][j]]> (0 in a slot without a row; NULL: not
 * written).  No two slots may have the same row. */
int moe_combine_rows_backward(int T, int topk, int H, int E, int64_t M, const void *dout, int64_t lddout, const void *y,
                              int dtype, const int32_t *rows, const float *w, const int32_t *offsets, void *dy,
                              float *dw, void *stream);

/* Products with one weight per expert, w [E][N][K], over rows in expert order (16-bit types
 * MOE_BF16 and MOE_F16, fp32 accumulation): for the rows r of expert e,
 *   moe_grouped_mm     out[r][n] = sum_k x[r][k] w[e][n][k]         x [M][K], out [M][N]
 *   moe_grouped_mm_dx  dx[r][k]  = sum_n dy[r][n] w[e][n][k]        dy [M][N], dx [M][K]
 *   moe_grouped_mm_dw  dw[e][n][k] = sum_r dy[r][n] x[r][k]         dw [E][N][K] of dtype or MOE_F32,
 *                      added to what dw holds if accumulate = 1; an expert without rows gets 0
 * offsets [E+1] is read by the GPU and taken as the non-decreasing sequence max(0, min(M, offsets))
 * that its running maximum gives, so no value of it leads out of the tensors; rows of out and dx
 * that belong to no expert are zeroed.  N and K multiples of 8 up to 2^20, E <= 1024, tensors
 * 16-byte aligned, row strides multiples of 8; workspaces 128-byte aligned.  moe_grouped_mm and
 * moe_grouped_mm_dx need theirs (one size serves both) where a small batch is split along the
 * contraction; 0 bytes otherwise.  Results do not depend on anything but the arguments: equal
 * inputs give equal bits.  The tensor core adds products to a 32-bit sum
 * by truncation, so an fp32 dw is about 1e-6 off over a thousand rows and 2e-5 over 16000. */
int moe_grouped_mm_workspace(int64_t M, int E, int N, int K, uint64_t *bytes);
int moe_grouped_mm(int64_t M, int E, int N, int K, const void *x, int64_t ldx, const void *w, const int32_t *offsets,
                   void *out, int64_t ldo, int dtype, void *workspace, uint64_t workspace_bytes, void *stream);
int moe_grouped_mm_dx(int64_t M, int E, int N, int K, const void *dy, int64_t lddy, const void *w, const int32_t *offsets,
                      void *dx, int64_t lddx, int dtype, void *workspace, uint64_t workspace_bytes, void *stream);
int moe_grouped_mm_dw_workspace(int64_t M, int E, int N, int K, uint64_t *bytes);
int moe_grouped_mm_dw(int64_t M, int E, int N, int K, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                      const int32_t *offsets, void *dw, int dtype, int dw_dtype, int accumulate, void *workspace,
                      uint64_t workspace_bytes, void *stream);

/* RMS norm of each of T rows with the residual's addition: h = x + residual, rounded to their type (the
 * residual stream, written to h [T][H]; without a residual, NULL, h is not written and stands for x),
 * rstd = 1 / sqrt(sum(h^2)/H + eps) in fp32, y = h * rstd * weight [T][H] of x's type.  weight [H] is of
 * w_dtype (x's type or MOE_F32) or NULL; rstd [T] fp32 (NULL: not written) is what the backward call reads.
 * 1 <= H <= 16384. */
int moe_rms_norm(int T, int H, const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, const void *weight,
                 int w_dtype, float eps, void *h, void *y, float *rstd, void *stream);

/* The same written as the FP8 rows and 1x128 scales that moe_forward reads (see moe_layer_norm_fp8).
 * H % 128 == 0; x, residual, weight, h and q 16-byte aligned, rows of x and residual too. */
int moe_rms_norm_fp8(int T, int H, const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, const void *weight,
                     int w_dtype, float eps, int pow2_scales, void *h, uint8_t *q, float *sf, void *stream);

/* Gradients of moe_rms_norm from h (x where there was no residual): dx [T][H] of its type, of x and of the
 * residual alike, dh [T][H] (the gradient of h from elsewhere; NULL: none) added to it, and the sums
 * over the rows dweight [H] of w_dtype (may be NULL).  Sums as in moe_layer_norm_backward; the workspace
 * is needed when dweight is asked for (16-byte aligned). */
int moe_rms_norm_backward_workspace(int T, int H, uint64_t *bytes);
int moe_rms_norm_backward(int T, int H, const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *dh, int64_t lddh,
                          int dtype, const void *weight, int w_dtype, const float *rstd, void *dx, void *dweight, void *workspace,
                          uint64_t workspace_bytes, void *stream);

/* The router over scores s of the logits ([T][E], rows ld apart): sigmoid, or softmax over all experts.
 * The choice goes by c = s + bias (fp32 [E], NULL: none).  With groups > 1, of E/groups neighbouring
 * experts each, a group's score is the sum of its group_top (1 or 2) largest c (of the one, where but one
 * of its experts can be chosen; a group with none is left out), the topk_groups best groups stay, and the
 * topk experts with the largest c are chosen from theirs, in descending order; ties go to the lowest group
 * and expert.  c and its sums are compared as computed in 64 bits (without a bias, unless sums of two choose
 * among the groups, as the logits are): the lowest finite logit has a score of 0.  The gate weights are scale * s, or with renormalize = 1 scale * s / sum of s over the chosen ones.  -inf, NaN, fewer
 * candidates than topk, and token_mask as in moe_route_topk (a bias of -inf excludes its expert).
 * E <= 1024, topk <= 32, groups <= 32 and a divisor of E, topk <= topk_groups * E/groups, scale finite and
 * not 0. */
enum moe_score { MOE_SCORE_SIGMOID = 0, MOE_SCORE_SOFTMAX = 1 };
int moe_route_scores(int T, int E, int topk, const void *logits, int64_t ld, int dtype, int score, const float *bias, int groups,
                     int topk_groups, int group_top, const uint8_t *token_mask, int renormalize, float scale, int64_t *topk_idx,
                     float *topk_w, void *stream);

/* Gradient of the logits ([T][E], of `dtype`) from that of the gate weights, dw [T][topk] fp32, with the
 * indices and weights that the forward call gave, and its score, renormalize and scale.  The choice is
 * constant.  logits is not read for renormalised softmax scores (may be NULL).  dw in a slot of
 * index -1 is not read. */
int moe_route_scores_backward(int T, int E, int topk, const float *dw, const int64_t *topk_idx, const float *topk_w,
                              const void *logits, int64_t ld, int dtype, int score, int renormalize, float scale, void *dlogits,
                              void *stream);

/* The experts' activation over rows of gate and up, gu [M][2*I] (gate first): act = silu(gate) * up, [M][I],
 * in fp32 and rounded once (0 for gates below -88.7, where exp(-gate) is past fp32).  With codes and scales (both or neither) gate and up are also kept in 8 bits
 * for the backward call: codes [M][2*I], scales [M][2*ceil(I/32)].  The format (of MX blocks with INT8
 * elements): 32 neighbours of a row (of gate, of up; the last group may be shorter) have a byte b, and a code n
 * stands for n * 2^(b - 133); b = 127 + floor(log2 of the largest magnitude), at least 7; n is the nearest in
 * -127 .. 127, ties to even.  A NaN or an infinity makes its group NaN (b = 255). */
int moe_swiglu(int64_t M, int I, const void *gu, int64_t ldg, int dtype, void *act, int8_t *codes, uint8_t *scales, void *stream);

/* Gradient of moe_swiglu's gate and up, dgu [M][2*I] of `dtype`, from dact [M][I] and either gu or the codes
 * and scales that stand for it (the other NULL); act [M][I] (NULL: not wanted) gets the activation again. */
int moe_swiglu_backward(int64_t M, int I, const void *dact, int64_t ldd, const void *gu, int64_t ldg, const int8_t *codes,
                        const uint8_t *scales, int dtype, void *dgu, void *act, void *stream);

/* Rows x [M][H] in the 8-bit format of moe_swiglu, codes [M][H] and scales [M][ceil(H/32)], and back (any byte
 * and code; rounded to `dtype`).  M <= 2^30, and H and I <= 2^20 here and in the calls above. */
int moe_checkpoint_rows(int64_t M, int H, const void *x, int64_t ldx, int dtype, int8_t *codes, uint8_t *scales, void *stream);
int moe_restore_rows(int64_t M, int H, const int8_t *codes, const uint8_t *scales, int dtype, void *x, void *stream);

/* Waits for `stream`, then returns and clears the sticky status of the operators' device-side
 * waits on the current device: MOE_OK, or MOE_ERR_TIMEOUT if a wait of a grouped product ran
 * past its limit (2 s, and 2 us for each 64 of the contraction; its outputs are then undefined).  The
 * status is the device's, not a stream's or a thread's: who asks first has it, and clears it for all.  Not inside a stream capture. */
int moe_ops_get_error(int *device_status, void *stream);

/* Release every device buffer of the handle (after syncing its last stream): the teardown
 * of the buffers the layer object of "DeepGEMM Mega MoE 对称内存（Symmetric Memory）深度分析"
 * §10.1 allocates. */
int moe_destroy(moe_handle_t h);

/* Static description of a status code. */
const char *moe_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* CPW_MOE_H */
