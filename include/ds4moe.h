/*
 * ds4moe.h -- C ABI of libds4moe: the routed mixture-of-experts FFN of one
 * DeepSeek-V4-Flash-shaped layer on one GB300 GPU (sm_103a).
 *
 * What the layer computes (by page title and section):
 *   - "DeepSeek V4 Flash -- DFlash Integration", Model Architecture: hidden
 *     4096; 256 routed experts, top-6, plus 1 shared; expert FFN 2048; the
 *     first 3 layers route by a token-ID -> expert table, the others by
 *     "top-k over learned router + optional bias"; Execution Modes
 *     (--ds4-expert-top-k): the kept experts' weights are renormalised.
 *   - "Baekpica/ds4 dfm Edition" README, two-bank batching notes: the router
 *     returns selected expert IDs and normalized weights; the expert path is
 *     gate/up, weighted SwiGLU, expert down, plus the shared expert.
 *   - DwarfStar README, Model Weights: routed experts 2-bit, shared experts
 *     and router kept at higher precision (Q8_0, "SExpQ8").
 *   - ds4-rocm fork README, __launch_bounds__ list: activations are
 *     pre-quantised to int8 for the Q8_0 matmuls ("_preq" kernels).
 *
 * Every float operation follows one fixed binary32 order (the canonical
 * arithmetic spec): the library's results are bit-identical to a scalar
 * CPU evaluation of the same spec, for every token count and every code path.
 *
 * Conventions for every entry point:
 *   - Pointers are CUDA device pointers unless the name says host.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).
 *   - Argument and shape errors are detected on the host before anything is
 *     enqueued; the call then returns an error status and changes nothing.
 *   - ds4moe_route / ds4moe_forward enqueue work only: no allocation, no
 *     host synchronisation, so they may be captured in a CUDA graph.
 *   - Data errors found on the device (a hash token id outside [0, vocab),
 *     a non-finite activation) never trap: the device sets a flag that
 *     ds4moe_get_device_error reports; an out-of-range token contributes
 *     nothing to y.
 *   - One handle must not be used on two streams at once; distinct handles
 *     are independent.
 */
#ifndef DS4MOE_H
#define DS4MOE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DS4MOE_ABI_VERSION 1

typedef enum {
  DS4MOE_OK = 0,
  DS4MOE_ERR_INVALID_ARG = 1, /* bad pointer, shape, format or token count */
  DS4MOE_ERR_UNSUPPORTED = 2, /* valid request the library does not handle */
  DS4MOE_ERR_OOM = 3,         /* device allocation failed                  */
  DS4MOE_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed      */
  DS4MOE_ERR_DEVICE = 5       /* the device error flag was set             */
} ds4moe_status;

/* Weight formats (canonical byte layouts; all little endian).
 *   DS4MOE_F32  : row-major binary32 (router only).
 *   DS4MOE_Q8_0 : blocks of 32 weights, 34 bytes: fp16 d, int8 q[32];
 *                 w_i = d * q_i.
 *   DS4MOE_Q2S  : superblocks of 256 weights, 84 bytes:
 *                 uint8 sm[16] | uint8 qs[64] | fp16 d | fp16 dmin;
 *                 group g = i/16, sc = sm[g] & 15, mn = sm[g] >> 4,
 *                 q_i = (qs[i/4] >> 2*(i%4)) & 3,
 *                 w_i = d*sc*q_i - dmin*mn   (2.625 bits per weight).
 *   DS4MOE_Q4S  : superblocks of 256 weights, 148 bytes (routed experts of
 *                 the 4-bit layers; this library's own layout -- the DwarfStar
 *                 README, Model Weights, names a "q2 with the last 6 layers
 *                 q4" variant but not its bytes):
 *                 uint8 sm[16] | uint8 qs[128] | fp16 d | fp16 dmin;
 *                 group g = i/16, sc = sm[g] & 15, mn = sm[g] >> 4,
 *                 q_i = (qs[i/2] >> 4*(i%2)) & 15,
 *                 w_i = d*sc*q_i - dmin*mn   (4.625 bits per weight).
 * A matrix [R][K] is R rows of K/32 (Q8_0) or K/256 (Q2S, Q4S) blocks, rows
 * contiguous; expert tensors stack their E matrices contiguously. */
typedef enum { DS4MOE_F32 = 0, DS4MOE_Q8_0 = 1, DS4MOE_Q2S = 2, DS4MOE_Q4S = 3 } ds4moe_fmt;

typedef enum { DS4MOE_ROUTE_LEARNED = 0, DS4MOE_ROUTE_HASH = 1 } ds4moe_route_kind;

/* Element types of activations (and of 16-bit weights and caches). */
typedef enum { DS4MOE_DT_F32 = 0, DS4MOE_DT_BF16 = 1, DS4MOE_DT_F16 = 2 } ds4moe_dtype;

/* Device error flag bits (ds4moe_get_device_error). */
#define DS4MOE_DEVERR_TOKEN_ID 1u   /* hash token id outside [0, vocab)     */
#define DS4MOE_DEVERR_NONFINITE 2u  /* non-finite activation quantised      */
#define DS4MOE_DEVERR_TIMEOUT 4u    /* a bounded on-chip wait gave up       */
#define DS4MOE_DEVERR_INTERNAL 8u   /* an internal consistency check failed */
#define DS4MOE_DEVERR_PAGE 16u      /* block-table entry outside the cache  */
#define DS4MOE_DEVERR_LENGTH 32u    /* length or count outside its buffers  */
#define DS4MOE_DEVERR_ADAPTER 64u   /* adapter slot outside [-1, n_slots)   */

typedef struct {
  uint32_t abi_version; /* = DS4MOE_ABI_VERSION */
  int32_t hidden;       /* H: multiple of 256 (4096 for DeepSeek-V4-Flash)          */
  int32_t n_experts;    /* E routed experts, 1..1024 (256)                          */
  int32_t top_k;        /* k, 1..min(E, 16) (6)                                     */
  int32_t ffn;          /* F: multiple of 64; of 256 with Q2S/Q4S matrices (2048)   */
  int32_t n_shared;     /* 0 or 1 shared expert, always added with weight 1         */
  int32_t route;        /* ds4moe_route_kind                                        */
  int32_t vocab;        /* hash routing: table rows (129280); ignored otherwise     */
  int32_t router_fmt;   /* DS4MOE_F32 or DS4MOE_Q8_0 (learned routing)              */
  int32_t routed_fmt;   /* DS4MOE_Q8_0, DS4MOE_Q2S or DS4MOE_Q4S                    */
  int32_t shared_fmt;   /* DS4MOE_Q8_0, DS4MOE_Q2S or DS4MOE_Q4S                    */
  float route_scale;    /* multiplies the renormalised routed weights (1.0)         */
  int32_t max_tokens;   /* largest n_tok of any later call, 1..1048576. A call of   */
                        /* fewer than 65 tokens runs on the decode path in chunks  */
                        /* of at most 64 tokens; a larger one (when hidden and ffn */
                        /* are multiples of 128) on the prefill path in chunks of  */
                        /* at most 4096 tokens. Scratch is sized at create for     */
                        /* Ts = max(min(max_tokens, 64), min(max_tokens, 4096))    */
                        /* tokens: about 560 MB at 4096 tokens and the DS4 shape   */
} ds4moe_layer_desc;

/* Canonical weight buffers, DEVICE memory, read only during ds4moe_create
 * (the library keeps its own re-laid-out copy; the caller may free these
 * when create returns). Unused pointers may be NULL. */
typedef struct {
  const void *router_w;       /* [E][H] router_fmt                (learned)   */
  const float *router_bias;   /* [E] selection bias               (learned)   */
  const int32_t *hash_table;  /* [vocab][k] expert ids in [0, E)  (hash)      */
  const void *gate, *up;      /* [E][F][H] routed_fmt                         */
  const void *down;           /* [E][H][F] routed_fmt                         */
  const void *sh_gate, *sh_up;/* [F][H] shared_fmt                (n_shared)  */
  const void *sh_down;        /* [H][F] shared_fmt                (n_shared)  */
} ds4moe_weights;

typedef struct ds4moe_layer ds4moe_layer; /* opaque handle */

/* Validate `desc`, allocate the handle's device memory on the current device
 * (weights in the library's layout plus scratch for one chunk of tokens),
 * re-lay out the weights, and synchronise. On success *out owns all of it;
 * on error *out is NULL and nothing stays allocated.
 * Errors: INVALID_ARG (desc, missing or non-device pointer), UNSUPPORTED
 * (a shape whose kernels do not fit one SM, e.g. more than ~700 experts),
 * OOM, CUDA. */
ds4moe_status ds4moe_create(const ds4moe_layer_desc *desc, const ds4moe_weights *w,
                            ds4moe_layer **out);

/* Release everything the handle owns (synchronises the device). NULL is a no-op. */
void ds4moe_destroy(ds4moe_layer *h);

/* Routing only (steps: int8 quantisation of x, router GEMV, sigmoid,
 * bias-for-selection top-k, renormalisation; or the hash-table lookup).
 * Passages: "DeepSeek V4 Flash -- DFlash Integration", Model Architecture
 * (routed experts chosen by top-k over a learned router plus an optional
 * bias; the first layers route by a token-ID table) and Execution Modes
 * (--ds4-expert-top-k: the kept experts' weights are renormalised).
 *   x        [n_tok][H] fp32 (learned routing; may be NULL for hash)
 *   token_ids[n_tok] int32 (hash routing; may be NULL for learned)
 *   ids_out  [n_tok][k] int32: expert ids in descending key order
 *            (hash: table order); -1 for an out-of-range token id
 *   w_out    [n_tok][k] fp32: renormalised weights * route_scale (0 for -1)
 * n_tok in 0..max_tokens. Enqueued on `stream`. */
ds4moe_status ds4moe_route(ds4moe_layer *h, const float *x, const int32_t *token_ids, int32_t n_tok,
                           int32_t *ids_out, float *w_out, void *stream);

/* Routing without a handle and without any device allocation.
 * No counterpart in the pages: they describe no allocation-free entry point.
 * It exists for callers that cannot call cudaMalloc: plug-ins and embedders
 * whose host application owns all device memory (for example a serving engine
 * that reserves the GPU's memory up front and accounts for every byte, so an
 * allocation behind its back fails or breaks its budget), and code paths that
 * cannot afford cudaMalloc's implicit device-wide synchronisation.
 *
 * Computes exactly what ds4moe_route computes (same ids, same weight bits)
 * from the caller's canonical buffers, read on every call:
 *   desc: hidden, n_experts, top_k, route, vocab, router_fmt and route_scale
 *         are used (same rules as ds4moe_create); the other fields are ignored.
 *   w:    router_w + router_bias (learned) or hash_table (hash), device memory;
 *         other members are ignored.
 *   x, token_ids, ids_out, w_out: as for ds4moe_route.
 *   err_flags: device uint32, may be NULL; DS4MOE_DEVERR_* bits are OR-ed in
 *         (a hash-table entry outside [0, n_experts) gives id -1, weight 0
 *         and DS4MOE_DEVERR_INTERNAL).
 * Scratch: one fixed device array of DS4MOE_NOALLOC_SCRATCH_BYTES (512 KiB)
 * per device, built into the library. Learned routing needs
 * n_tok * 32 * E_pad bytes of it (E_pad = n_experts rounded up to 32): at most
 * 64 tokens per call for 256 experts. A larger n_tok returns
 * DS4MOE_ERR_UNSUPPORTED and enqueues nothing. Hash routing uses no scratch.
 * Nothing in the array has to start at zero; a call reads only what it wrote.
 * Every call on a device shares the one array, so calls whose work can
 * overlap on the GPU (issued on different streams without an order between
 * them, or from several host threads) race and give wrong results: issue
 * them on one stream, or order them.
 * The first call on each device, with that device current, looks up the
 * array's address (cudaGetSymbolAddress) and sets a kernel attribute; make
 * that first call before any stream capture.
 * Errors: INVALID_ARG (desc, pointers, n_tok < 0), UNSUPPORTED (scratch too
 * small for n_tok), CUDA. */
#define DS4MOE_NOALLOC_SCRATCH_BYTES (512u * 1024u)
ds4moe_status ds4moe_route_noalloc(const ds4moe_layer_desc *desc, const ds4moe_weights *w, const float *x,
                                   const int32_t *token_ids, int32_t n_tok, int32_t *ids_out, float *w_out,
                                   uint32_t *err_flags, void *stream);

/* The whole layer: y[t] += MoE(x[t]) for t < n_tok, i.e.
 * Passages: "DeepSeek V4 Flash -- DFlash Integration", Model Architecture
 * (256 routed experts top-6 plus 1 shared, expert FFN 2048) and Forward Pass
 * (the MoE FFN adds its output to the residual stream); "Baekpica/ds4 dfm
 * Edition" README, two-bank batching notes (router -> top-k -> gate/up ->
 * weighted SwiGLU -> expert down, plus the shared expert).
 *   y[t] += sum_j w_j * down_j(hq_j) + shared(x[t])
 * with hq_j the int8-requantised silu(gate_j x) * (up_j x).
 *   x         [n_tok][H] fp32, read only
 *   token_ids [n_tok] int32, required for hash routing, else may be NULL
 *   y         [n_tok][H] fp32, read and written (must not alias x)
 * n_tok in 0..max_tokens. Enqueued on `stream`; no host synchronisation.
 * Calls of fewer than 65 tokens take the decode path (router, gate/up and
 * down kernels, chunks of at most 64 tokens; units of eight tokens take
 * their int8 block dots from the tensor cores); larger calls the prefill
 * path (tensor-core grouped GEMMs, chunks of at most 4096 tokens; when hidden
 * and ffn are multiples of 128, else the decode path). All give the same
 * bits. */
ds4moe_status ds4moe_forward(ds4moe_layer *h, const float *x, int32_t n_tok, const int32_t *token_ids,
                             float *y, void *stream);

/* One layer of a stack: the RMSNorm with unit gain of ds4moe_rmsnorm (same
 * arithmetic, same bits) folded into the forward,
 *   y[t] += MoE(x[t] / sqrt(mean(x[t]^2) + eps)),
 * for a residual stream that passes RMSNorm, then the MoE FFN added to it
 * ("DeepSeek V4 Flash -- DFlash Integration", Forward Pass). From two tokens
 * on (and on the prefill path) the router kernel normalises the rows as it
 * quantises them, so no normalised copy is written and no extra kernel runs;
 * a one-token decode call runs the RMSNorm kernel into a row buffer of the
 * handle first (faster there). Bit-identical to ds4moe_rmsnorm into a
 * buffer followed by ds4moe_forward on it.
 *   x  [n_tok][H] fp32, read only, 16-byte aligned
 *   y  [n_tok][H] fp32, read and written; may be x itself (y += on the
 *      residual in place: every read of x completes before any write of y),
 *      else must not overlap it
 * Other arguments, paths, errors and stream behaviour as ds4moe_forward;
 * DS4MOE_ERR_INVALID_ARG also for a NaN eps, an unaligned x or a partial
 * overlap of x and y. */
ds4moe_status ds4moe_forward_rmsnorm(ds4moe_layer *h, const float *x, int32_t n_tok, const int32_t *token_ids,
                                     float eps, float *y, void *stream);

/* ds4moe_forward on HOST buffers (pinned or pageable): y_host += MoE(x_host),
 * synchronising `stream` before it returns. Decode-sized calls (n_tok up to
 * min(max_tokens, 64)) on pinned buffers: the kernels read x and token_ids
 * and update y in them directly over the CPU-GPU link. Decode-sized calls on
 * pageable buffers copy them into mapped pinned buffers owned by the handle
 * and replay one CUDA graph per token count (captured on the first call of
 * that count; kept until ds4moe_destroy). Larger calls copy x, the token
 * ids and y to device staging buffers chunk by chunk (Ts tokens at a time,
 * see max_tokens), run the layer on each chunk and copy y back.
 * Memory: the first call allocates, and keeps until ds4moe_destroy, device
 * staging of 2 * Ts * hidden * 4 + Ts * 4 bytes (about 128 MB at Ts = 4096,
 * hidden 4096) and, for pageable callers, 2 * min(max_tokens, 64) * hidden * 4
 * + min(max_tokens, 64) * 4 bytes of mapped pinned host memory. Not reentrant
 * on one handle. Same arguments otherwise. */
ds4moe_status ds4moe_forward_host(ds4moe_layer *h, const float *x_host, int32_t n_tok,
                                  const int32_t *token_ids_host, float *y_host, void *stream);

/* RMSNorm with unit gain between stacked layers:
 *   out[t] = x[t] / sqrt(mean(x[t]^2) + eps)   (x, out [n_tok][hidden] fp32;
 * out may equal x). hidden must be a multiple of 32. (DFlash Integration page,
 * Forward Pass, step 5: RMSNorm before the output projection.) */
ds4moe_status ds4moe_rmsnorm(const float *x, float *out, int32_t n_tok, int32_t hidden, float eps,
                             void *stream);

/* Synchronise `stream`, read and clear the handle's device error flag.
 * *flags_out (may be NULL) receives the DS4MOE_DEVERR_* bits.
 * When DS4MOE_DEVERR_TIMEOUT is among them, a kernel gave up a bounded wait
 * and left some cross-block completion counters unfinished: this call also
 * zeroes them (and synchronises the device), so the next call starts from a
 * clean state. Outputs of calls made between the timeout and this call are
 * undefined.
 * Returns DS4MOE_ERR_DEVICE when any bit was set, else DS4MOE_OK. */
ds4moe_status ds4moe_get_device_error(ds4moe_layer *h, void *stream, uint32_t *flags_out);

/* Read-only device view of the handle's scratch after the last forward call,
 * for inspecting intermediate results. With C = Ts (see max_tokens) and
 * NS = k + n_shared, `which`:
 *   0 xq  int8  [C][H]        activation codes (CAS step 1)
 *   1 dx  fp32  [C][H/32]     activation scales
 *   2 gs  int16 [C][H/16]     16-group sums of xq
 *   3 ids int32 [C][k]        routed expert ids
 *   4 w   fp32  [C][k]        renormalised weights
 *   5 hq  int8  [C*NS][F]     SwiGLU codes, row t*NS+slot (slot k = shared)
 *   6 dh  fp32  [C*NS][F/32]  SwiGLU scales
 *   7 a   fp32  [C*NS][H]     per-slot down-projection outputs
 * Rows refer to the tokens of the last chunk of that call (64 tokens at most
 * on the decode path, 4096 on the prefill path); other rows are undefined.
 * Errors: INVALID_ARG for an unknown `which`. */
ds4moe_status ds4moe_debug_scratch(ds4moe_layer *h, int32_t which, const void **ptr_out, uint64_t *bytes_out);

/* Per-stage timing with CUDA events recorded on the call's stream.
 * ds4moe_profile_enable(h, 1) makes every later ds4moe_forward record an
 * event before each stage and after the last one; ds4moe_profile_collect
 * waits for the last forward's events and adds the stage durations to the
 * handle's totals; ds4moe_profile_read copies the totals (milliseconds,
 * summed over collected calls) for the stages
 *   0 quantise x, 1 route (router GEMV + top-k, or hash), 2 bucket,
 *   3 gate/up, 4 down, 5 combine
 * into ms_out[0..n) and the number of collected calls into *calls.
 * ds4moe_profile_enable(h, 0) stops recording and zeroes the totals.
 * Profiling adds event records to the stream; it is off by default. */
#define DS4MOE_N_STAGES 6
ds4moe_status ds4moe_profile_enable(ds4moe_layer *h, int32_t on);
ds4moe_status ds4moe_profile_collect(ds4moe_layer *h);
ds4moe_status ds4moe_profile_read(const ds4moe_layer *h, double *ms_out, int32_t n, int64_t *calls);

/* ---------------------------------------------------------------------------
 * Dense Q8_0 product beside the MoE: y = W x for the output head (129280 x
 * 4096, "OutQ8") and the attention projections, on activations pre-quantised
 * to int8 per 32-block.
 * Passages: ds4-rocm fork README, Performance optimizations (the
 * matmul_q8_0_preq_* kernels: Q8_0 matmuls on pre-quantised activations, the
 * largest share of decode time beside the MoE); DwarfStar README, Model
 * Weights (the OutQ8 model name).
 * Arithmetic (canonical spec): x quantised as for the MoE (CAS step 1); each
 * output is the CAS row sum of its Q8_0 block terms (d * dx) * I over
 * S = min(8, n_in/32) contiguous segments, as for an expert row.
 *
 * ds4moe_dense_create: w_q8 is the canonical [n_out][n_in] Q8_0 matrix (rows
 *   of n_in/32 blocks of 34 bytes) in DEVICE memory, read only during the call
 *   (re-laid out into a handle-owned copy; rows padded to a multiple of 32).
 *   n_out 1..2^24; n_in a multiple of 32, up to 65536, with n_in/32 a multiple
 *   of min(8, n_in/32); max_tokens 1..65536 sizes the activation scratch
 *   and the segment-sum scratch of split rows (min(8, n_in/32) x
 *   min(max_tokens, 8) x n_out floats). Synchronises. Errors: INVALID_ARG,
 *   UNSUPPORTED (n_in too wide for a block's shared memory), OOM, CUDA; on
 *   error *out is NULL.
 * ds4moe_dense_forward: y[t][n] = sum_k W[n][k] x[t][k] for t < n_tok
 *   (x [n_tok][n_in] fp32, y [n_tok][n_out] fp32, overwritten; device
 *   pointers), enqueued on `stream` (two launches, three for split rows; no
 *   allocation, no host synchronisation). Built for decode-sized n_tok: the
 *   matrix is streamed once per pass of up to 8 tokens (fewer for very wide
 *   n_in); from two tokens on the integer block dots run on the tensor
 *   cores (the int8 codes as fp16 with f32 accumulation: every partial sum
 *   is an integer below 2^24, so the dots are exact and the bits the same);
 *   a call of one pass may split rows over several warps by whole
 *   segments, whose sums a third launch adds in segment order (the same bits
 *   as unsplit). Calls on one handle must not run concurrently (shared
 *   scratch).
 *   Errors: INVALID_ARG (pointers, n_tok outside 0..max_tokens), CUDA.
 * ds4moe_dense_get_device_error: as ds4moe_get_device_error, for the dense
 *   handle's flag (DS4MOE_DEVERR_NONFINITE, DS4MOE_DEVERR_TIMEOUT).
 * ds4moe_dense_destroy: releases everything (synchronises); NULL is a no-op. */
typedef struct ds4moe_dense ds4moe_dense;
ds4moe_status ds4moe_dense_create(int32_t n_out, int32_t n_in, int32_t max_tokens, const void *w_q8,
                                  ds4moe_dense **out);
ds4moe_status ds4moe_dense_forward(ds4moe_dense *h, const float *x, int32_t n_tok, float *y, void *stream);
ds4moe_status ds4moe_dense_get_device_error(ds4moe_dense *h, void *stream, uint32_t *flags_out);
void ds4moe_dense_destroy(ds4moe_dense *h);
uint64_t ds4moe_dense_device_bytes(const ds4moe_dense *h);
uint64_t ds4moe_dense_launch_count(const ds4moe_dense *h);
/* ds4moe_dense_debug_config: overrides the dense kernel's launch geometry for
 *   later calls (a tuning and test hook; the results are the same bits under
 *   every setting): ks = K steps per ring stage (a divisor of n_in/32/S, at
 *   most 8), nst = ring stages per warp (2..6, within shared memory), ns =
 *   units per 32-row item (a divisor of S), tc = the block-dot step: 1 the
 *   dp4a step only, 2 the tensor-core step for every call (where eight
 *   tokens' fp16 codes fit a pass; the automatic choice takes it from two tokens
 *   on). 0 keeps the automatic choice of that value. A call whose tokens do
 *   not fit one pass of the segment-sum scratch runs unsplit (ns = 1)
 *   whatever ns says; a (ks, nst) that does not fit a call's shared memory
 *   falls back to the automatic ring.
 *   Errors: INVALID_ARG (NULL, a value outside its range). */
ds4moe_status ds4moe_dense_debug_config(ds4moe_dense *h, int32_t ks, int32_t nst, int32_t ns, int32_t tc);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection: every token
 * brings the slot of its request's adapter,
 *   y[t] = base[t] + scale_s * B_s (A_s x[t]),  s = slots[t];  s = -1: base[t].
 * (The pages have no adapters; the projection is ds4moe_dense_forward, whose
 * output is the base.) x and weights as they are, products and sums in 32 bits:
 * no rounding to fewer bits on the way (many tokens: a product's fp32 operand
 * is taken as the sum of two 11-bit numbers, off by 2^-20 of it at most, and the
 * tensor cores cut sums to 24 bits instead of rounding them: for terms of random
 * sign the matrix that is added to base is off by less than 2^-19 of its norm at
 * any rank and width; token by token by less than 2^-20).
 *
 * ds4moe_adapters_create: places for n_slots (1..4096) adapters of up to max_rank
 *   (1..256) in `dtype` (DS4MOE_DT_BF16 or DS4MOE_DT_F16) on the current device,
 *   all empty; n_out 1..2^24, n_in a multiple of 32 up to 65536, max_tokens
 *   1..65536. Device memory: n_slots * 2 bytes * (max_rank to 32 * n_in + max_rank
 *   to 8 * n_out), and max_tokens * (max_rank to 32) * 4 of workspace.
 *   Synchronises. Errors: INVALID_ARG, UNSUPPORTED (more slots or a larger rank),
 *   OOM, CUDA; on error *out is NULL.
 * ds4moe_adapters_set: copies an adapter of `rank` (0..max_rank; 0 empties the
 *   slot, a and b may be NULL) into a slot: a [rank][n_in], b [n_out][rank],
 *   contiguous, device. scale finite. Enqueued on `stream`: calls there before
 *   it use the old adapter, calls after it the new one. Ranks of the slots may
 *   differ.
 * ds4moe_adapters_forward: n_tok 0..max_tokens.
 *   x      [n_tok][n_in] of x_dtype (DS4MOE_DT_F32 or the adapters' type), rows
 *          x_stride elements apart: 16-byte aligned rows
 *   slots  [n_tok] int32, in any order; an empty slot adds nothing; one outside
 *          [-1, n_slots) adds nothing and raises DS4MOE_DEVERR_ADAPTER
 *   base   [n_tok][n_out] fp32, base_stride apart; NULL or y itself (with its
 *          stride): y is added to
 *   y      [n_tok][n_out] fp32, y_stride apart; must not overlap x, nor base
 *          otherwise (columns of one matrix do not; rows in gaps of another
 *          distance in bytes are taken for overlapping: INVALID_ARG)
 *   Strides are below 2^31 elements.
 *   Enqueued on `stream` (one launch for few tokens, three for many, four where the
 *   number of adapters that the call uses decides, on the device; the slots that
 *   the handle has do not), no allocation, no synchronisation. Calls on one handle must not run concurrently (shared
 *   workspace). Errors: INVALID_ARG, CUDA.
 * ds4moe_adapters_debug_path: 1: every later call token by token, 2: by tiles of
 *   tokens of one adapter, 0: by the number of tokens (a test hook; results differ by
 *   roundings). Errors: INVALID_ARG.
 * The others as their ds4moe_dense_* namesakes. */
typedef struct ds4moe_adapters ds4moe_adapters;
ds4moe_status ds4moe_adapters_create(int32_t n_out, int32_t n_in, int32_t n_slots, int32_t max_rank, int32_t dtype,
                                     int32_t max_tokens, ds4moe_adapters **out);
ds4moe_status ds4moe_adapters_set(ds4moe_adapters *h, int32_t slot, int32_t rank, const void *a, const void *b,
                                  float scale, void *stream);
ds4moe_status ds4moe_adapters_forward(ds4moe_adapters *h, const void *x, int64_t x_stride, int32_t x_dtype,
                                      const int32_t *slots, int32_t n_tok, const float *base, int64_t base_stride,
                                      float *y, int64_t y_stride, void *stream);
ds4moe_status ds4moe_adapters_debug_path(ds4moe_adapters *h, int32_t path);
ds4moe_status ds4moe_adapters_get_device_error(ds4moe_adapters *h, void *stream, uint32_t *flags_out);
void ds4moe_adapters_destroy(ds4moe_adapters *h);
uint64_t ds4moe_adapters_device_bytes(const ds4moe_adapters *h);
uint64_t ds4moe_adapters_launch_count(const ds4moe_adapters *h);

/* ---------------------------------------------------------------------------
 * Attention beside the MoE: a paged key-value cache, its append, and the
 * attention that reads it. Forward only.
 * Passages: "DeepSeek V4 Flash -- DFlash Integration", Model Architecture (64
 * heads over 1 key-value head of dimension 512), the paged 128-token cache and
 * the sliding-window ring of the same page, and its verification of drafted
 * tokens (2 to 5 rows per sequence).
 *
 * Formula. The query of position i sees position j when
 *   j <= i  and  (window == 0  or  j > i - window  or  j < n_sink),
 * that is, the last `window` positions and the first n_sink ones. For head h
 * (key-value head g = h / (n_heads / n_kv_heads)):
 *   s_j = scale * <q_h, k_j,g>,  out_h = sum_j exp(s_j) v_j,g / sum_j exp(s_j)
 * over the visible j. No visible position (i < 0), or no score above
 * -infinity: zeros. Keys and values of positions that a row does not see never
 * reach its output, whatever they hold (infinities and NaN among them); where
 * rows of one tile differ in what they see of such a value, those that do not
 * see it take some 1000 cycles per position. Scores, softmax and sums
 * are held in 32 bits; the weights are rounded to the 16-bit type before they
 * multiply the values, and the output once at the end.
 *
 * Cache: k, v are pools of n_pages pages of page_size positions each. Element
 * (page, row, head, d) of k lies at k + page * k_page_stride + row *
 * k_row_stride + head * k_head_stride + d (strides in elements; v likewise; k
 * and v may be the same memory). Position pos of sequence b is in page
 * block_table[b * table_stride + pos / page_size], row pos % page_size; table
 * entries of pages without a visible position are not read. page_size: a
 * multiple of 16, up to 65536. Base pointers 16-byte aligned, strides multiples
 * of 8 elements.
 *
 * Data errors on the device set a flag of the handle: DS4MOE_DEVERR_PAGE (a
 * table entry outside [0, n_pages): its keys and values are read as zeros, and
 * an append to it is dropped), DS4MOE_DEVERR_LENGTH (kv_len outside
 * [0, max_pages * page_size]: clamped; a cu_q that is not ascending in
 * [0, n_tok]: each entry is clamped to that and raised to the largest before
 * it, so that sequences never share a row; a row appended at a position
 * outside the table is dropped). */
#define DS4MOE_ATTN_MAX_NEW 16 /* new tokens per sequence of a decode call */

typedef struct {
  uint32_t abi_version; /* = DS4MOE_ABI_VERSION                                  */
  int32_t n_heads;      /* query heads: a multiple of n_kv_heads, at most 128x   */
  int32_t n_kv_heads;   /* 1..1024                                               */
  int32_t head_dim;     /* 64, 128, 256 or 512                                   */
  int32_t dtype;        /* DS4MOE_DT_BF16 or DS4MOE_DT_F16: q, cache and out     */
  int32_t window;       /* last positions visible to a query; 0: all             */
  int32_t n_sink;       /* first positions that stay visible (with a window)     */
  float scale;          /* of the scores; > 0, usually 1 / sqrt(head_dim)        */
  int32_t max_seqs;     /* largest n_seq of any later call, 1..65536             */
  int32_t max_tokens;   /* largest number of rows of any later call, 1..1048576  */
} ds4moe_attn_desc;

typedef struct {
  void *k, *v;
  int64_t n_pages;
  int64_t k_page_stride, k_row_stride, k_head_stride;
  int64_t v_page_stride, v_row_stride, v_head_stride;
  const int32_t *block_table; /* [n_seq][table_stride]                           */
  int64_t table_stride;
  int32_t page_size;
  int32_t max_pages;          /* entries of a table row (<= table_stride)        */
} ds4moe_kv_cache;

/* Opaque handle: shape and workspace, nothing of a cache. One handle serves any
 * number of layers of its shape whose calls run one after another on a stream
 * (its workspace is 21 MB for heads of 64 and 41 MB for longer ones, and little
 * more with max_tokens). */
typedef struct ds4moe_attn ds4moe_attn;

/* Validates `desc` and allocates the handle's workspace on the current device
 * (synchronises). Errors: INVALID_ARG, UNSUPPORTED (another head_dim, more
 * than 128 heads per key-value head), OOM, CUDA; on error *out is NULL. */
ds4moe_status ds4moe_attn_create(const ds4moe_attn_desc *desc, ds4moe_attn **out);
/* Releases everything (synchronises the device). NULL is a no-op. */
void ds4moe_attn_destroy(ds4moe_attn *h);

/* Writes the new tokens' keys and values into the pages.
 *   k_new, v_new [n_tok][n_kv_heads][head_dim], rows k_stride / v_stride
 *           elements apart; src_dtype DS4MOE_DT_F32 (rounded to the cache's
 *           type, to nearest even) or the cache's own type. v_new NULL: only k.
 *   cu_q    [n_seq + 1] ascending: sequence b has rows cu_q[b] .. cu_q[b+1] - 1.
 *           NULL: n_tok / n_seq rows each.
 *   kv_len  [n_seq] positions of each sequence INCLUDING the new ones: the j-th
 *           of n rows goes to position kv_len - n + j.
 * Enqueued on `stream`, no allocation, no synchronisation, as the two calls
 * below. Errors: INVALID_ARG, CUDA. */
ds4moe_status ds4moe_kv_append(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *k_new, int64_t k_stride,
                               const void *v_new, int64_t v_stride, int32_t src_dtype, const int32_t *cu_q,
                               const int32_t *kv_len, int32_t n_seq, int32_t n_tok, void *stream);

/* The same append with the position rotation on the way, for the keys and, in
 * the same launch, the queries of the new tokens. Passage: "DeepSeek V4 Flash --
 * DFlash Integration", Model Architecture (partial rope of 64 of 512 elements;
 * YaRN, whose frequencies and factor are the caller's here).
 * The pair (x, y) number i of a head's rotated elements becomes, at position p,
 *   x' = scale * (x cos - y sin),  y' = scale * (y cos + x sin),
 *   angle = p * inv_freq[i],
 * in 32 bits, rounded once to the cache's type; elements outside
 * [offset, offset + rot_dim) and values pass as in ds4moe_kv_append. Angles are
 * those of the fp32 frequencies as they are, at any position: p * inv_freq / 2 pi
 * is reduced to one turn in 64-bit fixed point, exact to |inv_freq| * 2^-33 turns
 * at p = 2^31. A frequency that is not finite gives NaN.
 *   q_new   [n_tok][n_heads][head_dim], rows q_stride elements apart, of
 *           src_dtype; may be NULL (then q_out too)
 *   q_out   the same rows in the cache's type, q_out_stride apart; may be q_new
 *           itself (of the cache's type, with the same stride), must not overlap
 *           the inputs otherwise (columns of one matrix do not; rows in gaps of
 *           another distance in bytes are taken for overlapping). Rows of no sequence are left as they are; a
 *           row whose position the cache has no place for is rotated all the same.
 * Other arguments, flags and errors as ds4moe_kv_append; INVALID_ARG also for a
 * rope that is not as below. */
typedef struct {
  const float *inv_freq; /* device, [rot_dim / 2], 16-byte aligned: radians per position */
  int32_t rot_dim;       /* rotated elements of a head: a multiple of 16, 16..head_dim  */
  int32_t offset;        /* the first of them: a multiple of 8                          */
  int32_t interleaved;   /* pair i: 0: elements i and i + rot_dim/2; 1: 2i and 2i + 1   */
  float scale;           /* of cosine and sine, usually 1                               */
} ds4moe_rope;

ds4moe_status ds4moe_kv_append_rope(ds4moe_attn *h, const ds4moe_kv_cache *cache, const ds4moe_rope *rope,
                                    const void *q_new, int64_t q_stride, void *q_out, int64_t q_out_stride,
                                    const void *k_new, int64_t k_stride, const void *v_new, int64_t v_stride,
                                    int32_t src_dtype, const int32_t *cu_q, const int32_t *kv_len, int32_t n_seq,
                                    int32_t n_tok, void *stream);

/* Attention of n_new (1..DS4MOE_ATTN_MAX_NEW) new tokens of every sequence.
 *   q, out  [n_seq * n_new][n_heads][head_dim], rows q_stride / out_stride
 *           elements apart, 16-byte aligned; out must not overlap q or the
 *           cache. Row b * n_new + j has position kv_len[b] - n_new + j.
 *   kv_len  [n_seq] positions including the new ones (already appended). */
ds4moe_status ds4moe_attn_decode(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *q, int64_t q_stride,
                                 const int32_t *kv_len, int32_t n_seq, int32_t n_new, void *out, int64_t out_stride,
                                 void *stream);

/* The same, of a batch whose sequences begin with the same positions (a system
 * prompt, a document): the same formula and results, but the shared keys and
 * values are read once for all sequences of a group.
 *   shared_len  [n_groups] positions that the group's sequences have in common:
 *           all their tables lead to the same keys and values there (the same
 *           pages, or copies: shared_len may lie inside a page). They are read
 *           through the table of the first sequence that shares. A sequence whose
 *           first new token does not see all of them (kv_len - n_new + 1 <
 *           shared_len) shares nothing. 0: nothing is shared.
 *   group_start [n_groups + 1] ascending: group g is sequences group_start[g] ..
 *           group_start[g+1] - 1; a sequence of no group shares nothing. NULL:
 *           one group of all (n_groups = 1).
 * n_groups 1..n_seq. Both are read on the device as kv_len is; DS4MOE_DEVERR_LENGTH
 * for shared_len outside the table (clamped) and bounds out of order (as cu_q).
 * Where sharing would gain nothing (few shared positions or sequences; shapes whose
 * sequences fill the products' tiles by themselves; handles with a window, which
 * see little of what is shared) every sequence reads its positions itself: the
 * argument never changes a result but by its roundings (the weights of shared
 * positions of fp16 are scaled as ds4moe_attn_prefill does it: one below 2^-31 of
 * the largest is 0, in ds4moe_attn_decode's kernel of few rows one below 2^-39).
 * That is decided twice. On the host, by the table's capacity max_pages *
 * page_size, the most that can be shared: where that would gain nothing, and with
 * a window, the call is ds4moe_attn_decode, launch for launch and bit for bit, and
 * neither array is read or flagged. Else on the device for every group, and a call
 * that shares nothing there still has the launches of one that does (8 sequences
 * of 1700, 32/8 heads of 128: 16 us plain, 28 to 31 so; 8 of 25000: 134 and 148;
 * 64 of 5000: 196 and 211). So give max_pages no larger than the batch's longest
 * sequence needs, in a table of any table_stride.
 * ds4moe_attn_reserve_shared: workspace for such calls of up to max_tokens
 * (n_seq * n_new) rows, at most the handle's: max_tokens * n_heads * (head_dim +
 * 1) * 4 bytes. Allocates, synchronises; a smaller number than before changes
 * nothing. Calls captured before it must not be replayed after it. Errors:
 * INVALID_ARG, OOM, CUDA. A call of more rows than reserved: INVALID_ARG. */
ds4moe_status ds4moe_attn_reserve_shared(ds4moe_attn *h, int32_t max_tokens);
ds4moe_status ds4moe_attn_decode_shared(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *q, int64_t q_stride,
                                        const int32_t *kv_len, const int32_t *shared_len, const int32_t *group_start,
                                        int32_t n_groups, int32_t n_seq, int32_t n_new, void *out, int64_t out_stride,
                                        void *stream);

/* ds4moe_attn_debug_share(h, 1): later calls share wherever two sequences have a
 *   position in common, whether it gains anything or not (a test hook); 0: as
 *   above. Errors: INVALID_ARG. */
ds4moe_status ds4moe_attn_debug_share(ds4moe_attn *h, int32_t always);

/* Attention of ragged runs of new tokens: sequence b has rows cu_q[b] ..
 * cu_q[b+1] - 1 (none is allowed), the last of them at position
 * kv_len[b] - 1. Rows of no sequence are left as they are. */
ds4moe_status ds4moe_attn_prefill(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *q, int64_t q_stride,
                                  const int32_t *cu_q, const int32_t *kv_len, int32_t n_seq, int32_t n_tok, void *out,
                                  int64_t out_stride, void *stream);

/* As ds4moe_get_device_error, for the attention handle's flag. */
ds4moe_status ds4moe_attn_get_device_error(ds4moe_attn *h, void *stream, uint32_t *flags_out);
uint64_t ds4moe_attn_device_bytes(const ds4moe_attn *h);
uint64_t ds4moe_attn_launch_count(const ds4moe_attn *h);

/* ---------------------------------------------------------------------------
 * After the output head.
 *
 * ds4moe_token_probs: probs[r] = softmax(logits[r] / temperature) over vocab
 *   (fp32, rows `stride` elements apart; probs may be logits itself with the
 *   same stride). temperature 1e-6 .. 1e6, or 0: 1 at the lowest index of the row's maximum, 0
 *   elsewhere. A NaN in a row, or a maximum of +-infinity (temperature > 0),
 *   gives NaN.
 * ds4moe_verify_drafts: which of a sequence's drafted tokens x_0, x_1, ... stay,
 *   and the token after them ("DeepSeek V4 Flash -- DFlash Integration", the
 *   speculative decoding sections). With target probabilities p_i and the
 *   drafter's q_i for draft i:
 *     draft i is accepted when u_accept[i] * q_i(x_i) < p_i(x_i); n is the first
 *     draft that is not (or n_draft);
 *     the token after them is drawn from r = max(p_n - q_n, 0) (p_n where that
 *     is 0 everywhere; p_n when all were accepted): the lowest v with
 *     r(0) + ... + r(v) > u_sample * sum(r).
 *   target  [n_seq][max_draft + 1] rows of vocab, target_stride apart
 *   draft   [n_seq][max_draft] rows, draft_stride apart; NULL: a drafter that
 *           is sure of its tokens (q_i = 1 at x_i, 0 elsewhere)
 *   draft_tokens [n_seq][max_draft]; n_draft [n_seq] (NULL: max_draft each)
 *   u_accept [n_seq][max_draft], u_sample [n_seq]: uniform numbers in [0, 1)
 *   n_accepted [n_seq]: n; tokens_out [n_seq][max_draft + 1]: the accepted
 *           drafts, the drawn token (-1 where p_n is 0 everywhere), then -1.
 *   Probabilities are taken in [0, 1] (others are clamped, NaN is 0) and
 *   summed exactly, in multiples of 2^-45 (of 2^(ceil(log2 vocab) - 62) above
 *   131072 entries).
 *   err_flags (device, may be NULL): DS4MOE_DEVERR_TOKEN_ID for a drafted token
 *   outside [0, vocab) (rejected), DS4MOE_DEVERR_LENGTH for n_draft outside
 *   [0, max_draft] (clamped).
 * Both are enqueued on `stream` without allocation or synchronisation.
 * Errors: INVALID_ARG, CUDA. */
#define DS4MOE_MAX_DRAFT 64
ds4moe_status ds4moe_token_probs(const float *logits, int64_t logits_stride, int32_t n_rows, int32_t vocab,
                                 float temperature, float *probs, int64_t probs_stride, void *stream);
ds4moe_status ds4moe_verify_drafts(const float *target, int64_t target_stride, const float *draft, int64_t draft_stride,
                                   const int32_t *draft_tokens, const int32_t *n_draft, const float *u_accept,
                                   const float *u_sample, int32_t n_seq, int32_t max_draft, int32_t vocab,
                                   int32_t *n_accepted, int32_t *tokens_out, uint32_t *err_flags, void *stream);

/* Test hooks for failure detection (no counterpart in the pages; they make
 * failures happen on the host side or through a short wait bound, never by
 * faulting the GPU).
 * ds4moe_debug_set_wait_limit: bound, in SM cycles, of the hand-off waits of
 *   the decode path's expert kernels (a warp waiting for another warp of its
 *   block, or for the router's count of quantised x); 0 restores the default
 *   (about 2^31 cycles). A wait that runs out raises DS4MOE_DEVERR_TIMEOUT
 *   and its block leaves; waits for the block's own copies keep the default
 *   bound, so no copy is left in flight. Errors: INVALID_ARG (NULL, < 0).
 * ds4moe_debug_fail_alloc: the n-th device allocation the library makes
 *   from now on (in ds4moe_create, or the first ds4moe_forward_host) fails
 *   as if the device were out of memory; 0 turns it off. Process-wide.
 *   Errors: INVALID_ARG (n < 0). */
ds4moe_status ds4moe_debug_set_wait_limit(ds4moe_layer *h, int64_t cycles);
ds4moe_status ds4moe_debug_fail_alloc(int32_t n);

/* Number of kernels this handle has launched since create. */
uint64_t ds4moe_launch_count(const ds4moe_layer *h);

/* Bytes of device memory the handle owns (weights + scratch). */
uint64_t ds4moe_device_bytes(const ds4moe_layer *h);

/* Human-readable status name (static storage). */
const char *ds4moe_status_string(ds4moe_status s);

/* = DS4MOE_ABI_VERSION of the loaded library. */
uint32_t ds4moe_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* DS4MOE_H */
