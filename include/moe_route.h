/*
 * moe_route.h -- C interface of the MI355X (gfx950) routed mixture-of-experts layer.
 *
 * The layer, as the pages describe it:
 *   - Betelgeuse news article (fanjiajia.top, "Betelgeuse: RTX 3060 12GB + 16GB ..."),
 *     section "mechanism: VRAM expert-slot pool, in-stream doorbell and victim cache":
 *     48 layers x 512 routed experts; each token takes 10 routed experts + 1 shared one;
 *     router and shared expert always resident; routed experts sit in a per-layer pool
 *     of HBM slots; a GPU-side check finds the misses and rings the host only on a miss;
 *     HBM and host copies of an expert are exclusive.  Section "what bit-exact means":
 *     the top-10 selection is exact and never altered; a failed expert read is an error,
 *     never a silent zero weight.
 *   - halogen-flash-server README, section "Bring your own GGUF": expert weights are a
 *     small set of values times a per-block scale (the Q4_0 family), repacked losslessly
 *     into the kernels' own layout; unsupported formats are refused by name.
 *   - Basalt README, section "The .basalt model file": quantized bytes used as stored.
 *
 * Readings where the pages are silent: router weights = softmax over the k selected
 * logits (they sum to 1 over the chosen experts); equal logits -> lower expert id first;
 * the optional per-expert bias is added to the logits before selection; the shared expert
 * has weight 1; the expert FFN is SwiGLU, y_e = Wd (silu(Wg x) * (Wu x)); the layer output
 * is y = sum_j w_j y_{e_j} (j = 0..k-1, selection order) + y_shared, with no residual.
 *
 * Conventions for every entry point
 *   - Tensor pointers are device pointers owned by the caller (allocated by any means);
 *     the library never allocates or frees device memory.  The activations x, the outputs y
 *     and the router matrix are moved with 16-byte vector accesses and must be 16-byte
 *     aligned (a hipMalloc'd buffer, and a whole-token slice of one, is); a misaligned one is
 *     MOE_EINVAL.  Its only process-wide state is
 *     the profiling selection of moe_debug_kernel_events (off unless a caller sets it).
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Work is
 *     enqueued asynchronously on it; the call returns once it is enqueued.
 *   - Every call validates its arguments on the host first and enqueues nothing when
 *     it returns an error.  Return value: MOE_OK (0) or a negative MOE_E* code.
 *   - n_tokens >= 1 wherever a token count is taken: an empty batch is MOE_EINVAL.
 *   - `ws` is a caller-owned device workspace of `ws_bytes` bytes (256-byte aligned),
 *     at least moe_workspace_bytes(dims, n_tokens).  It must be cleared once with
 *     moe_workspace_init before its first use; calls leave it reusable.  Calls that
 *     share one workspace must be ordered on one stream.
 *   - Faults the device detects (an expert id out of range, a slot index out of range,
 *     a selected expert that is not resident when its weights are needed, a NaN logit,
 *     an expert named twice in one token's top-k list, a value outside the fp16 range on
 *     the prefill path) set bits of an error word in `ws`; the outputs of that call are
 *     then invalid, never silently computed (Betelgeuse article, "what bit-exact means":
 *     a failed expert read is an error, not a zero weight).  moe_check_device_error reads
 *     and clears the word.
 *
 * Expert blob (one routed or shared expert; H = hidden, F = ffn), six sections in this order:
 *   [gate codes F*H/2][up codes F*H/2][down codes H*F/2]
 *   [gate scales F*H/16][up scales F*H/16][down scales H*F/16]          (bytes)
 * Gate and up have R = F rows over K = H inputs, down R = H rows over K = F inputs.  A code
 * u (0..15) stands for q = u - 8; blocks of 32 consecutive inputs of a row share one fp16
 * scale (little-endian), and the weight is q * scale (halogen README, "Bring your own GGUF":
 * a small set of values times a per-block scale, moved losslessly into the kernels' layout).
 * Each row is cut into K/128 groups of 128 inputs (four blocks), stored group-major:
 *   - codes of group c of row r: the 64-byte record at byte 64 * (c * R + r) of the section,
 *     sixteen little-endian 32-bit words.  Word 4g + i (g, i = 0..3) holds slice g of block i,
 *     that is inputs 128c + 32i + 8g .. 128c + 32i + 8g + 7: input 128c + 32i + 8g + 2j in bits
 *     4j..4j+3 and input 128c + 32i + 8g + 2j + 1 in bits 16+4j..16+4j+3 (j = 0..3);
 *   - scales of group c of row r: four fp16 values (blocks 4c .. 4c+3 of the row) at byte
 *     8 * (c * R + r) of the scale section.
 * With MOE_FMT_AFFINE4 three more sections follow, [gate mins][up mins][down mins], laid out
 * as the scales.  Model shape (H 2048, F 768): 2,654,208 bytes = 648 x 4 KiB (affine: 2,949,120).
 */
#ifndef MOE_ROUTE_H
#define MOE_ROUTE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_API __attribute__((visibility("default")))

enum moe_status {
  MOE_OK = 0,
  MOE_EINVAL = -1,        /* a NULL pointer, a size out of range, inconsistent dimensions */
  MOE_EUNSUPPORTED = -2,  /* valid request this library does not implement (dtype, block, shape) */
  MOE_EWORKSPACE = -3,    /* ws NULL, misaligned or smaller than moe_workspace_bytes */
  MOE_EHIP = -4,          /* a HIP runtime call failed (launch, copy, stream wait) */
  MOE_EDEVICE = -5,       /* the device error word was set (moe_check_device_error) */
  MOE_EFILL = -6          /* a slot-pool fill (host -> HBM expert copy) failed */
};

/* MOE_F16 is an operand type of the dense operators (moe_linear_*, moe_gated_*) and of those after them only. */
enum moe_dtype { MOE_F32 = 0, MOE_BF16 = 1, MOE_F16 = 2 };

/* Device error word bits (moe_check_device_error). */
enum moe_device_error {
  MOE_DERR_EXPERT_ID = 1,     /* a selected / given expert id outside [0, n_experts) */
  MOE_DERR_SLOT = 2,          /* a slot-table entry >= n_slots */
  MOE_DERR_NOT_RESIDENT = 4,  /* an expert needed by an FFN call has no slot (-1) */
  MOE_DERR_NAN = 8,           /* a NaN logit reached the selection */
  MOE_DERR_FILL = 16,         /* the slot-pool service reported a failed fill */
  MOE_DERR_DUP_ID = 32,       /* a token's top-k list names one expert twice */
  MOE_DERR_RANGE = 64,        /* prefill: an activation, SwiGLU output or weighted expert row
                                 beyond the fp16 range (|v| > 65504) or not finite */
  MOE_DERR_ROWS = 128,        /* rows by expert: a pair out of range or in two rows, a row out of
                                 range, perm and inv at odds, offsets that descend or leave the rows */
  MOE_DERR_TARGET = 256       /* loss: a target outside [0, vocab) that is not `ignore` */
};

/* Largest token count of a decode call.  The pages' decode batches: concurrent streams (Basalt
 * README, "Concurrent requests: --parallel N", N = 1..8) and speculative verify batches, whose
 * tokens must come out byte-identical to the same request decoded alone and serially (halogen
 * README, "Quality: what is measured, and what is not", identity properties).  On the decode
 * path a token's output is bitwise the same at every batch size up to the limit:
 *   MOE_DECODE_MAX_TOKENS (16) with bf16 activations (and a bf16 router, for the calls that
 *   route) and F <= 2048;
 *   MOE_DECODE_MAX_TOKENS_NARROW (8) otherwise: an fp32 token takes two matrix-core rows, and 16
 *   tokens' SwiGLU rows of a wider F do not fit a workgroup's LDS.
 * Above the limit moe_layer_forward takes the prefill kernels. */
#define MOE_DECODE_MAX_TOKENS 16
#define MOE_DECODE_MAX_TOKENS_NARROW 8

/* Layer dimensions.  hidden = H, ffn = F (expert FFN width, shared expert too),
 * n_experts = E routed experts, top_k = k, n_shared = 0 or 1, block = 32 (the only
 * supported quantization block; anything else is MOE_EUNSUPPORTED).
 * Supported: H and F multiples of 128 (whole groups of the code layout; else MOE_EINVAL)
 * and at most 4096; 1 <= k <= 16; k <= E <= 1024 (beyond: MOE_EUNSUPPORTED).  The prefill
 * path (more than MOE_DECODE_MAX_TOKENS tokens) further needs H % 256 == 0, bf16
 * activations and router, and n_tokens * H < 2^31 (1,048,575 tokens at H = 2048; beyond:
 * MOE_EUNSUPPORTED). */
typedef struct moe_dims {
  int32_t hidden;
  int32_t ffn;
  int32_t n_experts;
  int32_t top_k;
  int32_t n_shared;
  int32_t block;
  int32_t format;        /* weight format (moe_format); 0 = MOE_FMT_Q4_0, so a zeroed tail is the default */
  int8_t codebook[16];   /* MOE_FMT_CB4: the 16 values a code stands for (times the block scale) */
} moe_dims;

/* Weight formats (halogen README, "Bring your own GGUF": the engine reads the IQ4_NL / IQ4_XS /
 * IQ3_S / Q4_0 family as a small set of values times a per-block scale, and Q4_K / Q5_K / Q5_1
 * as exact affine planes; other block layouts are refused by name).  With a block scale s (fp16):
 *   MOE_FMT_Q4_0     w = (u - 8) * s;
 *   MOE_FMT_CB4      w = codebook[u] * s, codebook = dims.codebook (16 signed 8-bit values);
 *   MOE_FMT_AFFINE4  w = u * s - m, with a second fp16 plane m per block (the blob's mins).
 * Any other value of dims.format is MOE_EUNSUPPORTED.  Q4_0 runs on every kernel; the other two
 * run on the general (non-pipelined) decode and prefill kernels. */
enum moe_format { MOE_FMT_Q4_0 = 0, MOE_FMT_CB4 = 1, MOE_FMT_AFFINE4 = 2 };

/* One layer's weights (all device pointers).
 *   router       [E][H], dtype router_dtype (MOE_F32 or MOE_BF16); row e scores expert e.
 *   router_bias  [E] fp32 added to the logits, or NULL.
 *   arena        expert blobs; the blob in slot s starts at arena + s * slot_stride.
 *   slot_stride  bytes; >= moe_expert_blob_bytes and a multiple of 4096 (the Betelgeuse
 *                article stores each expert as one 4 KB-aligned blob).
 *   n_slots      number of slots in the arena.
 *   shared_blob  the shared expert's blob when n_shared == 1 (always resident), else NULL. */
typedef struct moe_layer_weights {
  const void* router;
  int32_t router_dtype;
  const float* router_bias;
  const uint8_t* arena;
  int64_t slot_stride;
  int32_t n_slots;
  const uint8_t* shared_blob;
} moe_layer_weights;

/* Miss notification for a slot pool served by the host (Betelgeuse article, "mechanism":
 * the in-stream check rings a host doorbell only on a miss).
 *   host_miss_ids    host-mapped pinned int32[E]: the step's miss list (ascending ids).
 *   host_miss_count  host-mapped pinned int32[3]: [0] = number of misses, [2] = number of
 *                    selections written to host_step_ids, [1] = epoch, written last (the
 *                    host polls [1] == epoch, then reads the rest).
 *   ready            device-visible uint32 the stream waits on: work after the check
 *                    runs once *ready >= epoch.  With no miss the check kernel writes
 *                    *ready = epoch itself; otherwise the host writes it after the fills.
 *   epoch            this call's epoch (strictly increasing over calls).
 *   host_step_ids    optional host-mapped pinned int32[n_tokens * k] (or NULL): the step's
 *                    selections in (token, choice) order, written by the decode path
 *                    (<= MOE_DECODE_MAX_TOKENS tokens) before the epoch; a pool's
 *                    recency policy needs the hits as well as the misses. */
typedef struct moe_doorbell {
  int32_t* host_miss_ids;
  int32_t* host_miss_count;
  uint32_t* ready;
  uint32_t epoch;
  int32_t* host_step_ids;
} moe_doorbell;

/* Bytes of one expert blob (layout above) for `dims`; 0 if dims are invalid. */
MOE_API size_t moe_expert_blob_bytes(const moe_dims* dims);

/* Workspace bytes that every entry point below needs for up to `max_tokens` tokens;
 * 0 if dims are invalid or max_tokens < 1. */
MOE_API size_t moe_workspace_bytes(const moe_dims* dims, int32_t max_tokens);

/* Static message for a status code (never NULL). */
MOE_API const char* moe_strerror(int code);

/* Clears the control area at the start of `ws` (its first 4 KiB: error word, counters, miss
 * flags) with a fill kernel on `stream`.  Call once before the workspace's first use. */
MOE_API int moe_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* Synchronizes `stream`, reads the device error word of `ws` into *bits_out (may be NULL)
 * and clears it.  Returns MOE_OK when the word was 0, MOE_EDEVICE otherwise. */
MOE_API int moe_check_device_error(void* ws, void* stream, int32_t* bits_out);

/* Profiling aid.  Until the next call, every launch of kernel `which` (1 = decode gate/up GEMV,
 * 2 = decode down GEMV, 3 = prefill gate/up grouped GEMM, 4 = prefill down grouped
 * GEMM, 5 = decode router GEMV; 0 = off) records the hipEvent_t `start_event` / `stop_event` (created by the caller with
 * timing enabled) around that kernel alone, via hipExtLaunchKernel.  Process-wide setting,
 * not for concurrent use from several threads. */
MOE_API int moe_debug_kernel_events(int32_t which, void* start_event, void* stop_event);

/* Prefill plan (halogen README, "Measured": the engine's GEMM plan carries choices measured on
 * the hardware).  How a prefill call of n_tokens runs: the rows per grouped-GEMM work item (64 or
 * 128), the grouped-GEMM kernel of the gate/up and of the down projection, and the router GEMM's
 * rows per work (32 or 64).  The library takes the plan from a table measured on MI355X per shape
 * and token range (tune.py in the package writes it), else a default.  Kernels:
 *   MOE_GEMM_PIPE128      8 waves x 512 weight rows, up to 128-row items, weights 1 chunk ahead;
 *   MOE_GEMM_PIPE64_DEEP  the same with up to 64-row items and weights 3 chunks ahead;
 *   MOE_GEMM_GENERAL      4 waves x 256 weight rows, every width and weight format.
 * The pipelined kernels exist at the model's reduction widths (gate/up over H = 2048, down over
 * F = 768), for every weight format except the affine one on MOE_GEMM_PIPE128; elsewhere the
 * general kernel runs whatever the plan says. */
enum moe_gemm_kernel { MOE_GEMM_PIPE128 = 0, MOE_GEMM_PIPE64_DEEP = 1, MOE_GEMM_GENERAL = 2 };
typedef struct moe_prefill_plan {
  int32_t item_rows;
  int32_t gate_up_kernel;
  int32_t down_kernel;
  int32_t router_rows;
} moe_prefill_plan;

/* The plan a prefill call of n_tokens with these dims runs (the kernels as they will run). */
MOE_API int moe_prefill_plan_get(const moe_dims* dims, int32_t n_tokens, moe_prefill_plan* out);

/* Tuning aid: every prefill call of the process runs `plan` (validated: item_rows 64 or 128,
 * MOE_GEMM_PIPE64_DEEP only with 64, router_rows 32 or 64; else MOE_EINVAL) until the next call;
 * NULL returns to the table.  Process-wide, not for concurrent use from several threads. */
MOE_API int moe_debug_force_prefill_plan(const moe_prefill_plan* plan_or_null);

/* Test entry point: dequantizes matrix `matrix` (0 = gate [F][H], 1 = up [F][H],
 * 2 = down [H][F]) of the expert blob at `blob` into fp32 `out` (row-major), exactly
 * (q * scale is exact in fp32).  Follows halogen README "Bring your own GGUF" (a small
 * set of values times a per-block scale). */
MOE_API int moe_debug_dequant(const moe_dims* dims, const uint8_t* blob, int32_t matrix,
                              float* out, void* stream);

/* Router and top-k selection (Betelgeuse article, "mechanism": 10 routed experts of 512
 * per token; "what bit-exact means": the selection is exact).
 *   x        [n_tokens][H], dtype x_dtype (MOE_F32 or MOE_BF16).
 *   router   [E][H], dtype router_dtype; bias [E] fp32 or NULL.
 *   topk_ids [n_tokens][k] int32 out: ids ranked by (logit desc, id asc).
 *   topk_w   [n_tokens][k] fp32 out: softmax over the k selected logits.
 *   logits   [n_tokens][E] fp32 out (x . router_e + bias_e), or NULL.
 * Logits accumulate in fp32 (bf16 x bf16 products are exact).  With more than
 * MOE_DECODE_MAX_TOKENS_NARROW tokens both x and router must be bf16. */
MOE_API int moe_route(const moe_dims* dims, const void* x, int32_t x_dtype, int32_t n_tokens,
                      const void* router, int32_t router_dtype, const float* bias,
                      int32_t* topk_ids, float* topk_w, float* logits_or_null,
                      void* ws, size_t ws_bytes, void* stream);

/* In-stream residency check (Betelgeuse article, "mechanism", scheduling row: expert id ->
 * slot on the GPU, host notified only on a miss).
 *   layer_table [E] int32: slot of each expert, -1 = not resident (cached in LDS).
 *   topk_ids    [n_tokens][k].
 *   slots       [n_tokens][k] int32 out: layer_table[id] (-1 for a miss).
 *   miss_ids    [E] int32 out: the distinct missing ids, ascending; miss_count [1] out.
 *   bell        optional doorbell (see moe_doorbell), or NULL.  With a doorbell the call also
 *               publishes the selections to bell->host_step_ids (when not NULL), so a pool
 *               knows the step's hits; it then takes at most MOE_DECODE_MAX_TOKENS tokens
 *               (more: MOE_EUNSUPPORTED).
 * Entries >= n_slots set MOE_DERR_SLOT; ids outside [0, E) set MOE_DERR_EXPERT_ID. */
MOE_API int moe_slot_lookup(const moe_dims* dims, const int32_t* layer_table, int32_t n_slots,
                            const int32_t* topk_ids, int32_t n_tokens, int32_t* slots,
                            int32_t* miss_ids, int32_t* miss_count, const moe_doorbell* bell_or_null,
                            void* ws, size_t ws_bytes, void* stream);

/* Grouping of the (token, choice) pairs p = t*k + j by expert: a stable counting sort.
 *   counts [E] out, offsets [E+1] out (exclusive prefix sums), perm [n_tokens*k] out:
 *   pair indices in (expert, p) order.  (halogen README, "Measured": the ordering step
 *   of the tokens moves prefill speed.)  A token's k ids must be distinct (as moe_route
 *   writes them); a repeated id sets MOE_DERR_DUP_ID and the outputs are invalid. */
MOE_API int moe_group_tokens(const moe_dims* dims, const int32_t* topk_ids, int32_t n_tokens,
                             int32_t* counts, int32_t* offsets, int32_t* perm,
                             void* ws, size_t ws_bytes, void* stream);

/* Expert FFNs + combine for a small batch (1..MOE_DECODE_MAX_TOKENS tokens with bf16 x and
 * F <= 2048, else 1..MOE_DECODE_MAX_TOKENS_NARROW; more: MOE_EINVAL).  Betelgeuse
 * article, "mechanism": every token runs its 10 routed experts and the shared expert, all of
 * them, none dropped; halogen README, "Bring your own GGUF": decode pays per byte of weights
 * read.  So each distinct selected expert's blob is streamed once per call, whatever the
 * number of tokens that chose it: 4-bit GEMVs, codes entering the matrix cores exactly,
 * fp32 accumulation, bandwidth-bound.
 *   layer_table [E] or NULL (NULL: expert e sits in slot e, all resident).
 *   x [n_tokens][H] (MOE_F32 or MOE_BF16); topk_ids / topk_w [n_tokens][k] (as moe_route
 *   writes them: a token's ids distinct, else MOE_DERR_DUP_ID); y [n_tokens][H] fp32 out.
 * Every expert a token selected must be resident (else MOE_DERR_NOT_RESIDENT). */
MOE_API int moe_expert_ffn_decode(const moe_dims* dims, const moe_layer_weights* w,
                                  const int32_t* layer_table_or_null, const void* x, int32_t x_dtype,
                                  int32_t n_tokens, const int32_t* topk_ids, const float* topk_w,
                                  float* y, void* ws, size_t ws_bytes, void* stream);

/* Expert FFNs + combine for a long batch (prefill).  halogen README, "Measured": prefill is
 * compute-bound and the ordering of tokens moves its speed; Basalt README, "Prompt chunks":
 * a chunk's cost per token keeps falling up to a few thousand tokens.  Tokens are grouped by
 * expert (a stable counting sort), and each expert's rows run as a grouped GEMM on MFMA with
 * dequantized fp16 tiles and fp32 accumulation, SwiGLU fused into the gate/up epilogue.
 * x must be MOE_BF16.  Arguments as moe_expert_ffn_decode, any n_tokens >= 1.  The fp16
 * operands and intermediates hold |v| <= 65504: a bf16 activation, a SwiGLU output or a
 * router-weighted expert row beyond that sets MOE_DERR_RANGE (the output is then invalid). */
MOE_API int moe_expert_ffn_prefill(const moe_dims* dims, const moe_layer_weights* w,
                                   const int32_t* layer_table_or_null, const void* x, int32_t x_dtype,
                                   int32_t n_tokens, const int32_t* topk_ids, const float* topk_w,
                                   float* y, void* ws, size_t ws_bytes, void* stream);

/* The whole layer (Betelgeuse article, "mechanism": router and shared expert resident, 10
 * routed experts of 512 per token, the residency check in the stream and the host rung only
 * on a miss): route -> residency check -> (wait for fills) -> expert FFNs -> combine.
 * Uses the decode kernels up to the decode limit (MOE_DECODE_MAX_TOKENS for bf16 x and router
 * and F <= 2048, else MOE_DECODE_MAX_TOKENS_NARROW) and the prefill kernels above.  With a layer_table and a doorbell, misses are reported to the host and the FFNs
 * run after *bell->ready >= bell->epoch (the host fills the slots and updates the table
 * meanwhile); a doorbell is taken only by a decode-sized call (n_tokens within the decode
 * limit; more: MOE_EUNSUPPORTED), since the host's recency policy needs the
 * step's selections.  topk_ids_out / topk_w_out [n_tokens][k] receive the routing if not
 * NULL. */
MOE_API int moe_layer_forward(const moe_dims* dims, const moe_layer_weights* w,
                              const int32_t* layer_table_or_null, const moe_doorbell* bell_or_null,
                              const void* x, int32_t x_dtype, int32_t n_tokens, float* y,
                              int32_t* topk_ids_out_or_null, float* topk_w_out_or_null,
                              void* ws, size_t ws_bytes, void* stream);

/* The whole layer without a caller workspace, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid allocation).  Same
 * arguments and results as moe_layer_forward, with two differences:
 *   - the workspace is a library-owned static device array of MOE_STATIC_SCRATCH_BYTES per GPU
 *     (held from the first call on that GPU until the process ends); a call whose workspace
 *     would exceed it (moe_workspace_bytes(dims, n_tokens) > MOE_STATIC_SCRATCH_BYTES; the
 *     model shape fits up to about 100 tokens) returns MOE_EWORKSPACE, enqueueing nothing;
 *   - device_error_out (device int32[1], required) receives the call's device error bits
 *     (0 = none; the moe_device_error bits otherwise), copied from the array and cleared there
 *     by the call's last kernel.
 * It calls no hipMalloc, hipFree or allocating routine.  Every call on one GPU shares that GPU's
 * array: calls that may overlap on one GPU (different streams, or other threads) race and must be
 * ordered by the caller.  The first call on a GPU looks the array up and clears its control words
 * on `stream`. */
#define MOE_STATIC_SCRATCH_BYTES (8u << 20)
MOE_API int moe_layer_forward_static(const moe_dims* dims, const moe_layer_weights* w,
                                     const int32_t* layer_table_or_null, const moe_doorbell* bell_or_null,
                                     const void* x, int32_t x_dtype, int32_t n_tokens, float* y,
                                     int32_t* topk_ids_out_or_null, float* topk_w_out_or_null,
                                     int32_t* device_error_out, void* stream);

/* ---- Host service of a per-layer expert-slot pool (decode calls) ----------------------------
 * Betelgeuse news article, section "mechanism: VRAM expert-slot pool, in-stream doorbell and
 * victim cache": a layer keeps a fixed number of HBM slots, the in-stream check rings the host
 * only on a miss, a miss is filled from host memory, and the HBM and host copies of an expert
 * are exclusive.  Policy (the article names none): least recently used among the slots whose
 * expert is not selected in the step, ties to the lower slot; misses placed in ascending id
 * order; recency stamped per selection in (token, choice) order.
 *
 * Use per layer call: moe_pool_arm -> moe_layer_forward(..., table, &bell, ...) on the compute
 * stream -> moe_pool_serve on the host (it blocks until the call's check has run, then
 * enqueues the copies, the table update and the release of the compute stream on its copy
 * streams).  Several layers' calls may be enqueued before their serves; serve them in the
 * same order.  A pool is used from one host thread and one pair of copy streams (or one).
 *
 * The compute stream's wait stalls whatever the runtime has queued behind it on the same
 * hardware queue, and the runtime spreads streams over a few such queues (4 by default).
 * Create the compute stream and the copy streams together, non-blocking, before other
 * streams (a framework's stream pool, graph capture streams) exist: a copy stream that ends
 * up behind the wait never runs, and the next serve then times out.  Each serve failure is
 * also reported on stderr with its epoch and reason. */
typedef struct moe_pool moe_pool;

#define MOE_POOL_MAX_SPARES 64

typedef struct moe_pool_stats {
  int64_t calls;       /* served calls */
  int64_t selections;  /* (token, choice) selections seen */
  int64_t misses;      /* distinct misses filled */
  int64_t bytes_h2d;   /* expert bytes copied host -> HBM */
  int64_t bytes_d2h;   /* expert bytes copied HBM -> host (exclusive swap) */
} moe_pool_stats;

/* Creates the service for one layer.  All memory is the caller's and must outlive the pool:
 *   arena, slot_stride, n_slots  device slots (as in moe_layer_weights), n_slots <= E;
 *   table          device int32[E]: written here (slot of each expert, -1 elsewhere) and kept
 *                  up to date by moe_pool_serve; pass it as the layer_table of the calls;
 *   initial        host int32[n_slots]: the distinct expert held by each slot, hottest first
 *                  (colder ones are evicted first); their blobs must already be in the slots;
 *   host_home      host array [E] of pinned host pointers: the blob of every expert not in
 *                  `initial`, NULL for those in it (the pool permutes these buffers);
 *   spares, n_spares  n_spares (1..MOE_POOL_MAX_SPARES) pinned host buffers holding no
 *                  expert, at spares + i * slot_stride; the pool permutes them with host_home
 *                  (a miss's victim goes to the oldest, the missed expert's buffer becomes the
 *                  newest); more spares let the copies out run ahead of the copies in;
 *   host_miss_ids  host-mapped pinned int32[E]; host_counts host-mapped pinned int32[3];
 *   host_step_ids  host-mapped pinned int32[MOE_DECODE_MAX_TOKENS * k];
 *   ready          device uint32 (set to 0 here).
 * Copies the table and the ready word synchronously.  Returns MOE_EINVAL on inconsistent
 * arguments (a slot holding an id out of range or twice, an expert with no or two homes). */
MOE_API int moe_pool_create(const moe_dims* dims, uint8_t* arena, int64_t slot_stride, int32_t n_slots,
                            int32_t* table, const int32_t* initial, uint8_t* const* host_home, uint8_t* spares,
                            int32_t n_spares, int32_t* host_miss_ids, int32_t* host_counts,
                            int32_t* host_step_ids, uint32_t* ready, moe_pool** pool_out);

/* Frees the pool object and its events (not the caller's memory).  Synchronize the pool's copy
 * streams first: the copies it enqueued and their event waits must have completed. */
MOE_API int moe_pool_destroy(moe_pool* pool);

/* The doorbell of the pool's next call (next epoch).  MOE_EINVAL if the previous call was
 * armed but not served. */
MOE_API int moe_pool_arm(moe_pool* pool, moe_doorbell* bell_out);

/* Serves the armed call: waits on the host until the check kernel has written the epoch
 * (polling host memory, at most timeout_us microseconds if > 0), places every miss, and
 * enqueues per miss a device->host copy of the victim into a spare buffer on d2h_stream and a
 * host->device copy of the missed expert into the victim's slot on h2d_stream (ordered after
 * that device->host copy by an event), then on h2d_stream the table and *ready = epoch.
 * h2d_stream_or_null NULL puts everything on d2h_stream.  With two streams the copies of the
 * two PCIe directions overlap; a device->host copy into a buffer waits for the host->device
 * copy that last read it, and a serve's first one waits for the previous serve's copies in
 * (its victims may be slots those filled).  fills_out (host int32[E][3] or NULL)
 * receives (expert, slot, evicted expert) per fill, n_fills_out their number.  On a timeout,
 * a bad doorbell or a failed copy the compute stream is still released (*ready = epoch), the
 * fill error bit is set in ws (when not NULL) and MOE_EFILL is returned. */
MOE_API int moe_pool_serve(moe_pool* pool, void* ws_or_null, void* d2h_stream, void* h2d_stream_or_null,
                           int32_t* fills_out, int32_t* n_fills_out, int64_t timeout_us);

/* Counters since creation. */
MOE_API int moe_pool_get_stats(const moe_pool* pool, moe_pool_stats* out);

/* The pool's current slot table (host int32[E]). */
MOE_API int moe_pool_get_table(const moe_pool* pool, int32_t* table_out);

/* Hot-expert profile (Betelgeuse article, "limits and licence": a profile file only seeds the
 * cache with hot experts; "mechanism": the package carries a hot-expert profile).
 * moe_pool_get_profile: host int64[E], the selections of every expert the pool has served
 * (hits and misses) since creation.
 * moe_profile_seed: from such counts, the initial residency of a pool of n_slots slots: the
 * n_slots experts with the most selections, hottest first (ties: lower id first), as
 * moe_pool_create's `initial` takes it (host int32[n_slots] out).  1 <= n_slots <= n_experts. */
MOE_API int moe_pool_get_profile(const moe_pool* pool, int64_t* counts_out);
MOE_API int moe_profile_seed(const int64_t* counts, int32_t n_experts, int32_t n_slots, int32_t* initial_out);

/* Slot lending (Basalt README, "Prompt chunks: --prefill": a prompt chunk's buffers are carved
 * from the expert cache's last slots for the length of the prompt, and the experts in those slots
 * are copied back afterwards).  moe_pool_lend lends the pool's last n slots (n_slots - n ..
 * n_slots - 1, one contiguous region of n * slot_stride bytes at *region_out, e.g. another call's
 * workspace): on `stream` it copies their experts out to host_bufs (caller's pinned host memory,
 * n * slot_stride bytes, which holds them meanwhile: the tiers stay exclusive) and marks them not
 * resident in the table.  Use the region only after those copies (same stream, or an event).
 * moe_pool_unlend copies the experts back on `stream` (after the caller's last use of the region
 * in that stream's order) and restores the table; the recency policy is as if nothing had been
 * lent.  Neither may be called while a call is armed; moe_pool_arm refuses while slots are lent
 * (MOE_EINVAL).  A failed copy enqueue returns MOE_EFILL with the lend state unchanged. */
MOE_API int moe_pool_lend(moe_pool* pool, int32_t n, uint8_t* host_bufs, void* stream, uint8_t** region_out);
MOE_API int moe_pool_unlend(moe_pool* pool, void* stream);

/* Test hook for the failure path: after `after_n` more successful copy enqueues, the pool treats
 * the next one as failed (the copy is not enqueued), as a failed hipMemcpyAsync would be: serve
 * then releases the compute stream with MOE_DERR_FILL set and returns MOE_EFILL (Betelgeuse article,
 * "what bit-exact means": a failed expert read is an error, never zero weights).  -1 = off. */
MOE_API int moe_pool_debug_fail_copies(moe_pool* pool, int32_t after_n);

/* ---- Dense operators ------------------------------------------------------------------------
 * What stands beside the routed experts in a model and has plain 16-bit weights: a dense shared
 * expert or the dense feed-forward blocks of its first layers, projections, the output head; each
 * with its backward pass.  Row-major matrices, one row per token; a weight is [n_out][n_in]:
 *
 *   linear  z = x W^T + b               y = act(z) + r                       (b, r optional)
 *           dz = dy * act'(z)           dx = dz W    dW = dz^T x    db = sum_t dz
 *   gated   g = x Wg^T + bg, u = x Wu^T + bu         h = act(g) * u
 *           dg = dh * u * act'(g)       du = dh * act(g)
 *           dx = dg Wg + du Wu          dWg = dg^T x   dWu = du^T x   dbg = sum_t dg   dbu = sum_t du
 *
 * A gated block whose h goes through a linear (W [hidden][F], r = the routed layer's fp32 y) adds a
 * dense shared expert to moe_layer_forward's output.
 *
 * Conventions, beyond those at the top of this file (whose 16-byte rule for x and y does not hold here):
 *   - dims->dtype is the type of x, every weight, bias, saved pre-activation, h, incoming gradient
 *     and result of a backward pass: MOE_BF16 or MOE_F16 (anything else: MOE_EUNSUPPORTED).  y and r of the
 *     linear share y_dtype: dims->dtype or MOE_F32.
 *   - ld* is a matrix's row stride in elements, at least its row length and at most MOE_DENSE_MAX_LD;
 *     rows may start at any element-aligned address (a slice of a wider tensor, an odd width; an odd
 *     address is MOE_EINVAL).  Operands on 16-byte addresses with strides (and n_in) a multiple of 8 run the
 *     asynchronous-copy kernels, whatever each one's stride is.  Otherwise x (and the weights, where n_in is no
 *     multiple of 8) is first copied into the workspace where that pays, and the rest runs kernels of about half the rate.
 *   - 1 <= n_in, n_out <= MOE_DENSE_MAX_WIDTH; 1 <= n_tokens <= MOE_DENSE_MAX_TOKENS (beyond:
 *     MOE_EUNSUPPORTED).
 *   - Sums are fp32 in a fixed order, so equal calls give equal bits.  Up to
 *     MOE_DENSE_ROW_TOKENS tokens a forward pass gives a token the same bits alone and in any batch.
 *     Results are rounded to their type once (to nearest even); a value beyond fp16's range becomes
 *     infinite, as the type has it.  The backward passes round dz (dg, du) to dims->dtype before the
 *     matrix products; the bias gradients sum it unrounded.  In fp16 a dz past 65504 is thus an infinity to its token's
 *     dx and its output's dW, finite though they may be, and one below 2^-25 is zero: scale the incoming gradient.
 *   - silu and sigmoid are 0 below z = -87 (by definition less than 2^-118 from it).
 *   - A NaN or an infinity stays in the rows and columns that its definition reaches; nothing between the
 *     rows of a matrix (ld > row length) is used, nor written.
 *   - A pre-activation past dims->dtype's range is saved as an infinity.  The backward passes take the limits
 *     there: act' is 0 or 1, act is 0, 1 or infinite; a zero gradient (or act') times an infinite factor is 0.
 *   - Outputs must not overlap inputs or each other, except y on r exactly (same address and
 *     stride).  A NULL output of a backward pass is not computed; at least one must be given.
 *   - A launch that fails (MOE_EHIP) may leave a call's earlier launches enqueued.
 *   - `ws` as everywhere: moe_dense_workspace_bytes(dims, n_tokens, backward) bytes, cleared once
 *     with moe_workspace_init.  The layer's calls and these may share one, ordered on one stream.
 */
#define MOE_DENSE_MAX_WIDTH (1 << 20)
#define MOE_DENSE_MAX_LD (1 << 22)
#define MOE_DENSE_MAX_TOKENS (1 << 24)
#define MOE_DENSE_ROW_TOKENS 16

/* MOE_ACT_GELU is z * Phi(z) (erf), MOE_ACT_GELU_TANH its tanh form; relu'(0) = 0.  The gated block
 * takes any of them as its act (MOE_ACT_NONE: the bilinear block h = g * u). */
enum moe_act { MOE_ACT_NONE = 0, MOE_ACT_SILU = 1, MOE_ACT_GELU = 2, MOE_ACT_GELU_TANH = 3, MOE_ACT_RELU = 4,
               MOE_ACT_SIGMOID = 5 };

typedef struct moe_dense_dims {
  int32_t n_in;   /* row length of x and of every weight */
  int32_t n_out;  /* rows of each weight; row length of y, z (g, u, h) */
  int32_t dtype;  /* MOE_BF16 or MOE_F16 */
  int32_t act;    /* moe_act */
} moe_dense_dims;

/* Workspace bytes that the forward calls (backward = 0) or all calls (backward = 1) with `dims` need
 * for up to `max_tokens` tokens; 0 if dims are invalid or max_tokens out of range. */
MOE_API size_t moe_dense_workspace_bytes(const moe_dense_dims* dims, int32_t max_tokens, int32_t backward);

/* Tuning aid: every dense product of the process runs this tile kernel (MOE_DENSE_AUTO: chosen by size, the
 * default; the MOE_DENSE_TILE ones only where the rows are whole 16-byte chunks), and every dense call this many
 * splits of its reductions (1..8, as far as the workspace holds their sums; 0: chosen by size).  Process-wide,
 * not for concurrent use from several threads. */
enum moe_dense_kernel { MOE_DENSE_AUTO = 0, MOE_DENSE_TILE64 = 1, MOE_DENSE_TILE128 = 2, MOE_DENSE_TILE256 = 3,
                        MOE_DENSE_ANY64 = 4, MOE_DENSE_ANY128 = 5 };
MOE_API int moe_debug_force_dense_plan(int32_t kernel, int32_t splits);

/* y [n_tokens][n_out] (y_dtype) = act(x W^T + bias) + residual.
 *   x [n_tokens][n_in]; w [n_out][n_in]; bias [n_out] or NULL; residual [n_tokens][n_out] of
 *   y_dtype or NULL (ld_residual is then ignored); pre [n_tokens][n_out] or NULL receives z for the
 *   backward pass (ld_pre ignored when NULL). */
MOE_API int moe_linear_forward(const moe_dense_dims* dims, const void* x, int64_t ldx, int32_t n_tokens, const void* w,
                               int64_t ldw, const void* bias_or_null, const void* residual_or_null, int64_t ld_residual,
                               void* y, int64_t ldy, int32_t y_dtype, void* pre_or_null, int64_t ld_pre, void* ws,
                               size_t ws_bytes, void* stream);

/* Gradients of moe_linear_forward's act(x W^T + bias); the residual's is dy itself.
 *   pre = the saved z (required unless act is MOE_ACT_NONE; then ignored); dy [n_tokens][n_out];
 *   dx [n_tokens][n_in], dw [n_out][n_in], dbias [n_out]: NULL = not wanted. */
MOE_API int moe_linear_backward(const moe_dense_dims* dims, const void* x, int64_t ldx, int32_t n_tokens, const void* w,
                                int64_t ldw, const void* pre_or_null, int64_t ld_pre, const void* dy, int64_t ld_dy,
                                void* dx_or_null, int64_t ld_dx, void* dw_or_null, int64_t ld_dw, void* dbias_or_null,
                                void* ws, size_t ws_bytes, void* stream);

/* h [n_tokens][n_out] = act(x Wg^T + bias_gate) * (x Wu^T + bias_up); both projections, the activation and the
 * product in one pass.  w_gate and w_up [n_out][n_in] may be the halves of one [2 n_out][n_in]
 * tensor.  gate / up [n_tokens][n_out] or NULL receive g and u for the backward pass (both or neither). */
MOE_API int moe_gated_forward(const moe_dense_dims* dims, const void* x, int64_t ldx, int32_t n_tokens,
                              const void* w_gate, int64_t ld_wg, const void* w_up, int64_t ld_wu,
                              const void* bias_gate_or_null, const void* bias_up_or_null, void* h, int64_t ldh,
                              void* gate_or_null, int64_t ld_gate, void* up_or_null, int64_t ld_up, void* ws,
                              size_t ws_bytes, void* stream);

/* Gradients of moe_gated_forward.  gate, up = the saved g and u; dh [n_tokens][n_out]; every output
 * NULL = not wanted. */
MOE_API int moe_gated_backward(const moe_dense_dims* dims, const void* x, int64_t ldx, int32_t n_tokens,
                               const void* w_gate, int64_t ld_wg, const void* w_up, int64_t ld_wu, const void* gate,
                               int64_t ld_gate, const void* up, int64_t ld_up, const void* dh, int64_t ld_dh,
                               void* dx_or_null, int64_t ld_dx, void* dw_gate_or_null, int64_t ld_dwg,
                               void* dw_up_or_null, int64_t ld_dwu, void* dbias_gate_or_null, void* dbias_up_or_null,
                               void* ws, size_t ws_bytes, void* stream);

/* ---- Rows by expert ---------------------------------------------------------------------------
 * The routed layer's data movement where its experts are not the 4-bit blobs of moe_layer_forward, for
 * training and for 16-bit experts: token rows laid out by expert and back, with the router weights
 * applied, each with its gradient.  With the pairs p = t*k + j of moe_group_tokens, perm[r] the pair in
 * row r, inv[p] the row of pair p:
 *
 *   dispatch  xs[r] = x[perm[r] / k]                   dx[t] = sum_j dxs[inv[t*k+j]] + r[t]    (r optional)
 *   combine   y[t] = sum_j w[t][j] ys[inv[t*k+j]] + r[t]                                       (r optional)
 *             dys[r] = w[perm[r]] dy[perm[r] / k]      dw[t][j] = sum_i dy[t][i] ys[inv[t*k+j]][i]
 *
 * Conventions, beyond those at the top of this file and those of the dense operators for types, strides,
 * alignment, overlap and rounding:
 *   - perm [n_rows] is moe_group_tokens' or a caller's own.  A negative entry is a padding row (groups
 *     padded to a multiple, room behind the last group): zero in xs and dys, read by nobody.  A pair that no
 *     row has (a dropped one) has inv = -1: it adds nothing, its dw is 0.
 *   - A pair >= n_tokens * k in perm, a pair in two rows, an inv entry >= n_rows and, in the combine's backward
 *     pass, an inv that is not perm's set MOE_DERR_ROWS: what they name is taken as absent, no access
 *     leaves the arrays, and the call's outputs are invalid.
 *   - Sums are fp32, over j (or i) in a fixed order: equal calls give equal bits.
 *   - 1 <= k <= 16; 1 <= width <= MOE_DENSE_MAX_WIDTH; 1 <= n_tokens <= MOE_DENSE_MAX_TOKENS;
 *     1 <= n_rows <= MOE_ROWS_MAX (beyond: MOE_EUNSUPPORTED).
 *   - `ws`: moe_rows_workspace_bytes(dims, n_tokens) bytes, or any larger workspace of the library's.
 */
#define MOE_ROWS_MAX (1 << 28)

typedef struct moe_rows_dims {
  int32_t width;  /* row length of x, xs, ys, y and their gradients */
  int32_t top_k;  /* pairs per token */
  int32_t dtype;  /* of x, xs, ys, dxs, dys: MOE_BF16 or MOE_F16 */
} moe_rows_dims;

/* Workspace bytes of the calls below; 0 if dims are invalid or max_tokens out of range. */
MOE_API size_t moe_rows_workspace_bytes(const moe_rows_dims* dims, int32_t max_tokens);

/* xs [n_rows][width] = the rows of x [n_tokens][width] that perm [n_rows] names; inv [n_tokens][k] out. */
MOE_API int moe_dispatch_forward(const moe_rows_dims* dims, const void* x, int64_t ldx, int32_t n_tokens,
                                 const int32_t* perm, int32_t n_rows, void* xs, int64_t ld_xs, int32_t* inv, void* ws,
                                 size_t ws_bytes, void* stream);

/* dx [n_tokens][width] (dx_dtype: dims->dtype or MOE_F32) = each token's sum of its rows of dxs [n_rows][width],
 * plus residual of dx_dtype, if not NULL (the gradient that reaches x by another way). */
MOE_API int moe_dispatch_backward(const moe_rows_dims* dims, const void* dxs, int64_t ld_dxs, int32_t n_rows,
                                  const int32_t* inv, int32_t n_tokens, const void* residual_or_null,
                                  int64_t ld_residual, void* dx, int64_t ld_dx, int32_t dx_dtype, void* ws,
                                  size_t ws_bytes, void* stream);

/* y [n_tokens][width] (y_dtype: dims->dtype or MOE_F32) from ys [n_rows][width] and topk_w [n_tokens][k] fp32;
 * residual of y_dtype or NULL (a shared expert's output, the stream it is added to). */
MOE_API int moe_combine_forward(const moe_rows_dims* dims, const void* ys, int64_t ld_ys, int32_t n_rows,
                                const int32_t* inv, const float* topk_w, int32_t n_tokens, const void* residual_or_null,
                                int64_t ld_residual, void* y, int64_t ldy, int32_t y_dtype, void* ws, size_t ws_bytes,
                                void* stream);

/* Gradients of moe_combine_forward from dy [n_tokens][width] of dy_dtype (dims->dtype or MOE_F32); the residual's is
 * dy itself.  dys [n_rows][width] and dtopk_w [n_tokens][k] fp32: NULL = not wanted (not both).  ys is needed for
 * dtopk_w only (else ignored, may be NULL). */
MOE_API int moe_combine_backward(const moe_rows_dims* dims, const void* dy, int64_t ld_dy, int32_t dy_dtype,
                                 int32_t n_tokens, const int32_t* perm, const int32_t* inv, int32_t n_rows,
                                 const float* topk_w, const void* ys_or_null, int64_t ld_ys, void* dys_or_null,
                                 int64_t ld_dys, float* dtopk_w_or_null, void* ws, size_t ws_bytes, void* stream);

/* ---- Experts' products with 16-bit weights -----------------------------------------------------
 * What runs between moe_dispatch_forward and moe_combine_forward: expert e's matrices on its rows offsets[e] ..
 * offsets[e+1] - 1 of the rows laid out by expert (moe_group_tokens' offsets, or a caller's own), and the gradients:
 *
 *   linear  y_r = W_e x_r                              dx_r = W_e^T dy_r               dW_e = sum_r dy_r x_r^T
 *   gated   g_r = Wg_e x_r, u_r = Wu_e x_r             h_r = act(g_r) * u_r
 *           dg = dh * u * act'(g), du = dh * act(g)    dx_r = Wg_e^T dg_r + Wu_e^T du_r
 *           dWg_e = sum_r dg_r x_r^T                   dWu_e = sum_r du_r x_r^T
 *
 * Conventions, beyond those of the dense operators (types, strides, alignment, rounding, saved infinities, overlap):
 *   - weights and their gradients are [E][n_out][n_in]: row stride ld, matrices `stride` elements apart (both matrices
 *     of a gated block alike; they may be the halves of one [E][2 n_out][n_in] tensor).
 *   - offsets [E+1] lives on the device; no call waits for it.  An expert may have any number of rows, none among them:
 *     its dW is then zero.  Rows before offsets[0] and from offsets[E] on belong to nobody: no result of theirs is
 *     written.  Padding rows of a group are rows like any other.  The backward passes make dz of every one of the n_rows
 *     rows in the workspace, but use those of groups only.
 *   - Offsets that descend or leave 0 .. n_rows set MOE_DERR_ROWS: they are clamped, no access leaves the arrays, the
 *     results are invalid.
 *   - Sums are fp32 in an order that depends on the shapes (n_rows among them) and an expert's rows, not on where its rows lie.
 *   - 1 <= n_experts <= 1024; 1 <= n_rows <= MOE_ROWS_MAX.  The linear takes MOE_ACT_NONE only.
 *   - moe_debug_force_dense_plan's kernel holds here too.
 *   - `ws`: moe_experts_workspace_bytes(dims, n_rows, backward) bytes.
 */
typedef struct moe_experts_dims {
  int32_t n_experts;
  int32_t n_in;   /* row length of xs and of every weight */
  int32_t n_out;  /* rows of each weight; row length of ys, g, u, h */
  int32_t dtype;  /* MOE_BF16 or MOE_F16 */
  int32_t act;    /* moe_act; linear: MOE_ACT_NONE */
} moe_experts_dims;

/* Workspace bytes that the forward calls (backward = 0) or all calls (backward = 1) need for up to `max_rows` rows;
 * 0 if dims are invalid or max_rows out of range. */
MOE_API size_t moe_experts_workspace_bytes(const moe_experts_dims* dims, int32_t max_rows, int32_t backward);

/* ys [n_rows][n_out] = each row of xs [n_rows][n_in] through its expert's matrix. */
MOE_API int moe_experts_linear_forward(const moe_experts_dims* dims, const void* xs, int64_t ld_xs, int32_t n_rows,
                                       const int32_t* offsets, const void* w, int64_t ldw, int64_t w_stride, void* ys,
                                       int64_t ld_ys, void* ws, size_t ws_bytes, void* stream);

/* Gradients of moe_experts_linear_forward from dys [n_rows][n_out]; dxs [n_rows][n_in], dw: NULL = not wanted (not both). */
MOE_API int moe_experts_linear_backward(const moe_experts_dims* dims, const void* xs, int64_t ld_xs, int32_t n_rows,
                                        const int32_t* offsets, const void* w, int64_t ldw, int64_t w_stride,
                                        const void* dys, int64_t ld_dys, void* dxs_or_null, int64_t ld_dxs,
                                        void* dw_or_null, int64_t ld_dw, int64_t dw_stride, void* ws, size_t ws_bytes,
                                        void* stream);

/* h [n_rows][n_out] = the gated block of each row's expert, in one pass.  gate / up [n_rows][n_out] (one stride,
 * ld_saved) or NULL receive g and u for the backward pass (both or neither). */
MOE_API int moe_experts_gated_forward(const moe_experts_dims* dims, const void* xs, int64_t ld_xs, int32_t n_rows,
                                      const int32_t* offsets, const void* w_gate, const void* w_up, int64_t ldw,
                                      int64_t w_stride, void* h, int64_t ldh, void* gate_or_null, void* up_or_null,
                                      int64_t ld_saved, void* ws, size_t ws_bytes, void* stream);

/* Gradients of moe_experts_gated_forward from dh [n_rows][n_out] and the saved gate and up; dw_gate and dw_up share
 * ld_dw and dw_stride; every output NULL = not wanted (not all). */
MOE_API int moe_experts_gated_backward(const moe_experts_dims* dims, const void* xs, int64_t ld_xs, int32_t n_rows,
                                       const int32_t* offsets, const void* w_gate, const void* w_up, int64_t ldw,
                                       int64_t w_stride, const void* gate, const void* up, int64_t ld_saved,
                                       const void* dh, int64_t ld_dh, void* dxs_or_null, int64_t ld_dxs,
                                       void* dw_gate_or_null, void* dw_up_or_null, int64_t ld_dw, int64_t dw_stride,
                                       void* ws, size_t ws_bytes, void* stream);

/* ---- Loss over an output head ------------------------------------------------------------------
 * Softmax cross entropy of z = x W^T over a vocabulary, with its gradient, in pieces of the vocabulary: the logits are
 * never kept (a moe_linear_forward of the same sizes writes them; this is its training form).
 *
 *   lse_t = log sum_v exp(z_tv)        loss_t = lse_t - z_t,target
 *   dz_tv = dloss_t (exp(z_tv - lse_t) - [v = target])      dx = dz W      dW = dz^T x
 *
 * Conventions, beyond those of the dense operators (types, strides, alignment, rounding, overlap):
 *   - targets [n_tokens] int32.  A token whose target is `ignore` has loss and lse 0 and no gradient (x may hold
 *     anything finite).  Any other target outside [0, vocab) sets MOE_DERR_TARGET: its loss and lse are NaN, it adds
 *     nothing to the gradients.
 *   - loss, lse, dloss [n_tokens] fp32.  Reductions over the tokens are the caller's: dloss is 1 / count for their mean, a
 *     token's weight for a weighted one.
 *   - Logits are fp32 sums and are not rounded.  loss is formed from what the other columns add to the target's, so
 *     that a small loss keeps its relative precision; the gradient takes both saved values for the same reason
 *     (exp(z - lse) - 1 at the target is expm1(-loss)).
 *   - The backward pass computes the logits again and rounds dz to dims->dtype before the products, with dloss taken
 *     relative to the largest |dloss| of the call (undone in fp32 afterwards).  fp16: relative to a power of two near the
 *     token's own, so that its probabilities keep fp16's precision down to 2^-27 and are zero below 2^-38, however its dloss
 *     compares; dW then takes x times the token's share of the largest |dloss| (a power of two), rounded to fp16 with the call's
 *     largest |x| at 2^14: exact down to 2^-28 of that, zero below 2^-39.  A result past 65504 is an infinity, one below 2^-25
 *     zero: scale dloss.
 *   - An infinite logit gives the limits: loss 0 where it is the target's alone, infinite where it is another's (the
 *     gradient of that column is then NaN), NaN where it is both; a NaN stays in its token, its dx and the dW it reaches.
 *   - Sums are in a fixed order: equal calls give equal bits.
 *   - 1 <= n_in, vocab <= MOE_DENSE_MAX_WIDTH; 1 <= n_tokens <= MOE_LOSS_MAX_TOKENS (beyond: MOE_EUNSUPPORTED).
 *   - moe_debug_force_dense_plan holds here too.
 *   - `ws`: moe_loss_workspace_bytes(dims, n_tokens or more, backward) bytes.  Forward: 8 bytes per 64 columns and a copy of x,
 *     both for 8192 tokens at most, and a copy of W where n_in is no multiple of 8.  Backward: that with a copy of all of x, up
 *     to 256 MiB of dz (beyond 2^19 tokens 512 bytes per token), with more than one piece dx in fp32, up to 32 MiB of split sums;
 *     fp16: another copy of x.
 */
#define MOE_LOSS_MAX_TOKENS (1 << 20)

typedef struct moe_loss_dims {
  int32_t n_in;    /* row length of x and W */
  int32_t vocab;   /* rows of W */
  int32_t dtype;   /* of x, W, dx, dW: MOE_BF16 or MOE_F16 */
  int32_t ignore;  /* target of tokens that are left out: any value, inside [0, vocab) too (a padding token's id) */
} moe_loss_dims;

/* Workspace bytes that the forward call (backward = 0) or both calls (backward = 1) need for up to `max_tokens`
 * tokens; 0 if dims are invalid or max_tokens out of range. */
MOE_API size_t moe_loss_workspace_bytes(const moe_loss_dims* dims, int32_t max_tokens, int32_t backward);

/* loss and lse [n_tokens] of x [n_tokens][n_in] against w [vocab][n_in]. */
MOE_API int moe_loss_forward(const moe_loss_dims* dims, const void* x, int64_t ldx, int32_t n_tokens, const void* w,
                             int64_t ldw, const int32_t* targets, float* loss, float* lse, void* ws, size_t ws_bytes,
                             void* stream);

/* dx [n_tokens][n_in] and dw [vocab][n_in] (NULL = not wanted, not both) from moe_loss_forward's loss and lse. */
MOE_API int moe_loss_backward(const moe_loss_dims* dims, const void* x, int64_t ldx, int32_t n_tokens, const void* w,
                              int64_t ldw, const int32_t* targets, const float* loss, const float* lse,
                              const float* dloss, void* dx_or_null, int64_t ld_dx, void* dw_or_null, int64_t ld_dw,
                              void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTE_H */
