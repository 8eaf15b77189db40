/*
 * megamoe.h -- C ABI of the GB300 (sm_103a) NVFP4 MegaMoE routed-expert forward,
 * with, around it, the router (megamoe_router_topk, and
 * megamoe_forward_from_logits for the whole layer from router logits, a
 * shared expert included) and the dense NVFP4 linear with a measured-amax
 * scale (megamoe_linear_nvfp4); and the scored router and the MXFP4 operators
 * (megamoe_router_scored_topk, megamoe_quantize_mxfp4, megamoe_linear_mxfp4,
 * megamoe_forward_mxfp4 and their companions), the experts' operators in 16 bits
 * with their gradients (megamoe_grouped_linear and its companions) and the linear
 * in 8-bit integers (megamoe_linear_int8), at the end of this file.
 *
 * What it computes (sources are the titles and sections of the pages the
 * method is taken from):
 *   "CURRENT_BUG.md -- DeepSeek-V4 Blackwell NVFP4"
 *     - "Architecture: DeepSeek-V4 MegaMoE": 384 experts with top-6 routing
 *       and a persistent grouped GEMM whose groups are the experts;
 *     - "What's Been Verified": the MoE is the L1 gate+up GEMM and the L2 down
 *       GEMM, both NVFP4;
 *     - "Test Plan -- Finding the NaN", Phase 1: the runner takes
 *       hidden_states, topk_ids, topk_weights and variable per-expert token
 *       counts padded to 128 rows, quantises the activations to NVFP4, and
 *       runs L1 GEMM -> SiLU -> L2 GEMM; Phase 2: zero-token experts and the
 *       expert_offsets / padded_expert_offsets arrays.
 *   "Current Bug: vLLM produces NaN from layer 0"
 *     - "What we've tried" item 1 and "Key evidence": the activation global
 *       scale must come from the measured amax, never from a stored
 *       input_scale.
 *
 * NVFP4 here: E2M1 element codes (two per byte, even element in the low
 * nibble), one unsigned E4M3 block scale per 16 elements along K, one FP32
 * global scale gs per tensor.  An element decodes to
 * e2m1(code) * e4m3(scale) / gs.  Activations are encoded with
 * gs = 2688 / amax (448 * 6), and with the float32 steps
 * s = (amax_b * gs) / 6, s8 = e4m3_rne_satfinite(s), enc = gs / decode(s8),
 * code = e2m1_rne_satfinite(x * enc), each a correctly rounded operation.
 *
 * Conventions for every entry point:
 *   - All pointers are DEVICE pointers unless a parameter says "host".  The
 *     caller owns every buffer (workspace included); the library never
 *     allocates or frees memory and never synchronises on the compute path.
 *   - All work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream).
 *   - Argument and shape errors are returned synchronously, before anything
 *     is enqueued.  A failed launch returns MEGAMOE_ERR_CUDA.  Problems only
 *     the device can see (an expert id >= E, a non-finite input, a spin-wait
 *     that ran out) set bits in a device status word and never trap; read it
 *     with megamoe_read_status.
 *   - Matrices are row-major.  "Atom layout" (MEGAMOE_SCALES_MMA) stores block
 *     scales in 512-byte atoms of 128 rows x 4 blocks: atom (a, c) covers rows
 *     128a..128a+127 and blocks 4c..4c+3 and holds row 128a + 32j + i, block
 *     4c + b at byte 16i + 4j + b; atoms are ordered [a][c].  This is the
 *     layout the tensor cores read block scales in.
 */
#ifndef MEGAMOE_H
#define MEGAMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* megamoe_stream_t; /* == cudaStream_t */

typedef enum megamoe_status {
  MEGAMOE_OK = 0,
  MEGAMOE_ERR_INVALID_ARG = 1,       /* null pointer, negative size, bad enum */
  MEGAMOE_ERR_UNSUPPORTED_SHAPE = 2, /* shape outside the supported set      */
  MEGAMOE_ERR_WORKSPACE_TOO_SMALL = 3,
  MEGAMOE_ERR_CUDA = 4,              /* a CUDA runtime/driver call failed     */
  MEGAMOE_ERR_DEVICE_STATUS = 5      /* megamoe_read_status found bits set    */
} megamoe_status;

/* Bits of the device status word. */
#define MEGAMOE_DEV_BAD_EXPERT_ID 0x1u /* a topk id >= E was seen (slot skipped) */
#define MEGAMOE_DEV_NONFINITE 0x2u     /* the amax of an input was not finite    */
#define MEGAMOE_DEV_TIMEOUT 0x4u       /* a bounded device wait gave up          */
#define MEGAMOE_DEV_BAD_OFFSETS 0x8u   /* an expert's rows outside the matrix, or another's */

/* Scale layouts. */
#define MEGAMOE_SCALES_ROWMAJOR 0 /* [rows, K/16] bytes                         */
#define MEGAMOE_SCALES_MMA 1      /* atom layout, ceil(rows/128)*128 rows          */

/* Grouped-GEMM epilogues. */
#define MEGAMOE_EPI_F32 0      /* out[r, n] = fp32 accumulator * alpha            */
#define MEGAMOE_EPI_SILU_MUL 1 /* out[r, i] = bf16(silu(gate) * up), amax of it   */
#define MEGAMOE_EPI_BF16 2     /* out[r, n] = bf16(fp32 accumulator * alpha)      */
#define MEGAMOE_EPI_BFP16 3    /* out = BFP16 matrix of fp32 accumulator * alpha */

/*
 * BFP16 (16-bit block floating point): the storage of the forward's L2
 * output y between the down GEMM and the combine (the pages fix no type for
 * it; fp32 would double its round trip through HBM).  A [rows, ld] BFP16
 * matrix (ld a multiple of 32) holds one power-of-two exponent per group of
 * 16 rows x 8 columns (rows 16g .. 16g + 15, columns 8c .. 8c + 7).  It is one
 * buffer of MEGAMOE_BFP16_BYTES(rows, ld) bytes:
 *   bytes [0, 2*rows*ld)                          uint16 values u[r*ld + c]
 *   bytes [2*rows*ld, + ceil(rows/16)*(ld/8))     int8 exponents s[(r/16)*(ld/8) + c/8]
 *   element (r, c) = (u - 32768) * 2^s              (s <= 114)
 *                  = fp16 value of the bits of u    (s = 127)
 * Writing the fp32 values v of a group's written rows: with m = max |v| and
 * E = floor(log2 m), s = max(E - 14, -126), plus one when m * 2^-s >= 32767.5,
 * and u = rint(v * 2^-s) + 32768 (ties to even; |rint| <= 32767), so the
 * group's largest values keep 15 significant bits (v * 2^-s is exact; the
 * only rounding is to the integer); s = 0 and u = 32768 when all are zero.
 * A group holding Inf or NaN gets s = 127 and the fp16 encoding of each
 * value, so non-finite values pass through.  Rows that are not written
 * (padding rows) take no part in their group's exponent.  (A value within
 * 2^-16 of the largest float decodes to Inf.)
 */
#define MEGAMOE_BFP16_BYTES(rows, ld) \
  ((size_t)(rows) * (size_t)(ld) * 2 + ((size_t)(rows) + 15) / 16 * ((size_t)(ld) / 8))

/* Limits. */
#define MEGAMOE_MAX_EXPERTS 1024
#define MEGAMOE_MAX_TOPK 16

/*
 * NVFP4 expert weights.  Expert e of W13 is [2I, d]: rows 0..I-1 are the gate
 * projection, rows I..2I-1 the up projection ("What's Been Verified": L1
 * gate+up).  W2 is [d, I] per expert (L2 down).
 *   w13_codes   [E*2I, d/2] E2M1 codes packed by megamoe_pack_weight_codes
 *               with half_rows = I
 *   w13_scales  atom layout of [E*2I, d/16] (from megamoe_swizzle_scales)
 *   w13_gs      [E, 2] float            global scales (gate, up)
 *   w2_codes    [E*d, I/2] packed by megamoe_pack_weight_codes, half_rows = 0
 *   w2_scales   atom layout of [E*d, I/16]
 *   w2_gs       [E] float
 * Supported: 1 <= E <= 1024, d and I multiples of 256.
 */
typedef struct megamoe_weights {
  int32_t num_experts;
  int32_t hidden;       /* d */
  int32_t intermediate; /* I */
  const uint8_t* w13_codes;
  const uint8_t* w13_scales;
  const float* w13_gs;
  const uint8_t* w2_codes;
  const uint8_t* w2_scales;
  const float* w2_gs;
} megamoe_weights;

/* Human-readable name of a status code (static storage). */
const char* megamoe_status_string(megamoe_status s);

/*
 * Largest number of padded rows routing can produce:
 * T*k + min(E, T*k) * (pad - 1).  Host-only, no device work.
 */
int64_t megamoe_max_padded_rows(int T, int k, int E, int pad);

/*
 * megamoe_route_permute -- bucket the (token, slot) pairs by expert.
 * ("Test Plan -- Finding the NaN", Phase 1: variable token counts per expert
 * padded to 128; Phase 2: zero-token experts, expert_offsets and
 * padded_expert_offsets.)
 *
 * Slot s = t*k + j is routed to expert topk_ids[t*k + j].  Slots are grouped
 * by expert with a stable counting sort (ascending s inside an expert).
 *   topk_ids        [T, k] int32; ids < 0 are skipped; ids >= E are skipped and
 *                   set MEGAMOE_DEV_BAD_EXPERT_ID in *status
 *   counts          [E]    valid slots per expert (out)
 *   offsets         [E+1]  exclusive prefix sum of counts (out)
 *   padded_offsets  [E+1]  exclusive prefix sum of counts rounded up to pad;
 *                          a zero count stays zero (out)
 *   row_src         [row_capacity] flat slot held by each padded row, -1 for
 *                   padding and for every row >= padded_offsets[E] (out)
 *   slot_dst        [T*k]  padded row of each slot, -1 if skipped (out)
 *   status          device uint32 status word (bits are OR-ed in; may be NULL)
 * Requires 1 <= E <= 1024, 1 <= k <= 16, pad >= 1, T >= 0 and
 * row_capacity >= megamoe_max_padded_rows(T, k, E, pad).  T*k above 2^30 or
 * megamoe_max_padded_rows at or above 2^31 (offsets are int32) returns
 * MEGAMOE_ERR_UNSUPPORTED_SHAPE; the forward checks the same.  One thread
 * block.
 */
megamoe_status megamoe_route_permute(const int32_t* topk_ids, int T, int k, int E, int pad,
                                     int32_t* counts, int32_t* offsets,
                                     int32_t* padded_offsets, int32_t* row_src,
                                     int64_t row_capacity, int32_t* slot_dst,
                                     uint32_t* status, megamoe_stream_t stream);

/*
 * megamoe_quantize_nvfp4 -- bf16 activations -> NVFP4
 * ("Test Plan -- Finding the NaN", Phase 1 item 4: quantize_activation_nvfp4;
 * global scale from the measured amax per "Current Bug: vLLM produces NaN
 * from layer 0", "What we've tried" item 1).
 *
 *   x          [rows, K] bf16 with row stride ld (elements), ld >= K
 *   amax_in    if non-NULL, the amax to use (device float, e.g. the amax the
 *              L1 epilogue measured); if NULL the amax of x over all rows is
 *              measured here (one extra read of x)
 *   amax_out   device float: the amax used (out; may be NULL if amax_in given)
 *   gs_out     device float: gs = 2688 / amax, or 1 if amax == 0 (out)
 *   codes      [out_rows, K/2] (out), scales in `scale_layout` (out)
 * Row mapping:
 *   slot_dst == NULL: out row r is x row r (out_rows == rows).
 *   slot_dst != NULL: x row t is written to out rows slot_dst[t*k + j],
 *                     j = 0..k-1, skipping -1 (the routed gather).
 *   row_src != NULL:  out rows with row_src[r] < 0 are written as zero codes
 *                     and zero scales instead (padding rows).
 *   live_rows != NULL: device int32; out rows >= *live_rows are not touched.
 * Requires rows >= 0, out_rows >= 0, ld >= K and, with slot_dst == NULL,
 * rows >= out_rows (else MEGAMOE_ERR_INVALID_ARG); K a multiple of 64, ld a
 * multiple of 8, x and codes 16-byte aligned, scales 4-byte aligned (else
 * MEGAMOE_ERR_UNSUPPORTED_SHAPE).
 */
megamoe_status megamoe_quantize_nvfp4(const uint16_t* x, int64_t rows, int K, int64_t ld,
                                      const int32_t* slot_dst, int k, const int32_t* row_src,
                                      const int32_t* live_rows, int64_t out_rows,
                                      const float* amax_in, float* amax_out, float* gs_out,
                                      uint8_t* codes, uint8_t* scales, int scale_layout,
                                      uint32_t* status, megamoe_stream_t stream);

/*
 * megamoe_swizzle_scales -- one-time weight preparation: row-major block
 * scales [rows, K/16] -> atom layout (see the file comment).  Rows are padded
 * to a multiple of 128 with zero bytes; dst holds ceil(rows/128)*128*K/16
 * bytes.  Requires K a multiple of 64 and 4-byte aligned src and dst.
 */
megamoe_status megamoe_swizzle_scales(const uint8_t* src, int64_t rows, int K, uint8_t* dst,
                                      megamoe_stream_t stream);

/*
 * megamoe_pack_weight_codes -- one-time weight preparation: row-major E2M1
 * codes [rows, K/2] -> tile-major blocks of 128 rows x 128 bytes (256
 * elements of K).  Within a block, row i sits at byte 128*i and its 16-byte
 * chunk j at chunk j XOR (i % 8): the 128-byte swizzle the tensor cores read
 * K-major operands in, so the GEMM copies a block to shared memory as is.
 *   half_rows == 0: blocks ordered [rows/128][K/256] (the W2 layout).
 *   half_rows == H: rows come in groups of 2H, H gate rows then H up rows (one
 *                   expert of W13, H = I); the gate and up blocks of the same
 *                   128 features and K step are adjacent:
 *                   [rows/2H][H/128][K/256][gate, up] (the W13 layout).
 * A stage of the grouped GEMM then reads one contiguous 16 KB (W2) or 32 KB
 * (W13) block with a single bulk copy.  Requires rows a multiple of 128 (of 2H when H > 0), H a
 * multiple of 128, K a multiple of 256, 16-byte alignment.
 */
megamoe_status megamoe_pack_weight_codes(const uint8_t* src, int64_t rows, int K, int half_rows,
                                         uint8_t* dst, megamoe_stream_t stream);

/*
 * megamoe_grouped_gemm -- one persistent grouped block-scaled GEMM over all
 * experts ("Architecture: DeepSeek-V4 MegaMoE": one problem per expert,
 * persistent tile scheduling across groups, token tile chosen from the
 * expected tokens per expert).  On tcgen05 tensor cores with TMEM
 * accumulators and TMA loads.
 *
 * For every expert e and every valid row r of e
 * (padded_offsets[e] <= r < padded_offsets[e] + offsets[e+1] - offsets[e]):
 *   acc[r, n] = sum_K dequant(act)[r, :] . dequant(w_e)[n, :]   (fp32 accumulate)
 *   act_codes   [act_rows, K/2]; act_scales row-major [act_rows, K/16];
 *               act_gs device float (one global scale)
 *   w_codes     [E*N, K/2] packed by megamoe_pack_weight_codes (half_rows =
 *               N/2 for MEGAMOE_EPI_SILU_MUL, 0 otherwise);
 *               w_scales atom layout of [E*N, K/16] (megamoe_swizzle_scales)
 *   w_gs        [E, G] float: G = 2 (gate, up) for MEGAMOE_EPI_SILU_MUL, else 1
 *   offsets, padded_offsets  [E+1] int32 as produced by megamoe_route_permute
 *               with a pad that is a multiple of 32
 * Epilogues:
 *   MEGAMOE_EPI_F32:      out float [act_rows, ld_out], out[r, n] = acc * alpha,
 *                         alpha = 1 / (act_gs * w_gs[e]).
 *   MEGAMOE_EPI_BF16:     out bf16 [act_rows, ld_out], out[r, n] = bf16(acc * alpha).
 *   MEGAMOE_EPI_BFP16:    out BFP16 [act_rows, ld_out] of acc * alpha (the
 *                         format above; ld_out a multiple of 32; a group's
 *                         rows are 16 padded rows of one expert; weights-on-M
 *                         tiles only: tile_n 256 runs as 128).
 *   MEGAMOE_EPI_SILU_MUL: N = 2I; out bf16 [act_rows, ld_out],
 *                         out[r, i] = bf16(silu(acc[r, i] * alpha_gate) *
 *                                          (acc[r, I + i] * alpha_up)),
 *                         out_amax (device float, zeroed here) = max |out| over
 *                         valid rows.
 * Padding rows of `out` are not written.  tile_n selects the tile shape
 * (0 = choose from the expected tokens per expert, expected_tokens = rows the
 * caller expects per active expert, may be 0):
 *   32, 64, 128  tiles of 128 weight rows x tile_n token rows (weights on the
 *                MMA's M side, tokens on N);
 *   256          token-major tiles: 128 token rows x 256 weight rows (tokens on
 *                M, weights on N; for SILU_MUL the gate and up rows of 128
 *                features in one MMA); requires N a multiple of 256.
 * Requires N a multiple of 128 (256 for SILU_MUL), K a multiple of 256,
 * 1 <= E <= 1024, 16-byte aligned pointers, ld_out >= output width and a
 * multiple of 16 bytes (4 floats, 8 bf16), else MEGAMOE_ERR_UNSUPPORTED_SHAPE.
 */
megamoe_status megamoe_grouped_gemm(const uint8_t* act_codes, const uint8_t* act_scales,
                                    const float* act_gs, int64_t act_rows,
                                    const uint8_t* w_codes, const uint8_t* w_scales,
                                    const float* w_gs, int E, int N, int K,
                                    const int32_t* offsets, const int32_t* padded_offsets,
                                    int epilogue, void* out, int64_t ld_out, float* out_amax,
                                    int tile_n, double expected_tokens, uint32_t* status,
                                    megamoe_stream_t stream);

/*
 * megamoe_router_topk -- the router step ahead of megamoe_route_permute
 * ("CURRENT_BUG.md -- DeepSeek-V4 Blackwell NVFP4", "Test Plan -- Finding the
 * NaN", Phase 1 item 1: topk_ids and topk_weights come from the router; the
 * pages do not spell the router out: this is the plain top-k + softmax):
 *   score[t, e] = fl32(logits[t, e] + bias[e])   (bias nullable: score = logit)
 *   topk_ids[t, 0..k-1]     = the k experts of highest score, in descending
 *                             score, ties to the lower expert index
 *   topk_weights[t, j]      = softmax over the k selected *logits* (fp32)
 * With shared_expert >= 0 one more column is appended to both outputs:
 * id shared_expert with weight 1 (a shared expert that every token visits,
 * to be run by megamoe_forward as one more expert).
 *   logits        float [T, ld_logits] (ld_logits >= E)
 *   topk_ids      int32 [T, k_out], topk_weights float [T, k_out],
 *                 k_out = k + (shared_expert >= 0)
 * Requires 1 <= k <= min(E, 16), E <= 1024, 4-byte aligned pointers.
 */
megamoe_status megamoe_router_topk(const float* logits, int64_t T, int E, int64_t ld_logits,
                                   const float* bias, int k, int shared_expert,
                                   int32_t* topk_ids, float* topk_weights,
                                   megamoe_stream_t stream);

/*
 * megamoe_forward_from_logits -- the MoE layer from router logits: the router
 * step of megamoe_router_topk (k routed experts among the first n_logits,
 * plus, with shared_expert >= 0, that expert for every token with weight 1)
 * followed by megamoe_forward over w's experts with k_out = k + (shared_expert
 * >= 0) slots per token.  For small batches (T * hidden <= 262144) the router
 * runs inside the forward's first thread block, ahead of the routing; larger
 * batches run it as its own kernel.  The ids and weights are written into the
 * workspace (sized by megamoe_workspace_size(T, k_out, w->num_experts, ...)).
 *   logits   float [T, ld_logits], n_logits <= w->num_experts columns used;
 *   bias     float [n_logits] or NULL (selection only)
 *   shared_expert  -1, or an expert index in [n_logits, w->num_experts)
 * Otherwise as megamoe_forward; k_out <= 16.
 */
megamoe_status megamoe_forward_from_logits(const megamoe_weights* w, const uint16_t* x,
                                           const float* logits, int64_t ld_logits,
                                           const float* bias, int n_logits, int k,
                                           int shared_expert, int T, int pad, uint16_t* out,
                                           void* ws, size_t ws_bytes, megamoe_stream_t stream);

/*
 * megamoe_linear_nvfp4 -- a dense NVFP4 linear layer whose activation global
 * scale comes from the measured amax of x, not from a stored input scale
 * ("Current Bug: vLLM produces NaN from layer 0", "Root Cause" and "Key
 * evidence": the attention projections quantised activations with the
 * checkpoint's input_scale, whose inverse (~4e3 to 1.6e4) overflowed
 * activations of amax 2-8).  The one-group case of the grouped GEMM:
 *   amax = max |x|, gs_x = 2688 / amax (1 if amax = 0), x -> NVFP4 as
 *   megamoe_quantize_nvfp4 does, then
 *   out[t, n] = sum_K dequant(x)[t, :] . dequant(w)[n, :]   (fp32 accumulate)
 * written as bf16 (out_dtype MEGAMOE_EPI_BF16) or float (MEGAMOE_EPI_F32).
 *   x          bf16 [T, K], row stride ld_x elements
 *   w_codes    [N, K/2] packed by megamoe_pack_weight_codes (half_rows 0)
 *   w_scales   atom layout of [N, K/16] (megamoe_swizzle_scales)
 *   w_gs       device float: the weight's global scale
 *   out        [T, ld_out] of out_dtype
 *   ws         device workspace of megamoe_linear_workspace_size(T, K, N) bytes,
 *              256-byte aligned, owned by the caller; it also receives the
 *              measured amax (float at ws + 0) and gs_x (float at ws + 4) and
 *              the status word (uint32 at ws + 8, read with megamoe_read_status)
 * Requires K a multiple of 256, N a multiple of 128, ld_x a multiple of 8
 * and ld_out of 16 bytes, 16-byte aligned pointers.  Argument errors return
 * before anything is enqueued; non-finite x sets MEGAMOE_DEV_NONFINITE.
 */
size_t megamoe_linear_workspace_size(int64_t T, int K, int N);
megamoe_status megamoe_linear_nvfp4(const uint16_t* x, int64_t T, int K, int64_t ld_x,
                                    const uint8_t* w_codes, const uint8_t* w_scales,
                                    const float* w_gs, int N, int out_dtype, void* out,
                                    int64_t ld_out, void* ws, size_t ws_bytes,
                                    megamoe_stream_t stream);

/*
 * megamoe_combine -- top-k weighted combine (topk_weights input of "Test Plan
 * -- Finding the NaN", Phase 1):
 *   out[t, :] = bf16( sum_{j=0..k-1, slot_dst[t*k+j] >= 0}
 *                     topk_weights[t*k+j] * y[slot_dst[t*k+j], :] )
 * summed in fp32 in ascending j.  y is float [*, ld_y]; out bf16 [T, d].
 * Requires d and ld_y multiples of 4, y 16-byte and out 8-byte aligned
 * (else MEGAMOE_ERR_UNSUPPORTED_SHAPE).
 */
megamoe_status megamoe_combine(const float* y, int64_t ld_y, const int32_t* slot_dst,
                               const float* topk_weights, int T, int k, int d, uint16_t* out,
                               megamoe_stream_t stream);

/*
 * megamoe_combine_bfp16 -- the same combine over a BFP16 y of y_rows rows and
 * leading dimension ld_y (the forward's own form of y): each element is
 * decoded exactly into fp32, then summed in fp32 in ascending j and rounded
 * once to bf16.  Requires d and ld_y multiples of 32, y 16-byte and out
 * 8-byte aligned (else MEGAMOE_ERR_UNSUPPORTED_SHAPE); a slot_dst entry at or
 * past y_rows is skipped like a negative one.
 */
megamoe_status megamoe_combine_bfp16(const void* y, int64_t ld_y, int64_t y_rows,
                                     const int32_t* slot_dst, const float* topk_weights, int T,
                                     int k, int d, uint16_t* out, megamoe_stream_t stream);

/*
 * Workspace bytes megamoe_forward needs for these sizes (host-only).
 */
size_t megamoe_workspace_size(int T, int k, int E, int d, int I, int pad);

/*
 * megamoe_forward -- the whole routed-expert forward on one stream:
 * route -> amax(x) -> quantise x into routed rows -> L1 grouped GEMM with
 * SiLU(gate)*up and amax(h) in its epilogue -> requantise h -> L2 grouped
 * GEMM into a BFP16 y -> top-k weighted combine (y decoded exactly, fp32
 * sums, one bf16 rounding).
 *   x             [T, d] bf16 hidden_states
 *   topk_ids      [T, k] int32 (ids < 0 skipped)
 *   topk_weights  [T, k] float (used as given)
 *   pad           rows per expert are padded to a multiple of pad; must be a
 *                 multiple of 32 (32, 64, 128, ...)
 *   out           [T, d] bf16 (out)
 *   ws, ws_bytes  workspace, at least megamoe_workspace_size(...) bytes,
 *                 256-byte aligned; its first 4 bytes are the device status
 *                 word, cleared at the start of every call.
 * Requires the weight shapes above, 1 <= k <= 16, T >= 0, x and the weight
 * codes and scales 16-byte aligned, out 8-byte aligned.  Every step is a
 * kernel launch on `stream` (no host synchronisation, no memory allocation),
 * so the call can be recorded into a CUDA graph and replayed.
 */
megamoe_status megamoe_forward(const megamoe_weights* w, const uint16_t* x,
                               const int32_t* topk_ids, const float* topk_weights, int T, int k,
                               int pad, uint16_t* out, void* ws, size_t ws_bytes,
                               megamoe_stream_t stream);

/*
 * megamoe_set_wait_limit_ns -- bound of every pipeline wait inside the
 * grouped GEMM kernels launched afterwards (host setting of this library,
 * all devices; 0 restores the default of 4 s).  A wait that runs out raises
 * the kernel's abort flag and MEGAMOE_DEV_TIMEOUT; the kernel then lets its
 * copies and MMAs in flight land (waiting up to 4 s), frees its tensor memory
 * and returns, so the context stays usable.  For failure-detection tests and
 * diagnosis; the default never fires in normal operation.
 */
void megamoe_set_wait_limit_ns(uint64_t ns);

/*
 * megamoe_set_fused_requant -- where megamoe_forward / _from_logits /
 * _static requantise h (the requantisation fused into the L1 GEMM's
 * epilogue, or after it; host setting of this library, all devices, for
 * forwards launched afterwards):
 *   0 (default)  a separate kernel after the L1 GEMM reads h once and encodes
 *                it with the global scale of amax(h);
 *   1            the L1 GEMM kernel does it: after its last tile each CTA
 *                arrives on a grid-wide count in the workspace and waits
 *                (bounded by the pipeline wait limit; MEGAMOE_DEV_TIMEOUT on
 *                expiry) until every CTA with tiles has, so amax(h) is
 *                final, then encodes the h rows of its own tiles.
 * Both give bit-identical results.  The default is the faster on GB300 (the
 * separate kernel lets CTAs that finish early free their SM for the next
 * kernel); an L1 GEMM split along K always uses the separate kernel.
 */
void megamoe_set_fused_requant(int enable);

/*
 * Expert-parallel forward, one shard (one process and GPU) of G: the shard
 * holds experts [expert_base, expert_base + w_shard->num_experts) of
 * num_experts_total ("CURRENT_BUG.md -- DeepSeek-V4 Blackwell NVFP4", "Test
 * Plan -- Finding the NaN", Phase 2: the EP8 slice of 48 of the 384 experts).
 * The layer's tokens are first gathered on every shard (x, topk_ids and
 * topk_weights of all T tokens, global expert ids); then:
 *
 *   megamoe_ep_forward_begin  routes the shard's slots (ids of other shards
 *     skipped, ids >= num_experts_total flagged MEGAMOE_DEV_BAD_EXPERT_ID and
 *     skipped), takes amax(x) over all T tokens (the same on every shard, so
 *     x's global scale needs no exchange), quantises x and runs the L1 GEMM
 *     with SiLU(gate)*up; the shard's amax(h) is left as a float at bytes
 *     [12, 16) of ws.
 *   The caller replaces that float on every shard by the maximum over all
 *     shards (an all-reduce(max) of 4 bytes): h has one global scale over
 *     every valid row of the layer's intermediate, whichever shard holds it.
 *   megamoe_ep_forward_end  requantises h with that global amax, runs the L2
 *     GEMM and writes out_partial [T, d] fp32 = sum over the shard's slots j
 *     (ascending) of topk_weights[t, j] * y (0 for tokens with no slot on the
 *     shard), before any rounding.
 *   The caller sums the shards' out_partial (an all-reduce or reduce-scatter)
 *     and rounds once with megamoe_round_bf16.
 *
 * With the same inputs the result equals megamoe_forward's up to the order of
 * the fp32 additions across shards.  w_shard, T, k, pad and ws are those of
 * megamoe_forward on the shard's experts (ws: megamoe_workspace_size(T, k,
 * w_shard->num_experts, d, I, pad) bytes, 256-byte aligned, the same buffer
 * for begin and end); out_partial is 16-byte aligned.  Errors as
 * megamoe_forward, plus MEGAMOE_ERR_INVALID_ARG when the shard's range does
 * not fit in [0, num_experts_total).
 */
megamoe_status megamoe_ep_forward_begin(const megamoe_weights* w_shard, const uint16_t* x,
                                        const int32_t* topk_ids, int T, int k, int expert_base,
                                        int num_experts_total, int pad, void* ws, size_t ws_bytes,
                                        megamoe_stream_t stream);
megamoe_status megamoe_ep_forward_end(const megamoe_weights* w_shard, const float* topk_weights,
                                      int T, int k, int num_experts_total, int pad,
                                      float* out_partial, void* ws, size_t ws_bytes,
                                      megamoe_stream_t stream);

/*
 * megamoe_round_bf16 -- out[i] = bf16(in[i]), round to nearest even, i < n
 * (the single rounding of the expert-parallel sum).  n a multiple of 4, in
 * 16-byte and out 8-byte aligned, else MEGAMOE_ERR_UNSUPPORTED_SHAPE.
 */
megamoe_status megamoe_round_bf16(const float* in, int64_t n, uint16_t* out,
                                  megamoe_stream_t stream);

/*
 * megamoe_forward_scan_stages -- debug aid: which stage of the last forward
 * run with this workspace produced a non-finite value ("CURRENT_BUG.md --
 * DeepSeek-V4 Blackwell NVFP4", "Test Plan -- Finding the NaN", Phase 1
 * item 3: check after the L1 GEMM and SiLU, and after the L2 GEMM).  ws and
 * (T, k, E = w->num_experts, d, I, pad) are those of a megamoe_forward /
 * _from_logits call already enqueued on `stream`; out its output.  Scans
 * the valid rows (padding rows are never written and may hold anything) and
 * writes to *flags (device uint32, cleared here) the bits of every stage
 * that holds one:
 *   MEGAMOE_STAGE_XQ_SCALE  a block scale of the quantised x is an E4M3 NaN byte
 *   MEGAMOE_STAGE_H         h = bf16(SiLU(gate) * up) holds Inf or NaN
 *   MEGAMOE_STAGE_HQ_SCALE  a block scale of the requantised h is an E4M3 NaN byte
 *   MEGAMOE_STAGE_Y         the L2 output y holds Inf or NaN (a BFP16 group
 *                           of valid rows with exponent 127)
 *   MEGAMOE_STAGE_OUT       the combined output holds Inf or NaN
 * Reads every intermediate once (~3.7 GB at 16384 tokens): for diagnosis,
 * not the forward's path.  Asynchronous on `stream`.
 */
#define MEGAMOE_STAGE_XQ_SCALE 0x01u
#define MEGAMOE_STAGE_H 0x02u
#define MEGAMOE_STAGE_HQ_SCALE 0x04u
#define MEGAMOE_STAGE_Y 0x08u
#define MEGAMOE_STAGE_OUT 0x10u
megamoe_status megamoe_forward_scan_stages(const megamoe_weights* w, int T, int k, int pad,
                                           const uint16_t* out, const void* ws, size_t ws_bytes,
                                           uint32_t* flags, megamoe_stream_t stream);

/*
 * megamoe_read_status -- synchronise `stream`, copy the device status word at
 * `status` (for megamoe_forward: the first 4 bytes of ws) into *bits (host),
 * and return MEGAMOE_ERR_DEVICE_STATUS if any bit is set, else MEGAMOE_OK.
 */
megamoe_status megamoe_read_status(const uint32_t* status, uint32_t* bits,
                                   megamoe_stream_t stream);

/*
 * megamoe_forward_static -- megamoe_forward without a caller-provided
 * workspace, for callers that cannot allocate device memory where they run
 * the forward: plugins in a host process that owns every device allocation
 * (an inference server with its own memory pool, which forbids side
 * allocations), embedded callers that link only this library and have no
 * allocator at hand, hot loops that must never enter the allocator.  (The
 * source pages have no counterpart: this is a deployment variant of
 * megamoe_forward, not a step of the method.)
 *
 * The workspace is a fixed device array inside the library of
 * MEGAMOE_STATIC_WS_BYTES (64 MiB), held by every GPU that loads the library
 * until the process exits.  Nothing is allocated or freed by this call.
 * Arguments are those of megamoe_forward, minus ws/ws_bytes, plus:
 *   status_out  device uint32 (may be NULL): receives the forward's device
 *               status word (see MEGAMOE_DEV_*), copied on `stream`; written
 *               only when the call returns MEGAMOE_OK.
 * Argument and shape errors are those of megamoe_forward and are reported
 * first; then MEGAMOE_ERR_WORKSPACE_TOO_SMALL when
 * megamoe_workspace_size(T, k, E, d, I, pad) exceeds MEGAMOE_STATIC_WS_BYTES
 * (for E = 384, d = 7168, I = 2048, k = 6, pad = 32 that is T > 9 tokens).
 * The first call on a device looks the array up for that device (with it
 * current) and should come before any stream capture; a call under a new
 * driver context of the device (after cudaDeviceReset, or a context made
 * current through the driver API) looks it up again.  All calls share the
 * array: calls that overlap on the GPU race, so the caller serialises them
 * (one stream per device, or its own ordering).
 */
#define MEGAMOE_STATIC_WS_BYTES (64u << 20)
megamoe_status megamoe_forward_static(const megamoe_weights* w, const uint16_t* x,
                                      const int32_t* topk_ids, const float* topk_weights, int T,
                                      int k, int pad, uint16_t* out, uint32_t* status_out,
                                      megamoe_stream_t stream);

/* ------------------------------------------------------------------------
 * Scored router
 *
 * Scores of every expert, s_e = 1 / (1 + exp(-l_e)) or softmax(l)_e, in fp32;
 * the choice is by c_e = s_e + bias_e (bias may be null), the weights by s_e:
 *   - the E experts form n_group equal runs; a group's score is the sum of
 *     its group_top (1 or 2) largest c, and the topk_group groups of highest
 *     score stay;
 *   - the k experts of largest c among them, in descending order;
 *   - w_j = scale * s_j / sum_i s_i (renormalize), or scale * s_j.  Softmax shares
 *     are taken of the logits, so they hold where the scores are 0 in fp32;
 *     sigmoid scores that are all 0 in fp32 (logits below -103) give weights 0.
 * Ties, of groups and of experts, go to the lower index.  An expert whose logit
 * is NaN or -inf scores 0; neither it nor one whose c is NaN or -inf is ever
 * taken; slots left over get id -1 and weight 0 (the forward skips them).  +inf
 * counts as the largest float.
 * ------------------------------------------------------------------------ */

/* Element types. */
#define MEGAMOE_TYPE_BF16 0
#define MEGAMOE_TYPE_F32 1
#define MEGAMOE_TYPE_F16 2
#define MEGAMOE_TYPE_I8 3 /* codes of the 8-bit integer linear */

/* Scores. */
#define MEGAMOE_SCORE_SIGMOID 0
#define MEGAMOE_SCORE_SOFTMAX 1

/*
 * megamoe_router_scored_topk
 *   logits        [T, ld_logits] of logits_type (BF16 or F32)
 *   bias          [E] float or null
 *   topk_ids      [T, k] int32 (out)
 *   topk_weights  [T, k] float (out)
 * Requires 1 <= E <= 1024, 1 <= k <= 16, k <= E, n_group a divisor of E and at
 * most 32, 1 <= topk_group <= n_group, group_top 1 or 2, T < 2^31.
 */
megamoe_status megamoe_router_scored_topk(const void* logits, int logits_type, int64_t T, int E,
                                          int64_t ld_logits, const float* bias, int score,
                                          int n_group, int topk_group, int group_top, int k,
                                          int renormalize, double scale, int32_t* topk_ids,
                                          float* topk_weights, megamoe_stream_t stream);

/*
 * megamoe_router_scored_topk_backward -- the gradient of the weights with
 * respect to the logits, for the ids that the forward call gave (distinct in a
 * row; ids < 0 or >= E take no part); the choice itself and the bias have none.
 *   grad_weights  [T, k] float
 *   grad_logits   [T, ld_grad] of logits_type (out; columns 0 .. E - 1)
 */
megamoe_status megamoe_router_scored_topk_backward(
    const void* logits, int logits_type, int64_t T, int E, int64_t ld_logits,
    const int32_t* topk_ids, const float* grad_weights, int score, int k, int renormalize,
    double scale, void* grad_logits, int64_t ld_grad, megamoe_stream_t stream);

/* ------------------------------------------------------------------------
 * MXFP4: E2M1 codes (two per byte, even element in the low nibble) and one
 * E8M0 scale byte per 32 elements, 2^(byte - 127), 255 = NaN.  No tensor-wide
 * scale.  Encoding: the scale is 2^(floor(log2(amax)) - 2), at least 2^-127;
 * elements to the nearest E2M1 value, ties to even, saturating at 6 (the rule
 * of the OCP Microscaling Formats specification 1.0).  A block that holds Inf
 * or NaN gets scale 255 and zero codes, and MEGAMOE_DEV_NONFINITE is set.
 *
 * Scales are [rows, K / 32] bytes (MEGAMOE_SCALES_ROWMAJOR) or in the atom
 * layout (MEGAMOE_SCALES_MMA): atoms of 128 rows x 4 blocks as above, with the
 * blocks of a row padded to a multiple of 8 (zero scales) and the rows to a
 * multiple of 128: MEGAMOE_MX_ATOM_BYTES(rows, K) bytes.
 * ------------------------------------------------------------------------ */
#define MEGAMOE_MX_ATOM_BYTES(rows, K) \
  (((size_t)(rows) + 127) / 128 * 128 * (((size_t)(K) + 255) / 256 * 8))

/*
 * megamoe_quantize_mxfp4 -- x [rows, K] of x_type, row stride ld.
 *   transpose 0: blocks along the columns' direction of a row:
 *                codes [rows, K / 2], scales of [rows, K]
 *   transpose 1: x^T, blocks along the rows of x: codes [K, R / 2], scales of
 *                [K, R], R = rows up to a multiple of 32 (the last block's
 *                missing elements count as zeros)
 *   status       device status word or null
 * Requires K a multiple of 32 below 2^30, rows < 2^31, ld * element size a multiple
 * of 16, x and codes 16-byte aligned.
 */
megamoe_status megamoe_quantize_mxfp4(const void* x, int x_type, int64_t rows, int K, int64_t ld,
                                      int transpose, uint8_t* codes, uint8_t* scales,
                                      int scale_layout, uint32_t* status, megamoe_stream_t stream);

/*
 * megamoe_dequantize_mxfp4 -- values of row-major codes and scales as bf16
 * (exact) or fp32.  Requires K a multiple of 32, out 16-byte aligned and
 * ld * element size a multiple of 16.
 */
megamoe_status megamoe_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                        int K, void* out, int out_type, int64_t ld,
                                        megamoe_stream_t stream);

/* Row-major MXFP4 scales [rows, K / 32] -> atom layout (weights, once). */
megamoe_status megamoe_swizzle_scales_mxfp4(const uint8_t* src, int64_t rows, int K, uint8_t* dst,
                                            megamoe_stream_t stream);

/*
 * megamoe_linear_mxfp4 -- out [T, N] = MXFP4(x) w^T, fp32 accumulation.
 *   x         [T, K] of x_type, row stride ld_x
 *   w_codes   [N, K / 2] row-major, w_scales atom layout
 *   out       [T, N] bf16 (MEGAMOE_EPI_BF16) or fp32 (MEGAMOE_EPI_F32)
 *   ws        at least megamoe_linear_mxfp4_workspace_size(T, K, N) bytes,
 *             256-byte aligned; its first 4 bytes are the status word
 * Requires K and N multiples of 32, T, K and N below 2^30, pointers 16-byte aligned
 * and rows on 16-byte boundaries.
 */
size_t megamoe_linear_mxfp4_workspace_size(int64_t T, int K, int N);
megamoe_status megamoe_linear_mxfp4(const void* x, int x_type, int64_t T, int K, int64_t ld_x,
                                    const uint8_t* w_codes, const uint8_t* w_scales, int N,
                                    int out_dtype, void* out, int64_t ld_out, void* ws,
                                    size_t ws_bytes, megamoe_stream_t stream);

/*
 * megamoe_linear_mxfp4_backward -- the gradients of the linear for training,
 * each a product of operands quantised along the dimension it sums over (the
 * quantisers' own derivative taken as 1):
 *   grad_x [T, K] = MXFP4(grad_out) MXFP4(w along N)
 *   grad_w [N, K] = MXFP4(grad_out along T)^T MXFP4(x along T)
 *   grad_out  [T, N], x [T, K], w [N, K]: of their types, row strides ld_*
 *             (w the master weight)
 *   grad_x, grad_w  bf16 or fp32 (MEGAMOE_EPI_*); either may be null and is
 *             then not computed
 *   ws        at least megamoe_linear_mxfp4_backward_workspace_size bytes,
 *             256-byte aligned; its first 4 bytes are the status word
 * Requires K and N multiples of 32.  T = 0 gives a zero grad_w.
 */
size_t megamoe_linear_mxfp4_backward_workspace_size(int64_t T, int K, int N);
megamoe_status megamoe_linear_mxfp4_backward(
    const void* grad_out, int grad_type, int64_t ld_grad, const void* x, int x_type, int64_t ld_x,
    const void* w, int w_type, int64_t ld_w, int64_t T, int K, int N, void* grad_x,
    int grad_x_dtype, int64_t ld_grad_x, void* grad_w, int grad_w_dtype, int64_t ld_grad_w,
    void* ws, size_t ws_bytes, megamoe_stream_t stream);

/*
 * MXFP4 expert weights: as megamoe_weights, without global scales.
 *   w13_codes   packed by megamoe_pack_weight_codes with half_rows = I
 *   w13_scales  atom layout of [E*2I, d] (megamoe_swizzle_scales_mxfp4)
 *   w2_codes    packed with half_rows = 0
 *   w2_scales   atom layout of [E*d, I]
 */
typedef struct megamoe_mx_weights {
  int32_t num_experts;
  int32_t hidden;       /* d */
  int32_t intermediate; /* I */
  const uint8_t* w13_codes;
  const uint8_t* w13_scales;
  const uint8_t* w2_codes;
  const uint8_t* w2_scales;
} megamoe_mx_weights;

/*
 * megamoe_forward_mxfp4 -- the routed-expert forward with MXFP4 weights and
 * activations: route -> quantise x into routed rows -> L1 grouped GEMM with
 * SiLU(gate)*up, quantised to MXFP4 in its epilogue -> L2 grouped GEMM into y
 * -> top-k weighted combine in fp32, rounded once to bf16.  Arguments, shapes and
 * errors as megamoe_forward; workspace of megamoe_workspace_size_mxfp4 bytes.
 *
 * y, the down product of each slot between the fp32 sum and the combine, is held
 * in 16 bits: one power-of-two exponent for 32 neighbouring columns of a row, so
 * that a value is off by at most 2^-15 of the largest of the 32 and no token
 * depends on another.  Inf and NaN are kept and leave the others as they are.
 */
size_t megamoe_workspace_size_mxfp4(int T, int k, int E, int d, int I, int pad);
megamoe_status megamoe_forward_mxfp4(const megamoe_mx_weights* w, const uint16_t* x,
                                     const int32_t* topk_ids, const float* topk_weights, int T,
                                     int k, int pad, uint16_t* out, void* ws, size_t ws_bytes,
                                     megamoe_stream_t stream);

/*
 * megamoe_forward_mxfp4_from_logits -- megamoe_router_scored_topk over the
 * weights' E experts (its ids and weights in the workspace), then
 * megamoe_forward_mxfp4.
 */
megamoe_status megamoe_forward_mxfp4_from_logits(
    const megamoe_mx_weights* w, const uint16_t* x, const void* logits, int logits_type,
    int64_t ld_logits, const float* bias, int score, int n_group, int topk_group, int group_top,
    int renormalize, double scale, int T, int k, int pad, uint16_t* out, void* ws, size_t ws_bytes,
    megamoe_stream_t stream);

/* ------------------------------------------------------------------------
 * Experts in 16 bits: products grouped by expert, the activation between them
 * and the movement of rows, with the gradients that training needs.  Types are
 * MEGAMOE_TYPE_BF16 or MEGAMOE_TYPE_F16 (one of them for all operands of a
 * call); sums are fp32, each output rounded once.  Row matrices may have any row
 * stride that keeps rows on 16-byte boundaries; widths are multiples of 8.
 *
 * Results, here and in the linear in 8-bit integers below, have no memory in common
 * with each other, a workspace or what the call reads: such calls are refused
 * (MEGAMOE_ERR_INVALID_ARG; rows of one stride may lie between each other).  In place,
 * at the same address and stride, are allowed: the activation's result in the gate or
 * up columns of a, its gradient's two halves in those of a or in grad, combine's grad_y
 * in y and its grad_topk_weights in topk_weights.
 * ------------------------------------------------------------------------ */

/*
 * megamoe_grouped_linear -- out[r, n] = sum_k x[r, k] w[e, n, k] for the rows r of
 * each expert e: offsets[e + 1] - offsets[e] of them from padded_offsets[e] on, as
 * megamoe_route_permute gives both with any pad (padded_offsets null: from
 * offsets[e] on, which is pad 1).  Any counts, none among them.
 *   x        [rows, K], row stride ld_x; w [E, N, K]
 *   out      [rows, N] of `type` or MEGAMOE_TYPE_F32, row stride ld_out; rows of no
 *            expert are left as they are
 *   status   device status word or null: MEGAMOE_DEV_BAD_OFFSETS where an expert's
 *            rows are not all inside the matrix (those outside are left out), or an
 *            expert shares a row with one before it (which is treated as without rows)
 * Values of other experts' rows and of rows of no expert have no part in an expert's
 * product; the order of its sums is fixed by the call's sizes.
 * Requires K and N multiples of 8, 1 <= E <= 1024, rows, K and N below 2^30 (and tiles
 * of 256 x 256, with all rows in every expert, as well), pointers 16-byte and rows
 * 16-byte aligned.
 */
megamoe_status megamoe_grouped_linear(const void* x, int type, int64_t rows, int64_t ld_x,
                                      const void* w, int E, int N, int K, const int32_t* offsets,
                                      const int32_t* padded_offsets, int out_type, void* out,
                                      int64_t ld_out, uint32_t* status, megamoe_stream_t stream);

/*
 * megamoe_grouped_linear_backward -- its gradients:
 *   grad_x [rows, K]  grad_x[r, k] = sum_n grad_out[r, n] w[e, n, k], of `type`; rows
 *                     of no expert are left as they are
 *   grad_w [E, N, K]  grad_w[e, n, k] = sum_r grad_out[r, n] x[r, k] over e's rows, of
 *                     `type` or MEGAMOE_TYPE_F32; zeros for an expert without rows
 * Either may be null and is then not computed (w may then be null for grad_x, x for
 * grad_w).
 */
megamoe_status megamoe_grouped_linear_backward(
    const void* grad_out, int64_t ld_grad, const void* x, int64_t ld_x, const void* w, int type,
    int64_t rows, int E, int N, int K, const int32_t* offsets, const int32_t* padded_offsets,
    void* grad_x, int64_t ld_grad_x, int grad_w_type, void* grad_w, uint32_t* status,
    megamoe_stream_t stream);

/*
 * megamoe_silu_mul -- out[r, i] = g / (1 + exp(-g)) * u with g = a[r, i] and u =
 * a[r, I + i]; a [rows, 2 I], out [rows, I].  live_rows (device int32, may be null):
 * rows from *live_rows on are neither read nor written (offsets + E with pad 1).
 * megamoe_silu_mul_backward -- grad_a [rows, 2 I] from grad [rows, I]: of g
 * grad u s (1 + g (1 - s)), of u grad g s, with s = 1 / (1 + exp(-g)).
 */
megamoe_status megamoe_silu_mul(const void* a, int type, int64_t rows, int I, int64_t ld_a,
                                const int32_t* live_rows, void* out, int64_t ld_out,
                                megamoe_stream_t stream);
megamoe_status megamoe_silu_mul_backward(const void* grad, int64_t ld_grad, const void* a, int type,
                                         int64_t rows, int I, int64_t ld_a,
                                         const int32_t* live_rows, void* grad_a, int64_t ld_grad_a,
                                         megamoe_stream_t stream);

/*
 * megamoe_gather_rows -- tokens into the experts' order: out[r] = x[row_src[r] / k], zeros
 * where row_src[r] < 0 (row_src as megamoe_route_permute gives it; a source past the
 * T tokens counts as none).  Its gradient with respect to x is
 * megamoe_combine_rows of the rows' gradients without weights.
 *   x [T, d], row_src [rows], out [rows, d]
 */
megamoe_status megamoe_gather_rows(const void* x, int type, int64_t T, int d, int64_t ld_x,
                                   const int32_t* row_src, int64_t rows, int k, void* out,
                                   int64_t ld_out, megamoe_stream_t stream);

/*
 * megamoe_combine_rows -- out[t] = sum_j topk_weights[t, j] y[slot_dst[t k + j]] in
 * ascending j, one rounding at the end; slots whose row is negative or past the
 * matrix are skipped; topk_weights null: all 1.
 *   y [rows, d], slot_dst [T, k], topk_weights [T, k], out [T, d] of `type`
 */
megamoe_status megamoe_combine_rows(const void* y, int type, int64_t rows, int64_t ld_y,
                                    const int32_t* slot_dst, const float* topk_weights, int64_t T,
                                    int k, int d, void* out, int64_t ld_out,
                                    megamoe_stream_t stream);

/*
 * megamoe_combine_rows_backward -- its gradients for slot_dst whose rows are all
 * different, as megamoe_route_permute gives them:
 *   grad_y [rows, d]           grad_y[slot_dst[t k + j]] = topk_weights[t, j]
 *                              grad_out[t], of `type`; rows of no slot are left
 *   grad_topk_weights [T, k]   sum_i grad_out[t, i] y[slot_dst[t k + j], i], 0 for a
 *                              skipped slot; may be null (y may then be null)
 */
megamoe_status megamoe_combine_rows_backward(const void* grad_out, int64_t ld_grad, const void* y,
                                             int type, int64_t rows, int64_t ld_y,
                                             const int32_t* slot_dst, const float* topk_weights,
                                             int64_t T, int k, int d, void* grad_y,
                                             int64_t ld_grad_y, float* grad_topk_weights,
                                             megamoe_stream_t stream);

/* ------------------------------------------------------------------------
 * Linear in 8-bit integers: a scale for each token (row of x) and one for each
 * output channel (row of w), symmetric, integers -127 .. 127 (-128 is taken as it
 * is where the caller brings it).
 *   scale[t] = amax_t / 127 (correctly rounded), code = rint(127 x / amax_t), ties to
 *   even, decided as in exact arithmetic.  A row of zeros has scale 0.  A row that
 *   holds Inf or NaN gets scale NaN and codes 0, and MEGAMOE_DEV_NONFINITE is set.
 * ------------------------------------------------------------------------ */

/* x [rows, K] of MEGAMOE_TYPE_BF16, F16 or F32 -> codes int8 [rows, K], scales [rows];
 * status: device status word or null.  Requires K a multiple of 16, x and codes
 * 16-byte aligned, rows of x on 16-byte boundaries. */
megamoe_status megamoe_quantize_int8(const void* x, int x_type, int64_t rows, int K, int64_t ld,
                                     int8_t* codes, float* scales, uint32_t* status,
                                     megamoe_stream_t stream);

/*
 * megamoe_linear_int8 -- out[t, n] = (sum_k q_x[t, k] w_codes[n, k]) s_x[t] w_scales[n].
 *   x         [T, K], row stride ld_x: BF16, F16 or F32, quantised here as above, or
 *             MEGAMOE_TYPE_I8 codes with x_scales [T] (null otherwise)
 *   w_codes   int8 [N, K], w_scales float [N]
 *   out       [T, N] bf16 (MEGAMOE_EPI_BF16) or fp32 (MEGAMOE_EPI_F32)
 *   ws        at least megamoe_linear_int8_workspace_size(T, K, N) bytes, 256-byte
 *             aligned; its first 4 bytes are the status word
 * The integers' sum of an fp32 result is exact for K below 131072, whatever T is, and
 * rounded once.  That of a bf16 result is so for few tokens, whose integers fit on chip
 * (up to 16, with T K up to some 96000); else it is exact while no partial sum passes
 * 2^24 in magnitude, and past that cut towards zero at each 16 of K, by up to 2^-23 of
 * what has been added up.
 * Requires K a multiple of 16, N of 8, T, K and N below 2^30, pointers 16-byte
 * aligned (scales 4-byte) and rows on 16-byte boundaries.
 */
size_t megamoe_linear_int8_workspace_size(int64_t T, int K, int N);
megamoe_status megamoe_linear_int8(const void* x, int x_type, int64_t T, int K, int64_t ld_x,
                                   const float* x_scales, const int8_t* w_codes,
                                   const float* w_scales, int N, int out_dtype, void* out,
                                   int64_t ld_out, void* ws, size_t ws_bytes,
                                   megamoe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MEGAMOE_H */
