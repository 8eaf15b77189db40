// Host-side launchers of the MegaMoE kernels (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/megamoe.h"

namespace megamoe {

// Launch on `stream` with programmatic stream serialization: the kernel may be
// scheduled while its predecessor finishes; every kernel of this library
// executes griddepcontrol.wait before touching global memory.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// The same with clusters of `cluster` blocks.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                      int cluster, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

size_t route_smem_bytes(int E);
// Routing over many blocks (three passes) when the caller passes a block_hist
// scratch of kRouteMaxBlocks * E ints: megamoe_forward from this many slots on
// (its workspace holds the scratch from there), the MXFP4 forward from
// kMxRouteMultiMinSlots (api_mx.cu).
constexpr int kRouteMultiMinSlots = 16384;
constexpr int kRouteMaxBlocks = 256;
// zero_words (may be null): n_zero 32-bit words cleared before anything else
// (the forward's status word and amax accumulators).
// row_src may be null: it is not written then.
cudaError_t launch_route(const int32_t* ids, int n_slots, int E, int pad, int32_t* counts,
                         int32_t* offsets, int32_t* padded_offsets, int32_t* row_src,
                         int64_t row_capacity, int32_t* slot_dst, uint32_t* status,
                         uint32_t* zero_words, int n_zero, cudaStream_t stream,
                         int32_t* block_hist = nullptr);

// zero_first: clear *amax first (false when the caller already cleared it).
cudaError_t launch_amax(const uint16_t* x, int64_t rows, int K, int64_t ld, float* amax,
                        uint32_t* status, bool zero_first, cudaStream_t stream);
// Dense linear prologue (one block): status cleared, single-group offsets
// {0, rows, 0, rows}, and the amax of x when linear_prologue_full_amax (else
// amax = 0 for a following launch_amax with zero_first = false).
bool linear_prologue_full_amax(int64_t rows, int K);
cudaError_t launch_linear_prologue(const uint16_t* x, int64_t rows, int K, int64_t ld,
                                   float* amax, uint32_t* status, int32_t* groups,
                                   cudaStream_t stream);
cudaError_t launch_quant(const uint16_t* x, int64_t rows_in, int K, int64_t ld,
                         const int32_t* slot_dst, int k, const int32_t* row_src,
                         const int32_t* live_rows, int64_t out_rows, const float* amax,
                         float* gs_out, uint8_t* codes, uint8_t* scales, int scale_layout,
                         cudaStream_t stream, bool slot_rows = false);

// Small-batch prologue of the forward in one thread block: route and the amax
// of x.  Used when prologue_fits(T, d).
bool prologue_fits(int T, int d);
// Router fused into the prologue: ids/weights [T, k] (k = k_routed + shared
// column) are written from logits [T, ld] over n_logits experts, then routed.
struct RouterArgs {
  const float* logits = nullptr;
  int64_t ld = 0;
  const float* bias = nullptr;
  int n_logits = 0;
  int k_routed = 0;
  int shared = -1;
  int32_t* ids_out = nullptr;
  float* w_out = nullptr;
};
cudaError_t launch_prologue(const int32_t* ids, int T, int k, int E, int pad, int32_t* counts,
                            int32_t* offsets, int32_t* padded_offsets, int32_t* row_src,
                            int64_t row_capacity, int32_t* slot_dst, uint32_t* status,
                            uint32_t* zero_words, int n_zero, const uint16_t* x, int d,
                            float* amax, cudaStream_t stream, const RouterArgs* router = nullptr);
cudaError_t launch_swizzle(const uint8_t* src, int64_t rows, int K, uint8_t* dst,
                           cudaStream_t stream);

cudaError_t launch_pack(const uint8_t* src, int64_t rows, int K, int half_rows, uint8_t* dst,
                        cudaStream_t stream);

struct GemmLaunch {
  const uint8_t* act_codes;
  const uint8_t* act_scales;  // atom layout
  const float* act_gs;
  int64_t act_rows;
  const uint8_t* w_codes;   // tile-major (k_pack; gate/up paired for SILU_MUL)
  const uint8_t* w_scales;  // atom layout
  const float* w_gs;
  int E, N, K;
  const int32_t* offsets;
  const int32_t* padded_offsets;
  int epilogue;
  void* out;
  int64_t ld_out;
  float* out_amax;
  int tile_n;
  uint32_t* status;
  bool zero_amax = true;  // false when the caller already cleared out_amax
  // true only when the offsets were written by a kernel that finished before
  // the one immediately preceding the GEMM (the forward's order): the GEMM
  // then prefetches its first weight stages while that kernel runs
  bool early_weights = false;
  // split-K: ksplit > 1 cuts each tile's K range into ksplit pieces (token
  // tiles of 32 or 64 only); `partial` holds ksplit planes of
  // partial_plane >= offsets[E] * N floats; a finishing kernel sums them
  int ksplit = 1;
  float* partial = nullptr;
  int64_t partial_plane = 0;
  // requantisation of h fused into the SILU_MUL kernel (ksplit 1 only):
  // arrival counter zeroed before the launch, codes [rows, N/4], row-major
  // scales [rows, N/32], global scale out (all null: not fused)
  uint32_t* rq_arrivals = nullptr;
  uint8_t* rq_codes = nullptr;
  uint8_t* rq_scales = nullptr;
  float* rq_gs = nullptr;
  // MXFP4 operands: w_scales atoms of 128 rows x 4 blocks of 32, act_scales in
  // the routed layout (16 bytes per K step of 256, eight used), no global
  // scales; SILU_MUL writes rq_codes and rq_scales (routed layout) instead of
  // out, BFP16 is by rows; no split
  bool mx = false;
};
// Split-K choice for a GEMM of about `tiles` whole-K tiles of KT K steps: the
// smallest ksplit (<= 8, >= 2 K steps a piece) that minimises the waves of
// pieces over the SMs, in units of a whole tile.
int pick_ksplit(double tiles, int KT);
// Encodes the tensor maps and launches the persistent grouped GEMM.
cudaError_t launch_grouped_gemm(const GemmLaunch& g, cudaStream_t stream);
int pick_tile_n(double expected_tokens_per_expert);
// Bound of the grouped GEMM's pipeline waits (0 restores the default 4 s).
void set_wait_limit_ns(uint64_t ns);
uint64_t wait_limit_ns();

// Router: ids/weights [T, k (+1 with a shared expert)] from fp32 logits.
cudaError_t launch_router(const float* logits, int64_t T, int E, int64_t ld, const float* bias,
                          int k, int shared, int32_t* ids, float* weights, cudaStream_t stream);

// 2-D tensor map over a [rows, row_bytes] byte matrix, boxes of box_rows x 128
// bytes in the 128-byte swizzle.
bool make_codes_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_bytes,
                    uint32_t box_rows);

// 2-D tensor map of any type: [rows, cols] with a row stride of `stride` bytes.
bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t cols,
              uint64_t rows, uint64_t stride, uint32_t box_cols, uint32_t box_rows,
              CUtensorMapSwizzle swizzle);

// 3-D map, strides in bytes.
bool make_map_3d(CUtensorMap* map, const void* base, uint64_t n0, uint64_t n1, uint64_t n2,
                 uint64_t stride1, uint64_t stride2, uint32_t box0, uint32_t box1, uint32_t box2,
                 CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT32,
                 CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_NONE);

// Scored router (grouped top-k over sigmoid or softmax scores) and its gradient.
struct ScoredRouter {
  const void* logits;  // [T, ld], fp32 or bf16
  bool bf16;
  int64_t T, ld;
  int E;
  const float* bias;
  int softmax, n_group, topk_group, group_top, k, renormalize;
  float scale;
  int32_t* ids;  // [T, k]; read by the gradient
  float* weights;
};
cudaError_t launch_scored_router(const ScoredRouter& r, cudaStream_t stream);
// grad [T, k] -> out [T, ld_out] of the logits' type.
cudaError_t launch_scored_router_backward(const ScoredRouter& r, const float* grad, void* out,
                                          int64_t ld_out, cudaStream_t stream);

// MXFP4 quantisation of x [rows, K] along rows, or (transpose) along columns
// into codes [K, R / 2] with R = rows up to a multiple of 32.
struct MxQuant {
  const void* x;
  int type;  // MEGAMOE_TYPE_*
  int64_t rows, ld;
  int K;
  bool transpose;
  uint8_t* codes;
  uint8_t* scales;
  int layout;  // MEGAMOE_SCALES_*
  uint32_t* status;
  uint32_t* flags;  // one word a block for the product that follows, or null
};
// blocks (may be null): blocks of the launch, the words of flags.
cudaError_t launch_mx_quantize(const MxQuant& q, cudaStream_t s, int* blocks = nullptr);
// Matrices quantised tile by tile in one launch, each along its columns (codes
// of x^T), along its rows (atom layout of the scales), or both from one read.
struct MxTile {
  const void* x;
  int type;
  int64_t rows, ld;
  int K;
  uint8_t* row_codes;  // null: not along the rows
  uint8_t* row_scales;
  uint8_t* col_codes;  // null: not along the columns
  uint8_t* col_scales;
  int col_layout;
  int first, col_tiles;  // set by the launch
};
struct MxTiles {
  MxTile job[3];
  int count;
  uint32_t* status;
  uint32_t* flags;  // as MxQuant::flags
  int tiles;  // set by the launch
};
// Most words that a quantising launch leaves in its flags.
int mx_flags_words();
cudaError_t launch_mx_tiles(MxTiles jobs, cudaStream_t s, int* blocks = nullptr);
// x [T, d] bf16 into routed rows slot_dst[t k + j] (routed scale layout, or atoms).
cudaError_t launch_mx_routed(const uint16_t* x, int64_t T, int d, const int32_t* slot_dst, int k,
                             bool atoms, uint8_t* codes, uint8_t* scales, uint32_t* status,
                             cudaStream_t s);
// The routed experts' products on pairs of CTAs (large batches): experts' rows
// start at multiples of 128, scales of rows in the atom layout.  y null: gate and
// up (N = 2 I), SiLU * up quantised to h_codes and h_scales (atom layout); else
// down (N = d), y in BFP16 by rows and its exponents.
struct MxExperts {
  const uint8_t* act_codes;
  const uint8_t* act_scales;
  int64_t rows;
  const uint8_t* w_codes;
  const uint8_t* w_scales;
  int E, N, K;
  const int32_t* offsets;  // complete before the kernel ahead of this one started
  const int32_t* padded_offsets;
  uint8_t* h_codes;
  uint8_t* h_scales;
  uint16_t* y;
  int8_t* y_exp;
  uint32_t* status;
};
cudaError_t launch_mx_experts(const MxExperts& g, cudaStream_t stream);
// Row-major codes and scales -> values.
cudaError_t launch_mx_values(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K,
                             void* out, bool f32, int64_t ld, cudaStream_t s);
cudaError_t launch_mx_swizzle(const uint8_t* src, int64_t rows, int64_t K, uint8_t* dst,
                              cudaStream_t s);

// out [R, C] = P [R, K] Q [C, K]^T of MXFP4 operands (row-major codes, atom
// scales); K a multiple of 32, C of 16.
struct MxProduct {
  const uint8_t* r_codes;
  const uint8_t* r_scales;
  const uint8_t* c_codes;
  const uint8_t* c_scales;
  int64_t R, C, K;
  void* out;
  bool out_f32;
  int64_t ld_out;
  uint32_t* status;
  // findings of the quantising launch before it, for the status word
  const uint32_t* flags;
  int flag_count;
  // one of a linear's gradients: the launch before it ran with all of an SM's
  // shared memory (k_mx_tiles), and the other one may share the launch
  bool after_tiles;
};
cudaError_t launch_mx_product(const MxProduct& g, cudaStream_t stream);
// Two independent products, in one launch where their sizes allow it.
cudaError_t launch_mx_products(const MxProduct& g, const MxProduct& h, cudaStream_t stream);

// The MXFP4 linear for few tokens in one launch (clears *status first).
bool mx_linear_few_fits(int64_t T, int64_t K, int64_t N);
cudaError_t launch_mx_linear_few(const void* x, int x_type, int64_t T, int K, int64_t ld_x,
                                 const uint8_t* codes, const uint8_t* scales, int N, void* out,
                                 bool out_f32, int64_t ld_out, uint32_t* status,
                                 cudaStream_t stream);

// Products of 16-bit operands grouped by expert (grouped.cu): x [rows, K], grad
// [rows, N] in the experts' order, w [E, N, K].
struct Grouped {
  const void* x;
  const void* grad;
  const void* w;
  int type;  // MEGAMOE_TYPE_BF16 or _F16
  int64_t rows, ld_x, ld_grad;
  int E, N, K;
  const int32_t* offsets;
  const int32_t* padded_offsets;  // null: the same
  uint32_t* status;
};
cudaError_t launch_grouped_forward(const Grouped& g, void* out, int out_type, int64_t ld_out,
                                   cudaStream_t stream);
cudaError_t launch_grouped_grad_x(const Grouped& g, void* out, int64_t ld_out, cudaStream_t stream);
// after_grad_x: launched right behind launch_grouped_grad_x of the same operands.
cudaError_t launch_grouped_grad_w(const Grouped& g, void* out, int out_type, bool after_grad_x,
                                  cudaStream_t stream);
// Most tiles of the first two with `features` columns of output (counted in 31 bits).
inline int64_t grouped_tiles(int64_t rows, int E, int features) {
  return (rows / 256 + (rows < E ? rows : E)) * ((features + int64_t{255}) / 256);
}

// 8-bit integer linear (int8.cu).  x [T, K] of any MEGAMOE_TYPE_*; as I8 with
// x_scales [T].
struct Int8Quant {
  const void* x;
  int type;
  const float* x_scales;
  int64_t T, ld;
  int K;
  int8_t* codes;   // [T, K], or
  uint16_t* half;  // the integers as fp16, [T, K]
  float* scales;
  uint32_t* status;  // NONFINITE is set here unless clear
  bool clear;  // status = 0 (the product that follows sets what it finds)
};
cudaError_t launch_int8_quantize(const Int8Quant& q, cudaStream_t stream);
struct Int8Product {
  const uint16_t* x;  // fp16 integers [T, K]
  const float* x_scales;  // readable up to a multiple of 64
  int64_t T;
  const int8_t* w;  // [N, K]
  const float* w_scales;
  int N, K;
  void* out;
  bool out_f32;
  int64_t ld_out;
  float* partial;  // plan.split > 1: [split][T][N]
  uint32_t* status;
};
// How the product runs on pairs of CTAs.
struct Int8Plan {
  int per;        // tokens of a tile
  int64_t tiles;
  int split;      // shares of a tile's sum
};
constexpr int64_t kInt8Pairs = 76;  // of SMs (counted on for workspaces, which are sized without a device)
// Sums of fp32 results that are taken in parts: one part is exact, and 32 bits hold them.
inline bool int8_folds(int K) { return K > 1024 && K < 131072; }
Int8Plan int8_plan(int64_t T, int N, int K, bool fold);
cudaError_t launch_int8_product(const Int8Product& g, cudaStream_t stream);
// The same for few tokens.  Dots: up to four, quantised in the same launch (q's
// x, type, T, ld and x_scales; clears *status first).  Few: up to sixteen, q the
// quantised tokens (type I8).
bool int8_dots_fit(int64_t T, int64_t K);
cudaError_t launch_int8_dots(const Int8Quant& q, const Int8Product& g, cudaStream_t stream);
bool int8_few_fits(int64_t T, int64_t K);
cudaError_t launch_int8_few(const Int8Quant& q, const Int8Product& g, cudaStream_t stream);

// The gated activation and the movement of rows (rows.cu); 16-bit elements,
// widths multiples of 8.
struct Silu {
  const void* a;  // [rows, 2 I]: gate, up
  const void* grad;  // [rows, I], backward only
  int type;
  int64_t rows, ld_a, ld_grad, ld_out;
  int I;
  const int32_t* live_rows;  // may be null
  void* out;  // [rows, I], or backward [rows, 2 I]
};
cudaError_t launch_silu(const Silu& a, cudaStream_t stream);
cudaError_t launch_silu_backward(const Silu& a, cudaStream_t stream);
cudaError_t launch_gather_rows(const void* x, int64_t T, int d, int64_t ld_x,
                               const int32_t* row_src, int64_t rows, int k, void* out,
                               int64_t ld_out, cudaStream_t stream);
struct CombineRows {
  const void* y;
  int type;
  int64_t rows, ld_y;
  const int32_t* slot_dst;
  const float* weights;  // null: all one
  int64_t T;
  int k, d;
  const void* grad;  // backward: [T, d]
  int64_t ld_grad;
  void* out;  // [T, d], or backward the gradient of y
  int64_t ld_out;
  float* grad_weights;  // backward, may be null
};
cudaError_t launch_combine_rows(const CombineRows& c, cudaStream_t stream);
cudaError_t launch_combine_rows_backward(const CombineRows& c, cudaStream_t stream);

// Shape and weight-pointer checks of megamoe_forward.
megamoe_status check_forward_shape(const megamoe_weights* w, int T, int k, int pad);
// Argument and shape checks of megamoe_forward that do not involve the
// workspace (router: the ids and weights come from a fused router).
megamoe_status check_forward_args(const megamoe_weights* w, const uint16_t* x,
                                  const int32_t* topk_ids, const float* topk_weights, int T, int k,
                                  int pad, const uint16_t* out, bool router);

// Number of SMs of the current device (at least 1).
int num_sms();

// out: bf16 [T, d] (one rounding of the fp32 sum), or with out_f32 the fp32
// sum itself.
// y fp32 [*, ld_y] (y_exp null) or BFP16 (uint16 values at y, exponents
// [rows / 16, ld_y / 8] at y_exp), or with by_row BFP16 by rows (exponent
// words, 16 bits, [rows, ld_y / 32])
// (y_rows: rows of a BFP16 y; slots at or past it are skipped)
cudaError_t launch_combine(const void* y, const int8_t* y_exp, int64_t ld_y, int64_t y_rows,
                           const int32_t* slot_dst, const float* w, int T, int k, int d,
                           void* out, bool out_f32, cudaStream_t stream, bool by_row = false);
// Non-finite scan of a forward's stage outputs (MEGAMOE_STAGE_* bits in
// *flags, cleared first); valid rows only, every output row.
cudaError_t launch_stage_scan(const int32_t* row_src, const int32_t* padded_total,
                              const uint8_t* xq_sf, const uint16_t* h, const uint8_t* hq_sf,
                              const int8_t* y_exp, const uint16_t* out, int T, int d, int I,
                              uint32_t* flags, cudaStream_t stream);
// out[i] = bf16_rne(in[i]), n a multiple of 4.
cudaError_t launch_round_bf16(const float* in, int64_t n, uint16_t* out, cudaStream_t stream);
// Expert-parallel shard: ids in [base, base + E_local) -> id - base; other
// valid ids and ids < 0 -> -1 (skipped); ids >= E_total -> E_local (out of
// range for the shard, so the routing flags and skips them).
cudaError_t launch_ep_remap(const int32_t* ids, int64_t n, int base, int E_local, int E_total,
                            int32_t* out, cudaStream_t stream);

}  // namespace megamoe
