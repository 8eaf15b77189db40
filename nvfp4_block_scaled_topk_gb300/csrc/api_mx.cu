// C ABI of the scored router and the MXFP4 operators: argument checks,
// workspace layouts and the order of the launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/megamoe.h"
#include "kernels.h"

using namespace megamoe;

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline megamoe_status cuda_status(cudaError_t e) {
  return e == cudaSuccess ? MEGAMOE_OK : MEGAMOE_ERR_CUDA;
}
inline cudaStream_t as_stream(megamoe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Bytes of an element type, 0 if there is no such type.
inline int64_t type_bytes(int type) {
  return type == MEGAMOE_TYPE_F32 ? 4 : type == MEGAMOE_TYPE_BF16 || type == MEGAMOE_TYPE_F16 ? 2 : 0;
}
inline int64_t epi_bytes(int dtype) {
  return dtype == MEGAMOE_EPI_F32 ? 4 : dtype == MEGAMOE_EPI_BF16 ? 2 : 0;
}
// A matrix that is read or written in 16-byte vectors: base and rows on 16 bytes.
inline bool vectors_ok(const void* p, int64_t ld, int64_t bytes) {
  return aligned(p, 16) && ld * bytes % 16 == 0;
}

// Carves 256-byte aligned regions out of a workspace (sizes only when base is null).
struct Carver {
  uint8_t* base;
  size_t off = 0;
  uint8_t* take(size_t bytes) {
    uint8_t* p = base ? base + off : nullptr;
    off = (off + bytes + 255) / 256 * 256;
    return p;
  }
};

// An operand quantised into the workspace.
struct MxOperand {
  uint8_t* codes;
  uint8_t* scales;
};
MxOperand take_operand(Carver& c, int64_t rows, int64_t K) {
  MxOperand o;
  o.codes = c.take(static_cast<size_t>(rows) * (K / 2));
  o.scales = c.take(MEGAMOE_MX_ATOM_BYTES(rows, K));
  return o;
}

struct LinearWs {
  uint32_t* status;
  uint32_t* flags;  // of the quantising launch
  MxOperand x;
  size_t bytes;
};
LinearWs carve_linear(void* base, int64_t T, int K, int N) {
  Carver c{static_cast<uint8_t*>(base)};
  LinearWs w{};
  w.status = reinterpret_cast<uint32_t*>(c.take(256));
  if (!mx_linear_few_fits(T, K, N)) {
    w.flags = reinterpret_cast<uint32_t*>(c.take(4 * static_cast<size_t>(mx_flags_words())));
    w.x = take_operand(c, T, K);
  }
  w.bytes = c.off;
  return w;
}

struct BackwardWs {
  uint32_t* status;
  uint32_t* flags;
  MxOperand dy, dy_t, x_t, w_t;
  size_t bytes;
};
BackwardWs carve_backward(void* base, int64_t T, int K, int N) {
  Carver c{static_cast<uint8_t*>(base)};
  BackwardWs w{};
  const int64_t R = (T + 31) / 32 * 32;
  w.status = reinterpret_cast<uint32_t*>(c.take(256));
  w.flags = reinterpret_cast<uint32_t*>(c.take(4 * static_cast<size_t>(mx_flags_words())));
  w.dy = take_operand(c, T, N);
  w.dy_t = take_operand(c, N, R);
  w.x_t = take_operand(c, K, R);
  w.w_t = take_operand(c, K, N);
  w.bytes = c.off;
  return w;
}

// Rows and columns of the products are int, their tiles (of 128 x 128) and the
// quantisers' (of 128 x 64 at least, over all three matrices) counted in 31 bits.
constexpr int kMaxColumns = 1 << 30;  // columns rounded up to whole steps stay in 31 bits
bool linear_sizes_ok(int64_t T, int K, int N) {
  if (K % 32 != 0 || N % 32 != 0 || T >= (int64_t{1} << 30) || K >= kMaxColumns || N >= kMaxColumns)
    return false;
  const int64_t t = T / 128 + 1, k = K / 128 + 1, n = N / 128 + 1, most = int64_t{1} << 28;
  return t * k < most && t * n < most && n * k < most;
}

MxQuant quant_of(const void* x, int type, int64_t rows, int K, int64_t ld, bool transpose,
                 const MxOperand& o, uint32_t* status, uint32_t* flags) {
  return MxQuant{x, type, rows, ld, K, transpose, o.codes, o.scales, MEGAMOE_SCALES_MMA, status,
                 flags};
}

// Large batches run on pairs of CTAs with 256-row tiles (mx_experts.cu), from
// about this many rows an expert on: below, most experts' rows fit one 128-row
// tile of the single CTAs.  Single / pairs, us, at 90, 110 and 130 rows an expert:
// 48 experts of 7168 x 2048 with even loads 211 / 224, 223 / 232, 259 / 239, with
// uneven ones (weights of 1 / rank^0.3) 218 / 224, 236 / 234, 256 / 241; 64 experts
// of 2048 x 1024 even 65 / 66, 70 / 69, 93 / 72, uneven 68 / 67, 78 / 73, 84 / 75.
constexpr double kPairRows = 105.0;
bool pair_experts(int T, int k, int E) {
  return num_sms() >= 2 && static_cast<double>(T) * k / E >= kPairRows;
}
// Rows of an expert are padded to whole scale atoms of 128 rows there.
int padding(int T, int k, int E, int pad) {
  return pair_experts(T, k, E) ? (pad + 127) / 128 * 128 : pad;
}

// Routing over many blocks (three passes) from this many slots on.  A forward of
// small experts with one block / three passes (us): 384 experts, 2400 slots 32.4 /
// 33.7, 4200 34.9 / 34.4, 6000 37.4 / 35.2, 12018 49.5 / 40.2; 48 experts 20.3 /
// 21.4, 23.6 / 23.2, 28.0 / 26.4, 35.8 / 29.0.
constexpr size_t kMxRouteMultiMinSlots = 4096;

// Workspace of the MXFP4 forward.
struct ForwardWs {
  uint32_t* status;
  int32_t* counts;
  int32_t* offsets;
  int32_t* padded_offsets;
  int32_t* slot_dst;
  uint8_t* xq_codes;
  uint8_t* xq_scales;  // routed layout, 16 bytes per K step of 256, or (pairs) atoms
  uint8_t* hq_codes;
  uint8_t* hq_scales;
  uint16_t* y;  // BFP16 by rows: one exponent word per 32 columns of a row
  int8_t* y_exp;
  int32_t* r_ids;
  float* r_w;
  int32_t* route_hist;
  int64_t rows;
  size_t bytes;
};
ForwardWs carve_forward(void* base, int T, int k, int E, int d, int I, int pad) {
  Carver c{static_cast<uint8_t*>(base)};
  ForwardWs w{};
  const size_t slots = static_cast<size_t>(T) * k;
  w.rows = megamoe_max_padded_rows(T, k, E, padding(T, k, E, pad));
  const size_t rows = static_cast<size_t>(w.rows);
  auto ints = [&](size_t n) { return reinterpret_cast<int32_t*>(c.take(4 * n)); };
  w.status = reinterpret_cast<uint32_t*>(c.take(256));
  w.counts = ints(E);
  w.offsets = ints(E + 1);
  w.padded_offsets = ints(E + 1);
  w.slot_dst = ints(slots);
  w.xq_codes = c.take(rows * (d / 2));
  // (atoms take half of the routed layout's bytes, in whole groups of 128 rows)
  const size_t whole = (rows + 127) / 128 * 128;
  w.xq_scales = c.take(whole * (d / 16));
  w.hq_codes = c.take(rows * (I / 2));
  w.hq_scales = c.take(whole * (I / 16));
  uint8_t* y = c.take(rows * d * 2 + rows * (d / 32) * 2);
  w.y = reinterpret_cast<uint16_t*>(y);
  w.y_exp = y ? reinterpret_cast<int8_t*>(y + rows * d * 2) : nullptr;
  w.r_ids = ints(slots);
  w.r_w = reinterpret_cast<float*>(ints(slots));
  w.route_hist = slots >= kMxRouteMultiMinSlots
                     ? ints(static_cast<size_t>(kRouteMaxBlocks) * E)
                     : nullptr;
  w.bytes = c.off;
  return w;
}

megamoe_status check_router(const void* logits, int type, int64_t T, int E, int64_t ld, int score,
                            int k) {
  if (T < 0 || E < 1 || ld < E || k < 1 || k > E) return MEGAMOE_ERR_INVALID_ARG;
  if (type != MEGAMOE_TYPE_F32 && type != MEGAMOE_TYPE_BF16) return MEGAMOE_ERR_INVALID_ARG;
  if (score != MEGAMOE_SCORE_SIGMOID && score != MEGAMOE_SCORE_SOFTMAX)
    return MEGAMOE_ERR_INVALID_ARG;
  if (E > MEGAMOE_MAX_EXPERTS || k > MEGAMOE_MAX_TOPK || T >= (int64_t{1} << 31))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && !logits) return MEGAMOE_ERR_INVALID_ARG;
  if (logits && !aligned(logits, type_bytes(type))) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  return MEGAMOE_OK;
}
megamoe_status check_groups(int E, int n_group, int topk_group, int group_top, const float* bias) {
  if (n_group < 1 || E % n_group != 0 || topk_group < 1 || topk_group > n_group ||
      (group_top != 1 && group_top != 2))
    return MEGAMOE_ERR_INVALID_ARG;
  if (n_group > 32) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (bias && !aligned(bias, 4)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  return MEGAMOE_OK;
}

// Shapes of the MXFP4 forward (those of megamoe_forward).
megamoe_status check_mx_forward(const megamoe_mx_weights* w, const uint16_t* x, int T, int k,
                                int pad, const uint16_t* out, const void* ws, size_t ws_bytes) {
  if (!w) return MEGAMOE_ERR_INVALID_ARG;
  const float* none = reinterpret_cast<const float*>(sizeof(float));  // has no global scales
  const megamoe_weights shape{w->num_experts, w->hidden, w->intermediate, w->w13_codes,
                              w->w13_scales,  none,      w->w2_codes,     w->w2_scales, none};
  megamoe_status st = check_forward_args(&shape, x, nullptr, nullptr, T, k, pad, out, true);
  if (st != MEGAMOE_OK) return st;
  // weight blocks' rows are counted in 31 bits
  const int64_t E = w->num_experts, d = w->hidden, I = w->intermediate;
  if (E * 2 * I * (d / 256) >= (int64_t{1} << 31) || E * d * (I / 256) >= (int64_t{1} << 31))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  // and so are padded rows
  if (megamoe_max_padded_rows(T, k, w->num_experts, padding(T, k, w->num_experts, pad)) >=
      (int64_t{1} << 31))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (!ws || !aligned(ws, 256)) return MEGAMOE_ERR_INVALID_ARG;
  if (ws_bytes < megamoe_workspace_size_mxfp4(T, k, w->num_experts, w->hidden, w->intermediate, pad))
    return MEGAMOE_ERR_WORKSPACE_TOO_SMALL;
  return MEGAMOE_OK;
}

megamoe_status run_mx_forward(const megamoe_mx_weights* w, const uint16_t* x,
                              const int32_t* topk_ids, const float* topk_weights, int T, int k,
                              int pad, uint16_t* out, const ForwardWs& wk, cudaStream_t s) {
  const int E = w->num_experts, d = w->hidden, I = w->intermediate;
  const bool pairs = pair_experts(T, k, E);
  pad = padding(T, k, E, pad);
  // The routing clears the status word; no amax of x is needed, so there is
  // nothing between it and the quantiser.
  cudaError_t e = launch_route(topk_ids, T * k, E, pad, wk.counts, wk.offsets, wk.padded_offsets,
                               nullptr, 0, wk.slot_dst, wk.status, wk.status, 1, s,
                               wk.route_hist);
  if (e == cudaSuccess)
    e = launch_mx_routed(x, T, d, wk.slot_dst, k, pairs, wk.xq_codes, wk.xq_scales, wk.status, s);
  if (e != cudaSuccess) return MEGAMOE_ERR_CUDA;
  if (pairs) {
    MxExperts m{};
    m.act_codes = wk.xq_codes;
    m.act_scales = wk.xq_scales;
    m.rows = wk.rows;
    m.w_codes = w->w13_codes;
    m.w_scales = w->w13_scales;
    m.E = E;
    m.N = 2 * I;
    m.K = d;
    m.offsets = wk.offsets;
    m.padded_offsets = wk.padded_offsets;
    m.h_codes = wk.hq_codes;
    m.h_scales = wk.hq_scales;
    m.status = wk.status;
    e = launch_mx_experts(m, s);
    if (e != cudaSuccess) return MEGAMOE_ERR_CUDA;
    m.act_codes = wk.hq_codes;
    m.act_scales = wk.hq_scales;
    m.w_codes = w->w2_codes;
    m.w_scales = w->w2_scales;
    m.N = d;
    m.K = I;
    m.y = wk.y;
    m.y_exp = wk.y_exp;
    e = launch_mx_experts(m, s);
    if (e == cudaSuccess)
      e = launch_combine(wk.y, wk.y_exp, d, wk.rows, wk.slot_dst, topk_weights, T, k, d, out, false,
                         s, true);
    return cuda_status(e);
  }
  const int tile_n = pick_tile_n(static_cast<double>(T) * k / E);
  GemmLaunch g{};
  g.mx = true;
  g.act_codes = wk.xq_codes;
  g.act_scales = wk.xq_scales;
  g.act_rows = wk.rows;
  g.w_codes = w->w13_codes;
  g.w_scales = w->w13_scales;
  g.E = E;
  g.N = 2 * I;
  g.K = d;
  g.offsets = wk.offsets;
  g.padded_offsets = wk.padded_offsets;
  g.epilogue = MEGAMOE_EPI_SILU_MUL;
  g.rq_codes = wk.hq_codes;
  g.rq_scales = wk.hq_scales;
  g.ld_out = I;
  // token-major tiles where 128-token tiles would be chosen, as in megamoe_forward
  g.tile_n = tile_n == 128 ? 256 : tile_n;
  g.status = wk.status;
  // the offsets were complete before the quantiser started
  g.early_weights = true;
  e = launch_grouped_gemm(g, s);
  if (e != cudaSuccess) return MEGAMOE_ERR_CUDA;
  g.act_codes = wk.hq_codes;
  g.act_scales = wk.hq_scales;
  g.w_codes = w->w2_codes;
  g.w_scales = w->w2_scales;
  g.N = d;
  g.K = I;
  g.epilogue = MEGAMOE_EPI_BFP16;
  g.out = wk.y;
  g.ld_out = d;
  g.tile_n = tile_n;
  e = launch_grouped_gemm(g, s);
  if (e == cudaSuccess)
    e = launch_combine(wk.y, wk.y_exp, d, wk.rows, wk.slot_dst, topk_weights, T, k, d, out, false, s,
                       true);
  return cuda_status(e);
}

}  // namespace

extern "C" {

megamoe_status megamoe_router_scored_topk(const void* logits, int logits_type, int64_t T, int E,
                                          int64_t ld_logits, const float* bias, int score,
                                          int n_group, int topk_group, int group_top, int k,
                                          int renormalize, double scale, int32_t* topk_ids,
                                          float* topk_weights, megamoe_stream_t stream) {
  megamoe_status st = check_router(logits, logits_type, T, E, ld_logits, score, k);
  if (st == MEGAMOE_OK) st = check_groups(E, n_group, topk_group, group_top, bias);
  if (st != MEGAMOE_OK) return st;
  if (T > 0 && (!topk_ids || !topk_weights)) return MEGAMOE_ERR_INVALID_ARG;
  if (!aligned(topk_ids, 4) || !aligned(topk_weights, 4)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const ScoredRouter r{logits, logits_type == MEGAMOE_TYPE_BF16, T, ld_logits, E, bias,
                       score == MEGAMOE_SCORE_SOFTMAX, n_group, topk_group, group_top, k,
                       renormalize != 0, static_cast<float>(scale), topk_ids, topk_weights};
  return cuda_status(launch_scored_router(r, as_stream(stream)));
}

megamoe_status megamoe_router_scored_topk_backward(
    const void* logits, int logits_type, int64_t T, int E, int64_t ld_logits,
    const int32_t* topk_ids, const float* grad_weights, int score, int k, int renormalize,
    double scale, void* grad_logits, int64_t ld_grad, megamoe_stream_t stream) {
  megamoe_status st = check_router(logits, logits_type, T, E, ld_logits, score, k);
  if (st != MEGAMOE_OK) return st;
  if (ld_grad < E || (T > 0 && (!topk_ids || !grad_weights || !grad_logits)))
    return MEGAMOE_ERR_INVALID_ARG;
  if (!aligned(topk_ids, 4) || !aligned(grad_weights, 4) ||
      !aligned(grad_logits, type_bytes(logits_type)))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const ScoredRouter r{logits, logits_type == MEGAMOE_TYPE_BF16, T, ld_logits, E, nullptr,
                       score == MEGAMOE_SCORE_SOFTMAX, 1, 1, 1, k, renormalize != 0,
                       static_cast<float>(scale), const_cast<int32_t*>(topk_ids), nullptr};
  return cuda_status(
      launch_scored_router_backward(r, grad_weights, grad_logits, ld_grad, as_stream(stream)));
}

megamoe_status megamoe_quantize_mxfp4(const void* x, int x_type, int64_t rows, int K, int64_t ld,
                                      int transpose, uint8_t* codes, uint8_t* scales,
                                      int scale_layout, uint32_t* status, megamoe_stream_t stream) {
  const int64_t size = type_bytes(x_type);
  if (rows < 0 || K <= 0 || ld < K || !size) return MEGAMOE_ERR_INVALID_ARG;
  if (scale_layout != MEGAMOE_SCALES_ROWMAJOR && scale_layout != MEGAMOE_SCALES_MMA)
    return MEGAMOE_ERR_INVALID_ARG;
  if (K % 32 != 0 || K >= kMaxColumns || rows >= (int64_t{1} << 31))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  // the tiles of a transposed launch are counted in 31 bits
  if (transpose && (rows + 127) / 128 * ((K + 63) / 64) >= (int64_t{1} << 30))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (rows > 0 && (!x || !codes || !scales)) return MEGAMOE_ERR_INVALID_ARG;
  if (rows > 0 && (!vectors_ok(x, ld, size) || !aligned(codes, 16)))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  return cuda_status(launch_mx_quantize(
      MxQuant{x, x_type, rows, ld, K, transpose != 0, codes, scales, scale_layout, status, nullptr},
      as_stream(stream)));
}

megamoe_status megamoe_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                        int K, void* out, int out_type, int64_t ld,
                                        megamoe_stream_t stream) {
  if (rows < 0 || K <= 0 || ld < K) return MEGAMOE_ERR_INVALID_ARG;
  if (out_type != MEGAMOE_TYPE_BF16 && out_type != MEGAMOE_TYPE_F32) return MEGAMOE_ERR_INVALID_ARG;
  if (K % 32 != 0) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (rows > 0 && (!codes || !scales || !out)) return MEGAMOE_ERR_INVALID_ARG;
  if (rows > 0 && (!aligned(codes, 16) || !vectors_ok(out, ld, type_bytes(out_type))))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  return cuda_status(launch_mx_values(codes, scales, rows, K, out, out_type == MEGAMOE_TYPE_F32, ld,
                                      as_stream(stream)));
}

megamoe_status megamoe_swizzle_scales_mxfp4(const uint8_t* src, int64_t rows, int K, uint8_t* dst,
                                            megamoe_stream_t stream) {
  if (rows < 0 || K <= 0) return MEGAMOE_ERR_INVALID_ARG;
  if (K % 32 != 0) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (rows > 0 && (!src || !dst)) return MEGAMOE_ERR_INVALID_ARG;
  return cuda_status(launch_mx_swizzle(src, rows, K, dst, as_stream(stream)));
}

size_t megamoe_linear_mxfp4_workspace_size(int64_t T, int K, int N) {
  if (T < 0 || K <= 0 || N <= 0) return 0;
  return carve_linear(nullptr, T, K, N).bytes;
}

megamoe_status megamoe_linear_mxfp4(const void* x, int x_type, int64_t T, int K, int64_t ld_x,
                                    const uint8_t* w_codes, const uint8_t* w_scales, int N,
                                    int out_dtype, void* out, int64_t ld_out, void* ws,
                                    size_t ws_bytes, megamoe_stream_t stream) {
  const int64_t x_size = type_bytes(x_type), out_size = epi_bytes(out_dtype);
  if (T < 0 || K <= 0 || N <= 0 || ld_x < K || ld_out < N || !x_size || !out_size)
    return MEGAMOE_ERR_INVALID_ARG;
  if (!linear_sizes_ok(T, K, N)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (!w_codes || !w_scales || !ws || (T > 0 && (!x || !out))) return MEGAMOE_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || !aligned(w_codes, 16) || !aligned(w_scales, 16) ||
      (T > 0 && (!vectors_ok(x, ld_x, x_size) || !vectors_ok(out, ld_out, out_size))))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const LinearWs wk = carve_linear(ws, T, K, N);
  if (ws_bytes < wk.bytes) return MEGAMOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = as_stream(stream);
  if (T > 0 && mx_linear_few_fits(T, K, N))
    return cuda_status(launch_mx_linear_few(x, x_type, T, K, ld_x, w_codes, w_scales, N, out,
                                              out_dtype == MEGAMOE_EPI_F32, ld_out, wk.status, s));
  if (T == 0) return cuda_status(cudaMemsetAsync(wk.status, 0, sizeof(uint32_t), s));
  int blocks = 0;
  cudaError_t e = launch_mx_quantize(
      quant_of(x, x_type, T, K, ld_x, false, wk.x, wk.status, wk.flags), s, &blocks);
  if (e == cudaSuccess)
    e = launch_mx_product(MxProduct{wk.x.codes, wk.x.scales, w_codes, w_scales, T, N, K, out,
                                    out_dtype == MEGAMOE_EPI_F32, ld_out, wk.status, wk.flags,
                                    blocks, false},
                          s);
  return cuda_status(e);
}

size_t megamoe_linear_mxfp4_backward_workspace_size(int64_t T, int K, int N) {
  if (T < 0 || K <= 0 || N <= 0) return 0;
  return carve_backward(nullptr, T, K, N).bytes;
}

megamoe_status megamoe_linear_mxfp4_backward(
    const void* grad_out, int grad_type, int64_t ld_grad, const void* x, int x_type, int64_t ld_x,
    const void* w, int w_type, int64_t ld_w, int64_t T, int K, int N, void* grad_x,
    int grad_x_dtype, int64_t ld_grad_x, void* grad_w, int grad_w_dtype, int64_t ld_grad_w,
    void* ws, size_t ws_bytes, megamoe_stream_t stream) {
  const int64_t g_size = type_bytes(grad_type), x_size = type_bytes(x_type),
                w_size = type_bytes(w_type);
  const int64_t gx_size = epi_bytes(grad_x_dtype), gw_size = epi_bytes(grad_w_dtype);
  if (T < 0 || K <= 0 || N <= 0 || ld_grad < N || !g_size || !ws) return MEGAMOE_ERR_INVALID_ARG;
  if (grad_x && (ld_w < K || !w_size || !gx_size || ld_grad_x < K || !w))
    return MEGAMOE_ERR_INVALID_ARG;
  if (grad_w && (ld_x < K || !x_size || !gw_size || ld_grad_w < K)) return MEGAMOE_ERR_INVALID_ARG;
  if (!linear_sizes_ok(T, K, N)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && (!grad_out || (grad_w && !x))) return MEGAMOE_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || (T > 0 && !vectors_ok(grad_out, ld_grad, g_size)) ||
      (grad_x && (!vectors_ok(w, ld_w, w_size) || !vectors_ok(grad_x, ld_grad_x, gx_size))) ||
      (grad_w && ((T > 0 && !vectors_ok(x, ld_x, x_size)) ||
                  !vectors_ok(grad_w, ld_grad_w, gw_size))))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const BackwardWs wk = carve_backward(ws, T, K, N);
  if (ws_bytes < wk.bytes) return MEGAMOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = as_stream(stream);
  cudaError_t e = cudaSuccess;
  if (T == 0 || (!grad_x && !grad_w)) {  // sums over nothing
    e = cudaMemsetAsync(wk.status, 0, sizeof(uint32_t), s);
    if (e == cudaSuccess && grad_w)
      e = cudaMemset2DAsync(grad_w, ld_grad_w * gw_size, 0, K * gw_size, N, s);
    return cuda_status(e);
  }
  // one launch reads grad_out once for both products, x and w once each
  MxTiles jobs{};
  auto add = [&](const void* p, int type, int64_t rows, int cols, int64_t ld, const MxOperand* row,
                 const MxOperand* col) {
    MxTile& t = jobs.job[jobs.count++];
    t.x = p;
    t.type = type;
    t.rows = rows;
    t.K = cols;
    t.ld = ld;
    if (row) {
      t.row_codes = row->codes;
      t.row_scales = row->scales;
    }
    if (col) {
      t.col_codes = col->codes;
      t.col_scales = col->scales;
    }
    t.col_layout = MEGAMOE_SCALES_MMA;
  };
  jobs.status = wk.status;
  jobs.flags = wk.flags;
  add(grad_out, grad_type, T, N, ld_grad, grad_x ? &wk.dy : nullptr, grad_w ? &wk.dy_t : nullptr);
  if (grad_w) add(x, x_type, T, K, ld_x, nullptr, &wk.x_t);
  if (grad_x) add(w, w_type, N, K, ld_w, nullptr, &wk.w_t);
  int blocks = 0;
  e = launch_mx_tiles(jobs, s, &blocks);
  const int64_t R = (T + 31) / 32 * 32;
  const MxProduct px{wk.dy.codes, wk.dy.scales, wk.w_t.codes, wk.w_t.scales, T, K, N, grad_x,
                     grad_x_dtype == MEGAMOE_EPI_F32, ld_grad_x, wk.status, wk.flags, blocks,
                     true};
  const MxProduct pw{wk.dy_t.codes, wk.dy_t.scales, wk.x_t.codes, wk.x_t.scales, N, K, R, grad_w,
                     grad_w_dtype == MEGAMOE_EPI_F32, ld_grad_w, wk.status, wk.flags,
                     grad_x ? 0 : blocks, true};
  if (e == cudaSuccess) {
    if (grad_x && grad_w) e = launch_mx_products(px, pw, s);
    else if (grad_x) e = launch_mx_product(px, s);
    else if (grad_w) e = launch_mx_product(pw, s);
  }
  return cuda_status(e);
}

size_t megamoe_workspace_size_mxfp4(int T, int k, int E, int d, int I, int pad) {
  if (T < 0 || k < 1 || E < 1 || d <= 0 || I <= 0 || pad < 1) return 0;
  return carve_forward(nullptr, T, k, E, d, I, pad).bytes;
}

megamoe_status megamoe_forward_mxfp4(const megamoe_mx_weights* w, const uint16_t* x,
                                     const int32_t* topk_ids, const float* topk_weights, int T,
                                     int k, int pad, uint16_t* out, void* ws, size_t ws_bytes,
                                     megamoe_stream_t stream) {
  megamoe_status st = check_mx_forward(w, x, T, k, pad, out, ws, ws_bytes);
  if (st != MEGAMOE_OK) return st;
  if (T > 0 && (!topk_ids || !topk_weights)) return MEGAMOE_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  if (T == 0) return cuda_status(cudaMemsetAsync(ws, 0, 256, s));
  const ForwardWs wk = carve_forward(ws, T, k, w->num_experts, w->hidden, w->intermediate, pad);
  return run_mx_forward(w, x, topk_ids, topk_weights, T, k, pad, out, wk, s);
}

megamoe_status megamoe_forward_mxfp4_from_logits(
    const megamoe_mx_weights* w, const uint16_t* x, const void* logits, int logits_type,
    int64_t ld_logits, const float* bias, int score, int n_group, int topk_group, int group_top,
    int renormalize, double scale, int T, int k, int pad, uint16_t* out, void* ws, size_t ws_bytes,
    megamoe_stream_t stream) {
  megamoe_status st = check_mx_forward(w, x, T, k, pad, out, ws, ws_bytes);
  if (st == MEGAMOE_OK) st = check_router(logits, logits_type, T, w->num_experts, ld_logits, score, k);
  if (st == MEGAMOE_OK) st = check_groups(w->num_experts, n_group, topk_group, group_top, bias);
  if (st != MEGAMOE_OK) return st;
  cudaStream_t s = as_stream(stream);
  if (T == 0) return cuda_status(cudaMemsetAsync(ws, 0, 256, s));
  const ForwardWs wk = carve_forward(ws, T, k, w->num_experts, w->hidden, w->intermediate, pad);
  const ScoredRouter r{logits, logits_type == MEGAMOE_TYPE_BF16, T, ld_logits, w->num_experts, bias,
                       score == MEGAMOE_SCORE_SOFTMAX, n_group, topk_group, group_top, k,
                       renormalize != 0, static_cast<float>(scale), wk.r_ids, wk.r_w};
  if (launch_scored_router(r, s) != cudaSuccess) return MEGAMOE_ERR_CUDA;
  return run_mx_forward(w, x, wk.r_ids, wk.r_w, T, k, pad, out, wk, s);
}

}  // extern "C"
