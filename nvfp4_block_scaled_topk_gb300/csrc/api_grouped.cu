// C ABI of the 16-bit experts' operators and the 8-bit integer linear: argument
// checks, workspace layouts and the order of the launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <array>

#include "../../include/megamoe.h"
#include "kernels.h"

using namespace megamoe;

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline megamoe_status cuda_status(cudaError_t e) {
  return e == cudaSuccess ? MEGAMOE_OK : MEGAMOE_ERR_CUDA;
}
inline cudaStream_t as_stream(megamoe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline bool half_type(int type) { return type == MEGAMOE_TYPE_BF16 || type == MEGAMOE_TYPE_F16; }
inline int64_t type_bytes(int type) {
  return type == MEGAMOE_TYPE_F32 ? 4 : half_type(type) ? 2 : type == MEGAMOE_TYPE_I8 ? 1 : 0;
}
// Base and rows on 16 bytes; row strides that a tensor map takes (below 2^40 bytes).
inline bool rows_ok(const void* p, int64_t ld, int64_t bytes) {
  return aligned(p, 16) && ld * bytes % 16 == 0 && ld < (int64_t{1} << 36);
}

// Rows of a matrix in memory, in bytes.
struct Place {
  uintptr_t at;
  int64_t rows, pitch, width;
  Place(const void* p, int64_t n, int64_t ld, int64_t cols, int64_t bytes)
      : at(reinterpret_cast<uintptr_t>(p)), rows(p ? n : 0), pitch(ld * bytes), width(cols * bytes) {}
  Place(const void* p, int64_t n, int64_t bytes) : Place(p, 1, n, n, bytes) { rows = p && n > 0; }
  bool same(const Place& o) const {
    return at == o.at && width == o.width && rows == o.rows && (rows == 1 || pitch == o.pitch);
  }
};
// Whether they have a byte in common.  Rows of one pitch may lie between each other;
// of two pitches they count as meeting where their spans do.
bool meet(Place a, Place b) {
  if (a.rows == 0 || b.rows == 0) return false;
  auto span = [](const Place& m) {
    return static_cast<unsigned __int128>(m.rows - 1) * m.pitch + m.width;
  };
  if (a.at + span(a) <= b.at || b.at + span(b) <= a.at) return false;
  if (a.rows == 1 && a.width <= b.pitch) a.pitch = b.pitch;
  if (b.rows == 1 && b.width <= a.pitch) b.pitch = a.pitch;
  if (a.pitch != b.pitch) return true;
  const int64_t off = b.at >= a.at ? static_cast<int64_t>((b.at - a.at) % a.pitch)
                                   : a.pitch - 1 - static_cast<int64_t>((a.at - b.at - 1) % a.pitch);
  return off < a.width || off + b.width > a.pitch;
}
// Read and written at the same place by the same thread, or nowhere in common.
bool meet_elsewhere(const Place& a, const Place& b) { return !a.same(b) && meet(a, b); }

constexpr int64_t kMaxRows = int64_t{1} << 31;
constexpr int kMaxWidth = 1 << 30;

// Sizes of the grouped products.  Tiles are counted in 31 bits, for offsets of any
// values (every expert with all of the rows).
megamoe_status check_grouped(int type, int64_t rows, int E, int N, int K, const int32_t* offsets,
                             const int32_t* padded_offsets, const uint32_t* status) {
  if (!half_type(type) || rows < 0 || E < 1 || N < 1 || K < 1 || !offsets)
    return MEGAMOE_ERR_INVALID_ARG;
  if (E > MEGAMOE_MAX_EXPERTS || rows >= kMaxWidth || N % 8 != 0 || K % 8 != 0 || N >= kMaxWidth ||
      K >= kMaxWidth)
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const int64_t most = int64_t{1} << 30, mt = (N + 255) / 256, kt = (K + 255) / 256;
  const int64_t per = (rows + 255) / 256 * E;
  if (per > most / std::max(mt, kt) || mt * kt > most / E) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  // the stride between experts' weights is below 2^40 bytes
  if (static_cast<int64_t>(N) * K >= (int64_t{1} << 39)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(offsets, 4) || !aligned(padded_offsets, 4) || !aligned(status, 4))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  return MEGAMOE_OK;
}

megamoe_status check_silu(const void* a, int type, int64_t rows, int I, int64_t ld_a,
                          const int32_t* live_rows) {
  if (!half_type(type) || rows < 0 || I < 1 || ld_a < 2 * static_cast<int64_t>(I))
    return MEGAMOE_ERR_INVALID_ARG;
  if (rows > 0 && !a) return MEGAMOE_ERR_INVALID_ARG;
  if (rows >= kMaxRows || I % 8 != 0 || I >= kMaxWidth || !rows_ok(a, ld_a, 2) ||
      !aligned(live_rows, 4))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  return MEGAMOE_OK;
}

// The gates' columns and the others'.
std::array<Place, 2> halves(const void* a, int64_t rows, int64_t ld, int I) {
  return {Place(a, rows, ld, I, 2),
          Place(a ? static_cast<const uint16_t*>(a) + I : nullptr, rows, ld, I, 2)};
}

megamoe_status check_rows(int type, int64_t rows, int64_t T, int k, int d) {
  if (!half_type(type) || rows < 0 || T < 0 || d < 1 || k < 1) return MEGAMOE_ERR_INVALID_ARG;
  if (rows >= kMaxRows || T >= kMaxRows || T * k > kMaxRows || d % 8 != 0 || d >= kMaxWidth ||
      k > MEGAMOE_MAX_TOPK)
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  return MEGAMOE_OK;
}

// Workspace of the integer linear: status, the tokens' scales (the product reads
// them in whole vectors past the last) and their integers, as fp16 or (few tokens)
// as they are.
struct Int8Ws {
  uint32_t* status;
  float* scales;
  void* integers;
  float* partial;  // of tiles whose sums are shared
  size_t bytes;
};
Int8Ws carve_int8(void* base, int64_t T, int K, int N) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  uint8_t* p = static_cast<uint8_t*>(base);
  const size_t scales = up(4 * static_cast<size_t>(T) + 256);
  const bool few = int8_few_fits(T, K);
  Int8Ws w{};
  w.status = reinterpret_cast<uint32_t*>(p);
  w.bytes = 256;
  if (int8_dots_fit(T, K)) return w;  // quantised inside the product
  w.scales = reinterpret_cast<float*>(p + w.bytes);
  w.bytes += scales;
  w.integers = p + w.bytes;
  w.bytes += up((few ? 1 : 2) * static_cast<size_t>(T) * K);
  if (few) return w;
  // (for either type of result)
  const int split = std::max(int8_plan(T, N, K, false).split,
                             int8_folds(K) ? int8_plan(T, N, K, true).split : 1);
  if (split == 1) return w;
  w.partial = reinterpret_cast<float*>(p + w.bytes);
  w.bytes += up(4 * static_cast<size_t>(split) * T * N);
  return w;
}

bool int8_sizes_ok(int64_t T, int K, int N) {
  if (K % 16 != 0 || N % 8 != 0 || T >= (int64_t{1} << 30) || K >= kMaxWidth || N >= kMaxWidth)
    return false;
  return (T / 16 + 1) * (N / 256 + 1) < (int64_t{1} << 31);
}

}  // namespace

extern "C" {

megamoe_status megamoe_grouped_linear(const void* x, int type, int64_t rows, int64_t ld_x,
                                      const void* w, int E, int N, int K, const int32_t* offsets,
                                      const int32_t* padded_offsets, int out_type, void* out,
                                      int64_t ld_out, uint32_t* status, megamoe_stream_t stream) {
  const megamoe_status st = check_grouped(type, rows, E, N, K, offsets, padded_offsets, status);
  if (st != MEGAMOE_OK) return st;
  if (ld_x < K || ld_out < N || !w || (out_type != type && out_type != MEGAMOE_TYPE_F32))
    return MEGAMOE_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !out)) return MEGAMOE_ERR_INVALID_ARG;
  if (!rows_ok(x, ld_x, 2) || !rows_ok(out, ld_out, type_bytes(out_type)) || !aligned(w, 16))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const Place to(out, rows, ld_out, N, type_bytes(out_type));
  if (meet(to, Place(x, rows, ld_x, K, 2)) || meet(to, Place(w, static_cast<int64_t>(E) * N * K, 2)))
    return MEGAMOE_ERR_INVALID_ARG;
  const Grouped g{x, nullptr, w, type, rows, ld_x, 0, E, N, K, offsets, padded_offsets, status};
  return cuda_status(launch_grouped_forward(g, out, out_type, ld_out, as_stream(stream)));
}

megamoe_status megamoe_grouped_linear_backward(
    const void* grad_out, int64_t ld_grad, const void* x, int64_t ld_x, const void* w, int type,
    int64_t rows, int E, int N, int K, const int32_t* offsets, const int32_t* padded_offsets,
    void* grad_x, int64_t ld_grad_x, int grad_w_type, void* grad_w, uint32_t* status,
    megamoe_stream_t stream) {
  const megamoe_status st = check_grouped(type, rows, E, N, K, offsets, padded_offsets, status);
  if (st != MEGAMOE_OK) return st;
  if (ld_grad < N || (rows > 0 && !grad_out)) return MEGAMOE_ERR_INVALID_ARG;
  if (!rows_ok(grad_out, ld_grad, 2)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (grad_x) {
    if (!w || ld_grad_x < K) return MEGAMOE_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !rows_ok(grad_x, ld_grad_x, 2)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (grad_w) {
    if ((rows > 0 && !x) || ld_x < K || (grad_w_type != type && grad_w_type != MEGAMOE_TYPE_F32))
      return MEGAMOE_ERR_INVALID_ARG;
    if (!rows_ok(x, ld_x, 2) || !aligned(grad_w, 16)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  }
  // grad_w is under way before grad_x is done: neither may lie where the other reads
  const int64_t values = static_cast<int64_t>(E) * N * K;
  const Place from(grad_out, rows, ld_grad, N, 2), weights(grad_x ? w : nullptr, values, 2);
  const Place tokens(grad_w ? x : nullptr, rows, ld_x, K, 2), to_x(grad_x, rows, ld_grad_x, K, 2);
  const Place to_w(grad_w, values, type_bytes(grad_w_type));
  if (meet(to_x, from) || meet(to_x, weights) || meet(to_x, tokens) || meet(to_x, to_w) ||
      meet(to_w, from) || meet(to_w, weights) || meet(to_w, tokens))
    return MEGAMOE_ERR_INVALID_ARG;
  const Grouped g{x, grad_out, w, type, rows, ld_x, ld_grad, E, N, K, offsets, padded_offsets, status};
  cudaError_t e = cudaSuccess;
  if (grad_x) e = launch_grouped_grad_x(g, grad_x, ld_grad_x, as_stream(stream));
  if (e == cudaSuccess && grad_w)
    e = launch_grouped_grad_w(g, grad_w, grad_w_type, grad_x != nullptr, as_stream(stream));
  return cuda_status(e);
}

megamoe_status megamoe_silu_mul(const void* a, int type, int64_t rows, int I, int64_t ld_a,
                                const int32_t* live_rows, void* out, int64_t ld_out,
                                megamoe_stream_t stream) {
  const megamoe_status st = check_silu(a, type, rows, I, ld_a, live_rows);
  if (st != MEGAMOE_OK) return st;
  if (ld_out < I || (rows > 0 && !out)) return MEGAMOE_ERR_INVALID_ARG;
  if (!rows_ok(out, ld_out, 2)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const Place to(out, rows, ld_out, I, 2);
  for (const Place& from : halves(a, rows, ld_a, I))
    if (meet_elsewhere(to, from)) return MEGAMOE_ERR_INVALID_ARG;
  return cuda_status(launch_silu(Silu{a, nullptr, type, rows, ld_a, 0, ld_out, I, live_rows, out},
                                 as_stream(stream)));
}

megamoe_status megamoe_silu_mul_backward(const void* grad, int64_t ld_grad, const void* a, int type,
                                         int64_t rows, int I, int64_t ld_a,
                                         const int32_t* live_rows, void* grad_a, int64_t ld_grad_a,
                                         megamoe_stream_t stream) {
  const megamoe_status st = check_silu(a, type, rows, I, ld_a, live_rows);
  if (st != MEGAMOE_OK) return st;
  if (ld_grad < I || ld_grad_a < 2 * static_cast<int64_t>(I)) return MEGAMOE_ERR_INVALID_ARG;
  if (rows > 0 && (!grad || !grad_a)) return MEGAMOE_ERR_INVALID_ARG;
  if (!rows_ok(grad, ld_grad, 2) || !rows_ok(grad_a, ld_grad_a, 2))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const Place from_grad(grad, rows, ld_grad, I, 2);
  const auto from = halves(a, rows, ld_a, I), to = halves(grad_a, rows, ld_grad_a, I);
  for (const Place& t : to)
    if (meet_elsewhere(t, from[0]) || meet_elsewhere(t, from[1]) || meet_elsewhere(t, from_grad))
      return MEGAMOE_ERR_INVALID_ARG;
  return cuda_status(launch_silu_backward(
      Silu{a, grad, type, rows, ld_a, ld_grad, ld_grad_a, I, live_rows, grad_a}, as_stream(stream)));
}

megamoe_status megamoe_gather_rows(const void* x, int type, int64_t T, int d, int64_t ld_x,
                                   const int32_t* row_src, int64_t rows, int k, void* out,
                                   int64_t ld_out, megamoe_stream_t stream) {
  const megamoe_status st = check_rows(type, rows, T, k, d);
  if (st != MEGAMOE_OK) return st;
  if (ld_x < d || ld_out < d || (T > 0 && !x) || (rows > 0 && (!row_src || !out)))
    return MEGAMOE_ERR_INVALID_ARG;
  if (!rows_ok(x, ld_x, 2) || !rows_ok(out, ld_out, 2) || !aligned(row_src, 4))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const Place to(out, rows, ld_out, d, 2);
  if (meet(to, Place(x, T, ld_x, d, 2)) || meet(to, Place(row_src, rows, 4)))
    return MEGAMOE_ERR_INVALID_ARG;
  return cuda_status(launch_gather_rows(x, T, d, ld_x, row_src, rows, k, out, ld_out, as_stream(stream)));
}

megamoe_status megamoe_combine_rows(const void* y, int type, int64_t rows, int64_t ld_y,
                                    const int32_t* slot_dst, const float* topk_weights, int64_t T,
                                    int k, int d, void* out, int64_t ld_out,
                                    megamoe_stream_t stream) {
  const megamoe_status st = check_rows(type, rows, T, k, d);
  if (st != MEGAMOE_OK) return st;
  if (ld_y < d || ld_out < d || (rows > 0 && !y) || (T > 0 && (!slot_dst || !out)))
    return MEGAMOE_ERR_INVALID_ARG;
  if (!rows_ok(y, ld_y, 2) || !rows_ok(out, ld_out, 2) || !aligned(slot_dst, 4) ||
      !aligned(topk_weights, 4))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const Place to(out, T, ld_out, d, 2);
  if (meet(to, Place(y, rows, ld_y, d, 2)) || meet(to, Place(slot_dst, T * k, 4)) ||
      meet(to, Place(topk_weights, T * k, 4)))
    return MEGAMOE_ERR_INVALID_ARG;
  const CombineRows c{y, type, rows, ld_y, slot_dst, topk_weights, T, k, d,
                      nullptr, 0, out, ld_out, nullptr};
  return cuda_status(launch_combine_rows(c, as_stream(stream)));
}

megamoe_status megamoe_combine_rows_backward(const void* grad_out, int64_t ld_grad, const void* y,
                                             int type, int64_t rows, int64_t ld_y,
                                             const int32_t* slot_dst, const float* topk_weights,
                                             int64_t T, int k, int d, void* grad_y,
                                             int64_t ld_grad_y, float* grad_topk_weights,
                                             megamoe_stream_t stream) {
  const megamoe_status st = check_rows(type, rows, T, k, d);
  if (st != MEGAMOE_OK) return st;
  if (ld_grad < d || ld_grad_y < d || (T > 0 && (!grad_out || !slot_dst)) || (rows > 0 && !grad_y))
    return MEGAMOE_ERR_INVALID_ARG;
  if (!rows_ok(grad_out, ld_grad, 2) || !rows_ok(grad_y, ld_grad_y, 2) || !aligned(slot_dst, 4) ||
      !aligned(topk_weights, 4) || !aligned(grad_topk_weights, 4))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  if (grad_topk_weights) {
    if (ld_y < d || (rows > 0 && !y)) return MEGAMOE_ERR_INVALID_ARG;
    if (!rows_ok(y, ld_y, 2)) return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  }
  const Place from(grad_out, T, ld_grad, d, 2), to_y(grad_y, rows, ld_grad_y, d, 2);
  const Place slots(slot_dst, T * k, 4), weights(topk_weights, T * k, 4);
  const Place to_w(grad_topk_weights, T * k, 4), expert(grad_topk_weights ? y : nullptr, rows, ld_y, d, 2);
  if (meet(to_y, from) || meet(to_y, slots) || meet(to_y, weights) || meet(to_y, to_w) ||
      meet_elsewhere(to_y, expert) || meet(to_w, from) || meet(to_w, slots) || meet(to_w, expert) ||
      meet_elsewhere(to_w, weights))
    return MEGAMOE_ERR_INVALID_ARG;
  const CombineRows c{y, type, rows, ld_y, slot_dst, topk_weights, T, k, d,
                      grad_out, ld_grad, grad_y, ld_grad_y, grad_topk_weights};
  return cuda_status(launch_combine_rows_backward(c, as_stream(stream)));
}

megamoe_status megamoe_quantize_int8(const void* x, int x_type, int64_t rows, int K, int64_t ld,
                                     int8_t* codes, float* scales, uint32_t* status,
                                     megamoe_stream_t stream) {
  if (rows < 0 || K < 1 || ld < K || x_type == MEGAMOE_TYPE_I8 || !type_bytes(x_type))
    return MEGAMOE_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !codes || !scales)) return MEGAMOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || K >= kMaxWidth || rows >= kMaxRows || !rows_ok(x, ld, type_bytes(x_type)) ||
      !aligned(codes, 16) || !aligned(scales, 4) || !aligned(status, 4))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const Place from(x, rows, ld, K, type_bytes(x_type)), to(codes, rows, K, K, 1), to_s(scales, rows, 4);
  if (meet(to, from) || meet(to_s, from) || meet(to, to_s)) return MEGAMOE_ERR_INVALID_ARG;
  const Int8Quant q{x, x_type, nullptr, rows, ld, K, codes, nullptr, scales, status, false};
  return cuda_status(launch_int8_quantize(q, as_stream(stream)));
}

size_t megamoe_linear_int8_workspace_size(int64_t T, int K, int N) {
  if (T < 0 || K < 1 || N < 1 || !int8_sizes_ok(T, K, N)) return 0;
  return carve_int8(nullptr, T, K, N).bytes;
}

megamoe_status megamoe_linear_int8(const void* x, int x_type, int64_t T, int K, int64_t ld_x,
                                   const float* x_scales, const int8_t* w_codes,
                                   const float* w_scales, int N, int out_dtype, void* out,
                                   int64_t ld_out, void* ws, size_t ws_bytes,
                                   megamoe_stream_t stream) {
  if (T < 0 || K < 1 || N < 1 || ld_x < K || ld_out < N || !type_bytes(x_type))
    return MEGAMOE_ERR_INVALID_ARG;
  if (out_dtype != MEGAMOE_EPI_BF16 && out_dtype != MEGAMOE_EPI_F32) return MEGAMOE_ERR_INVALID_ARG;
  if (!w_codes || !w_scales || !ws || (T > 0 && (!x || !out))) return MEGAMOE_ERR_INVALID_ARG;
  if ((x_type == MEGAMOE_TYPE_I8) != (x_scales != nullptr) && T > 0) return MEGAMOE_ERR_INVALID_ARG;
  const int64_t out_bytes = out_dtype == MEGAMOE_EPI_F32 ? 4 : 2;
  if (!int8_sizes_ok(T, K, N) || !rows_ok(x, ld_x, type_bytes(x_type)) ||
      !rows_ok(out, ld_out, out_bytes) || !aligned(w_codes, 16) || !aligned(w_scales, 4) ||
      !aligned(x_scales, 4) || !aligned(ws, 256))
    return MEGAMOE_ERR_UNSUPPORTED_SHAPE;
  const Int8Ws wk = carve_int8(ws, T, K, N);
  if (ws_bytes < wk.bytes) return MEGAMOE_ERR_WORKSPACE_TOO_SMALL;
  const Place from[] = {Place(x, T, ld_x, K, type_bytes(x_type)), Place(w_codes, N, K, K, 1),
                        Place(w_scales, N, 4), Place(x_scales, T, 4)};
  const Place to(out, T, ld_out, N, out_bytes), own(ws, static_cast<int64_t>(wk.bytes), 1);
  for (const Place& f : from)
    if (meet(to, f) || meet(own, f)) return MEGAMOE_ERR_INVALID_ARG;
  if (meet(to, own)) return MEGAMOE_ERR_INVALID_ARG;
  const cudaStream_t s = as_stream(stream);
  if (T == 0) return cuda_status(cudaMemsetAsync(wk.status, 0, 4, s));
  const bool few = int8_few_fits(T, K), codes = x_type == MEGAMOE_TYPE_I8;
  Int8Quant q{x, x_type, x_scales, T, ld_x, K, nullptr, nullptr, wk.scales, wk.status, true};
  if (few) q.codes = static_cast<int8_t*>(wk.integers);
  else q.half = static_cast<uint16_t*>(wk.integers);
  const Int8Product g{q.half, wk.scales, T, w_codes, w_scales, N, K, out,
                      out_dtype == MEGAMOE_EPI_F32, ld_out, wk.partial, wk.status};
  if (int8_dots_fit(T, K) || (few && codes)) {  // in one launch
    return cuda_status(few ? launch_int8_few(q, g, s) : launch_int8_dots(q, g, s));
  }
  cudaError_t e = launch_int8_quantize(q, s);
  if (e != cudaSuccess) return MEGAMOE_ERR_CUDA;
  if (few) {
    q.x = q.codes;
    q.type = MEGAMOE_TYPE_I8;
    q.x_scales = wk.scales;
    q.ld = K;
    return cuda_status(launch_int8_few(q, g, s));
  }
  return cuda_status(launch_int8_product(g, s));
}

}  // extern "C"
