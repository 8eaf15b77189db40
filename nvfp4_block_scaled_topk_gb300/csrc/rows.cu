// Around the 16-bit grouped products: the gated activation between an expert's
// two products and the movement of rows between token and expert order, each
// with its gradient.  Sums are fp32 in ascending slot order, one rounding at the end.
//
// All are bound by their bytes, or with few rows by the launch (1.5 us for the
// activation of 48 rows, 2.1 for the sums of eight tokens, in a stream of calls).  At
// the copy rate / measured, us: gradient of the activation, 49152 x 2048, 148.6 / 151.5;
// 2003 tokens of 7168 into 11777 rows 29.2 / 33.2; their sums 29.7 / 38.5; gradient of
// the sums of 8192 tokens 221 / 230.  8192 tokens (117 MB) into 49152 rows take 181 us
// where 121 are needed: the experts' rows come to each token six times, and it has left
// L2 in between.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace megamoe {

namespace {

template <typename X>
__device__ __forceinline__ float2 widen(uint32_t v);
template <>
__device__ __forceinline__ float2 widen<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 widen<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <typename X>
__device__ __forceinline__ uint32_t narrow(float a, float b);
template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t narrow<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// exp(-|g|) of a 16-bit number: its product with the leading bits of log2 e (15 of them
// with 8 of bf16, 13 with 11 of fp16) is exact, and what those leave out of log2 e follows
// as the factor exp(d), 1 + d and, where d is larger, d^2 / 2 (a split constant after Cody
// and Waite; multiplied by log2 e in one, the rounding of the product alone puts the
// result off by |g| 2^-24).
template <typename X>
__device__ __forceinline__ float exp_minus(float g);
__device__ __forceinline__ float ex2(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}
template <>
__device__ __forceinline__ float exp_minus<__nv_bfloat16>(float g) {
  const float a = fabsf(g), e = ex2(a * -0x1.7154p+0f);
  return fmaf(e, a * -4.888495e-6f, e);
}
template <>
__device__ __forceinline__ float exp_minus<__half>(float g) {
  const float a = fminf(fabsf(g), 128.f), e = ex2(a * -0x1.715p+0f), d = a * -4.7194842e-5f;
  return fmaf(e, fmaf(0.5f * d, d, d), e);
}

// The largest magnitude of eight bf16 elements.
__device__ __forceinline__ float largest(const uint32_t (&v)[4]) {
  auto magnitudes = [](uint32_t w) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
  const __nv_bfloat162 m = __hmax2(__hmax2(magnitudes(v[0]), magnitudes(v[1])),
                                   __hmax2(magnitudes(v[2]), magnitudes(v[3])));
  return fmaxf(__low2float(m), __high2float(m));
}

// SiLU(g) u = g s u with s = 1 / (1 + exp(-g)); its gradient is grad u s (1 + g (1 - s))
// by g and grad g s by u.  The exponential is taken of -|g|, so that neither s nor 1 - s
// overflows or cancels; it and the products are off by a few units of fp32, the
// hardware's reciprocal of a number in [1, 2] by one.
//
// Near: the gates' magnitudes are below 80 (past 87 the exponential is no normal number),
// those of the other factors, of which two are multiplied, below 2^60.  fp16 values are
// always near enough: gates further down give less than the type's smallest number.
// (Two forms because the far one for all takes 161 us for the gradient of 49152 x 2048,
// 151.5 so.)
template <typename X>
__device__ __forceinline__ void sigmoid(float g, float* s, float* rest) {
  const float e = exp_minus<X>(g);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  const float er = e * r;
  *s = g >= 0.f ? r : er;
  *rest = g >= 0.f ? er : r;
}
template <typename X>
__device__ __forceinline__ float silu_near(float g, float u) {
  float s, rest;
  sigmoid<X>(g, &s, &rest);
  return g * s * u;
}
template <typename X>
__device__ __forceinline__ void silu_grad_near(float g, float u, float grad, float* dg, float* du) {
  float s, rest;
  sigmoid<X>(g, &s, &rest);
  *dg = grad * u * (s * fmaf(g, rest, 1.f));
  *du = grad * (g * s);
}

// Far: s in the factors p p r: with h = exp(-|g| / 2), which fp32 holds down to |g| = 174,
// and r = 1 / (1 + h h), p is 1 or (g below 0) h.  The products are ordered so that no
// step leaves fp32's range where the result does not.
struct FarGate {
  float p, r, rest;
  __device__ explicit FarGate(float g) {
    const float h = expf(-0.5f * fabsf(g)), e = h * h;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    p = g >= 0.f ? 1.f : h;
    rest = g >= 0.f ? e * r : r;
  }
};
__device__ __forceinline__ float silu_far(float g, float u) {
  const FarGate s(g);
  return g * s.p * s.r * (u * s.p);
}
// The larger of grad and u meets the gate's factor first (halved: it can be 1.1; the
// smaller one is doubled), all of it where the smaller one is 1 at most, else each of the
// two takes a p.
__device__ __forceinline__ void silu_grad_far(float g, float u, float grad, float* dg, float* du) {
  const FarGate s(g);
  const bool first = fabsf(grad) > fabsf(u);
  const float big = first ? grad : u, small = first ? u : grad;
  const bool all = fabsf(small) <= 1.f;
  *dg = big * s.p * (s.r * fmaf(0.5f * g, s.rest, 0.5f)) * (all ? s.p : 1.f) *
        (small * (all ? 2.f : 2.f * s.p));
  *du = g * s.p * s.r * (grad * s.p);
}

// Eight elements of each.
template <typename X, bool BACKWARD, bool FAR>
__device__ __forceinline__ void silu_eight(const uint32_t (&g)[4], const uint32_t (&u)[4],
                                           const uint32_t (&h)[4], uint32_t (&o)[4], uint32_t (&q)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 gv = widen<X>(g[j]), uv = widen<X>(u[j]);
    if (!BACKWARD) {
      o[j] = FAR ? narrow<X>(silu_far(gv.x, uv.x), silu_far(gv.y, uv.y))
                 : narrow<X>(silu_near<X>(gv.x, uv.x), silu_near<X>(gv.y, uv.y));
      continue;
    }
    const float2 hv = widen<X>(h[j]);
    float2 dg, du;
    if (FAR) {
      silu_grad_far(gv.x, uv.x, hv.x, &dg.x, &du.x);
      silu_grad_far(gv.y, uv.y, hv.y, &dg.y, &du.y);
    } else {
      silu_grad_near<X>(gv.x, uv.x, hv.x, &dg.x, &du.x);
      silu_grad_near<X>(gv.y, uv.y, hv.y, &dg.y, &du.y);
    }
    o[j] = narrow<X>(dg.x, dg.y);
    q[j] = narrow<X>(du.x, du.y);
  }
}

// 16 bytes (eight elements) a thread and step; vectors of all rows in one line, so
// that short rows leave no lane idle.  Blocks an SM: 49152 x 2048 bf16 take 91.4 us with
// eight and 95 with six (and more registers) forward, the gradient 155.7 and 151.5.
template <typename X, bool BACKWARD>
__global__ void __launch_bounds__(256, BACKWARD ? 6 : 8) k_silu(const Silu p) {
  pdl_wait();
  pdl_trigger();
  const uint32_t vecs = static_cast<uint32_t>(p.I) / 8;
  int64_t rows = p.rows;
  if (p.live_rows) rows = min(rows, static_cast<int64_t>(max(__ldg(p.live_rows), 0)));
  const int64_t total = rows * vecs;
  const X* a = static_cast<const X*>(p.a);
  for (int64_t i = blockIdx.x * int64_t{256} + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = (i >> 32) == 0 ? static_cast<uint32_t>(i) / vecs : i / vecs;
    const int col = static_cast<int>(i - row * vecs) * 8;
    const X* at = a + row * p.ld_a + col;
    const uint4 g4 = __ldcs(reinterpret_cast<const uint4*>(at));
    const uint4 u4 = __ldcs(reinterpret_cast<const uint4*>(at + p.I));
    uint4 h4 = make_uint4(0, 0, 0, 0);
    if (BACKWARD)
      h4 = __ldcs(reinterpret_cast<const uint4*>(static_cast<const X*>(p.grad) + row * p.ld_grad + col));
    const uint32_t g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
    const uint32_t h[4] = {h4.x, h4.y, h4.z, h4.w};
    uint32_t o[4], q[4];
    bool near = true;
    if constexpr (!std::is_same_v<X, __half>) {
      near = largest(g) < 80.f;
      if (BACKWARD) near = near && largest(u) < 0x1p60f && largest(h) < 0x1p60f;
    }
    if (near) silu_eight<X, BACKWARD, false>(g, u, h, o, q);
    else silu_eight<X, BACKWARD, true>(g, u, h, o, q);
    X* to = static_cast<X*>(p.out) + row * p.ld_out + col;
    *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
    if (BACKWARD) *reinterpret_cast<uint4*>(to + p.I) = make_uint4(q[0], q[1], q[2], q[3]);
  }
}

// A warp copies 2 KB of a row at a time, four loads in flight; streaming stores, which
// leave the tokens in L2 for the next expert that wants them (36.1 us without, 33.6).
__global__ void __launch_bounds__(256) k_gather_rows(const uint16_t* __restrict__ x, int64_t T,
                                                     int vecs, int64_t ld_x,
                                                     const int32_t* __restrict__ row_src,
                                                     int64_t rows, int k, uint16_t* out,
                                                     int64_t ld_out) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int chunks = (vecs + 127) / 128;
  const int64_t total = rows * chunks;
  for (int64_t i = blockIdx.x * int64_t{8} + (threadIdx.x >> 5); i < total;
       i += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t row = i / chunks;
    const int v0 = static_cast<int>(i - row * chunks) * 128 + lane;
    const int src = __ldg(row_src + row);
    const int64_t t = src >= 0 ? src / k : -1;
    const bool some = t >= 0 && t < T;
    const uint4* from = reinterpret_cast<const uint4*>(x + (some ? t : 0) * ld_x);
    uint4* to = reinterpret_cast<uint4*>(out + row * ld_out);
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = some && v0 + 32 * j < vecs ? __ldg(from + v0 + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v0 + 32 * j < vecs) __stcs(to + v0 + 32 * j, v[j]);
  }
}

// A warp sums `run` chunks of 256 elements of a token, one after another with the
// token's rows and weights in registers; eight slots' loads in flight at a time.
template <typename X, bool MANY>  // MANY: more than eight slots
__global__ void __launch_bounds__(256, 4) k_combine_rows(const CombineRows p, int run) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, vecs = p.d / 8;
  const int chunks = (vecs + 31) / 32, runs = (chunks + run - 1) / run;
  const int64_t total = p.T * runs;
  const uint4* y = static_cast<const uint4*>(p.y);
  const int64_t ld = p.ld_y / 8;
  for (int64_t i = blockIdx.x * int64_t{8} + (threadIdx.x >> 5); i < total;
       i += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t t = i / runs;
    const int c0 = static_cast<int>(i - t * runs) * run;
    int r[8];
    float w[8];
    auto slots = [&](int j0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = j0 + j < p.k ? __ldg(p.slot_dst + t * p.k + j0 + j) : -1;
        w[j] = p.weights && j0 + j < p.k ? __ldg(p.weights + t * p.k + j0 + j) : 1.f;
        if (r[j] >= p.rows) r[j] = -1;
      }
    };
    slots(0);
    for (int c = c0; c < min(c0 + run, chunks); ++c) {
      const int v = c * 32 + lane;
      if (v >= vecs) break;
      float2 acc[4] = {};
      for (int j0 = 0;; j0 += 8) {
        uint4 q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r[j] >= 0) q[j] = __ldcs(y + r[j] * ld + v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (r[j] < 0) continue;
          const uint32_t u[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = widen<X>(u[e]);
            acc[e].x = fmaf(w[j], f.x, acc[e].x);
            acc[e].y = fmaf(w[j], f.y, acc[e].y);
          }
        }
        if (!MANY || j0 + 8 >= p.k) break;
        slots(j0 + 8);
      }
      if (MANY) slots(0);
      reinterpret_cast<uint4*>(static_cast<X*>(p.out) + t * p.ld_out)[v] =
          make_uint4(narrow<X>(acc[0].x, acc[0].y), narrow<X>(acc[1].x, acc[1].y),
                     narrow<X>(acc[2].x, acc[2].y), narrow<X>(acc[3].x, acc[3].y));
    }
  }
}

// A block takes a token: its gradient is read once, each slot's row of y gives a
// share of that slot's weight's gradient and its place takes w grad.  The shares
// are summed lane by lane, then over the warps in order.  Four blocks an SM keep
// enough loads in flight (8192 tokens of six slots, 7168: 260 us with two, 236);
// streaming stores took 345.
template <typename X, int K>
__global__ void __launch_bounds__(256, K <= 8 ? 4 : 2) k_combine_rows_grad(const CombineRows p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_part[K][8];
  const int vecs = p.d / 8, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    int r[K];
    float w[K], dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      r[j] = j < p.k ? __ldg(p.slot_dst + t * p.k + j) : -1;
      w[j] = j < p.k && p.weights ? __ldg(p.weights + t * p.k + j) : 1.f;
      if (r[j] >= p.rows) r[j] = -1;
      dot[j] = 0.f;
    }
    const uint4* grad = reinterpret_cast<const uint4*>(static_cast<const X*>(p.grad) + t * p.ld_grad);
    for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
      const uint4 g4 = __ldcs(grad + v);
      uint4 q[K];
      if (p.grad_weights) {
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (r[j] >= 0)
            q[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const X*>(p.y) + r[j] * p.ld_y) + v);
      }
      const uint32_t g[4] = {g4.x, g4.y, g4.z, g4.w};
      float2 f[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) f[c] = widen<X>(g[c]);
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (r[j] < 0) continue;
        if (p.grad_weights) {
          const uint32_t u[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 z = widen<X>(u[c]);
            dot[j] = fmaf(f[c].x, z.x, fmaf(f[c].y, z.y, dot[j]));
          }
        }
        reinterpret_cast<uint4*>(static_cast<X*>(p.out) + r[j] * p.ld_out)[v] =
            make_uint4(narrow<X>(w[j] * f[0].x, w[j] * f[0].y), narrow<X>(w[j] * f[1].x, w[j] * f[1].y),
                       narrow<X>(w[j] * f[2].x, w[j] * f[2].y), narrow<X>(w[j] * f[3].x, w[j] * f[3].y));
      }
    }
    if (!p.grad_weights) continue;
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (lane == 0) s_part[j][warp] = dot[j];
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < p.k) {
      float sum = 0.f;
      for (int i = 0; i < warps; ++i) sum += s_part[threadIdx.x][i];
      p.grad_weights[t * p.k + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

// Up to `per_sm` blocks an SM, grid-stride beyond that.
unsigned blocks_for(int64_t tasks, int per_block, int per_sm) {
  return static_cast<unsigned>(std::min((tasks + per_block - 1) / per_block,
                                        static_cast<int64_t>(num_sms()) * per_sm));
}

template <bool BACKWARD>
cudaError_t silu_any(const Silu& a, cudaStream_t stream) {
  const int64_t total = a.rows * (a.I / 8);
  if (total == 0) return cudaSuccess;
  auto kern = a.type == MEGAMOE_TYPE_F16 ? k_silu<__half, BACKWARD> : k_silu<__nv_bfloat16, BACKWARD>;
  return launch_pdl(kern, dim3(blocks_for(total, 256, 32)), dim3(256), 0, stream, a);
}

}  // namespace

cudaError_t launch_silu(const Silu& a, cudaStream_t stream) { return silu_any<false>(a, stream); }
cudaError_t launch_silu_backward(const Silu& a, cudaStream_t stream) {
  return silu_any<true>(a, stream);
}

cudaError_t launch_gather_rows(const void* x, int64_t T, int d, int64_t ld_x,
                               const int32_t* row_src, int64_t rows, int k, void* out,
                               int64_t ld_out, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  const int vecs = d / 8;
  return launch_pdl(k_gather_rows, dim3(blocks_for(rows * ((vecs + 127) / 128), 8, 32)), dim3(256),
                    0, stream, static_cast<const uint16_t*>(x), T, vecs, ld_x, row_src, rows, k,
                    static_cast<uint16_t*>(out), ld_out);
}

cudaError_t launch_combine_rows(const CombineRows& c, cudaStream_t stream) {
  if (c.T == 0) return cudaSuccess;
  const bool many = c.k > 8;
  auto kern = c.type == MEGAMOE_TYPE_F16
                  ? (many ? k_combine_rows<__half, true> : k_combine_rows<__half, false>)
                  : (many ? k_combine_rows<__nv_bfloat16, true> : k_combine_rows<__nv_bfloat16, false>);
  // Up to four chunks of a token by one warp as long as every SM keeps its warps:
  // 8192 tokens of six slots and 7168 elements took 172, 144, 139, 143 and 154 us with
  // 1, 2, 4, 8 and 28.
  const int64_t chunks = (c.d / 8 + 31) / 32;
  const int run = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(4, c.T * chunks / (num_sms() * int64_t{32}))));
  const int64_t tasks = c.T * ((chunks + run - 1) / run);
  return launch_pdl(kern, dim3(blocks_for(tasks, 8, 32)), dim3(256), 0, stream, c, run);
}

template <typename X>
static cudaError_t combine_grad(const CombineRows& c, dim3 grid, dim3 block, cudaStream_t stream) {
  auto kern = c.k <= 4   ? k_combine_rows_grad<X, 4>
              : c.k <= 8 ? k_combine_rows_grad<X, 8>
                         : k_combine_rows_grad<X, 16>;
  return launch_pdl(kern, grid, block, 0, stream, c);
}

cudaError_t launch_combine_rows_backward(const CombineRows& c, cudaStream_t stream) {
  if (c.T == 0) return cudaSuccess;
  const int vecs = c.d / 8, steps = (vecs + 255) / 256;  // threads that divide the row evenly
  const dim3 block(static_cast<unsigned>(((vecs + steps - 1) / steps + 31) / 32 * 32));
  const dim3 grid(blocks_for(c.T, 1, 16));
  return c.type == MEGAMOE_TYPE_F16 ? combine_grad<__half>(c, grid, block, stream)
                                    : combine_grad<__nv_bfloat16>(c, grid, block, stream);
}

}  // namespace megamoe
