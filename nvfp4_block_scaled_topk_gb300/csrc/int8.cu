// Linear in 8-bit integers: y[t, n] = (sum_k q_x[t, k] q_w[n, k]) s_x[t] s_w[n].
//
// A token's scale is amax / 127 (rounded to fp32) and its integers
// rint(127 x / amax), ties to even, decided as in exact arithmetic.
//
// The tensor cores of sm_103a have no integer kind.  An 8-bit integer is exact in
// fp16 and a product of two in fp32, so the integers are multiplied as fp16
// (kind::f16) and a sum of up to 1024 products is exact.  Longer ones are taken in parts
// of 1024 that are added up as 32-bit integers (K below 131072), for few tokens and for
// fp32 results: the same bits whatever the number of tokens.  A bf16 result of more
// tokens has its sum in one part, exact while no partial sum passes 2^24; past that each
// of the K / 16 additions drops what lies below fp32's last bit, up to K / 16 2^-23 of
// the sum in all, where half a step of bf16 is 2^-9 at least.
//
// Weights stay in memory as bytes.  A pair of CTAs has 256 features on the MMA's
// M side: four warps of each read a stage's bytes from shared memory, widen them
// in registers (a byte with its sign bit flipped under 0x64 is the fp16 value 1024
// + 128 + q) and put them into tensor memory, from where the MMA takes its A
// operand; the tokens' integers come as fp16 by tensor map.  Per 128 of K a CTA
// so takes in 16 KB of weights and up to 32 KB of tokens.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace megamoe {

namespace {

// ---------------------------------------------------------------------------
// Quantisation of tokens: a block a row, which it holds between the search for the
// largest magnitude and the rounding (rows past 8192 elements are read again).  8192 x
// 7168 bf16 take 37 us, 117 MB read and 117 written as fp16 (62 % of DRAM, 56 % of the
// issue slots, the barrier between the two in the way of the rest); 51 us with halves
// decided by a comparison, which many rows have hundreds of.
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 256;
constexpr int kHeld = 4;  // eights of elements a thread keeps between the two passes

// Eight elements as they lie, and as fp32.
template <typename X>
struct Eight {
  uint4 q[sizeof(X) / 2];
  __device__ void load(const X* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(X) / 2); ++i)
      q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ void values(float (&v)[8]) const;
};
template <>
__device__ __forceinline__ void Eight<__nv_bfloat16>::values(float (&v)[8]) const {
  const uint32_t u[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void Eight<__half>::values(float (&v)[8]) const {
  const uint32_t u[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void Eight<float>::values(float (&v)[8]) const {
  const uint32_t u[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
}
// The largest magnitude so far, NaN and Inf the largest of all: as bits of fp32, or
// of two 16-bit elements at a time.
template <typename X>
__device__ __forceinline__ void take_largest(const Eight<X>& e, uint32_t* m) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(X) / 2); ++i) {
    const uint32_t u[4] = {e.q[i].x, e.q[i].y, e.q[i].z, e.q[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *m = sizeof(X) == 4 ? max(*m, u[j] & 0x7fffffffu) : __vmaxu2(*m, u[j] & 0x7fff7fffu);
  }
}
template <typename X>
__device__ __forceinline__ uint32_t fp32_bits(uint32_t m);
template <>
__device__ __forceinline__ uint32_t fp32_bits<float>(uint32_t m) { return m; }
template <>
__device__ __forceinline__ uint32_t fp32_bits<__nv_bfloat16>(uint32_t m) {
  return max(m & 0xffffu, m >> 16) << 16;
}
template <>
__device__ __forceinline__ uint32_t fp32_bits<__half>(uint32_t m) {
  const uint32_t h = max(m & 0xffffu, m >> 16);
  return h >= 0x7c00u ? 0x7f800000u
                      : __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
}

// A row's divisor.  Rows of very small or large magnitudes are scaled by a power of
// two first (exact wherever it could change an integer), so that no step below
// leaves fp32's normal range.
struct RowScale {
  float amax;  // of the scaled row
  float inv;   // 1 / amax, fp32 elements: 127 / amax
  float by;         // 1, 2^100 or 2^-20
};
template <typename X>
__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  r.by = amax < 0x1p-90f ? 0x1p100f : amax > 0x1p118f ? 0x1p-20f : 1.f;
  r.amax = amax * r.by;
  r.inv = (sizeof(X) == 2 ? 1.f : 127.f) / r.amax;
  return r;
}

// rint(127 x / amax) of one fp32 element by comparing |127 x| with (k + 1/2) amax, k =
// floor |t|, each as a rounded product and its error: both errors have ten bits at
// most and the products are within a factor of two of each other, so every
// difference is exact.
__device__ __noinline__ float compared(float x, float amax, float t) {
  const float k = floorf(fabsf(t)), h = k + 0.5f, a = fabsf(x);
  const float p = __fmul_rn(127.f, a), q = __fmul_rn(h, amax);
  const float d = __fadd_rn(__fsub_rn(p, q), __fsub_rn(__fmaf_rn(127.f, a, -p), __fmaf_rn(h, amax, -q)));
  const bool odd = (static_cast<int>(k) & 1) != 0;
  return copysignf(d > 0.f || (d == 0.f && odd) ? k + 1.f : k, x);
}

// rint(127 x / amax) of eight as in exact arithmetic, ties to even.
//
// 16-bit elements: p = 127 x is exact, t = p inv is off by 2 units, the remainder p - t
// amax is exact, and adding its share gives the quotient Q rounded once, exactly Q
// where fp32 holds it, so at every half.  Any other Q is further from a half than
// that rounding: with mantissas of 11 bits, by Q 2^-20 at least.  (Halves are common:
// where amax is 2^n, one in a few hundred.)
//
// fp32: t = x (127 / amax) is off by at most 2^-23 Q, below 2^-15; a fraction that
// near to a half is compared.
template <typename X>
__device__ __forceinline__ void quantised(float (&x)[8], const RowScale& r, float (&q)[8]) {
  if (r.by != 1.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= r.by;
  }
  const uint64_t inv2 = pack2(r.inv, r.inv);
  const uint64_t up = pack2(12582912.f, 12582912.f), down = pack2(-12582912.f, -12582912.f);
  float off = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint64_t v = pack2(x[j], x[j + 1]);
    uint64_t t;
    if constexpr (sizeof(X) == 2) {
      const uint64_t p = mul2(v, pack2(127.f, 127.f));
      t = mul2(p, inv2);
      t = fma2(fma2(t, pack2(-r.amax, -r.amax), p), inv2, t);
    } else {
      t = mul2(v, inv2);
    }
    const uint64_t n2 = add2(add2(t, up), down);  // 1.5 * 2^23: to the nearest integer
    const float2 n = unpack2(n2);
    q[j] = n.x;
    q[j + 1] = n.y;
    if constexpr (sizeof(X) == 4) {
      const float2 d = unpack2(fma2(n2, pack2(-1.f, -1.f), t));
      off = fmaxf(off, fmaxf(fabsf(d.x), fabsf(d.y)));
    }
  }
  if constexpr (sizeof(X) == 4) {
    if (off < 0.5f - 0x1p-15f) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = x[j] * r.inv;
      if (!(fabsf(t - q[j]) < 0.5f - 0x1p-15f)) q[j] = compared(x[j], r.amax, t);
    }
  }
}

template <typename X>
__global__ void __launch_bounds__(kQuantThreads) k_int8_quantize(const Int8Quant p) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t s_amax[2][kQuantThreads / 32];
  const int vecs = p.K / 8, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
    const X* row = static_cast<const X*>(p.x) + t * p.ld;
    Eight<X> held[kHeld];
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const int i = threadIdx.x + h * kQuantThreads;
      if (i < vecs) held[h].load(row + i * 8);
    }
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (threadIdx.x + h * kQuantThreads < vecs) take_largest(held[h], &m);
    for (int i = threadIdx.x + kHeld * kQuantThreads; i < vecs; i += kQuantThreads) {
      Eight<X> e;
      e.load(row + static_cast<int64_t>(i) * 8);
      take_largest(e, &m);
    }
    m = __reduce_max_sync(0xffffffffu, fp32_bits<X>(m));
    if (lane == 0) s_amax[turn][warp] = m;  // two sets in turn: one barrier a row
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) m = max(m, s_amax[turn][i]);
    const bool finite = m < 0x7f800000u;
    const float amax = __uint_as_float(m);
    const bool zero = !finite || m == 0;
    const RowScale scale = row_scale<X>(amax);
    if (threadIdx.x == 0) {
      p.scales[t] = finite ? amax / 127.f : __uint_as_float(0x7fffffffu);
      if (!finite && !p.clear) set_status(p.status, MEGAMOE_DEV_NONFINITE);
    }
    auto put = [&](int i, const Eight<X>& e) {
      float v[8], q[8];
      e.values(v);
      if (!zero) quantised<X>(v, scale, q);
      const int64_t at = t * p.K + static_cast<int64_t>(i) * 8;
      if (p.half) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2 h = __floats2half2_rn(q[2 * j], q[2 * j + 1]);
          w[j] = zero ? 0u : *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p.half + at) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j >> 2] |= zero ? 0u : static_cast<uint32_t>(__float2int_rn(q[j]) & 0xff) << (8 * (j & 3));
        *reinterpret_cast<uint2*>(p.codes + at) = make_uint2(w[0], w[1]);
      }
    };
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const int i = threadIdx.x + h * kQuantThreads;
      if (i < vecs) put(i, held[h]);
    }
    for (int i = threadIdx.x + kHeld * kQuantThreads; i < vecs; i += kQuantThreads) {
      Eight<X> e;
      e.load(row + static_cast<int64_t>(i) * 8);
      put(i, e);
    }
  }
}

// Four integers -> four fp16 values: with its sign bit flipped a byte is q + 128,
// and under 0x64 the fp16 number 1024 + 128 + q, of which 1152 is taken off exactly.
__device__ __forceinline__ void widen4(uint32_t bytes, uint32_t* lo, uint32_t* hi) {
  const uint32_t u = bytes ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  *lo = *reinterpret_cast<const uint32_t*>(&x);
  *hi = *reinterpret_cast<const uint32_t*>(&y);
}

// Integers that the caller brings, as fp16, and their scales.
__global__ void __launch_bounds__(kQuantThreads) k_int8_widen(const Int8Quant p) {
  pdl_wait();
  pdl_trigger();
  if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  const int vecs = p.K / 16;
  const int64_t total = p.T * vecs;
  for (int64_t i = blockIdx.x * int64_t{kQuantThreads} + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kQuantThreads) {
    const int64_t t = i / vecs;
    const int v = static_cast<int>(i - t * vecs);
    if (v == 0) p.scales[t] = __ldg(p.x_scales + t);
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const int8_t*>(p.x) + t * p.ld) + v);
    uint4 a, b;
    widen4(q.x, &a.x, &a.y);
    widen4(q.y, &a.z, &a.w);
    widen4(q.z, &b.x, &b.y);
    widen4(q.w, &b.z, &b.w);
    uint4* to = reinterpret_cast<uint4*>(p.half + t * p.K + static_cast<int64_t>(v) * 16);
    to[0] = a;
    to[1] = b;
  }
}

// sum sx sw with the token's scale last where it is large, so that nothing overflows that
// the other scale would have brought back.  (A small one first loses nothing: the sum is
// whole, so their product is exact wherever it is no normal number.)
constexpr float kLoud = 0x1p64f;
__device__ __forceinline__ float scaled(float sum, float sx, float sw) {
  const bool loud = fabsf(sx) > kLoud;
  return sum * (loud ? sw : sx) * (loud ? sx : sw);
}

// ---------------------------------------------------------------------------
// Few tokens: 256-row tiles would leave most SMs without work, or each with a long
// sum.  Bound by the weights' bytes and by the launch; the first of a block's
// weights are on their way to L2 before the kernel ahead is done (they are the
// caller's constants).
//
// us (K -> N; dots / MMA / pairs of CTAs, the last two with the quantiser before them):
//              1 token      4 tokens     8 tokens     16 tokens
//   1536 24576  9.4 / 14.1  11.5 / 14.2  14.3 / 24.2  18.1 / 22.9
//   7168  7168 11.6 / 18.6  15.8 / 18.9  19.2 / 29.9     - / 22.5
//   7168  2048  7.3 / 11.1  10.5 / 11.9  12.5 / 15.6     - / 13.8
//   4096  4096  5.3 /  8.4   7.6 /  8.3   8.9 / 15.5  11.4 / 13.4
// 1536 -> 24576 are 37.7 MB, 5.6 us at the copy rate; 7.3 us in a stream of calls.
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewBlocks = 2;        // an SM
constexpr int kFewSmem = 96 * 1024;  // of tokens' integers

struct Int8Few {
  const void* x;  // integers [T, K], or (dots) of `type`
  int type;
  const float* x_scales;
  int T;
  int64_t ld;
  const int8_t* w;
  const float* w_scales;
  int N, K;
  int split;  // (MMA) warps that share a row's sum, a power of two up to 8
  void* out;
  bool out_f32;
  int64_t ld_out;
  uint32_t* status;
};

__device__ __forceinline__ void few_store(const Int8Few& p, int t, int n, float sum, float scale) {
  const float y = scaled(sum, scale, __ldg(p.w_scales + n));
  if (p.out_f32) static_cast<float*>(p.out)[t * p.ld_out + n] = y;
  else static_cast<__nv_bfloat16*>(p.out)[t * p.ld_out + n] = __float2bfloat16_rn(y);
}
__device__ __forceinline__ void few_status(const Int8Few& p, const float* scales) {
  bool bad = false;
  for (int t = 0; t < p.T; ++t) bad |= !(fabsf(scales[t]) <= 0x1.fffffep127f);
  *p.status = bad ? MEGAMOE_DEV_NONFINITE : 0u;
}

// Up to four tokens in one launch: every block quantises them into its shared
// memory; a warp then multiplies its rows by them, F at a time, with dp4a: sums
// exact in 32-bit integers, no rounding but that of the sum to fp32.
template <typename X, int T>
__device__ __forceinline__ void few_quantise(const Int8Few& p, int8_t* s_codes,
                                             uint32_t (*s_amax)[kFewWarps], float* s_scale) {
  const X* x = static_cast<const X*>(p.x);
  const int vecs = p.K / 8;
  uint32_t m[T] = {};
#pragma unroll 2
  for (int i = threadIdx.x; i < vecs; i += kFewThreads) {
    Eight<X> e[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
      if (t < p.T) e[t].load(x + t * p.ld + i * 8);
#pragma unroll
    for (int t = 0; t < T; ++t)
      if (t < p.T) take_largest(e[t], &m[t]);
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    m[t] = __reduce_max_sync(0xffffffffu, fp32_bits<X>(m[t]));
    if ((threadIdx.x & 31) == 0) s_amax[t][threadIdx.x >> 5] = m[t];
  }
  __syncthreads();
#pragma unroll 1
  for (int t = 0; t < T; ++t) {  // (a token that is not there: zeros)
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < kFewWarps; ++i) a = max(a, s_amax[t][i]);
    const bool finite = a < 0x7f800000u, zero = !finite || a == 0;
    const float amax = __uint_as_float(a);
    const RowScale scale = row_scale<X>(amax);
    if (threadIdx.x == 0) s_scale[t] = finite ? amax / 127.f : __uint_as_float(0x7fffffffu);
#pragma unroll 2
    for (int i = threadIdx.x; i < vecs; i += kFewThreads) {
      uint32_t w[2] = {0, 0};
      if (!zero) {
        Eight<X> e;
        e.load(x + t * p.ld + i * 8);
        float v[8], q[8];
        e.values(v);
        quantised<X>(v, scale, q);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j >> 2] |= static_cast<uint32_t>(__float2int_rn(q[j]) & 0xff) << (8 * (j & 3));
      }
      *reinterpret_cast<uint2*>(s_codes + t * p.K + i * 8) = make_uint2(w[0], w[1]);
    }
  }
}

template <int T, int F>
__global__ void __launch_bounds__(kFewThreads, kFewBlocks) k_int8_dots(const Int8Few p) {
  extern __shared__ __align__(16) int8_t s_codes[];  // [T][K]
  __shared__ uint32_t s_amax[T][kFewWarps];
  __shared__ float s_scale[T];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kFewWarps;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kFewWarps + warp;
  const int n0 = static_cast<int>(p.N * me / warps), n1 = static_cast<int>(p.N * (me + 1) / warps);
  if (lane == 0 && n0 < n1)
    bulk_prefetch_l2(p.w + static_cast<int64_t>(n0) * p.K,
                     static_cast<uint32_t>(min(static_cast<int64_t>(n1 - n0) * p.K, int64_t{16384})));
  pdl_wait();
  pdl_trigger();
  if (p.type == MEGAMOE_TYPE_I8) {
#pragma unroll 1
    for (int t = 0; t < T; ++t) {
      const uint4* row = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(p.x) + t * p.ld);
#pragma unroll 4
      for (int i = threadIdx.x; i < p.K / 16; i += kFewThreads)
        reinterpret_cast<uint4*>(s_codes + t * p.K)[i] = t < p.T ? __ldg(row + i) : make_uint4(0, 0, 0, 0);
      if (threadIdx.x == 0) s_scale[t] = t < p.T ? __ldg(p.x_scales + t) : 0.f;
    }
  } else if (p.type == MEGAMOE_TYPE_F32) {
    few_quantise<float, T>(p, s_codes, s_amax, s_scale);
  } else if (p.type == MEGAMOE_TYPE_F16) {
    few_quantise<__half, T>(p, s_codes, s_amax, s_scale);
  } else {
    few_quantise<__nv_bfloat16, T>(p, s_codes, s_amax, s_scale);
  }
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) few_status(p, s_scale);

  const int pieces = p.K / 16;  // of 16 bytes
  for (int n = n0; n < n1; n += F) {
    const uint4* row = reinterpret_cast<const uint4*>(p.w + static_cast<int64_t>(n) * p.K);
    int acc[F][T] = {};
#pragma unroll(8 / F)
    for (int i = lane; i < pieces; i += 32) {
      uint4 q[F];
#pragma unroll
      for (int f = 0; f < F; ++f)
        q[f] = n + f < n1 ? __ldcs(row + static_cast<int64_t>(f) * pieces + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const uint4 c = *reinterpret_cast<const uint4*>(s_codes + t * p.K + i * 16);
#pragma unroll
        for (int f = 0; f < F; ++f) {
          acc[f][t] = __dp4a(static_cast<int>(q[f].x), static_cast<int>(c.x), acc[f][t]);
          acc[f][t] = __dp4a(static_cast<int>(q[f].y), static_cast<int>(c.y), acc[f][t]);
          acc[f][t] = __dp4a(static_cast<int>(q[f].z), static_cast<int>(c.z), acc[f][t]);
          acc[f][t] = __dp4a(static_cast<int>(q[f].w), static_cast<int>(c.w), acc[f][t]);
        }
      }
    }
    int mine = 0;  // lane F t + f: token t of row n + f
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int sum = __reduce_add_sync(0xffffffffu, acc[f][t]);
        if (lane == F * t + f) mine = sum;
      }
    const int t = lane / F, c = n + lane % F;
    if (t < p.T && c < n1) few_store(p, t, c, static_cast<float>(mine), s_scale[t < T ? t : 0]);
  }
}

template <int T, int F>
cudaError_t launch_dots(const Int8Few& a, int64_t blocks, cudaStream_t stream) {
  auto kern = k_int8_dots<T, F>;
  const size_t smem = static_cast<size_t>(T) * a.K;
  if (smem > 48 * 1024 - 256) {  // more, with the kernel's own, than a kernel has unasked
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kFewThreads), smem, stream, a);
}
template <int F>
cudaError_t launch_dots_t(const Int8Few& a, int64_t blocks, cudaStream_t stream) {
  return a.T == 1 ? launch_dots<1, F>(a, blocks, stream)
         : a.T == 2 ? launch_dots<2, F>(a, blocks, stream)
                    : launch_dots<4, F>(a, blocks, stream);
}

// Up to sixteen tokens, their integers as k_int8_quantize leaves them: the warps'
// own MMA (16 rows x 8 tokens, fp16 with fp32 sums), since the tensor cores have next
// to nothing to do.  A row's bytes go from memory to the lanes that multiply them: a
// lane has 16 of the 64 bytes of a step, and the order in which the MMA takes them is
// the same for the tokens' integers.
//
// Rows of integers in shared memory: whole steps, and 64 bytes more so that two
// tokens' pieces fall into different banks.
__host__ __device__ constexpr int few_pitch(int K) { return (K + 127) / 128 * 128 + 64; }

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), fp16.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Sixteen integers as eight pairs.
__device__ __forceinline__ void widen16(uint4 q, uint32_t (&v)[8]) {
  widen4(q.x, &v[0], &v[1]);
  widen4(q.y, &v[2], &v[3]);
  widen4(q.z, &v[4], &v[5]);
  widen4(q.w, &v[6], &v[7]);
}

// NT: eights of tokens.
template <int NT>
__global__ void __launch_bounds__(kFewThreads, kFewBlocks) k_int8_few(const Int8Few p) {
  extern __shared__ __align__(16) int8_t s_codes[];  // [8 NT][pitch]
  __shared__ float s_scale[8 * NT];
  __shared__ int s_part[2][kFewWarps][NT * 4][32];  // sums of the warps that share a row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = static_cast<int>(static_cast<int64_t>(p.N) * blockIdx.x / gridDim.x);
  const int r1 = static_cast<int>(static_cast<int64_t>(p.N) * (blockIdx.x + 1) / gridDim.x);
  const int pitch = few_pitch(p.K);
  if (lane == 0) {  // a warp's eighth of the block's rows
    const int a = r0 + (r1 - r0) * warp / kFewWarps, b = r0 + (r1 - r0) * (warp + 1) / kFewWarps;
    if (a < b)
      bulk_prefetch_l2(p.w + static_cast<int64_t>(a) * p.K,
                       static_cast<uint32_t>(min(static_cast<int64_t>(b - a) * p.K, int64_t{16384})));
  }
  pdl_wait();
  pdl_trigger();
  for (int t = warp; t < 8 * NT; t += kFewWarps) {
    const uint4* row = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(p.x) + t * p.ld);
    uint4* codes = reinterpret_cast<uint4*>(s_codes + t * pitch);
#pragma unroll 8
    for (int i = lane; i < pitch / 16; i += 32)
      codes[i] = t < p.T && i < p.K / 16 ? __ldg(row + i) : make_uint4(0, 0, 0, 0);
    if (lane == 0) s_scale[t] = t < p.T ? __ldg(p.x_scales + t) : 0.f;
  }
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) few_status(p, s_scale);

  // The block's rows in turns of up to 16 for each group of warps that share a sum,
  // of equal size.
  const int groups = kFewWarps / p.split, group = warp / p.split, share = warp % p.split;
  const int turns = (r1 - r0 + 16 * groups - 1) / (16 * groups);
  const int per = turns ? (r1 - r0 + turns * groups - 1) / (turns * groups) : 0;
  const int pieces = p.K / 16, steps = (pieces + 3) / 4;  // of 16 and of 64 bytes
  const int g = lane >> 2, j = lane & 3;
  const int8_t* codes = s_codes + g * pitch + j * 16;
  for (int turn = 0; turn < turns; ++turn) {
    const int n0 = r0 + (turn * groups + group) * per;
    const int live = min(per, r1 - n0);  // rows n0 + g and n0 + g + 8 are this lane's
    const uint4* lo = reinterpret_cast<const uint4*>(p.w + static_cast<int64_t>(n0 + g) * p.K) + j;
    const uint4* hi = reinterpret_cast<const uint4*>(p.w + static_cast<int64_t>(n0 + g + 8) * p.K) + j;
    float acc[NT][4] = {};
    int sum[NT][4] = {};  // parts of 1024 terms: 16 steps of this warp
#pragma unroll 1
    for (int c0 = share, turns4 = 0; c0 < steps; c0 += 4 * p.split, ++turns4) {
      uint4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + i * p.split;
        const bool in = 4 * c + j < pieces;
        a[i] = in && g < live ? __ldcs(lo + 4 * c) : make_uint4(0, 0, 0, 0);
        b[i] = in && g + 8 < live ? __ldcs(hi + 4 * c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + i * p.split;
        if (c >= steps) break;
        uint32_t u[8], v[8];
        widen16(a[i], u);
        widen16(b[i], v);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t x[8];
          widen16(*reinterpret_cast<const uint4*>(codes + n * 8 * pitch + c * 64), x);
#pragma unroll
          for (int h = 0; h < 8; h += 2)
            mma_16x8x16(acc[n], u[h], v[h], u[h + 1], v[h + 1], x[h], x[h + 1]);
        }
      }
      if ((turns4 & 3) != 3 && c0 + 4 * p.split < steps) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[n][i] += __float2int_rn(acc[n][i]);
          acc[n][i] = 0.f;
        }
    }
    if (p.split > 1) {  // the shares in order
      int(*part)[NT * 4][32] = s_part[turn & 1];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][n * 4 + i][lane] = sum[n][i];
      __syncthreads();
      if (share != 0) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          for (int s = 1; s < p.split; ++s) sum[n][i] += part[warp + s][n * 4 + i][lane];
    }
    // rows g and g + 8 of tokens 2 j and 2 j + 1
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 8 * n + 2 * j + (i & 1), r = g + 8 * (i >> 1);
        if (t < p.T && r < live) few_store(p, t, n0 + r, static_cast<float>(sum[n][i]), s_scale[t]);
      }
  }
}

template <int NT>
cudaError_t launch_few(const Int8Few& a, int64_t blocks, cudaStream_t stream) {
  auto kern = k_int8_few<NT>;
  const size_t smem = static_cast<size_t>(8 * NT) * few_pitch(a.K);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kFewThreads), smem, stream, a);
}

// ---------------------------------------------------------------------------
// The product on pairs of CTAs: 256 features x up to 256 tokens a tile.  8192 x 7168
// -> 2048 take 128 us (240 GFLOP: 1.88 PFLOP/s of fp16 MMAs, the tensor pipe 86 % busy;
// a library's bf16 product takes 133 on operands of twice the bytes), 296 tiles in four
// turns of the 76 pairs.  Handing a stage of widened weights to the other CTA by a
// releasing arrival took 310 us: the tensor-memory stores have been waited for, and
// tcgen05's own fences order them.
// ---------------------------------------------------------------------------
struct Int8Maps {
  CUtensorMap w, x, x8;  // tokens in boxes of 32 and of 8
};

struct Int8Args {
  const float* x_scales;
  const float* w_scales;
  int T, N, K;
  int per;    // tokens of a tile, a multiple of 16 up to 256
  int split;  // shares of a tile's sum, each with a pair of CTAs
  void* out;
  int64_t ld_out;
  float* partial;  // split > 1: [split][T][N], added up by k_int8_sum (FOLD: integers)
  uint32_t* status;
  uint64_t wait_limit_ns;
};

// What a pair of CTAs does at a time: steps k0 .. k1 of a tile's sum.
struct Item {
  int tile, mt, nt, share, k0, k1;
};

struct Cfg {
  static constexpr int THREADS = 576;  // producer, MMA issuer, 8 epilogue warps, 8 that widen
  static constexpr int STAGES = 4;     // of 128 of K
  static constexpr int W = 128 * 128;  // a CTA's bytes of weights
  static constexpr int X = 128 * 128;  // its tokens' fp16, 64 of K
  static constexpr int STAGE = W + 2 * X;
  static constexpr int STG = 2048;  // staged output of an epilogue warp
  static constexpr int STG_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = STG_OFF + kEpiWarps * STG;
  static constexpr int SMEM = 1024 + BAR_OFF + 256;
  // tensor memory: accumulators in turn at columns 0 and 128 (128 in common), then
  // two buffers of widened weights
  static constexpr int ACC1 = 128;
  static constexpr int A_COL0 = 384;
  static constexpr int A_COLS = 64;
  static_assert(SMEM <= 232448, "shared memory budget");
};

// kind::f16 over the pair with A in each CTA's tensor memory (its 128 rows).
__device__ __forceinline__ void mma_f16_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
      "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void store_rounded(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_rounded(float v, float* p) { *p = v; }

// Tile q: bands of eight tiles of tokens, feature tile by feature tile within a
// band, so that tiles in work at a time share few rows of either operand.
__device__ __forceinline__ void int8_tile(int q, int MT, int NT, int* mt, int* nt) {
  const int band = q / (8 * MT), r = q - band * 8 * MT;
  const int wide = min(8, NT - band * 8);
  *mt = r / wide;
  *nt = band * 8 + r - *mt * wide;
}

__device__ __forceinline__ Item int8_item(int q, int split, int MT, int NT, int KT) {
  Item t;
  t.tile = q / split;
  t.share = q - t.tile * split;
  int8_tile(t.tile, MT, NT, &t.mt, &t.nt);
  t.k0 = t.share * KT / split;
  t.k1 = (t.share + 1) * KT / split;
  return t;
}

// FOLD: sums in parts of PART steps (1024 terms), which the epilogue's warps add up as
// integers in registers, 96 each: tiles have 192 tokens at most, and the accumulators no
// columns in common.  (8192 x 7168 -> 2048: 185 us for fp32 results; 222 with 128 tokens,
// 170 in one part.)  Those warps then take registers from the others, a warpgroup each, so
// that the first one has two idle warps.
struct FoldCfg {
  static constexpr int TOKENS = 192;
  static constexpr int THREADS = 640;
  static constexpr int FEW_REGS = 40, WIDEN_REGS = 80, MANY_REGS = 136;  // of a thread; 96 at launch
};

template <typename O, bool FOLD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FOLD ? FoldCfg::THREADS : Cfg::THREADS, 1)
    k_int8_pair(const __grid_constant__ Int8Maps maps, const Int8Args p) {
  using C = Cfg;
  constexpr int STAGES = C::STAGES, PART = FOLD ? 8 : 1 << 30;
  constexpr int EPI = FOLD ? 4 : 2, WIDEN = EPI + kEpiWarps;  // the first warps of either
  constexpr int ACC1 = FOLD ? FoldCfg::TOKENS : C::ACC1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* w_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);  // this CTA's weights
  uint64_t* x_full = w_full + STAGES;  // rank 0's: the tokens of both
  uint64_t* empty = x_full + STAGES;
  uint64_t* a_full = empty + STAGES;  // rank 0's: the widening warps of both
  uint64_t* a_empty = a_full + 2;
  uint64_t* acc_full = a_empty + 2;
  uint64_t* acc_empty = acc_full + 2;  // rank 0's: the epilogue warps of both
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int MT = (p.N + 255) / 256, NT = (p.T + p.per - 1) / p.per;
  const int KT = (p.K + 127) / 128;
  const int total = MT * NT * p.split;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;  // items of this pair

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.w);
    prefetch_tensormap(&maps.x);
    prefetch_tensormap(&maps.x8);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&w_full[s], 1);
      mbar_init(&x_full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], 8);  // four warps of each CTA
      mbar_init(&a_empty[i], 1);
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are there before either is arrived on
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();
  pdl_trigger();

  if (warp < EPI) {
    if (FOLD) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FoldCfg::FEW_REGS));
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      // (the whole warp, one lane of it issuing: elect_one).  Weights are waited for
      // by this CTA's own warps, tokens by rank 0's MMAs.
      const bool leader = elect_one();
      const uint64_t pol_w = NT > 1 ? policy_evict_normal() : policy_evict_first();
      const uint64_t pol_x = policy_evict_normal();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int q = first; ok && q < total; q += step) {
        const Item it = int8_item(q, p.split, MT, NT, KT);
        const int rows = min(p.per, p.T - it.nt * p.per), half = (rows + 15) / 16 * 8;
        const RowBoxes mine(rows - rank * half, half), other(rows - (1 - rank) * half, half);
        const int t0 = it.nt * p.per + rank * half;
        const int m0 = it.mt * 256 + rank * 128;
        for (int i = it.k0; i < it.k1; ++i) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          uint8_t* sw = smem + stage * C::STAGE;
          uint8_t* sx = sw + C::W;
          if (leader) {
            mbar_arrive_expect_tx(&w_full[stage], C::W);
            tma_load_2d(sw, &maps.w, &w_full[stage], i * 128, m0, pol_w);
            if (rank == 0) mbar_arrive_expect_tx(&x_full[stage], 2 * (mine.bytes() + other.bytes()));
            const uint32_t bar = cluster_address(&x_full[stage], 0);
            for (int h = 0; h < 2; ++h) {
              for (int b = 0; b < mine.large; ++b)
                tma_load_2d_pair(sx + h * C::X + b * 4096, &maps.x, bar, i * 128 + h * 64,
                                 t0 + b * 32, pol_x);
              for (int b = 0; b < mine.small; ++b)
                tma_load_2d_pair(sx + h * C::X + b * 1024, &maps.x8, bar, i * 128 + h * 64, t0 + b * 8,
                                 pol_x);
            }
          }
          __syncwarp();
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      drain_copies(w_full, STAGES, issued);
      drain_pair_copies(x_full, STAGES, issued, rank, !ok);
      __syncwarp();
    } else if (warp == 1) {
      if (rank == 0) {
        // ---------------------------------------------------------- MMA issuer
        const bool leader = elect_one();
        const uint64_t dx = sdesc_sw128(smem_u32(smem) + C::W);
        // fp16 operands, K-major, fp32 sums, M = 256
        constexpr uint32_t idesc0 = (1u << 4) | (256u >> 4) << 24;
        int stage = 0, accs = 0, steps = 0;  // accs: accumulators taken
        uint32_t phase = 0;
        bool ok = true;
        for (int q = first; ok && q < total; q += step) {
          const Item it = int8_item(q, p.split, MT, NT, KT);
          const int n = (min(p.per, p.T - it.nt * p.per) + 15) / 16 * 16;
          const uint32_t idesc = idesc0 | static_cast<uint32_t>(n >> 3) << 17;
          for (int i0 = it.k0; ok && i0 < it.k1; i0 += min(PART, it.k1 - i0), ++accs) {
            // FOLD's accumulators have a barrier each; one that shares columns with the
            // last waits for that one's
            uint64_t* free = &acc_empty[FOLD ? accs & 1 : 0];
            const uint32_t turn = FOLD ? accs >> 1 & 1 : accs & 1;
            const uint32_t acc = tmem + (accs & 1) * ACC1;
            const int i1 = i0 + min(PART, it.k1 - i0);
            for (int i = i0; i < i1; ++i, ++steps) {
              const int buf = steps & 1;
              if (!mbar_wait(&x_full[stage], phase, abort_flag, p.status, p.wait_limit_ns) ||
                  !mbar_wait(&a_full[buf], steps >> 1 & 1, abort_flag, p.status, p.wait_limit_ns) ||
                  (i == i0 && !mbar_wait(free, turn ^ 1u, abort_flag, p.status, p.wait_limit_ns))) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint64_t cx = sdesc_at(dx, stage * C::STAGE);
              const uint32_t a = tmem + C::A_COL0 + buf * C::A_COLS;
              const int left = p.K - i * 128;  // a multiple of 16
              if (leader) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  if (16 * c < left)
                    mma_f16_pair_ts(acc, a + 8 * c, sdesc_at(cx, (c >> 2) * C::X + 32 * (c & 3)),
                                    idesc, (i != i0 || c != 0) ? 1u : 0u);
                tc_commit_pair(&empty[stage]);
                tc_commit_pair(&a_empty[buf]);
              }
              __syncwarp();
              if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
              }
            }
            if (!ok) break;
            if (leader) tc_commit_pair(&acc_full[FOLD ? accs & 1 : 0]);
            __syncwarp();
          }
        }
        // every MMA issued so far must finish before tensor memory is released
        if (leader) tc_commit_pair(drain);
        __syncwarp();
        mbar_drain(drain, 0);
      }
      __syncwarp();
    }
  } else if (warp >= WIDEN) {
    if (FOLD) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FoldCfg::WIDEN_REGS));
    // ---------------------------------------------------------- widening warps
    // A lane has a row of 128 bytes; its 16-byte piece j is at j ^ (row % 8).  Four
    // warps take the even stages and four the odd ones, each set with a buffer.
    const int quarter = warp & 3, buf = warp >= WIDEN + 4 ? 1 : 0;
    const uint32_t to = tmem + C::A_COL0 + buf * C::A_COLS + (static_cast<uint32_t>(quarter * 32) << 16);
    int64_t all = 0;  // stages of this pair's items
    for (int q = first; q < total; q += step) {
      const Item it = int8_item(q, p.split, MT, NT, KT);
      all += it.k1 - it.k0;
    }
    uint32_t phase = 0;
    for (int64_t i = buf; i < all; i += 2, phase ^= 1u) {
      const int stage = static_cast<int>(i % STAGES);
      if (!mbar_wait(&w_full[stage], static_cast<uint32_t>(i / STAGES) & 1u, abort_flag, p.status,
                     p.wait_limit_ns))
        break;
      const uint4* row = reinterpret_cast<const uint4*>(smem + stage * C::STAGE +
                                                        (quarter * 32 + lane) * 128);
      uint32_t v[64];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 b = row[j ^ (lane & 7)];
        widen4(b.x, &v[8 * j], &v[8 * j + 1]);
        widen4(b.y, &v[8 * j + 2], &v[8 * j + 3]);
        widen4(b.z, &v[8 * j + 4], &v[8 * j + 5]);
        widen4(b.w, &v[8 * j + 6], &v[8 * j + 7]);
      }
      if (!mbar_wait(&a_empty[buf], phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) break;
      tc_fence_after();
      tmem_st_32x32b_x32(to, v);
      tmem_st_32x32b_x32(to + 32, v + 32);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(&a_full[buf], 0);
      __syncwarp();
    }
  } else {
    if (FOLD) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FoldCfg::MANY_REGS));
    // -------------------------------------------------------------- epilogue
    // A lane has a feature, a column is a token: 64 or 128 bytes of 32 features of
    // a token at a time through shared memory.  The two warps of a quarter take
    // chunks of 32 tokens in turn, those first whose columns the next tile's
    // accumulator shares; its products may start once they have been read.
    const int quarter = warp & 3;
    const int half = warp >= EPI + 4 ? 1 : 0;
    uint8_t* stg = smem + C::STG_OFF + (warp - EPI) * C::STG;
    constexpr int SIZE = sizeof(O), PER = 16 / SIZE;
    constexpr int ROWS = C::STG / (32 * SIZE);  // staged at a time
    constexpr int LANES = 32 / PER;             // lanes of a token's 16-byte pieces
    const int piece = lane % LANES;
    O* out = static_cast<O*>(p.out);
    int accs = 0;
    bool bad = false, ok = true;
    for (int q = first; q < total; q += step) {
      const Item it = int8_item(q, p.split, MT, NT, KT);
      const int rows = min(p.per, p.T - it.nt * p.per), t0 = it.nt * p.per;
      const int m = it.mt * 256 + rank * 128 + quarter * 32;  // this warp's first feature
      const float sw = m + lane < p.N ? __ldg(p.w_scales + m + lane) : 0.f;
      const bool in = m + piece * PER < p.N;
      // tokens c .. c + 31: their sums (FOLD: integers) times the scales, or as they are
      auto put = [&](int c, const uint32_t(&v)[32]) {
        if (c >= rows) return;
        if (p.split > 1) {
          float* to = p.partial + (static_cast<int64_t>(it.share) * p.T + t0 + c) * p.N + m + lane;
          if (m + lane < p.N) {
#pragma unroll
            for (int j = 0; j < 32; ++j, to += p.N)
              if (c + j < rows) *to = __uint_as_float(v[j]);
          }
          return;
        }
        auto sum = [&](int j) {
          return FOLD ? static_cast<float>(static_cast<int>(v[j])) : __uint_as_float(v[j]);
        };
        const float4* xs = reinterpret_cast<const float4*>(p.x_scales + t0 + c);
        auto emit = [&](auto loud) {
#pragma unroll
          for (int g = 0; g < 32 / ROWS; ++g) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < ROWS; j += 4) {
              const float4 s = __ldg(xs + (g * ROWS + j) / 4);
              const float sx[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                store_rounded(loud ? scaled(sum(g * ROWS + j + i), sx[i], sw)
                                   : sum(g * ROWS + j + i) * sx[i] * sw,
                              reinterpret_cast<O*>(stg) + (j + i) * 32 + lane);
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < ROWS * LANES / 32; ++j) {
              const int r = j * (32 / LANES) + lane / LANES;
              const uint4 x = *reinterpret_cast<const uint4*>(stg + (r * LANES + piece) * 16);
              const int row = c + g * ROWS + r;
              if (in && row < rows)
                *reinterpret_cast<uint4*>(out + (t0 + static_cast<int64_t>(row)) * p.ld_out + m +
                                          piece * PER) = x;
            }
          }
        };
        // (a choice for each value costs 0.3 us)
        if (__any_sync(0xffffffffu, fabsf(__ldg(p.x_scales + t0 + c + lane)) > kLoud)) emit(std::true_type{});
        else emit(std::false_type{});
      };
      const uint32_t base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      if constexpr (FOLD) {
        uint32_t sum[3][32];
#pragma unroll
        for (int j = 0; j < 96; ++j) sum[j >> 5][j & 31] = 0;
        for (int i = it.k0; i < it.k1; i += PART, ++accs) {
          const uint32_t buf = accs & 1;
          if (!mbar_wait(&acc_full[buf], accs >> 1 & 1, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 6; ++h) {  // sixteen tokens at a time
            const int c = half * 32 + (h >> 1) * 64 + (h & 1) * 16;
            if (c >= rows) continue;
            uint32_t v[16];
            tmem_ld_32x32b_x16(base + buf * ACC1 + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              sum[h >> 1][(h & 1) * 16 + j] += static_cast<uint32_t>(__float2int_rn(__uint_as_float(v[j])));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(&acc_empty[buf], 0);
        }
        if (!ok) break;
        if (m < p.N) {  // warp-uniform
#pragma unroll
          for (int h = 0; h < 3; ++h) put(half * 32 + 64 * h, sum[h]);
        }
      } else {
        if (!mbar_wait(acc_full, accs & 1, abort_flag, p.status, p.wait_limit_ns)) break;
        tc_fence_after();
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {  // 128 tokens, the shared columns first
          const int c0 = ((accs & 1) ^ part ^ 1) * 128 + half * 32;
          uint32_t v[2][32];
          if (c0 < rows) tmem_ld_32x32b_x32(base + (accs & 1) * ACC1 + c0, v[0]);
          if (c0 + 64 < rows) tmem_ld_32x32b_x32(base + (accs & 1) * ACC1 + c0 + 64, v[1]);
          tmem_ld_wait();
          if (part == 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty, 0);
          }
          if (m >= p.N) continue;  // warp-uniform
          put(c0, v[0]);
          put(c0 + 64, v[1]);
        }
        ++accs;
      }
      if (it.mt == 0 && it.share == 0)  // once for each token
        for (int c = threadIdx.x - 32 * EPI; c < rows; c += 32 * kEpiWarps)
          bad |= !(fabsf(__ldg(p.x_scales + t0 + c)) <= 0x1.fffffep127f);
    }
    if (bad) set_status(p.status, MEGAMOE_DEV_NONFINITE);
    __syncwarp();
  }
  __syncthreads();
  // rank 0's commits arrive on rank 1's barriers too: none is on its way after the last
  if (warp == 1) mbar_drain(drain, 0);
  __syncwarp();
  cluster_sync();  // neither CTA leaves while the other still reaches into it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// The shares of a sum in their order (FOLD: integers), and the scales.  Four columns a
// thread.
template <typename O, bool FOLD>
__global__ void __launch_bounds__(256) k_int8_sum(const Int8Args p) {
  pdl_wait();
  pdl_trigger();
  const int quads = p.N / 4;
  const int64_t total = static_cast<int64_t>(p.T) * quads;
  for (int64_t i = blockIdx.x * int64_t{256} + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = i / quads;
    const int c = static_cast<int>(i - t * quads) * 4;
    const float* from = p.partial + t * p.N + c;
    using V = std::conditional_t<FOLD, int4, float4>;
    V all{};
#pragma unroll 4
    for (int s = 0; s < p.split; ++s) {
      const V v = __ldcg(reinterpret_cast<const V*>(from + static_cast<int64_t>(s) * p.T * p.N));
      all.x += v.x;
      all.y += v.y;
      all.z += v.z;
      all.w += v.w;
    }
    const float4 sum = make_float4(all.x, all.y, all.z, all.w);
    const float sx = __ldg(p.x_scales + t);
    O* to = static_cast<O*>(p.out) + t * p.ld_out + c;
    store_rounded(scaled(sum.x, sx, __ldg(p.w_scales + c)), to);
    store_rounded(scaled(sum.y, sx, __ldg(p.w_scales + c + 1)), to + 1);
    store_rounded(scaled(sum.z, sx, __ldg(p.w_scales + c + 2)), to + 2);
    store_rounded(scaled(sum.w, sx, __ldg(p.w_scales + c + 3)), to + 3);
  }
}

template <typename O, bool FOLD>
cudaError_t launch_pair(const Int8Maps& maps, const Int8Args& a, int64_t tiles, cudaStream_t stream) {
  auto kern = k_int8_pair<O, FOLD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  constexpr int kThreads = FOLD ? FoldCfg::THREADS : Cfg::THREADS;
  if (FOLD) {
    // what the warps hold after giving up and taking registers is what they start with
    static std::atomic<bool> fits{false};
    cudaFuncAttributes f;
    if (!fits.load(std::memory_order_relaxed)) {
      if ((e = cudaFuncGetAttributes(&f, kern)) != cudaSuccess) return e;
      if (f.numRegs * kThreads < 128 * FoldCfg::FEW_REGS + 256 * (FoldCfg::WIDEN_REGS + FoldCfg::MANY_REGS))
        return cudaErrorInvalidConfiguration;
      fits.store(true, std::memory_order_relaxed);
    }
  }
  const int64_t pairs = std::min<int64_t>(std::max(num_sms() / 2, 1), tiles);
  e = launch_pdl(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads), Cfg::SMEM, stream, maps, a);
  if (e != cudaSuccess || a.split == 1) return e;
  const int64_t blocks = (static_cast<int64_t>(a.T) * (a.N / 4) + 255) / 256;
  return launch_pdl(k_int8_sum<O, FOLD>,
                    dim3(static_cast<unsigned>(std::min<int64_t>(blocks, num_sms() * int64_t{16}))),
                    dim3(256), 0, stream, a);
}

}  // namespace

cudaError_t launch_int8_quantize(const Int8Quant& q, cudaStream_t stream) {
  if (q.T == 0) return cudaSuccess;
  const int64_t most = static_cast<int64_t>(num_sms()) * 16;
  if (q.type == MEGAMOE_TYPE_I8) {
    const int64_t blocks = (q.T * (q.K / 16) + kQuantThreads - 1) / kQuantThreads;
    return launch_pdl(k_int8_widen, dim3(static_cast<unsigned>(std::min(blocks, most))),
                      dim3(kQuantThreads), 0, stream, q);
  }
  auto kern = q.type == MEGAMOE_TYPE_F32   ? k_int8_quantize<float>
              : q.type == MEGAMOE_TYPE_F16 ? k_int8_quantize<__half>
                                           : k_int8_quantize<__nv_bfloat16>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(std::min(q.T, most))), dim3(kQuantThreads), 0,
                    stream, q);
}

// Tokens whose integers fit kFewSmem.  Dots: K up to 98304 for one token, 49152 for two,
// 24576 for three and four; few: 12160 for up to eight, 6016 for up to sixteen (16 x 7168
// do not fit).
bool int8_dots_fit(int64_t T, int64_t K) { return T <= 4 && (T == 3 ? 4 : T) * K <= kFewSmem; }
bool int8_few_fits(int64_t T, int64_t K) {
  return !int8_dots_fit(T, K) && T <= 16 && K <= kFewSmem &&
         (T + 7) / 8 * 8 * few_pitch(static_cast<int>(K)) <= kFewSmem;
}

static Int8Few few_of(const Int8Quant& q, const Int8Product& g) {
  return Int8Few{q.x, q.type, q.x_scales, static_cast<int>(q.T), q.ld,      g.w,      g.w_scales, g.N,
                 g.K, 1,      g.out,      g.out_f32,             g.ld_out,  g.status};
}
// Blocks of a launch: a row or more for each warp.
static int64_t few_blocks(int64_t N) {
  return std::min<int64_t>(static_cast<int64_t>(num_sms()) * kFewBlocks, (N + kFewWarps - 1) / kFewWarps);
}

cudaError_t launch_int8_dots(const Int8Quant& q, const Int8Product& g, cudaStream_t stream) {
  // Four rows at a time where a warp has three or more (1536 -> 24576: 9.4 us, 17.5 a
  // row at a time), else one (7168 -> 2048, four tokens: 10.5 us, 13.1 four at a time).
  const int64_t blocks = few_blocks(g.N);
  const Int8Few a = few_of(q, g);
  return g.N > 2 * blocks * kFewWarps ? launch_dots_t<4>(a, blocks, stream)
                                      : launch_dots_t<1>(a, blocks, stream);
}

cudaError_t launch_int8_few(const Int8Quant& q, const Int8Product& g, cudaStream_t stream) {
  // as many warps to a sum as leave each group of them 16 rows
  const int64_t blocks = few_blocks(g.N), rows = (g.N + blocks - 1) / blocks;
  Int8Few a = few_of(q, g);
  a.split = rows <= 16 ? 8 : rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
  return q.T <= 8 ? launch_few<1>(a, blocks, stream) : launch_few<2>(a, blocks, stream);
}

// Tokens of a tile and shares of its sum: those with which the pairs' turns take the
// fewest cycles.  A step of 128 of K takes four cycles a token in the tensor pipe, or
// what an SM takes in, 16 KB of weights and 128 bytes a token at some 48 bytes a cycle;
// a tile's start and end about 3000; adding up shares a kernel of its own and 8 bytes of
// each share's values through L2.  us, 256 tokens and one share / as chosen: 8192 x 7168
// -> 2048 178 / 168 (224 tokens: four turns of 296 tiles, not of 256), 3000 85 / 74, 1024
// 42 / 35 (two shares), 256 41 / 20, 64 31 / 15.
Int8Plan int8_plan(int64_t T, int N, int K, bool fold) {
  Int8Plan p{};
  double least = 0;
  const int64_t mt = (N + int64_t{255}) / 256, steps = (K + 127) / 128;
  for (int most = fold ? FoldCfg::TOKENS : 256; most >= 128; most -= 16) {
    const int64_t nt = (T + most - 1) / most;
    const int per = static_cast<int>(((T + nt - 1) / nt + 15) / 16 * 16);
    const int64_t tiles = (T + per - 1) / per * mt;
    const double step = std::max(4.0 * per, 341 + 2.67 * per);
    // shares of at least two steps where pairs would idle
    const int64_t shares = std::max<int64_t>(1, std::min({kInt8Pairs / tiles, steps / 2, int64_t{16}}));
    for (int64_t split = 1; split <= shares; split += std::max<int64_t>(1, shares - 1)) {
      const double turns = static_cast<double>((tiles * split + kInt8Pairs - 1) / kInt8Pairs);
      double cost = turns * (static_cast<double>((steps + split - 1) / split) * step + 3000);
      if (split > 1) cost += 4700 + static_cast<double>(split) * T * N * 8 / 2600;
      if (p.per == 0 || cost < least * 0.98) {
        least = cost;
        p.per = per;
        p.tiles = tiles;
        p.split = static_cast<int>(split);
      }
    }
  }
  return p;
}

cudaError_t launch_int8_product(const Int8Product& g, cudaStream_t stream) {
  if (g.T == 0) return cudaSuccess;
  Int8Maps maps;
  if (!make_map(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.w, g.K, g.N, g.K, 128, 128,
                CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&maps.x, CU_TENSOR_MAP_DATA_TYPE_UINT16, g.x, g.K, g.T,
                static_cast<uint64_t>(g.K) * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&maps.x8, CU_TENSOR_MAP_DATA_TYPE_UINT16, g.x, g.K, g.T,
                static_cast<uint64_t>(g.K) * 2, 64, 8, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const bool fold = g.out_f32 && int8_folds(g.K);
  const Int8Plan plan = int8_plan(g.T, g.N, g.K, fold);
  const Int8Args a{g.x_scales, g.w_scales, static_cast<int>(g.T), g.N, g.K, plan.per, plan.split,
                   g.out, g.ld_out, g.partial, g.status, wait_limit_ns()};
  const int64_t items = plan.tiles * plan.split;
  return fold        ? launch_pair<float, true>(maps, a, items, stream)
         : g.out_f32 ? launch_pair<float, false>(maps, a, items, stream)
                     : launch_pair<__nv_bfloat16, false>(maps, a, items, stream);
}

}  // namespace megamoe
