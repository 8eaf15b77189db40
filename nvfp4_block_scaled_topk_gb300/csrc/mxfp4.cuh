// MXFP4 codec and layouts (internal to the library): E2M1 elements, one
// power-of-two scale (E8M0 byte, 2^(byte - 127), 255 = NaN) per 32 elements.
//
// The scale of a block is 2^(floor(log2(amax)) - 2), at least 2^-127, so the
// largest element falls in [4, 8) and elements past 6 saturate (the rule of
// the OCP Microscaling Formats specification 1.0, section 6.3).  Every step is
// exact but the one rounding to E2M1: dividing by a power of two only moves
// the exponent.  A block that holds Inf or NaN gets scale 255 and zero codes,
// so it decodes to NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace megamoe {

constexpr uint32_t kMxNan = 255u;

// Scale byte from the bits of a block's largest |x| (as fp32).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return kMxNan;
  const uint32_t e = amax_bits >> 23;  // biased exponent; 0 for subnormals
  return e > 2u ? e - 2u : 0u;
}
// 2^(127 - byte), what elements are multiplied by before rounding (0 for NaN
// blocks, whose codes are zero).
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return byte == kMxNan ? 0.f : __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127)
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return byte == kMxNan ? __uint_as_float(0x7fffffffu)
                        : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}
// SiLU(g) * u to a few units of fp32 at every g: the exponential is taken of -|g|
// (the short form of it, __expf, is off by |g| units more), and the hardware's
// reciprocal of a number in [1, 2] by one.
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float e = expf(-fabsf(g));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return g * (g >= 0.f ? r : e * r) * u;
}
// Eight elements -> four bytes of codes (element 0 in the lowest nibble).
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], float inv) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 p = unpack2(mul2(pack2(v[i], v[i + 1]), pack2(inv, inv)));
    s[i] = p.x;
    s[i + 1] = p.y;
  }
  uint32_t c;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(c)
      : "f"(s[0]), "f"(s[1]), "f"(s[2]), "f"(s[3]), "f"(s[4]), "f"(s[5]), "f"(s[6]), "f"(s[7]));
  return inv != 0.f ? c : 0u;
}

// What a quantising kernel found, for a status word.  Alone it sets the word
// itself.  Ahead of a product (flags not null) its first block clears the word
// and every block leaves its own finding in flags[block]; the product's first
// block reads them (collect_flags) and sets the word, so that no other
// operation has to clear it beforehand.
__device__ __forceinline__ void report_nonfinite(bool bad, uint32_t* status, uint32_t* flags) {
  if (!flags) {
    if (bad) set_status(status, MEGAMOE_DEV_NONFINITE);
    return;
  }
  const int any = __syncthreads_or(bad ? 1 : 0);
  if (threadIdx.x == 0) {
    flags[blockIdx.x] = any ? MEGAMOE_DEV_NONFINITE : 0u;
    if (blockIdx.x == 0) *status = 0u;
  }
}

// By whole warps, `threads` threads of which this is number `index`.
__device__ __forceinline__ void collect_flags(const uint32_t* flags, int count, int index,
                                              int threads, uint32_t* status) {
  uint32_t bits = 0;
  for (int i = index; i < count; i += threads) bits |= __ldcg(flags + i);
  bits = __reduce_or_sync(0xffffffffu, bits);
  if ((index & 31) == 0 && bits) set_status(status, bits);
}

// Atoms along K of a matrix of row length K (a K step of 256 holds two).
__host__ __device__ __forceinline__ int64_t mx_atoms(int64_t K) { return (K + 255) / 256 * 2; }

// Byte of (row, block) in the atom layout: atoms of 128 rows x 4 blocks, the
// blocks of a row padded to whole K steps of 256.
__host__ __device__ __forceinline__ int64_t mx_atom_offset(int64_t row, int64_t block,
                                                           int64_t atoms) {
  return ((row >> 7) * atoms + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (block & 3);
}

// Byte of block b in a routed row's scales: 16 bytes for each K step of 256,
// the first eight used (a tensor-map box row is at least 16 bytes).
__host__ __device__ __forceinline__ int64_t mx_routed_offset(int b) {
  return static_cast<int64_t>(b >> 3) * 16 + (b & 7);
}

// The larger magnitudes of two pairs of 2-byte elements; NaN if either is.  The
// sign bits are of no use.
template <typename X>
__device__ __forceinline__ uint32_t wider_pair(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t wider_pair<__nv_bfloat16>(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
template <>
__device__ __forceinline__ uint32_t wider_pair<__half>(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}

// Eight consecutive elements: their bits, the largest |x| in a form that
// ordinary integer maxima keep ordered, and their values.
template <typename X>
struct Eight;
template <typename X>
struct Eight16 {  // 2-byte types: two magnitudes side by side in a word
  uint4 q;
  __device__ __forceinline__ void load(const X* p) { q = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { q = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint32_t widest() const {
    return wider_pair<X>(wider_pair<X>(q.x, q.y), wider_pair<X>(q.z, q.w)) & 0x7fff7fffu;
  }
  __device__ __forceinline__ static uint32_t wider(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
};
template <>
struct Eight<__nv_bfloat16> : Eight16<__nv_bfloat16> {
  __device__ __forceinline__ static uint32_t bits(uint32_t m) {  // as fp32
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Eight<__half> : Eight16<__half> {
  __device__ __forceinline__ static uint32_t bits(uint32_t m) {
    const uint16_t h = static_cast<uint16_t>(max(m & 0xffffu, m >> 16));
    return __float_as_uint(__half2float(__ushort_as_half(h)));
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Eight<float> {
  float v8[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v8[0] = a.x; v8[1] = a.y; v8[2] = a.z; v8[3] = a.w;
    v8[4] = b.x; v8[5] = b.y; v8[6] = b.z; v8[7] = b.w;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v8[i] = 0.f;
  }
  __device__ __forceinline__ uint32_t widest() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v8[i]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ static uint32_t wider(uint32_t a, uint32_t b) { return max(a, b); }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return m; }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v8[i];
  }
};

}  // namespace megamoe
