// MXFP4 quantisation along rows and along columns, the routed gather, the
// inverse, and the scales' atom layout (weights, once).
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "mxfp4.cuh"

namespace megamoe {

namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// Largest of the four lanes that share a 32-element block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, __shfl_xor_sync(kAll, m, 1));
  return max(m, __shfl_xor_sync(kAll, m, 2));
}

__device__ __forceinline__ int64_t scale_offset(int layout, int64_t row, int64_t b, int64_t K) {
  return layout == MEGAMOE_SCALES_MMA ? mx_atom_offset(row, b, mx_atoms(K)) : row * (K / 32) + b;
}

// Along rows.  Four lanes take a 32-element block, eight elements each, so a
// warp reads 256 consecutive elements with 16-byte loads and writes 128
// consecutive bytes of codes; the block's largest value is two shuffles.  One
// warp task is 256 elements of a row (a whole K step: its scale bytes past
// the row's end are written as zeros in the atom layout).
template <typename X>
__global__ void __launch_bounds__(256)
    k_mx_rows(const X* __restrict__ x, int64_t rows, int K, int64_t ld, uint8_t* __restrict__ codes,
              uint8_t* __restrict__ scales, int layout, uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int steps = (K + 255) / 256;
  const int64_t tasks = rows * steps;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
       w < tasks; w += warps) {
    const int64_t r = w / steps;
    const int col = static_cast<int>(w - r * steps) * 256 + 8 * lane;
    const bool in = col < K;
    float v[8] = {};
    if (in) mx_load8(x + r * ld + col, v);
    const uint32_t byte = mx_scale_byte(block_max(amax_bits8(v)));
    if (in) {
      *reinterpret_cast<uint32_t*>(codes + r * (K / 2) + col / 2) = mx_codes8(v, mx_inverse(byte));
      if (byte == kMxNan) set_status(status, MEGAMOE_DEV_NONFINITE);
    }
    if ((lane & 3) == 0 && (in || layout == MEGAMOE_SCALES_MMA))
      scales[scale_offset(layout, r, col >> 5, K)] = static_cast<uint8_t>(in ? byte : 0u);
  }
}

// Along columns: codes [K, R / 2] and scales of x^T, R = rows up to a multiple
// of 32 (elements past the last row count as zeros).  A block takes 256 rows
// x 64 columns through shared memory: rows come in with 16-byte loads, a
// thread then takes one pair of neighbouring columns down 32 rows (a 2-byte
// type: one 32-bit word per row, the warp's words consecutive), and the codes
// go out through shared memory as 128-byte runs along the columns' rows.
constexpr int kColRows = 256, kColCols = 64;

template <typename X>
struct ColPair;
template <>
struct ColPair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(const __nv_bfloat16* p) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
};
template <>
struct ColPair<__half> {
  static __device__ __forceinline__ float2 get(const __half* p) {
    return __half22float2(*reinterpret_cast<const __half2*>(p));
  }
};
template <>
struct ColPair<float> {
  static __device__ __forceinline__ float2 get(const float* p) {
    return *reinterpret_cast<const float2*>(p);
  }
};

template <typename X>
__global__ void __launch_bounds__(256)
    k_mx_columns(const X* __restrict__ x, int64_t rows, int K, int64_t ld,
                 uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int layout,
                 uint32_t* status) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  X* tile = reinterpret_cast<X*>(s_raw);  // [kColRows][kColCols]
  // [kColCols][kColRows / 2], 16-byte chunk q of column c at q ^ (c / 2 % 8),
  // so that both the chunks written (one block of 32 columns) and the chunks
  // read (eight blocks of a column) fall in different banks
  uint8_t* s_codes = s_raw + kColRows * kColCols * sizeof(X);
  constexpr int pitch = kColRows / 2;
  pdl_wait();
  pdl_trigger();
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kColRows;
  const int c0 = blockIdx.y * kColCols;
  const int64_t padded = (rows + 31) / 32 * 32;
  constexpr int per = 16 / sizeof(X);           // elements of a 16-byte load
  constexpr int vecs = kColCols / per;          // loads of a tile row
  constexpr int rounds = kColRows * vecs / 256;
#pragma unroll
  for (int i = 0; i < rounds; ++i) {
    const int t = threadIdx.x + 256 * i;
    const int r = t / vecs, c = (t % vecs) * per;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + r < rows && c0 + c < K)
      q = __ldg(reinterpret_cast<const uint4*>(x + (r0 + r) * ld + c0 + c));
    *reinterpret_cast<uint4*>(tile + r * kColCols + c) = q;
  }
  __syncthreads();
  const int pair = threadIdx.x & 31, blk = threadIdx.x >> 5;
  const X* from = tile + blk * 32 * kColCols + 2 * pair;
  uint32_t m0 = 0, m1 = 0;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    const float2 v = ColPair<X>::get(from + i * kColCols);
    m0 = max(m0, __float_as_uint(v.x) & 0x7fffffffu);
    m1 = max(m1, __float_as_uint(v.y) & 0x7fffffffu);
  }
  const uint32_t b0 = mx_scale_byte(m0), b1 = mx_scale_byte(m1);
  const float i0 = mx_inverse(b0), i1 = mx_inverse(b1);
  uint32_t q0[4], q1[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = ColPair<X>::get(from + (8 * g + i) * kColCols);
      a[i] = v.x;
      b[i] = v.y;
    }
    q0[g] = mx_codes8(a, i0);
    q1[g] = mx_codes8(b, i1);
  }
  uint8_t* to = s_codes + 2 * pair * pitch + ((blk ^ (pair & 7)) * 16);
  *reinterpret_cast<uint4*>(to) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
  *reinterpret_cast<uint4*>(to + pitch) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
  const int64_t block = (r0 >> 5) + blk;
  const int c = c0 + 2 * pair;
  if (c < K) {
    const bool in = block * 32 < rows;
    if (in || (layout == MEGAMOE_SCALES_MMA && block < mx_atoms(padded) * 4)) {
      scales[scale_offset(layout, c, block, padded)] = static_cast<uint8_t>(b0);
      scales[scale_offset(layout, c + 1, block, padded)] = static_cast<uint8_t>(b1);
      if (b0 == kMxNan || b1 == kMxNan) set_status(status, MEGAMOE_DEV_NONFINITE);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kColCols * 8 / 256; ++i) {
    const int t = threadIdx.x + 256 * i;
    const int col = t >> 3, part = t & 7;
    if (c0 + col < K && r0 + part * 32 < rows)
      *reinterpret_cast<uint4*>(codes + (c0 + col) * (padded / 2) + r0 / 2 + part * 16) =
          *reinterpret_cast<const uint4*>(s_codes + col * pitch + ((part ^ (col >> 1 & 7)) * 16));
  }
}

// Token rows into their routed rows: slot j of token t goes to row
// slot_dst[t k + j] (skipped when negative).  A row is encoded once.  Warp
// tasks of 256 elements as above; d is a multiple of 256.
__global__ void __launch_bounds__(256)
    k_mx_routed(const __nv_bfloat16* __restrict__ x, int64_t T, int d,
                const int32_t* __restrict__ slot_dst, int k, uint8_t* __restrict__ codes,
                uint8_t* __restrict__ scales, uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int steps = d / 256;
  const int64_t tasks = T * steps;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
       w < tasks; w += warps) {
    const int64_t t = w / steps;
    const int col = static_cast<int>(w - t * steps) * 256 + 8 * lane;
    const int my_dst = lane < k ? __ldg(slot_dst + t * k + lane) : -1;
    float v[8];
    mx_load8(x + t * d + col, v);
    const uint32_t byte = mx_scale_byte(block_max(amax_bits8(v)));
    const uint32_t c = mx_codes8(v, mx_inverse(byte));
    if (byte == kMxNan) set_status(status, MEGAMOE_DEV_NONFINITE);
    for (int j = 0; j < k; ++j) {
      const int64_t dst = __shfl_sync(kAll, my_dst, j);
      if (dst < 0) continue;  // warp-uniform
      *reinterpret_cast<uint32_t*>(codes + dst * (d / 2) + col / 2) = c;
      if ((lane & 3) == 0)
        scales[dst * (d / 16) + mx_routed_offset(col >> 5)] = static_cast<uint8_t>(byte);
    }
  }
}

// E2M1 code -> value: 0, 0.5, or (1 + m / 2) 2^(e - 1).
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const uint32_t m = code & 7u;
  const float v = m < 2u ? 0.5f * static_cast<float>(m)
                         : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
  return (code & 8u) ? -v : v;
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// The values: four bytes of codes in, eight elements out per thread.  bf16
// holds every MXFP4 value exactly.
template <typename O>
__global__ void __launch_bounds__(256)
    k_mx_values(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows,
                int K, O* __restrict__ out, int64_t ld) {
  pdl_wait();
  pdl_trigger();
  const int vecs = K / 8;
  const int64_t total = rows * vecs;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += stride) {
    const int64_t r = i / vecs;
    const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
    const float s = mx_scale_value(__ldg(scales + (i >> 2)));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e2m1_value(c >> (4 * j)) * s;
    store8(out + r * ld + (i - r * vecs) * 8, v);
  }
}

__global__ void __launch_bounds__(256)
    k_mx_swizzle(const uint8_t* __restrict__ src, int64_t rows, int64_t blocks, int64_t atoms,
                 uint8_t* __restrict__ dst) {
  pdl_wait();
  pdl_trigger();
  const int64_t total = (rows + 127) / 128 * 128 * atoms * 4;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += stride) {
    const int64_t r = i / (atoms * 4), b = i - r * (atoms * 4);
    dst[mx_atom_offset(r, b, atoms)] = r < rows && b < blocks ? __ldg(src + r * blocks + b) : 0;
  }
}

unsigned blocks_for(int64_t tasks, int64_t per_block) {
  return static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>((tasks + per_block - 1) / per_block, num_sms() * 16)));
}

template <typename X>
cudaError_t quantize_typed(const MxQuant& q, cudaStream_t s) {
  const X* x = static_cast<const X*>(q.x);
  if (!q.transpose) {
    const int64_t tasks = q.rows * ((q.K + 255) / 256);
    return launch_pdl(k_mx_rows<X>, dim3(blocks_for(tasks, 8)), dim3(256), 0, s, x, q.rows, q.K,
                      q.ld, q.codes, q.scales, q.layout, q.status);
  }
  const size_t smem = kColRows * kColCols * sizeof(X) + kColCols * (kColRows / 2);
  cudaError_t e = cudaFuncSetAttribute(k_mx_columns<X>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((q.rows + kColRows - 1) / kColRows),
                  static_cast<unsigned>((q.K + kColCols - 1) / kColCols));
  return launch_pdl(k_mx_columns<X>, grid, dim3(256), smem, s, x, q.rows, q.K, q.ld, q.codes,
                    q.scales, q.layout, q.status);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuant& q, cudaStream_t s) {
  if (q.rows == 0) return cudaSuccess;
  switch (q.type) {
    case MEGAMOE_TYPE_BF16: return quantize_typed<__nv_bfloat16>(q, s);
    case MEGAMOE_TYPE_F16: return quantize_typed<__half>(q, s);
    default: return quantize_typed<float>(q, s);
  }
}

cudaError_t launch_mx_routed(const uint16_t* x, int64_t T, int d, const int32_t* slot_dst, int k,
                             uint8_t* codes, uint8_t* scales, uint32_t* status, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  return launch_pdl(k_mx_routed, dim3(blocks_for(T * (d / 256), 8)), dim3(256), 0, s,
                    reinterpret_cast<const __nv_bfloat16*>(x), T, d, slot_dst, k, codes, scales,
                    status);
}

cudaError_t launch_mx_values(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K,
                             void* out, bool f32, int64_t ld, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const dim3 grid(blocks_for(rows * (K / 8), 256));
  return f32 ? launch_pdl(k_mx_values<float>, grid, dim3(256), 0, s, codes, scales, rows, K,
                          static_cast<float*>(out), ld)
             : launch_pdl(k_mx_values<__nv_bfloat16>, grid, dim3(256), 0, s, codes, scales, rows, K,
                          static_cast<__nv_bfloat16*>(out), ld);
}

cudaError_t launch_mx_swizzle(const uint8_t* src, int64_t rows, int64_t K, uint8_t* dst,
                              cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int64_t total = (rows + 127) / 128 * 128 * mx_atoms(K) * 4;
  return launch_pdl(k_mx_swizzle, dim3(blocks_for(total, 256)), dim3(256), 0, s, src, rows, K / 32,
                    mx_atoms(K), dst);
}

}  // namespace megamoe
