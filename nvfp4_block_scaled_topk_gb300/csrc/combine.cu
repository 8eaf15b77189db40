// Top-k weighted combine: out[t] = bf16( sum_j w[t, j] * y[slot_dst[t*k + j]] )
// (the topk_weights input of "CURRENT_BUG.md -- DeepSeek-V4 Blackwell NVFP4",
// "Test Plan -- Finding the NaN", Phase 1).  One thread per 4 consecutive
// features of one token: 128-bit loads of each routed row of y (up to eight
// slots' loads in flight at once), fp32 sums in ascending j, one bf16
// rounding, 64-bit stores.  y is fp32 (megamoe_combine), or (the forward)
// BFP16, then a warp per 256 features (k_combine_bfp16).  An expert-parallel
// shard writes the fp32 sum of its own slots instead, and the shards' sums
// are added and rounded once after the exchange (k_round_bf16).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace megamoe {

__global__ void __launch_bounds__(256) k_combine(const float* __restrict__ y, int64_t ld_y,
                                                 const int32_t* __restrict__ slot_dst,
                                                 const float* __restrict__ w, int T, int k, int d,
                                                 void* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int vecs = d / 4;
  const int64_t total = static_cast<int64_t>(T) * vecs;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int t = (i >> 32) == 0 ? static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(vecs))
                                 : static_cast<int>(i / vecs);
    const int v = static_cast<int>(i - static_cast<int64_t>(t) * vecs);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // eight slots at a time: all their row indices and weights, then all
    // their rows of y, are in flight together; the sums stay in ascending j
    for (int j0 = 0; j0 < k; j0 += 8) {
      int r[8];
      float wt[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = j0 + j < k ? __ldg(slot_dst + static_cast<int64_t>(t) * k + j0 + j) : -1;
        wt[j] = j0 + j < k ? __ldg(w + static_cast<int64_t>(t) * k + j0 + j) : 0.f;
      }
      float4 yv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        yv[j] = r[j] >= 0 ? __ldg(reinterpret_cast<const float4*>(y + r[j] * ld_y) + v)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (r[j] < 0) continue;
        acc.x = fmaf(wt[j], yv[j].x, acc.x);
        acc.y = fmaf(wt[j], yv[j].y, acc.y);
        acc.z = fmaf(wt[j], yv[j].z, acc.z);
        acc.w = fmaf(wt[j], yv[j].w, acc.w);
      }
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z, acc.w);
    uint2 pk;
    pk.x = *reinterpret_cast<const uint32_t*>(&lo);
    pk.y = *reinterpret_cast<const uint32_t*>(&hi);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + static_cast<int64_t>(t) * d)[v] = pk;
  }
}

// out[i] = bf16_rne(in[i]): four elements per thread, grid-stride.
__global__ void __launch_bounds__(256) k_round_bf16(const float4* __restrict__ in, int64_t n4,
                                                    uint2* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n4;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const float4 a = __ldg(in + i);
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(a.z, a.w);
    uint2 pk;
    pk.x = *reinterpret_cast<const uint32_t*>(&lo);
    pk.y = *reinterpret_cast<const uint32_t*>(&hi);
    out[i] = pk;
  }
}

// The combine over a BFP16 y: a warp takes 256 consecutive features of a token,
// a lane eight of them, which are one exponent group of each routed row.  Per
// slot one 16-byte load of values and one exponent byte (BY_ROW: BFP16 by rows, one
// exponent word for four lanes), the loads of SLOTS
// slots in flight; the slot's power of two is folded into its weight (w * 2^s is
// exact), so each element costs a byte permute and, two elements at a time, an
// exact subtraction and a fused multiply-add into the fp32 sum (the same sum as
// decoding first), in ascending j; one bf16 rounding (or the fp32 sum of a
// shard's slots).  Resident warps count for more than slots in flight: eight at
// a time (80 registers) took 46.2 us for 2003 tokens of 6 slots and 7168
// features, six 40.7, four (64 registers) 39.7, three 38.1 (5.3 TB/s), two 41.2;
// for 8 slots four took 45.4 and three 49.7.  So three or four, whichever leaves
// fewer places empty in the last round.
template <int SLOTS, bool F32_OUT, bool BY_ROW>
__global__ void __launch_bounds__(256) k_combine_bfp16(const uint16_t* __restrict__ y,
                                                       const int8_t* __restrict__ y_exp,
                                                       int64_t ld_y, int64_t y_rows,
                                                       const int32_t* __restrict__ slot_dst,
                                                       const float* __restrict__ w, int T, int k,
                                                       int d, bool out16,
                                                       void* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int vecs = d / 8, lane = threadIdx.x & 31;
  const int per = (vecs + 31) / 32;  // warp tasks of a token
  const int64_t total = static_cast<int64_t>(T) * per;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const uint64_t bias = pack2(-12615680.f, -12615680.f);  // as in bfp16_offset_value
  for (int64_t i = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) >> 5; i < total;
       i += warps) {
    const int t = (i >> 32) == 0 ? static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(per))
                                 : static_cast<int>(i / per);
    const int v = static_cast<int>(i - static_cast<int64_t>(t) * per) * 32 + lane;
    if (v < vecs) {
      uint64_t acc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = 0;
      for (int j0 = 0; j0 < k; j0 += SLOTS) {
        int r[SLOTS];
        float wt[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          r[j] = -1;
          if (j0 + j >= k) continue;
          r[j] = __ldg(slot_dst + static_cast<int64_t>(t) * k + j0 + j);
          wt[j] = __ldg(w + static_cast<int64_t>(t) * k + j0 + j);
          if (r[j] >= y_rows) r[j] = -1;  // outside y: skipped like a -1 slot
        }
        uint4 qv[SLOTS];
        int sv[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          if (r[j] >= 0) {
            qv[j] = __ldg(reinterpret_cast<const uint4*>(y + r[j] * ld_y) + v);
            sv[j] = BY_ROW ? __ldg(reinterpret_cast<const uint16_t*>(y_exp) +
                                   r[j] * (ld_y / kRowGroup) + v / (kRowGroup / 8))
                           : __ldg(y_exp + (r[j] >> 4) * (ld_y / 8) + v);
          }
        }
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          if (r[j] < 0) continue;
          const uint32_t qw[4] = {qv[j].x, qv[j].y, qv[j].z, qv[j].w};
          const int s = BY_ROW ? bfp16_row_exponent(sv[j]) : sv[j];
          if (BY_ROW ? (sv[j] & kRowSpecial) != 0 : s == kBfp16NonFinite) {  // a group holding Inf or NaN
            auto value = [&](int e, bool hi) {
              return BY_ROW ? bfp16_special_decode(qw[e], hi, s) : bfp16_decode(qw[e], hi, s);
            };
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[e] = fma2(pack2(wt[j], wt[j]), pack2(value(e, false), value(e, true)), acc[e]);
            continue;
          }
          const float wp = wt[j] * bfp16_pow2(s);
          const uint64_t wp2 = pack2(wp, wp);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[e] = fma2(wp2,
                          add2(pack2(__uint_as_float(__byte_perm(qw[e], 0x4B40u, 0x5410u)),
                                    __uint_as_float(__byte_perm(qw[e], 0x4B40u, 0x5432u))),
                               bias),
                          acc[e]);
        }
      }
      if (F32_OUT) {  // the sum before its rounding (one shard's share of the output)
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + static_cast<int64_t>(t) * d + 8 * v);
        const float2 a0 = unpack2(acc[0]), a1 = unpack2(acc[1]), a2 = unpack2(acc[2]), a3 = unpack2(acc[3]);
        __stcs(o, make_float4(a0.x, a0.y, a1.x, a1.y));
        __stcs(o + 1, make_float4(a2.x, a2.y, a3.x, a3.y));
      } else {
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = unpack2(acc[e]);
          const __nv_bfloat162 b2 = __floats2bfloat162_rn(a.x, a.y);
          pk[e] = *reinterpret_cast<const uint32_t*>(&b2);
        }
        uint16_t* o = static_cast<uint16_t*>(out) + static_cast<int64_t>(t) * d + 8 * v;
        if (out16) {
          *reinterpret_cast<uint4*>(o) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        } else {
          reinterpret_cast<uint2*>(o)[0] = make_uint2(pk[0], pk[1]);
          reinterpret_cast<uint2*>(o)[1] = make_uint2(pk[2], pk[3]);
        }
      }
    }
  }
}

// Up to 16 resident blocks of 256 threads per SM, grid-stride beyond that.
static unsigned stream_blocks(int64_t tasks) {
  int64_t blocks = (tasks + 255) / 256;
  const int64_t cap = static_cast<int64_t>(num_sms()) * 16;
  return static_cast<unsigned>(blocks > cap ? cap : blocks);
}

cudaError_t launch_combine(const void* y, const int8_t* y_exp, int64_t ld_y, int64_t y_rows,
                           const int32_t* slot_dst, const float* w, int T, int k, int d,
                           void* out, bool out_f32, cudaStream_t stream, bool by_row) {
  if (y_exp) {
    if (T == 0) return cudaSuccess;
    const int vecs = d / 8;
    const dim3 grid(stream_blocks(static_cast<int64_t>(T) * ((vecs + 31) / 32) * 32));
    const uint16_t* yq = static_cast<const uint16_t*>(y);
    const bool out16 = reinterpret_cast<uintptr_t>(out) % 16 == 0;
    const bool threes = (k + 2) / 3 * 3 < (k + 3) / 4 * 4;
    if (by_row && out_f32) return cudaErrorInvalidValue;  // no shards of the MXFP4 forward
    auto kern = by_row    ? (threes ? k_combine_bfp16<3, false, true> : k_combine_bfp16<4, false, true>)
                : out_f32 ? (threes ? k_combine_bfp16<3, true, false> : k_combine_bfp16<4, true, false>)
                          : (threes ? k_combine_bfp16<3, false, false>
                                    : k_combine_bfp16<4, false, false>);
    return launch_pdl(kern, grid, dim3(256), 0, stream, yq, y_exp, ld_y, y_rows, slot_dst, w, T, k, d,
                      out16, out);
  }
  // an fp32 y (megamoe_combine) always gives the bf16 output
  if (out_f32) return cudaErrorInvalidValue;
  const int64_t tasks = static_cast<int64_t>(T) * (d / 4);
  if (tasks == 0) return cudaSuccess;
  const dim3 grid(stream_blocks(tasks));
  return launch_pdl(k_combine, grid, dim3(256), 0, stream, static_cast<const float*>(y), ld_y,
                    slot_dst, w, T, k, d, out);
}

cudaError_t launch_round_bf16(const float* in, int64_t n, uint16_t* out, cudaStream_t stream) {
  const int64_t n4 = n / 4;
  if (n4 == 0) return cudaSuccess;
  return launch_pdl(k_round_bf16, dim3(stream_blocks(n4)), dim3(256), 0, stream,
                    reinterpret_cast<const float4*>(in), n4, reinterpret_cast<uint2*>(out));
}

}  // namespace megamoe
