// Scored router: sigmoid or softmax scores of every expert, a balance bias
// that moves the choice but not the weights, groups of experts, top-k, and
// the gradient of the weights with respect to the logits.
//
//   s_e = 1 / (1 + exp(-l_e))           or exp(l_e - m) / sum_i exp(l_i - m), in
//                                       fp32 to a few units, subnormal ones too
//   c_e = s_e + bias_e                  (an fp32 add)
//   a group's score is the sum of its group_top (1 or 2) largest c; the
//   topk_group groups of highest score stay; the k experts of largest c among
//   them are taken in descending order; ties go to the lower index
//   w_j = scale * s_j / sum_i s_i       (renormalised) or scale * s_j
//
// An expert whose logit is NaN or -inf scores 0; neither it nor one whose c is NaN
// or -inf is ever taken; slots left over get id -1 and weight 0, which the forward
// skips.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace megamoe {

namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}

// One logit, or four on a 16-byte (bf16: 8-byte) boundary.
__device__ __forceinline__ void load_logits(const float* p, float (&v)[1]) { v[0] = __ldg(p); }
__device__ __forceinline__ void load_logits(const __nv_bfloat16* p, float (&v)[1]) {
  v[0] = __bfloat162float(*p);
}
__device__ __forceinline__ void load_logits(const float* p, float (&v)[4]) {
  const float4 q = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
__device__ __forceinline__ void load_logits(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
  v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
  v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
}

// NaN -> -inf, +inf -> the largest float (so that exp(l - m) has a limit).
__device__ __forceinline__ float clean_logit(float l) {
  return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY;
}

// 1 / d for d in [1, 2]: the hardware's reciprocal, off by up to one unit, and a
// step of Newton's method, which leaves it within 2^-22 units of half a unit, so the
// order of two different d is kept.  (16384 tokens of 384 logits took 16.6 us with it,
// 18.7 with a correctly rounded reciprocal called for each score.)
__device__ __forceinline__ float reciprocal(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return __fmaf_rn(r, __fmaf_rn(-d, r, 1.f), r);
}

// The exponential is taken of -|l|, so that neither end overflows: a negative
// logit's score keeps its bits down to the subnormal numbers.
__device__ __forceinline__ float sigmoid(float l) {
  const float e = expf(-fabsf(l)), r = reciprocal(1.f + e);
  return l >= 0.f ? r : e * r;
}
// 1 - s, whose bits 1 - (s rounded) would lose.
__device__ __forceinline__ float sigmoid_rest(float l) { return sigmoid(-l); }

// Unsigned key in the order of the floats above -inf; 0 marks what cannot be taken.
__device__ __forceinline__ uint32_t order_key(float c) {
  if (!(c > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(c);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

constexpr int kWarps = 4;  // tokens per block

// The experts that a lane holds: of its group, V consecutive ones at a time,
// the group's lanes side by side.
template <int V>
__device__ __forceinline__ int lane_expert(int i, int sub, int lanes) {
  return (i / V * lanes + sub) * V + i % V;
}

// One warp per token, everything in registers.  The 32 lanes are cut into one
// run of `lanes` (a power of two) per group of experts, so a group's two largest
// scores are a shuffle reduction within its run, and dropping a group empties
// its lanes.  The choice:
//   - the k-th largest of the lanes' largest scores is a lower bound of the
//     k-th largest score (k lanes have one at least as large), found by k warp
//     maxima;
//   - the scores from the bound on, few more than k, go to shared memory, one
//     for each lane, and each lane counts those before its own (a larger score,
//     or an equal one at a lower index): its slot.
// More than 32 of them (ties) are taken one by one.  The work per token bounds
// this kernel, not its bytes: 16384 tokens of 384 fp32 logits in 8 groups, top-6,
// take 16.8 us (1.5 TB/s, 77 % of the issue slots); with the scores by the hardware's exponential alone, off
// by up to 2^-18 and none below the smallest normal number, 14.5, and then with all
// of the k taken by warp maxima 30.2.  One token takes 3.9 us, a launch's latency.
template <typename L, int NV, int V>
__global__ void __launch_bounds__(kWarps * 32)
    k_scored_router(const L* __restrict__ logits, int64_t T, int E, int64_t ld,
                    const float* __restrict__ bias, int softmax, int n_group, int lanes,
                    int topk_group, int group_top, int k, int renormalize, float scale,
                    int32_t* __restrict__ ids, float* __restrict__ weights) {
  __shared__ float2 s_taken[kWarps][32];  // score, expert (as bits)
  __shared__ int s_count[kWarps], s_id[kWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (t >= T) return;  // warp-uniform
  const L* row = logits + t * ld;
  const int size = E / n_group;
  const int group = lane / lanes, sub = lane & (lanes - 1);
  const int first = group * size;
  const int mine = group < n_group ? size : 0;  // experts within reach of this lane

  float c[NV];
#pragma unroll
  for (int i = 0; i < NV; i += V) {
    const int j = lane_expert<V>(i, sub, lanes);
    float v[V];
#pragma unroll
    for (int u = 0; u < V; ++u) v[u] = -INFINITY;
    if (j < mine) load_logits(row + first + j, v);
#pragma unroll
    for (int u = 0; u < V; ++u) c[i + u] = v[u];
  }
  float top = 0.f, total = 1.f;  // softmax: the largest logit, the sum of exp(l - top)
  if (softmax) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = clean_logit(c[i]);
      top = fmaxf(top, c[i]);
    }
    top = warp_max(top);
    if (top == -INFINITY) top = 0.f;  // no expert: every exp is 0
    total = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float e = expf(c[i] - top);
      total += e;
      c[i] = c[i] > -INFINITY ? e : -INFINITY;
    }
    total = warp_sum(total);
    const float inverse = total > 0.f ? __frcp_rn(total) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = c[i] > -INFINITY ? c[i] * inverse : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)  // NaN becomes -inf: not taken
      c[i] = c[i] > -INFINITY ? sigmoid(c[i]) : -INFINITY;
  }
  // scores plus bias; -inf: cannot be taken
  if (bias) {
#pragma unroll
    for (int i = 0; i < NV; i += V) {
      const int j = lane_expert<V>(i, sub, lanes);
      float b[V];
#pragma unroll
      for (int u = 0; u < V; ++u) b[u] = 0.f;
      if (j < mine) load_logits(bias + first + j, b);
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const float v = c[i + u] + b[u];
        c[i + u] = v > -INFINITY ? v : -INFINITY;  // NaN too
      }
    }
  }
  if (lane == 0) s_count[warp] = 0;
  if (n_group > 1) {
    float a = -INFINITY, b = -INFINITY;  // the group's two largest
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      b = fmaxf(b, fminf(a, c[i]));
      a = fmaxf(a, c[i]);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      const float oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
      b = fmaxf(fmaxf(b, ob), fminf(a, oa));
      a = fmaxf(a, oa);
    }
    const float g = group_top == 2 && b > -INFINITY ? __fadd_rn(a, b) : a;
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < n_group; ++o) {
      const float og = __shfl_sync(kAll, g, o * lanes);
      rank += og > g || (og == g && o < group);
    }
    if (rank >= topk_group) {
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] = -INFINITY;
    }
  }
  float most = c[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) most = fmaxf(most, c[i]);
  uint32_t key = order_key(most), bound = 0u;
  for (int j = 0; j < k; ++j) {
    bound = __reduce_max_sync(kAll, key);
    if (bound == 0u) break;  // fewer than k lanes have any
    if (key == bound) key = 0u;
  }
  const float least = bound == 0u ? -FLT_MAX : key_value(bound);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (c[i] >= least) {  // in any order: their slots do not depend on it
      const int at = atomicAdd(&s_count[warp], 1);
      if (at < 32)
        s_taken[warp][at] =
            make_float2(c[i], __int_as_float(first + lane_expert<V>(i, sub, lanes)));
    }
  }
  __syncwarp();
  const int n = s_count[warp];
  int my_id = -1;
  if (n <= 32) {
    const float2 own = s_taken[warp][min(lane, max(n - 1, 0))];
    const int e = __float_as_int(own.y);
    int slot = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float2 o = s_taken[warp][j];
      slot += o.x > own.x || (o.x == own.x && __float_as_int(o.y) < e);
    }
    if (lane < n) s_id[warp][slot] = e;
    __syncwarp();
    if (lane < min(k, n)) my_id = s_id[warp][lane];
  } else {
    for (int j = 0; j < k; ++j) {
      float best = -INFINITY;
      int e = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (c[i] > best) {  // experts ascend with i: the first of equals stays
          best = c[i];
          e = first + lane_expert<V>(i, sub, lanes);
        }
      }
      const uint32_t mk = order_key(best), m = __reduce_max_sync(kAll, mk);
      if (m == 0u) break;  // nothing left to take
      const int won = __reduce_min_sync(kAll, mk == m ? e : 0x7fffffff);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (first + lane_expert<V>(i, sub, lanes) == won && mine) c[i] = -INFINITY;
      if (lane == j) my_id = won;
    }
  }
  float w = 0.f;
  const float l = my_id >= 0 ? clean_logit(load_logit(row + my_id)) : -INFINITY;
  if (softmax && renormalize) {  // shares of the taken: the sum over all experts cancels
    const float most = warp_max(l);
    w = my_id >= 0 ? expf(l - most) : 0.f;
  } else if (my_id >= 0) {
    w = softmax ? __fdiv_rn(expf(l - top), total) : sigmoid(l);
  }
  if (renormalize) {
    const float sum = warp_sum(w);
    w = sum > 0.f ? __fdiv_rn(w, sum) : 0.f;
  }
  if (lane < k) {
    ids[t * k + lane] = my_id;
    weights[t * k + lane] = w * scale;
  }
}

__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Gradient, one warp per token.  With g_j = scale * dL/dw_j, p_j = s_j / sum s
// over the taken experts:
//   sigmoid, renormalised  dl_j = p_j (1 - s_j) (g_j - sum_i g_i p_i)
//   softmax, renormalised  dl_j = p_j (g_j - sum_i g_i p_i)  (the softmax's own
//                          sum cancels)
//   sigmoid                dl_j = g_j s_j (1 - s_j)
//   softmax                dl_e = s_e (g_e - sum_i g_i s_i) for every expert
// In the first three only the taken experts have a gradient and only their
// logits are read: the row is filled with zeros and the k values stored over
// them after a warp barrier.  Bound by those stores: 16384 tokens of 384 experts
// 6.2 us (25 MB written, 4.1 TB/s, most of it into L2; 10 MB of logits read).
template <typename L>
__global__ void __launch_bounds__(kWarps * 32)
    k_scored_router_backward(const L* __restrict__ logits, int64_t T, int E, int64_t ld,
                             const int32_t* __restrict__ ids, const float* __restrict__ grad,
                             int softmax, int k, int renormalize, float scale,
                             L* __restrict__ out, int64_t ld_out, int vectors) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= T) return;  // warp-uniform
  const L* row = logits + t * ld;
  L* orow = out + t * ld_out;
  int id = lane < k ? __ldg(ids + t * k + lane) : -1;
  if (id >= E) id = -1;
  const float g = id >= 0 ? __ldg(grad + t * k + lane) * scale : 0.f;
  const float l = id >= 0 ? clean_logit(load_logit(row + id)) : -INFINITY;
  const bool dense = softmax && !renormalize;
  float dl, dot = 0.f, top = 0.f, total = 1.f;
  if (dense) {
    top = -INFINITY;
    for (int e = lane; e < E; e += 32) top = fmaxf(top, clean_logit(load_logit(row + e)));
    top = warp_max(top);
    if (top == -INFINITY) top = 0.f;
    float sum = 0.f;
    for (int e = lane; e < E; e += 32) sum += expf(clean_logit(load_logit(row + e)) - top);
    total = warp_sum(sum);
    const float s = total > 0.f ? __fdiv_rn(expf(l - top), total) : 0.f;
    dot = warp_sum(g * s);
    dl = s * (g - dot);
  } else if (renormalize) {
    // softmax: the shares of the taken experts need only their own largest logit
    if (softmax) {
      top = warp_max(l);
      if (top == -INFINITY) top = 0.f;
    }
    const float s = softmax ? expf(l - top) : sigmoid(l);
    const float sum = warp_sum(s);
    const float p = sum > 0.f ? __fdiv_rn(s, sum) : 0.f;
    dl = p * (g - warp_sum(g * p));
    if (!softmax) dl *= sigmoid_rest(l);
  } else {
    dl = g * sigmoid(l) * sigmoid_rest(l);
  }
  if (dense) {
    for (int e = lane; e < E; e += 32) {
      const float s = __fdiv_rn(expf(clean_logit(load_logit(row + e)) - top), total);
      store_grad(orow + e, total > 0.f ? -s * dot : 0.f);
    }
  } else if (vectors) {  // rows start on 16-byte boundaries
    constexpr int per = 16 / sizeof(L);
    const int n = E / per;
    for (int v = lane; v < n; v += 32)
      reinterpret_cast<uint4*>(orow)[v] = make_uint4(0u, 0u, 0u, 0u);
    for (int e = n * per + lane; e < E; e += 32) store_grad(orow + e, 0.f);
  } else {
    for (int e = lane; e < E; e += 32) store_grad(orow + e, 0.f);
  }
  __syncwarp();
  if (id >= 0) store_grad(orow + id, dl);
}

template <typename L>
cudaError_t launch_router_typed(const ScoredRouter& r, cudaStream_t stream) {
  int runs = 1;  // groups, up to a power of two
  while (runs < r.n_group) runs *= 2;
  const int lanes = 32 / runs, size = r.E / r.n_group;
  const dim3 grid(static_cast<unsigned>((r.T + kWarps - 1) / kWarps)), block(kWarps * 32);
  auto run = [&](auto kern) {
    return launch_pdl(kern, grid, block, 0, stream, static_cast<const L*>(r.logits), r.T, r.E, r.ld,
                      r.bias, r.softmax, r.n_group, lanes, r.topk_group, r.group_top, r.k,
                      r.renormalize, r.scale, r.ids, r.weights);
  };
  // four experts a load where groups, rows and pointers are whole fours
  const bool fours = size % 4 == 0 && r.ld % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(r.logits) % (4 * sizeof(L)) == 0 &&
                     reinterpret_cast<uintptr_t>(r.bias) % 16 == 0;
  if (fours) {
    const int per_lane = (size + 4 * lanes - 1) / (4 * lanes) * 4;
    if (per_lane <= 4) return run(k_scored_router<L, 4, 4>);
    if (per_lane <= 8) return run(k_scored_router<L, 8, 4>);
    if (per_lane <= 12) return run(k_scored_router<L, 12, 4>);
    if (per_lane <= 16) return run(k_scored_router<L, 16, 4>);
    if (per_lane <= 32) return run(k_scored_router<L, 32, 4>);
    return run(k_scored_router<L, 64, 4>);
  }
  const int per_lane = (size + lanes - 1) / lanes;
  if (per_lane <= 4) return run(k_scored_router<L, 4, 1>);
  if (per_lane <= 12) return run(k_scored_router<L, 12, 1>);
  if (per_lane <= 32) return run(k_scored_router<L, 32, 1>);
  return run(k_scored_router<L, 64, 1>);
}

template <typename L>
cudaError_t launch_backward_typed(const ScoredRouter& r, const float* grad, void* out,
                                  int64_t ld_out, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((r.T + kWarps - 1) / kWarps)), block(kWarps * 32);
  const int vectors = reinterpret_cast<uintptr_t>(out) % 16 == 0 && ld_out * sizeof(L) % 16 == 0;
  return launch_pdl(k_scored_router_backward<L>, grid, block, 0, stream,
                    static_cast<const L*>(r.logits), r.T, r.E, r.ld,
                    static_cast<const int32_t*>(r.ids), grad, r.softmax, r.k, r.renormalize,
                    r.scale, static_cast<L*>(out), ld_out, vectors);
}

}  // namespace

cudaError_t launch_scored_router(const ScoredRouter& r, cudaStream_t stream) {
  if (r.T == 0) return cudaSuccess;
  return r.bf16 ? launch_router_typed<__nv_bfloat16>(r, stream)
                : launch_router_typed<float>(r, stream);
}

cudaError_t launch_scored_router_backward(const ScoredRouter& r, const float* grad, void* out,
                                          int64_t ld_out, cudaStream_t stream) {
  if (r.T == 0) return cudaSuccess;
  return r.bf16 ? launch_backward_typed<__nv_bfloat16>(r, grad, out, ld_out, stream)
                : launch_backward_typed<float>(r, grad, out, ld_out, stream);
}

}  // namespace megamoe
