// Scored router: sigmoid or softmax scores of every expert, a balance bias
// that moves the choice but not the weights, groups of experts, top-k, and
// the gradient of the weights with respect to the logits.
//
//   s_e = 1 / (1 + exp(-l_e))           or exp(l_e - m) / sum_i exp(l_i - m)
//   c_e = s_e + bias_e                  (an fp32 add)
//   a group's score is the sum of its group_top (1 or 2) largest c; the
//   topk_group groups of highest score stay; the k experts of largest c among
//   them are taken in descending order; ties go to the lower index
//   w_j = scale * s_j / sum_i s_i       (renormalised) or scale * s_j
//
// An expert whose logit is NaN or -inf, or whose c is, scores 0 and is never
// taken; slots left over get id -1 and weight 0, which the forward skips.
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

// NaN -> -inf, +inf -> the largest float (so that exp(l - m) has a limit).
__device__ __forceinline__ float clean_logit(float l) {
  return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY;
}

__device__ __forceinline__ float sigmoid(float l) { return __fdiv_rn(1.f, 1.f + expf(-l)); }

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

// One warp per token, everything in registers.  The 32 lanes are cut into one
// run of lanes_per_group (a power of two) per group of experts; a lane holds
// experts sub, sub + lanes_per_group, ... of its group (at most NV), so a
// group's two largest scores are a shuffle reduction within its run, and
// dropping a group empties its lanes.  A round of the top-k is two warp
// reductions: the largest key, then the lowest expert that has it.
template <typename L, int NV>
__global__ void __launch_bounds__(kWarps * 32)
    k_scored_router(const L* __restrict__ logits, int64_t T, int E, int64_t ld,
                    const float* __restrict__ bias, int softmax, int n_group, int lanes_per_group,
                    int topk_group, int group_top, int k, int renormalize, float scale,
                    int32_t* __restrict__ ids, float* __restrict__ weights) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= T) return;  // warp-uniform
  const L* row = logits + t * ld;
  const int size = E / n_group;
  const int group = lane / lanes_per_group, sub = lane & (lanes_per_group - 1);
  const bool mine = group < n_group;
  const int first = group * size;

  float c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = sub + i * lanes_per_group;
    c[i] = mine && j < size ? clean_logit(load_logit(row + first + j)) : -INFINITY;
  }
  float top = 0.f, total = 1.f;  // softmax: the largest logit, the sum of exp(l - top)
  if (softmax) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, c[i]);
    top = warp_max(top);
    if (top == -INFINITY) top = 0.f;  // no expert: every exp is 0
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) sum += expf(c[i] - top);
    total = warp_sum(sum);
  }
  auto score = [&](float l) {
    if (!softmax) return sigmoid(l);
    return total > 0.f ? __fdiv_rn(expf(l - top), total) : 0.f;
  };
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = sub + i * lanes_per_group;
    key[i] = 0u;
    if (c[i] > -INFINITY) {
      const float s = score(c[i]);
      key[i] = order_key(bias ? __fadd_rn(s, __ldg(bias + first + j)) : s);
    }
  }
  if (n_group > 1) {
    uint32_t a = 0u, b = 0u;  // the group's two largest keys
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      b = max(b, min(a, key[i]));
      a = max(a, key[i]);
    }
    for (int o = lanes_per_group >> 1; o > 0; o >>= 1) {
      const uint32_t oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
      b = max(max(b, ob), min(a, oa));
      a = max(a, oa);
    }
    uint32_t g = a;  // the group's score as a key
    if (group_top == 2 && b != 0u) g = order_key(__fadd_rn(key_value(a), key_value(b)));
    // rank among the groups (before it: a higher score, or an equal one at a
    // lower index); 0 keys (nothing to take) count as lowest
    int rank = 0;
    for (int o = 0; o < n_group; ++o) {
      const uint32_t og = __shfl_sync(kAll, g, o * lanes_per_group);
      rank += og > g || (og == g && o < group);
    }
    if (rank >= topk_group) {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = 0u;
    }
  }
  int my_id = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (key[i] > best) {  // experts ascend with i: the first of equals stays
        best = key[i];
        at = i;
      }
    }
    const uint32_t m = __reduce_max_sync(kAll, best);
    if (m == 0u) break;  // nothing left to take
    const int e = best == m ? first + sub + at * lanes_per_group : 0x7fffffff;
    const int won = __reduce_min_sync(kAll, e);
    if (e == won) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == at) key[i] = 0u;
    }
    if (lane == j) my_id = won;
  }
  float w = my_id >= 0 ? score(clean_logit(load_logit(row + my_id))) : 0.f;
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
// them after a warp barrier.
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
    if (!softmax) dl *= 1.f - s;
  } else {
    const float s = sigmoid(l);
    dl = g * s * (1.f - s);
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
  const int lanes = 32 / runs;
  const int per_lane = (r.E / r.n_group + lanes - 1) / lanes;
  const dim3 grid(static_cast<unsigned>((r.T + kWarps - 1) / kWarps)), block(kWarps * 32);
  auto run = [&](auto kern) {
    return launch_pdl(kern, grid, block, 0, stream, static_cast<const L*>(r.logits), r.T, r.E, r.ld,
                      r.bias, r.softmax, r.n_group, lanes, r.topk_group, r.group_top, r.k,
                      r.renormalize, r.scale, r.ids, r.weights);
  };
  if (per_lane <= 4) return run(k_scored_router<L, 4>);
  if (per_lane <= 8) return run(k_scored_router<L, 8>);
  if (per_lane <= 12) return run(k_scored_router<L, 12>);
  if (per_lane <= 16) return run(k_scored_router<L, 16>);
  if (per_lane <= 32) return run(k_scored_router<L, 32>);
  return run(k_scored_router<L, 64>);
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
