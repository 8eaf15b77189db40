// MXFP4 linear for up to 32 tokens in one launch, without a workspace.
//
//   out[t, n] = sum_k MXFP4(x)[t, k] w[n, k]
//
// What such a call has to do is stream the weights once; at these sizes that
// takes a few microseconds, as long as a launch or two.  So nothing runs before
// the product: the weights are the MMA's M side (128 features a CTA), their
// loads start at once, and while they are on their way each CTA quantises its
// own part of x (T tokens x its K range) straight into the swizzled operand
// tile and scale atoms that the MMA reads.  A cluster of up to eight CTAs shares
// a tile's K range; each leaves its fp32 partial sums in its shared memory and
// sums its share of the features over the cluster in rank order, so results do
// not depend on timing and no counter or partial plane in global memory is
// needed.
//
// Roles (256 threads): warp 0 producer of the weights' codes and scale atoms,
// warp 1 tensor-memory allocator and MMA issuer, warps 2..7 quantise x, warps
// 4..7 then drain the accumulator.
//
// 7168 -> 1536 (5.8 MB of weights, 0.9 us at the copy's bandwidth): 4.7 us at one
// token, 7.4 at 16, against 12.4 as three launches (status, quantiser, product);
// 1536 -> 24576 (20 MB, 3.0 us): 4.5 us at one token.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "mxfp4.cuh"

namespace megamoe {

namespace {

constexpr int kThreads = 256;
constexpr int kStages = 4;
constexpr int kSf = 1024;                   // scale atoms of 128 rows and a K step
constexpr int kStage = 128 * 128 + kSf;     // weights of a K step
constexpr int kMaxCluster = 8;
constexpr unsigned kAll = 0xffffffffu;

struct FewArgs {
  const void* x;
  int64_t ld_x;
  int T, K, N;
  const uint8_t* w_sf;  // atom layout
  void* out;
  int64_t ld_out;
  int cluster;
  uint32_t* status;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Bytes of a K step of x: BN rows of codes and two scale atoms.
template <int BN>
constexpr int kXStep = BN * 128 + kSf;

__device__ __forceinline__ float load_cluster(const float* p, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}

template <typename X, typename O, int BN>
__global__ void __launch_bounds__(kThreads) k_mx_linear_few(const __grid_constant__ CUtensorMap codes,
                                                            const FewArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kStages], empty[kStages], x_ready, acc_full;
  __shared__ uint32_t tmem_holder;
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;
  uint8_t* s_x = smem + kStages * kStage;  // [steps][kXStep]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.cluster;
  const int rank = S > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int mt = blockIdx.x / S;
  const int KT = (p.K + 255) / 256;
  const int k0 = rank * KT / S, k1 = (rank + 1) * KT / S;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&x_ready, 6);
    mbar_init(&acc_full, 1);
    s_abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&codes);
  }
  constexpr int cols = 64;  // 32 of accumulator, two sets of 16 of scales
  if (warp == 1) {
    tmem_alloc(&tmem_holder, cols);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_sync();  // the status word is clear before any rank sets it
  tc_fence_after();
  const uint32_t tmem = tmem_holder;

  if (warp == 0) {
    {
      // ------------------------------------------------ producer of the weights
      // (the whole warp, one lane of it issuing: elect_one)
      const bool leader = elect_one();
      const uint64_t pol = policy_evict_first();
      const uint8_t* sf = p.w_sf + mt * mx_atoms(p.K) * 512;
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int kt = k0; kt < k1; ++kt) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) break;
        uint8_t* sb = smem + stage * kStage;
        if (leader) {
          mbar_arrive_expect_tx(&full[stage], kStage);
          tma_load_2d(sb, &codes, &full[stage], kt * 128, mt * 128, pol);
          bulk_load(sb + 128 * 128, sf + static_cast<int64_t>(kt) * kSf, kSf, &full[stage], pol);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      drain_copies(full, kStages, issued);
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    const bool leader = elect_one();
    const uint64_t wd = sdesc_sw128(smem_u32(smem)), ws = sdesc_atom(smem_u32(smem) + 128 * 128);
    const uint64_t xd = sdesc_sw128(smem_u32(s_x)), xs = sdesc_atom(smem_u32(s_x) + BN * 128);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = mbar_wait(&x_ready, 0, abort_flag, p.status, p.wait_limit_ns);
    for (int kt = k0; ok && kt < k1; ++kt) {
      ok = mbar_wait(&full[stage], phase, abort_flag, p.status, p.wait_limit_ns);
      if (!ok) break;
      tc_fence_after();
      const int s = kt - k0;
      const uint32_t sf = tmem + 32 + 16 * (s & 1);
      const uint64_t wc = sdesc_at(wd, stage * kStage), wa = sdesc_at(ws, stage * kStage);
      const uint64_t xc = sdesc_at(xd, s * kXStep<BN>), xa = sdesc_at(xs, s * kXStep<BN>);
      if (leader) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tc_copy_atom(sf + 4 * h, sdesc_at(wa, 512 * h));
          tc_copy_atom(sf + 8 + 4 * h, sdesc_at(xa, 512 * h));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mma_mxf4(tmem, sdesc_at(wc, 32 * c), sdesc_at(xc, 32 * c), idesc_mxf4(128, BN, c & 1),
                   sf + 4 * (c >> 1), sf + 8 + 4 * (c >> 1), (s != 0 || c != 0) ? 1u : 0u);
        tc_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // also on the way out: every MMA issued so far finishes before tensor
    // memory is released
    if (leader) tc_commit(&acc_full);
    __syncwarp();
    mbar_drain(&acc_full, 0);
  } else {
    // ------------------------------------------------------ x into the operand
    const X* x = static_cast<const X*>(p.x);
    const int per = (k1 - k0) * 32;  // groups of eight elements in a row's part
    bool bad = false;
    constexpr int batch = 8;  // loads in flight
    for (int i0 = threadIdx.x - 64; i0 < p.T * per; i0 += batch * (kThreads - 64)) {  // whole warps
      Eight<X> v8[batch];
#pragma unroll
      for (int j = 0; j < batch; ++j) {
        const int i = i0 + j * (kThreads - 64);
        const int t = i / per, col = k0 * 256 + 8 * (i - t * per);
        if (t < p.T && col < p.K) v8[j].load(x + t * p.ld_x + col);
        else v8[j].clear();
      }
#pragma unroll
      for (int j = 0; j < batch; ++j) {
        const int i = i0 + j * (kThreads - 64);
        const int t = i / per, e = i - t * per;
        if (t >= p.T) break;  // warp-uniform
        uint32_t m = v8[j].widest();  // four lanes share a block
        m = Eight<X>::wider(m, __shfl_xor_sync(kAll, m, 1));
        m = Eight<X>::wider(m, __shfl_xor_sync(kAll, m, 2));
        const uint32_t byte = mx_scale_byte(Eight<X>::bits(m));
        float v[8];
        v8[j].values(v);
        uint8_t* step = s_x + (e >> 5) * kXStep<BN>;
        const int g = e & 31;  // group of the K step: 4 bytes of a 128-byte row
        *reinterpret_cast<uint32_t*>(step + (t >> 3) * 1024 + (t & 7) * 128 +
                                     (((g >> 2) ^ (t & 7)) * 16) + (g & 3) * 4) =
            mx_codes8(v, mx_inverse(byte));
        if ((g & 3) == 0)
          step[BN * 128 + (g >> 4) * 512 + t * 16 + (g >> 2 & 3)] = static_cast<uint8_t>(byte);
        bad |= byte == kMxNan;
      }
    }
    if (bad && mt == 0) set_status(p.status, MEGAMOE_DEV_NONFINITE);
    fence_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&x_ready);
  }

  // ----------------------------------------------------------------- epilogue
  // fp32 partial sums [BN][128]; the weights' stages are free by then
  float* part = reinterpret_cast<float*>(smem);
  bool done = true;
  if (warp >= 4) {
    done = mbar_wait(&acc_full, 0, abort_flag, p.status, p.wait_limit_ns);
    tc_fence_after();
    const int quarter = warp & 3, row = quarter * 32 + lane, n = mt * 128 + row;
#pragma unroll
    for (int c = 0; c < BN; c += 16) {
      uint32_t u[16];
      tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, u);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (S > 1) {
          if (c + j < p.T) part[(c + j) * 128 + row] = __uint_as_float(u[j]);
        } else if (done && c + j < p.T && n < p.N) {
          put(static_cast<O*>(p.out) + (c + j) * p.ld_out + n, __uint_as_float(u[j]));
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (S > 1) {
    cluster_sync();
    // this CTA's share of the features, each summed over the ranks in order
    const int share = 128 / S;
    for (int i = threadIdx.x; i < p.T * share; i += kThreads) {
      const int t = i / share, row = rank * share + i % share, n = mt * 128 + row;
      float sum = 0.f;
      for (int r = 0; r < S; ++r) sum += load_cluster(part + t * 128 + row, r);
      if (n < p.N) put(static_cast<O*>(p.out) + t * p.ld_out + n, sum);
    }
    cluster_sync();  // no CTA leaves while another reads its sums
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }
}

// CTAs of a cluster, where SMs would idle: a K step of weights and of x's
// quantisation (dearer with more tokens) against a cluster's start and sums,
// about three and a half steps.  Measured (us, 1 / 2 / 4 / 8 CTAs) at one token:
// 7168 -> 1536 9.0 / 7.1 / 5.6 / 4.7; 1024 -> 1024 3.3 / 4.0 / 3.8; more CTAs than
// SMs: 1536 -> 24576 4.5 / 9.0 / 14.0.
int few_cluster(int64_t T, int64_t N, int64_t K) {
  const int64_t mt = (N + 127) / 128, steps = (K + 255) / 256;
  const double step = 1.0 + static_cast<double>(T) / 8;
  int best = 1;
  double least = step * steps;
  for (int s = 2; s <= kMaxCluster && s <= steps && mt * s <= num_sms(); s *= 2) {
    const double cost = step * steps / s + 3.5;
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

int few_bytes(int bn, int64_t K, int cluster) {
  const int64_t steps = (K + 255) / 256;
  const int64_t bytes = 1024 + kStages * kStage + (steps + cluster - 1) / cluster * (bn * 128 + kSf);
  return static_cast<int>(std::min<int64_t>(bytes, int64_t{1} << 30));
}

template <typename X, typename O, int BN>
cudaError_t launch_few(const FewArgs& a, const uint8_t* w_codes, cudaStream_t stream) {
  CUtensorMap codes;
  if (!make_codes_map(&codes, w_codes, a.N, static_cast<uint64_t>(a.K) / 2, 128))
    return cudaErrorInvalidValue;
  auto kern = k_mx_linear_few<X, O, BN>;
  const int smem = few_bytes(BN, a.K, a.cluster);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kern, dim3(static_cast<unsigned>((a.N + 127) / 128 * a.cluster)),
                            dim3(kThreads), smem, a.cluster, stream, codes, a);
}

template <typename X>
cudaError_t launch_typed(const FewArgs& a, const uint8_t* w_codes, bool f32, cudaStream_t stream) {
  if (a.T <= 16)
    return f32 ? launch_few<X, float, 16>(a, w_codes, stream)
               : launch_few<X, __nv_bfloat16, 16>(a, w_codes, stream);
  return f32 ? launch_few<X, float, 32>(a, w_codes, stream)
             : launch_few<X, __nv_bfloat16, 32>(a, w_codes, stream);
}

}  // namespace

// Each CTA quantises the part of x that it needs: T tokens by its q K steps.
// Beyond T = 3.6 + 40 / q, quantising once in a kernel before the product is
// faster.  Measured (this form / that form, us): 7168 -> 1536 (q = 4) at 12 tokens
// 6.3 / 7.2, at 17 7.8 / 7.2; 1536 -> 24576 (q = 6) at 12 8.1 / 8.6, at 17 10.7 / 8.6;
// 7168 -> 16384 (q = 28) at 4 16.2 / 16.9, at 8 20.3 / 16.9; 2048 -> 7168 (q = 4) at
// 12 6.5 / 7.1, at 16 7.7 / 7.1.
bool mx_linear_few_fits(int64_t T, int64_t K, int64_t N) {
  if (T > 32) return false;
  const int64_t steps = (K + 255) / 256;
  const int cluster = few_cluster(T, N, K);
  const int64_t q = (steps + cluster - 1) / cluster;
  return static_cast<double>(T) <= 3.6 + 40.0 / static_cast<double>(q) &&
         few_bytes(T <= 16 ? 16 : 32, K, cluster) <= 226 * 1024;
}

cudaError_t launch_mx_linear_few(const void* x, int x_type, int64_t T, int K, int64_t ld_x,
                                 const uint8_t* codes, const uint8_t* scales, int N, void* out,
                                 bool out_f32, int64_t ld_out, uint32_t* status,
                                 cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const FewArgs a{x,   ld_x,   static_cast<int>(T),  K,      N,
                  scales, out, ld_out, few_cluster(T, N, K), status, wait_limit_ns()};
  switch (x_type) {
    case MEGAMOE_TYPE_BF16: return launch_typed<__nv_bfloat16>(a, codes, out_f32, stream);
    case MEGAMOE_TYPE_F16: return launch_typed<__half>(a, codes, out_f32, stream);
    default: return launch_typed<float>(a, codes, out_f32, stream);
  }
}

}  // namespace megamoe
