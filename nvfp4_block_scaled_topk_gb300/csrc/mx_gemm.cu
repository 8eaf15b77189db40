// MXFP4 product of two row-major matrices on tcgen05 tensor cores:
//   out[r, c] = sum_k P[r, k] Q[c, k]
// with E2M1 codes [rows, K / 2], one E8M0 scale per 32 elements along K (atom
// layout), fp32 accumulation in tensor memory (tcgen05.mma kind::mxf4,
// scale_vec::2X).  The linear's forward product and both of its gradients are
// this product of quantised operands.
//
// A tile is 128 rows of the M-side operand x BN rows of the N-side one.  The
// larger of few rows (tokens of a decode step) goes on N: the weights' rows
// are then M, and the tile is stored transposed.
//
// Roles (448 threads, one CTA per SM): warp 0 producer (codes by tensor map in
// the 128-byte swizzle, scale atoms by bulk copy), warp 1 tensor-memory
// allocator and MMA issuer, warps 6..9 scale writers (each moves a stage's
// scales into its own 32-lane quarter of tensor memory), warps 2..5 and
// 10..13 epilogue (two per quarter, half of the columns each).
//
// K beyond the matrix's end within the last step of 256: the tensor map fills
// codes with zeros, and the atom layout holds zero scales there.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "mxfp4.cuh"

namespace megamoe {

namespace {

struct MxGemmArgs {
  const uint8_t* m_sf;  // atom layouts of the two operands
  const uint8_t* n_sf;
  void* out;
  int64_t ld_out;
  int M, N, K;
  int transposed;  // out[n, m] instead of out[m, n]
  int ksplit;      // pieces of a tile's K range
  float* partial;  // [tiles][ksplit][BN][128] when split
  uint32_t* counters;  // [tiles][kEpiWarps], zero before the launch
  uint32_t* status;
  uint64_t wait_limit_ns;
};

struct MxMaps {
  CUtensorMap m, n;
};

template <int BN, int STAGES>
struct MxCfg {
  static constexpr int M_TILE = 128 * 128;
  static constexpr int N_TILE = BN * 128;
  static constexpr int GROUPS = BN > 128 ? BN / 128 : 1;  // 128-row scale groups of N
  static constexpr int SF = 1024;                         // a group's atoms of one K step
  static constexpr int OFF_N = M_TILE;
  static constexpr int OFF_SFM = OFF_N + N_TILE;
  static constexpr int OFF_SFN = OFF_SFM + SF;
  static constexpr int STAGE = OFF_SFN + GROUPS * SF;
  static constexpr uint32_t TX = M_TILE + N_TILE;
  static constexpr uint32_t SF_TX = SF + GROUPS * SF;
  // scale columns of a stage: 4 per 128 of K for M, BN / 32 (at least 4) for N
  static constexpr int SFN_COLS = BN / 32 > 4 ? BN / 32 : 4;
  static constexpr int SF_COLS = 2 * 4 + 2 * SFN_COLS;
  static constexpr int ACC_SLOTS = 2 * BN + STAGES * SF_COLS <= 512 ? 2 : 1;
  static constexpr int SF_COL0 = ACC_SLOTS * BN;
  static constexpr int BAR_OFF = STAGES * STAGE;
  static constexpr int SMEM = 1024 + BAR_OFF + 512;
  static_assert(SF_COL0 + STAGES * SF_COLS <= 512, "tensor memory budget");
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(STAGE % 1024 == 0, "128-byte swizzle atoms");
  static_assert((4 * STAGES + 2 * ACC_SLOTS + 1) * 8 + 8 <= 512, "barrier area");
};

struct Piece {
  int mt, nt, k0, k1, tile, ks;
};

__device__ __forceinline__ Piece decode_piece(int q, int S, int MT, int KT) {
  Piece p;
  p.tile = q / S;
  p.ks = q - p.tile * S;
  p.nt = p.tile / MT;
  p.mt = p.tile - p.nt * MT;
  p.k0 = p.ks * KT / S;
  p.k1 = (p.ks + 1) * KT / S;
  return p;
}

template <typename O>
__device__ __forceinline__ O to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// 16 consecutive columns c .. c + 15 of M-side row m.
template <typename O>
__device__ __forceinline__ void store16(const MxGemmArgs& p, int m, int c, const float (&v)[16]) {
  O* out = static_cast<O*>(p.out);
  if (p.transposed) {
    if (m >= p.M) return;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (c + j < p.N) out[static_cast<int64_t>(c + j) * p.ld_out + m] = to_out<O>(v[j]);
    return;
  }
  if (m >= p.M || c >= p.N) return;  // N is a multiple of 16
  uint4* dst = reinterpret_cast<uint4*>(out + static_cast<int64_t>(m) * p.ld_out + c);
  if (sizeof(O) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      dst[j] = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                          __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
  } else {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
    dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

template <int BN, int STAGES, typename O>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_mx_gemm(const __grid_constant__ MxMaps maps, const MxGemmArgs p) {
  using C = MxCfg<BN, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + STAGES;
  uint64_t* sf_full = empty + STAGES;
  uint64_t* sf_ready = sf_full + STAGES;
  uint64_t* acc_full = sf_ready + STAGES;
  uint64_t* acc_empty = acc_full + C::ACC_SLOTS;
  uint64_t* drain = acc_empty + C::ACC_SLOTS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int MT = (p.M + 127) / 128, NT = (p.N + BN - 1) / BN;
  const int KT = (p.K + 255) / 256;
  const int64_t atoms = mx_atoms(p.K);
  const int S = p.ksplit;
  const int total = MT * NT * S;

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.m);
    prefetch_tensormap(&maps.n);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_ready[s], 4);
    }
    for (int a = 0; a < C::ACC_SLOTS; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      const uint64_t pol = policy_evict_normal();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int q = blockIdx.x; ok && q < total; q += gridDim.x) {
        const Piece t = decode_piece(q, S, MT, KT);
        const int n0 = t.nt * BN;
        const uint8_t* sfm = p.m_sf + t.mt * atoms * 512;
        const uint8_t* sfn = p.n_sf + (n0 >> 7) * atoms * 512;
        for (int kt = t.k0; kt < t.k1; ++kt) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          uint8_t* sb = smem + stage * C::STAGE;
          // the atom layout's last row group is always whole, and the tile's
          // second group of 128 rows exists only where N reaches it
          const int groups = min(C::GROUPS, (p.N - n0 + 127) / 128);
          mbar_arrive_expect_tx(&sf_full[stage], C::SF + groups * C::SF);
          bulk_load(sb + C::OFF_SFM, sfm + kt * C::SF, C::SF, &sf_full[stage], pol);
          for (int g = 0; g < groups; ++g)
            bulk_load(sb + C::OFF_SFN + g * C::SF, sfn + (g * atoms * 512) + kt * C::SF, C::SF,
                      &sf_full[stage], pol);
          mbar_arrive_expect_tx(&full[stage], C::TX);
          tma_load_2d(sb, &maps.m, &full[stage], kt * 128, t.mt * 128, pol);
          tma_load_2d(sb + C::OFF_N, &maps.n, &full[stage], kt * 128, n0, pol);
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {  // unwinding: let every copy already in flight land first
        for (int s = 0; s < STAGES && s < issued; ++s) {
          const int i = issued - 1 - s;
          const uint32_t parity = static_cast<uint32_t>(i / STAGES) & 1u;
          mbar_drain(&full[i % STAGES], parity);
          mbar_drain(&sf_full[i % STAGES], parity);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int q = blockIdx.x; ok && q < total; q += gridDim.x) {
        const Piece t = decode_piece(q, S, MT, KT);
        if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, abort_flag, p.status, p.wait_limit_ns))
          break;
        tc_fence_after();
        const uint32_t d_col = tmem + acc * BN;
        for (int kt = t.k0; kt < t.k1; ++kt) {
          if (!mbar_wait(&full[stage], phase, abort_flag, p.status, p.wait_limit_ns) ||
              !mbar_wait(&sf_ready[stage], phase, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint8_t* sb = smem + stage * C::STAGE;
          const uint32_t sf = tmem + C::SF_COL0 + stage * C::SF_COLS;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            mma_mxf4(d_col, sdesc_sw128(smem_u32(sb) + 32 * c),
                     sdesc_sw128(smem_u32(sb + C::OFF_N) + 32 * c), idesc_mxf4(128, BN, c & 1),
                     sf + 4 * (c >> 1), sf + 8 + C::SFN_COLS * (c >> 1),
                     (kt != t.k0 || c != 0) ? 1u : 0u);
          tc_commit(&empty[stage]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit(&acc_full[acc]);
        if (++acc == C::ACC_SLOTS) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // every MMA issued so far must finish before tensor memory is released
      tc_commit(drain);
      mbar_drain(drain, 0);
    }
    __syncwarp();
  } else if (warp >= kSfWarp0 && warp < kEpiWarp1) {
    // ------------------------------------------------------- scale writers
    // An atom's bytes 16 i .. 16 i + 15 are rows i, 32 + i, 64 + i, 96 + i
    // (four blocks each): lane i of tensor memory, one column per row group.
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int q = blockIdx.x; ok && q < total; q += gridDim.x) {
      const Piece t = decode_piece(q, S, MT, KT);
      const int j0 = (t.nt * BN & 127) / 32;  // first 32-row group of a short N tile
      for (int kt = t.k0; kt < t.k1; ++kt) {
        if (!mbar_wait(&sf_full[stage], phase, abort_flag, p.status, p.wait_limit_ns)) {
          ok = false;
          break;
        }
        const uint8_t* sb = smem + stage * C::STAGE;
        const uint32_t sf = tmem + lane_off + C::SF_COL0 + stage * C::SF_COLS;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 a = reinterpret_cast<const uint4*>(sb + C::OFF_SFM + h * 512)[lane];
          tmem_st_32x32b_x4(sf + 4 * h, a.x, a.y, a.z, a.w);
#pragma unroll
          for (int g = 0; g < C::GROUPS; ++g) {
            uint4 b = reinterpret_cast<const uint4*>(sb + C::OFF_SFN + g * C::SF + h * 512)[lane];
            if (BN < 128) {
              if (j0 & 2) b = make_uint4(b.z, b.w, 0u, 0u);
              if (j0 & 1) b = make_uint4(b.y, b.z, 0u, 0u);
            }
            tmem_st_32x32b_x4(sf + 8 + C::SFN_COLS * h + 4 * g, b.x, b.y, b.z, b.w);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_ready[stage]);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int half = warp >= kEpiWarp1 ? 1 : 0;
    const int row = quarter * 32 + lane;  // M-side row of the tile
    constexpr int HALF = BN / 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int q = blockIdx.x; q < total; q += gridDim.x) {
      const Piece t = decode_piece(q, S, MT, KT);
      if (!mbar_wait(&acc_full[acc], acc_phase, abort_flag, p.status, p.wait_limit_ns)) break;
      tc_fence_after();
      const uint32_t base =
          tmem + acc * BN + half * HALF + (static_cast<uint32_t>(quarter * 32) << 16);
      const int m = t.mt * 128 + row, c0 = t.nt * BN + half * HALF;
      float* plane = S > 1 ? p.partial + (static_cast<int64_t>(q) * BN + half * HALF) * 128 + row
                           : nullptr;
#pragma unroll 1
      for (int c = 0; c < HALF; c += 16) {
        uint32_t u[16];
        tmem_ld_32x32b_x16(base + c, u);
        tmem_ld_wait();
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(u[j]);
        if (S > 1) {
#pragma unroll
          for (int j = 0; j < 16; ++j) __stcg(plane + (c + j) * 128, v[j]);
        } else {
          store16<O>(p, m, c0 + c, v);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
      if (++acc == C::ACC_SLOTS) {
        acc = 0;
        acc_phase ^= 1u;
      }
      if (S > 1) {
        // This warp's 32 x HALF part of the piece is in memory; the warp that
        // brings the last piece of the tile sums all of them in piece order.
        // No warp waits for another.
        __threadfence();
        __syncwarp();
        uint32_t before = 0;
        if (lane == 0)
          before = atomicAdd(p.counters + t.tile * kEpiWarps + half * 4 + quarter, 1u);
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before + 1 == static_cast<uint32_t>(S)) {
          __threadfence();
          const float* first =
              p.partial + (static_cast<int64_t>(t.tile) * S * BN + half * HALF) * 128 + row;
#pragma unroll 1
          for (int c = 0; c < HALF; c += 16) {
            float v[16] = {};
            for (int s = 0; s < S; ++s) {
              const float* pl = first + (static_cast<int64_t>(s) * BN + c) * 128;
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] += __ldcg(pl + j * 128);
            }
            store16<O>(p, m, c0 + c, v);
          }
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Large products: a pair of CTAs on one tile of 256 x 256.
//
// A stage of one CTA (a K step of 256) is 128 rows of each operand: 32 KB for
// 128 x 256 of output, where a CTA on its own loads 48 KB for the same.  All
// eight copies of a stage complete on one barrier of rank 0, whose one thread
// then copies the scales into tensor memory (tcgen05.cp, in order with the MMAs
// and hidden behind them: measured 128.4 cycles an MMA with and 128.3 without)
// and issues the MMAs of both CTAs.  Commits free the stage, and hand over the
// accumulator, in both.  The accumulator leaves tensor memory for registers
// before anything is stored, so the next tile's MMAs run under the stores,
// which go through shared memory as 128-byte rows by tensor map.
// ---------------------------------------------------------------------------
struct PairMaps {
  CUtensorMap m, n, sfm, sfn, out;
};

struct PairCfg {
  static constexpr int THREADS = 320;  // producer, MMA issuer, 8 epilogue warps
  static constexpr int STAGES = 5;
  static constexpr int TILE = 128 * 128;  // a CTA's rows of either operand
  static constexpr int SF = 1024;
  static constexpr int OFF_N = TILE;
  static constexpr int OFF_SFM = 2 * TILE;
  static constexpr int OFF_SFN = OFF_SFM + SF;  // all 256 rows of the N side
  static constexpr int STAGE = OFF_SFN + 2 * SF;
  static constexpr uint32_t TX = 2 * STAGE;  // both CTAs
  static constexpr int SF_COLS = 8 + 16;
  static constexpr int SF_COL0 = 256;  // two sets, taken in turn
  static constexpr int STG = 32 * 128;  // 32 rows x 128 bytes per epilogue warp
  static constexpr int STG_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = STG_OFF + kEpiWarps * STG;
  static constexpr int SMEM = 1024 + BAR_OFF + 256;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(STAGE % 1024 == 0, "128-byte swizzle atoms");
};

template <typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg::THREADS, 1)
    k_mx_gemm_pair(const __grid_constant__ PairMaps maps, const MxGemmArgs p) {
  using C = PairCfg;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);  // rank 0's
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + 1;  // rank 0's: the epilogue warps of both
  uint64_t* drain = acc_empty + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int MT = (p.M + 255) / 256, NT = (p.N + 255) / 256;
  const int KT = (p.K + 255) / 256;
  const int total = MT * NT;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;  // tiles of this pair

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.m);
    prefetch_tensormap(&maps.n);
    prefetch_tensormap(&maps.sfm);
    prefetch_tensormap(&maps.sfn);
    prefetch_tensormap(&maps.out);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * kEpiWarps);
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

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      const uint64_t pol = policy_evict_normal();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int q = first; ok && q < total; q += step) {
        const int nt = q / MT, mt = q - nt * MT;
        const int m0 = mt * 256 + rank * 128, n0 = nt * 256;
        for (int kt = 0; kt < KT; ++kt) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          uint8_t* sb = smem + stage * C::STAGE;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], C::TX);
          const uint32_t bar = cluster_address(&full[stage], 0);
          tma_load_2d_pair(sb, &maps.m, bar, kt * 128, m0, pol);
          tma_load_2d_pair(sb + C::OFF_N, &maps.n, bar, kt * 128, n0 + rank * 128, pol);
          tma_load_2d_pair(sb + C::OFF_SFM, &maps.sfm, bar, kt * 256, m0 >> 7, pol);
          tma_load_2d_pair(sb + C::OFF_SFN, &maps.sfn, bar, kt * 256, n0 >> 7, pol);
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {  // unwinding: let the copies in flight land first
        if (rank == 0) {
          for (int s = 0; s < STAGES && s < issued; ++s) {
            const int i = issued - 1 - s;
            mbar_drain(&full[i % STAGES], static_cast<uint32_t>(i / STAGES) & 1u);
          }
        } else {
          // rank 1's complete on rank 0's barriers, which may have moved on:
          // wait a time that no copy takes
          const uint64_t t0 = globaltimer();
          while (globaltimer() - t0 < 5000000) __nanosleep(1000);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------------------------------------------------- MMA issuer
      const bool leader = elect_one();
      const uint64_t codes = sdesc_sw128(smem_u32(smem));
      const uint64_t scales = sdesc_atom(smem_u32(smem) + C::OFF_SFM);
      int stage = 0, sets = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int q = first; ok && q < total; q += step) {
        if (!mbar_wait(acc_empty, acc_phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) break;
        tc_fence_after();
        for (int kt = 0; kt < KT; ++kt) {
          if (!mbar_wait(&full[stage], phase, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t cd = sdesc_at(codes, stage * C::STAGE);
          const uint64_t sd = sdesc_at(scales, stage * C::STAGE);
          const uint32_t sf = tmem + C::SF_COL0 + (sets & 1) * C::SF_COLS;
          ++sets;
          if (leader) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 128 of K each
              tc_copy_atom_pair(sf + 4 * h, sdesc_at(sd, 512 * h));
              tc_copy_atom_pair(sf + 8 + 8 * h, sdesc_at(sd, C::SF + 512 * h));
              tc_copy_atom_pair(sf + 12 + 8 * h, sdesc_at(sd, 2 * C::SF + 512 * h));
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
              mma_mxf4_pair(tmem, sdesc_at(cd, 32 * c), sdesc_at(cd, C::OFF_N + 32 * c),
                            idesc_mxf4(256, 256, c & 1), sf + 4 * (c >> 1), sf + 8 + 8 * (c >> 1),
                            (kt != 0 || c != 0) ? 1u : 0u);
            tc_commit_pair(&empty[stage]);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (leader) tc_commit_pair(acc_full);
        __syncwarp();
        acc_phase ^= 1u;
      }
      // every MMA issued so far must finish before tensor memory is released
      if (leader) tc_commit_pair(drain);
      mbar_drain(drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int half = warp >= 6 ? 1 : 0;
    uint8_t* stg = smem + C::STG_OFF + (warp - 2) * C::STG;
    constexpr bool F32 = sizeof(O) == 4;
    constexpr int COLS = F32 ? 32 : 64;  // columns of a staged chunk
    uint32_t acc_phase = 0;
    for (int q = first; q < total; q += step) {
      const int nt = q / MT, mt = q - nt * MT;
      if (!mbar_wait(acc_full, acc_phase, abort_flag, p.status, p.wait_limit_ns)) break;
      tc_fence_after();
      const uint32_t base = tmem + half * 128 + (static_cast<uint32_t>(quarter * 32) << 16);
      const int m = mt * 256 + rank * 128 + quarter * 32, c0 = nt * 256 + half * 128;
      uint32_t v[F32 ? 128 : 64];  // this lane's row: 128 values
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (F32) {
          tmem_ld_32x32b_x32(base + 32 * c, v + 32 * (F32 ? c : 0));
        } else {
          uint32_t u[32];
          tmem_ld_32x32b_x32(base + 32 * c, u);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(u[2 * j]),
                                                           __uint_as_float(u[2 * j + 1]));
            v[16 * c + j] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
      }
      if (F32) tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty, 0);
      acc_phase ^= 1u;
      if (m >= p.M) continue;  // warp-uniform
#pragma unroll
      for (int c = 0; c < 128 / COLS; ++c) {
        if (lane == 0) bulk_store_wait_read();  // the chunk before has left
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)  // 16-byte piece j of the row, swizzled
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) * 16)) =
              make_uint4(v[32 * c + 4 * j], v[32 * c + 4 * j + 1], v[32 * c + 4 * j + 2],
                         v[32 * c + 4 * j + 3]);
        fence_async_shared();
        __syncwarp();
        if (lane == 0 && c0 + c * COLS < p.N) tma_store_2d(&maps.out, stg, c0 + c * COLS, m);
      }
    }
    if (lane == 0) bulk_store_wait();
    __syncwarp();
  }
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other still reaches into it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <typename O>
cudaError_t launch_pair(const MxGemmArgs& a, const uint8_t* m_codes, const uint8_t* n_codes,
                        int tiles, cudaStream_t stream) {
  PairMaps maps;
  const uint64_t row = static_cast<uint64_t>(a.K) / 2;
  const uint64_t sf_row = static_cast<uint64_t>(mx_atoms(a.K)) * 512;
  const uint64_t m = a.M, n = a.N;
  if (!make_codes_map(&maps.m, m_codes, m, row, 128) ||
      !make_codes_map(&maps.n, n_codes, n, row, 128) ||
      !make_map(&maps.sfm, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.m_sf, sf_row / 4, (m + 127) / 128,
                sf_row, 256, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map(&maps.sfn, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.n_sf, sf_row / 4, (n + 127) / 128,
                sf_row, 256, 2, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map(&maps.out,
                sizeof(O) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                a.out, n, m, static_cast<uint64_t>(a.ld_out) * sizeof(O), 128 / sizeof(O), 32,
                CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = k_mx_gemm_pair<O>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PairCfg::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(2 * std::min(num_sms() / 2, tiles)), dim3(PairCfg::THREADS),
                    PairCfg::SMEM, stream, maps, a);
}

template <int BN, int STAGES, typename O>
cudaError_t launch_cfg(const MxGemmArgs& a, const uint8_t* m_codes, const uint8_t* n_codes,
                       int pieces, cudaStream_t stream) {
  using C = MxCfg<BN, STAGES>;
  MxMaps maps;
  const uint64_t row = static_cast<uint64_t>(a.K) / 2;
  if (!make_codes_map(&maps.m, m_codes, a.M, row, 128) ||
      !make_codes_map(&maps.n, n_codes, a.N, row, BN))
    return cudaErrorInvalidValue;
  auto kern = k_mx_gemm<BN, STAGES, O>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(std::min(num_sms(), pieces)), dim3(kGemmThreads), C::SMEM, stream,
                    maps, a);
}

// How a product of R x C with K steps KT runs: which side is M, the N tile and
// the pieces of K.
struct MxPlan {
  bool swap;  // rows of the output on the N side
  int bn, ksplit, tiles;  // bn 0: pairs of CTAs on tiles of 256 x 256
};

MxPlan plan_product(int64_t R, int64_t C, int64_t K) {
  MxPlan p{};
  const int sms = num_sms();
  const int KT = static_cast<int>((K + 255) / 256);
  // few output rows go on N: an M tile of 128 would be mostly empty
  p.swap = R <= 64;
  const int64_t M = p.swap ? C : R, N = p.swap ? R : C;
  const int64_t pairs = (M + 255) / 256 * ((N + 255) / 256);
  if (!p.swap && pairs * 2 >= sms) {
    p.tiles = static_cast<int>(pairs);
    p.ksplit = 1;
    return p;
  }
  const int64_t mt = (M + 127) / 128;
  p.bn = p.swap ? (N <= 32 ? 32 : 64) : mt * ((N + 255) / 256) >= sms ? 256 : 128;
  p.tiles = static_cast<int>(mt * ((N + p.bn - 1) / p.bn));
  // idle SMs take pieces of K, at least two steps each
  p.ksplit = 1;
  if (p.tiles * 2 <= sms) p.ksplit = std::max(1, std::min({sms / p.tiles, KT / 2, 16}));
  return p;
}

}  // namespace

size_t mx_product_bytes(int64_t R, int64_t C, int64_t K) {
  const MxPlan p = plan_product(R, C, K);
  return p.ksplit > 1 ? static_cast<size_t>(p.tiles) * p.ksplit * p.bn * 128 * 4 : 0;
}

int mx_product_counters(int64_t R, int64_t C, int64_t K) {
  const MxPlan p = plan_product(R, C, K);
  return p.ksplit > 1 ? p.tiles * kEpiWarps : 0;
}

cudaError_t launch_mx_product(const MxProduct& g, cudaStream_t stream) {
  if (g.R == 0 || g.C == 0) return cudaSuccess;
  const MxPlan p = plan_product(g.R, g.C, g.K);
  const uint8_t* m_codes = p.swap ? g.c_codes : g.r_codes;
  const uint8_t* n_codes = p.swap ? g.r_codes : g.c_codes;
  MxGemmArgs a{};
  a.m_sf = p.swap ? g.c_scales : g.r_scales;
  a.n_sf = p.swap ? g.r_scales : g.c_scales;
  a.out = g.out;
  a.ld_out = g.ld_out;
  a.M = static_cast<int>(p.swap ? g.C : g.R);
  a.N = static_cast<int>(p.swap ? g.R : g.C);
  a.K = static_cast<int>(g.K);
  a.transposed = p.swap;
  a.ksplit = p.ksplit;
  a.partial = g.partial;
  a.counters = g.counters;
  a.status = g.status;
  a.wait_limit_ns = wait_limit_ns();
  const int pieces = p.tiles * p.ksplit;
  auto run = [&](auto out) {
    using O = decltype(out);
    switch (p.bn) {
      case 0: return launch_pair<O>(a, m_codes, n_codes, p.tiles, stream);
      case 32: return launch_cfg<32, 8, O>(a, m_codes, n_codes, pieces, stream);
      case 64: return launch_cfg<64, 8, O>(a, m_codes, n_codes, pieces, stream);
      case 128: return launch_cfg<128, 6, O>(a, m_codes, n_codes, pieces, stream);
      default: return launch_cfg<256, 4, O>(a, m_codes, n_codes, pieces, stream);
    }
  };
  return g.out_f32 ? run(float{}) : run(__nv_bfloat16{});
}

}  // namespace megamoe
