// MXFP4 product of two row-major matrices on tcgen05 tensor cores:
//   out[r, c] = sum_k P[r, k] Q[c, k]
// with E2M1 codes [rows, K / 2], one E8M0 scale per 32 elements along K (atom
// layout), fp32 accumulation in tensor memory (tcgen05.mma kind::mxf4,
// scale_vec::2X).  The linear's forward product and both of its gradients are
// this product of quantised operands.
//
// Both kernels stage operand codes by tensor map in the 128-byte swizzle and
// scale atoms as they are; one converged warp copies a stage's scales into
// tensor memory (tcgen05.cp runs in order with the MMAs and hides behind them:
// measured 128.4 cycles an MMA of N = 256 with it and 128.2 without) and issues
// the MMAs.
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
  int out_f32;  // else bf16
  int cluster;  // CTAs that share a tile's K range
  int n_box;    // rows of an N-side box
  uint32_t* status;
  const uint32_t* flags;  // of the quantising launch before it (collect_flags)
  int flag_count;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ float4 load_cluster4(const float* p, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// ---------------------------------------------------------------------------
// Products of few tiles: one tile of 128 x BN a cluster of up to eight CTAs,
// which share its K range.  Each CTA leaves its fp32 partial sums in its shared
// memory (the stages are free by then) and sums its share of the tile over the
// cluster in rank order: the result does not depend on timing, and no partial
// sums or counters go through global memory.  Two CTAs fit an SM, so one's
// start and end run under the other's products.
//
// FLIP: few output rows (tokens) are the N side, so that no M tile is mostly
// empty, and the tile is stored transposed.  Its box holds only the rows that
// there are (up to eights): boxes that reach out of the matrix load more slowly
// (1536 -> 24576 at 17 tokens took longer than at 64).
//
// One launch takes one product or two (a linear's two gradients), each split as
// it would be alone: the launch's cluster is the larger of theirs, and the
// smaller one's CTAs form groups within it.
//
// Bound by latency: the loads' first arrival, the sums over the cluster and the
// launch.  Both gradients of 333 x 1536 -> 2048 take 13 us with their quantiser
// (its products' share 7 us), 512 x 7168 -> 2048 13.8 us without.
// ---------------------------------------------------------------------------
template <int BN, bool FLIP>
struct TileCfg {
  static constexpr int THREADS = 320;  // producer, MMA issuer, 8 epilogue warps
  static constexpr int STAGES = 3;
  static constexpr int M_TILE = 128 * 128;
  static constexpr int N_TILE = BN * 128;
  static constexpr int SF = 1024;  // scale atoms of 128 rows and a K step
  static constexpr int OFF_N = M_TILE;
  static constexpr int OFF_SFM = OFF_N + N_TILE;
  static constexpr int OFF_SFN = OFF_SFM + SF;
  static constexpr int STAGE = OFF_SFN + SF;
  static constexpr int COLS = BN + 32 <= 128 ? 128 : 256;  // tensor memory: a power of two
  static constexpr int SMEM = 1024 + STAGES * STAGE;
  // partial sums: rows of the output's row direction, padded against bank conflicts
  static constexpr int OUTER = FLIP ? BN : 128, INNER = FLIP ? 128 : BN;
  static constexpr int PITCH = INNER + 4;
  static_assert(BN <= 128, "one scale group");
  static_assert(OUTER * PITCH * 4 <= STAGES * STAGE, "partial sums fit the stages");
  static_assert(8 * 32 * 128 <= STAGES * STAGE, "staged rows fit the stages");
  static_assert(STAGE % 1024 == 0, "128-byte swizzle atoms");
};

struct TileMaps {
  CUtensorMap m, n, out;
};
struct TileJobs {
  TileMaps maps[2];
  MxGemmArgs args[2];
  int first;    // the second product's first block, a multiple of cluster
  int cluster;  // of the launch
};

template <int BN, bool FLIP>
__global__ void __launch_bounds__(320, 2) k_mx_gemm_tile(const __grid_constant__ TileJobs jobs) {
  const bool second = static_cast<int>(blockIdx.x) >= jobs.first;
  const TileMaps& maps = jobs.maps[second ? 1 : 0];
  const MxGemmArgs& p = jobs.args[second ? 1 : 0];
  const int block = blockIdx.x - (second ? jobs.first : 0);
  using C = TileCfg<BN, FLIP>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[STAGES], empty[STAGES], acc_full;
  __shared__ uint32_t tmem_holder;
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.cluster;
  const int MT = (p.M + 127) / 128, NT = (p.N + BN - 1) / BN;
  const int tile = block / S, rank = block - tile * S;  // rank within the tile's CTAs
  const int nt = tile / MT, mt = tile - nt * MT;
  const int KT = (p.K + 255) / 256;
  const int k0 = rank * KT / S, k1 = (rank + 1) * KT / S;
  if (tile >= MT * NT) {  // fills up the last cluster
    pdl_wait();
    pdl_trigger();
    cluster_sync();
    cluster_sync();
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    s_abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&maps.m);
    prefetch_tensormap(&maps.n);
    prefetch_tensormap(&maps.out);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  pdl_wait();
  pdl_trigger();

  bool done = true;
  if (warp == 0) {
    {
      // ------------------------------------------------------------ producer
      // (the whole warp, one lane of it issuing: elect_one)
      const bool leader = elect_one();
      const uint64_t pol = policy_evict_normal();
      const int64_t atoms = mx_atoms(p.K);
      const uint8_t* sfm = p.m_sf + mt * atoms * 512;
      const uint8_t* sfn = p.n_sf + (nt * BN >> 7) * atoms * 512;
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int kt = k0; kt < k1; ++kt) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) break;
        uint8_t* sb = smem + stage * C::STAGE;
        if (leader) {
          mbar_arrive_expect_tx(&full[stage], C::M_TILE + p.n_box * 128 + 2 * C::SF);
          tma_load_2d(sb, &maps.m, &full[stage], kt * 128, mt * 128, pol);
          tma_load_2d(sb + C::OFF_N, &maps.n, &full[stage], kt * 128, nt * BN, pol);
          bulk_load(sb + C::OFF_SFM, sfm + static_cast<int64_t>(kt) * C::SF, C::SF, &full[stage], pol);
          bulk_load(sb + C::OFF_SFN, sfn + static_cast<int64_t>(kt) * C::SF, C::SF, &full[stage], pol);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      drain_copies(full, STAGES, issued);
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    const bool leader = elect_one();
    const uint64_t codes = sdesc_sw128(smem_u32(smem));
    const uint64_t scales = sdesc_atom(smem_u32(smem) + C::OFF_SFM);
    int stage = 0;
    uint32_t phase = 0;
    for (int kt = k0; kt < k1; ++kt) {
      if (!mbar_wait(&full[stage], phase, abort_flag, p.status, p.wait_limit_ns)) break;
      tc_fence_after();
      const uint64_t cd = sdesc_at(codes, stage * C::STAGE);
      const uint64_t sd = sdesc_at(scales, stage * C::STAGE);
      const uint32_t sf = tmem + BN + 16 * (kt & 1);  // two sets, taken in turn
      if (leader) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 128 of K each
          tc_copy_atom(sf + 4 * h, sdesc_at(sd, 512 * h));
          tc_copy_atom(sf + 8 + 4 * h, sdesc_at(sd, C::SF + 512 * h));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mma_mxf4(tmem, sdesc_at(cd, 32 * c), sdesc_at(cd, C::OFF_N + 32 * c),
                   idesc_mxf4(128, BN, c & 1), sf + 4 * (c >> 1), sf + 8 + 4 * (c >> 1),
                   (kt != k0 || c != 0) ? 1u : 0u);
        tc_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == STAGES) {
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
    // ---------------------------------------------------------------- epilogue
    const int quarter = warp & 3, half = warp >= 6 ? 1 : 0;
    const int row = quarter * 32 + lane;
    constexpr int HALF = BN / 2;
    if (block == 0) collect_flags(p.flags, p.flag_count, threadIdx.x - 64, 256, p.status);
    done = mbar_wait(&acc_full, 0, abort_flag, p.status, p.wait_limit_ns);
    tc_fence_after();
    const uint32_t base = tmem + half * HALF + (static_cast<uint32_t>(quarter * 32) << 16);
    float* part = reinterpret_cast<float*>(smem);
    if (S > 1) {
#pragma unroll
      for (int c = 0; c < HALF; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(base + c, v);
        tmem_ld_wait();
        const int col = half * HALF + c;
        if (FLIP) {
#pragma unroll
          for (int j = 0; j < 32; ++j) part[(col + j) * C::PITCH + row] = __uint_as_float(v[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<uint4*>(part + row * C::PITCH + col + j) =
                make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      }
    } else if (FLIP) {
      const int m = mt * 128 + row;
#pragma unroll
      for (int c = 0; c < HALF; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(base + c, v);
        tmem_ld_wait();
        const int n = nt * BN + half * HALF + c;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (done && m < p.M && n + j < p.N) {
            const int64_t at = (n + j) * p.ld_out + m;
            if (p.out_f32) store1(static_cast<float*>(p.out) + at, __uint_as_float(v[j]));
            else store1(static_cast<__nv_bfloat16*>(p.out) + at, __uint_as_float(v[j]));
          }
      }
    } else {
      // 128-byte rows through shared memory and out by tensor map: 64 columns
      // of bf16 or 32 of fp32 at a time
      uint8_t* stg = smem + (warp - 2) * 4096;
      const int m = mt * 128 + quarter * 32, n = nt * BN + half * HALF;
      uint32_t w[32];
#pragma unroll
      for (int c = 0; c < HALF; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(base + c, v);
        tmem_ld_wait();
        if (p.out_f32) {
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = v[j];
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[2 * j]),
                                                           __uint_as_float(v[2 * j + 1]));
            w[(c & 32) / 2 + j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          if ((c & 32) == 0) continue;  // half of the chunk's columns
        }
        if (lane == 0) bulk_store_wait_read();  // the chunk before has left
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)  // 16-byte piece j of the row, swizzled
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) * 16)) =
              make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        fence_async_shared();
        __syncwarp();
        const int at = n + (p.out_f32 ? c : c & ~63);
        if (lane == 0 && done && m < p.M && at < p.N) tma_store_2d(&maps.out, stg, at, m);
      }
      if (lane == 0) bulk_store_wait();
      __syncwarp();
    }
    tc_fence_before();
  }
  __syncthreads();
  if (jobs.cluster > 1) cluster_sync();
  if (S > 1) {
    const uint32_t group = cluster_rank() - rank;  // the tile's first CTA
    const float* part = reinterpret_cast<const float*>(smem);
    constexpr int quads = C::INNER / 4;
    const int first = rank * C::OUTER / S, last = (rank + 1) * C::OUTER / S;
    for (int i = first * quads + threadIdx.x; i < last * quads; i += C::THREADS) {
      const int o = i / quads, q = i % quads * 4;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int r = 0; r < S; ++r) {
        const float4 v = load_cluster4(part + o * C::PITCH + q, group + r);
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
      // rows and columns of the output; whole fours along it
      const int r = (FLIP ? nt * BN : mt * 128) + o, c = (FLIP ? mt * 128 : nt * BN) + q;
      if (r < (FLIP ? p.N : p.M) && c < (FLIP ? p.M : p.N)) {
        if (p.out_f32) store4(static_cast<float*>(p.out) + r * p.ld_out + c, sum);
        else store4(static_cast<__nv_bfloat16*>(p.out) + r * p.ld_out + c, sum);
      }
    }
  }
  if (jobs.cluster > 1) cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

// A product as its kernel sees it.
struct MxJob {
  MxGemmArgs a;
  const uint8_t* m_codes;
  const uint8_t* n_codes;
  int tiles;
};

template <int BN, bool FLIP>
cudaError_t launch_tiles(const MxJob* jobs, int count, cudaStream_t stream) {
  using C = TileCfg<BN, FLIP>;
  TileJobs t{};
  t.cluster = jobs[0].a.cluster;
  if (count == 2) t.cluster = std::max(t.cluster, jobs[1].a.cluster);
  int blocks = 0;
  for (int i = 0; i < count; ++i) {
    const MxJob& j = jobs[i];
    const uint64_t row = static_cast<uint64_t>(j.a.K) / 2, m = j.a.M, n = j.a.N;
    const int size = j.a.out_f32 ? 4 : 2;
    t.args[i] = j.a;
    t.args[i].n_box = static_cast<int>(std::min<uint64_t>(BN, (n + 7) / 8 * 8));
    if (!make_codes_map(&t.maps[i].m, j.m_codes, m, row, 128) ||
        !make_codes_map(&t.maps[i].n, j.n_codes, n, row, t.args[i].n_box) ||
        !make_map(&t.maps[i].out,
                  size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  j.a.out, FLIP ? m : n, FLIP ? n : m, static_cast<uint64_t>(j.a.ld_out) * size,
                  128 / size, 32, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    blocks += (j.tiles * j.a.cluster + t.cluster - 1) / t.cluster * t.cluster;
    if (i == 0) t.first = blocks;
  }
  auto kern = k_mx_gemm_tile<BN, FLIP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kern, dim3(blocks), dim3(C::THREADS), C::SMEM, t.cluster, stream, t);
}

// ---------------------------------------------------------------------------
// Large products: a pair of CTAs on one tile of 256 x 256.
//
// A stage of one CTA (a K step of 256) is 128 rows of each operand: 32 KB for
// 128 x 256 of output, where a CTA on its own loads 48 KB for the same.  All
// eight copies of a stage complete on one barrier of rank 0, whose issuing warp
// then copies the scales into tensor memory (tcgen05.cp, in order with the MMAs
// and hidden behind them: measured 128.4 cycles an MMA with and 128.3 without)
// and issues the MMAs of both CTAs.  Commits free the stage, and hand over the
// accumulator, in both.
//
// Tensor memory holds two accumulators that have 48 of their 256 columns in
// common: a tile's products start as soon as those have been read from the one
// before, and the rest is read, rounded and stored meanwhile.  Stores go out as
// 128-byte rows through 2 KB of shared memory a warp, 16 rows at a time, by
// ordinary stores: stores by tensor map go through the same unit as the loads,
// which then stand behind them (1200 cycles at an issue that takes 130).  4096 x
// 1536 -> 24576 takes 60.3 us so, 63.2 with 8 rows at a time, 66 with 32 rows and
// the five stages that leave room for them, 71 with a lane storing its own row in
// sectors of 32 bytes.
//
// Tiles go in bands of four rows of tiles where there are more than 16, so that
// those in work at a time share few rows of either operand and find them in L2:
// 16384 x 7168 -> 7168 250 us with one band, 238 with bands of eight rows, 235 of
// four; with 16 rows of tiles one band is as good (66.6 against 67.2).
//
// 16384 x 7168 -> 7168 takes 220 us (7.65 PFLOP/s of the MMAs' 10), 4096 x 1536 ->
// 24576 60 us (201 MB of output alone are 30).  What bounds it: at long K the MMAs
// and the loads that they wait for (214 us with every operand load left out); at
// 6 and 8 K steps the epilogue, 4800 cycles a tile against the MMAs' 3100, which
// reads tensor memory and stages through shared memory under the MMAs' own use of
// both.
// ---------------------------------------------------------------------------
struct PairMaps {
  CUtensorMap m, n, sfm, sfn;
};

template <int S>
struct PairCfg {
  static constexpr int THREADS = 320;  // producer, MMA issuer, 8 epilogue warps
  static constexpr int STAGES = S;
  static constexpr int TILE = 128 * 128;  // a CTA's rows of either operand
  static constexpr int SF = 1024;
  static constexpr int OFF_N = TILE;
  static constexpr int OFF_SFM = 2 * TILE;
  static constexpr int OFF_SFN = OFF_SFM + SF;  // all 256 rows of the N side
  static constexpr int STAGE = OFF_SFN + 2 * SF;
  static constexpr uint32_t TX = 2 * STAGE;  // both CTAs
  static constexpr int SF_COLS = 8 + 16;
  // tensor memory: accumulators in turn at columns 0 and 208 (48 in common), then
  // two sets of scales, in turn
  static constexpr int ACC1 = 208;
  static constexpr int SF_COL0 = 464;
  static constexpr int STG = 16 * 128;  // 16 rows x 128 bytes per epilogue warp
  static constexpr int STG_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = STG_OFF + kEpiWarps * STG;
  static constexpr int SMEM = 768 + BAR_OFF + 256;  // from a multiple of 256 up to one of 1024
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(STAGE % 1024 == 0, "128-byte swizzle atoms");
};

// Tile q: bands of `tall` rows of tiles, column by column within a band.
__device__ __forceinline__ void pair_tile(int q, int tall, int MT, int NT, int* mt, int* nt) {
  const int band = q / (tall * NT), r = q - band * tall * NT;
  const int rows = min(tall, MT - band * tall);
  *nt = r / rows;
  *mt = band * tall + r - *nt * rows;
}

template <typename O, int S>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg<S>::THREADS, 1)
    k_mx_gemm_pair(const __grid_constant__ PairMaps maps, const MxGemmArgs p) {
  using C = PairCfg<S>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(256) uint8_t smem_pair[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_pair) + 1023) & ~static_cast<uintptr_t>(1023));
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
  const int tall = MT > 16 ? 4 : MT;  // rows of tiles in a band
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;  // tiles of this pair

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.m);
    prefetch_tensormap(&maps.n);
    prefetch_tensormap(&maps.sfm);
    prefetch_tensormap(&maps.sfn);
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
    {
      // ------------------------------------------------------------ producer
      // (the whole warp, one lane of it issuing: elect_one)
      const bool leader = elect_one();
      const uint64_t pol = policy_evict_normal();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int q = first; ok && q < total; q += step) {
        int mt, nt;
        pair_tile(q, tall, MT, NT, &mt, &nt);
        const int m0 = mt * 256 + rank * 128, n0 = nt * 256;
        for (int kt = 0; kt < KT; ++kt) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          uint8_t* sb = smem + stage * C::STAGE;
          if (leader) {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], C::TX);
            const uint32_t bar = cluster_address(&full[stage], 0);
            tma_load_2d_pair(sb, &maps.m, bar, kt * 128, m0, pol);
            tma_load_2d_pair(sb + C::OFF_N, &maps.n, bar, kt * 128, n0 + rank * 128, pol);
            tma_load_2d_pair(sb + C::OFF_SFM, &maps.sfm, bar, kt * 256, m0 >> 7, pol);
            tma_load_2d_pair(sb + C::OFF_SFN, &maps.sfn, bar, kt * 256, n0 >> 7, pol);
          }
          __syncwarp();
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      drain_pair_copies(full, STAGES, issued, rank, !ok);
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
        const uint32_t acc = tmem + acc_phase * C::ACC1;
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
          }
          __syncwarp();
          if (kt == 0) {
            if (!mbar_wait(acc_empty, acc_phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (leader) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              mma_mxf4_pair(acc, sdesc_at(cd, 32 * c), sdesc_at(cd, C::OFF_N + 32 * c),
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
    if (blockIdx.x == 0) collect_flags(p.flags, p.flag_count, threadIdx.x - 64, 256, p.status);
    uint32_t acc_phase = 0;
    for (int q = first; q < total; q += step) {
      int mt, nt;
      pair_tile(q, tall, MT, NT, &mt, &nt);
      if (!mbar_wait(acc_full, acc_phase, abort_flag, p.status, p.wait_limit_ns)) break;
      tc_fence_after();
      const uint32_t base =
          tmem + acc_phase * C::ACC1 + half * 128 + (static_cast<uint32_t>(quarter * 32) << 16);
      const int m = mt * 256 + rank * 128 + quarter * 32, c0 = nt * 256 + half * 128;
      // The next tile's products may start once the columns that the two
      // accumulators share have been read: the last of this one at column 0 (the
      // second half's), the first of the other.  The half without them lets go
      // at once: it has read the whole tile before.
      const bool shares = half != static_cast<int>(acc_phase);
      auto let_go = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty, 0);
      };
      if (!shares) let_go();
      acc_phase ^= 1u;
      constexpr int per = 16 / sizeof(O);
      const int piece = lane & 7;
      O* out = static_cast<O*>(p.out) + static_cast<int64_t>(m) * p.ld_out + c0 + piece * per;
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {  // 64 columns, the shared ones first
        const int at = 64 * (part ^ half);
        uint32_t u[64];  // this lane's row
        tmem_ld_32x32b_x32(base + at, u);
        tmem_ld_32x32b_x32(base + at + 32, u + 32);
        tmem_ld_wait();
        if (part == 0 && shares) let_go();
        if (m >= p.M) continue;  // warp-uniform
        if (!F32) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(u[2 * j]),
                                                            __uint_as_float(u[2 * j + 1]));
            u[j] = *reinterpret_cast<const uint32_t*>(&h2);
          }
        }
#pragma unroll
        for (int c = 0; c < 64 / COLS; ++c) {
          const int col = at + c * COLS;
          const bool in = c0 + col + piece * per < p.N;
#pragma unroll 1
          for (int g = 0; g < 2; ++g) {  // 16 rows
            __syncwarp();
            if (lane >> 4 == g) {
#pragma unroll
              for (int j = 0; j < 8; ++j)  // 16-byte piece j of the row, swizzled
                *reinterpret_cast<uint4*>(stg + (lane & 15) * 128 + ((j ^ piece) * 16)) =
                    make_uint4(u[32 * c + 4 * j], u[32 * c + 4 * j + 1], u[32 * c + 4 * j + 2],
                               u[32 * c + 4 * j + 3]);
            }
            __syncwarp();
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 4 * i + (lane >> 3);
              x[i] = *reinterpret_cast<const uint4*>(stg + r * 128 + ((piece ^ (r & 7)) * 16));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 16 * g + 4 * i + (lane >> 3);
              if (in && m + r < p.M)
                __stcs(reinterpret_cast<uint4*>(out + static_cast<int64_t>(r) * p.ld_out + col), x[i]);
            }
          }
        }
      }
      tc_fence_before();
    }
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

template <typename O, int S>
cudaError_t launch_pair(const MxJob& j, cudaStream_t stream) {
  const MxGemmArgs& a = j.a;
  PairMaps maps;
  const uint64_t row = static_cast<uint64_t>(a.K) / 2;
  const uint64_t sf_row = static_cast<uint64_t>(mx_atoms(a.K)) * 512;
  const uint64_t m = a.M, n = a.N;
  if (!make_codes_map(&maps.m, j.m_codes, m, row, 128) ||
      !make_codes_map(&maps.n, j.n_codes, n, row, 128) ||
      !make_map(&maps.sfm, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.m_sf, sf_row / 4, (m + 127) / 128,
                sf_row, 256, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map(&maps.sfn, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.n_sf, sf_row / 4, (n + 127) / 128,
                sf_row, 256, 2, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  auto kern = k_mx_gemm_pair<O, S>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PairCfg<S>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(2 * std::min(num_sms() / 2, j.tiles)), dim3(PairCfg<S>::THREADS),
                    PairCfg<S>::SMEM, stream, maps, a);
}

// How a product of R x C with K steps KT runs.
struct MxPlan {
  bool pair;  // pairs of CTAs on tiles of 256 x 256
  bool flip;  // output rows on the N side (tiles of 128 x 64)
  int tiles, cluster;
};

// CTAs that share a tile's K range, where SMs would idle: a cluster's sums cost
// as much as `sums` K steps, and more CTAs than SMs take turns.  Measured (us, 1
// / 2 / 4 / 8 CTAs): 128 x 7168 -> 1536 15.5 / 14.4 / 12.4 / 12.4; 512 x 7168 ->
// 2048 16.5 / 16.5 / 17.4 / 26.8; 333 x 1536 -> 2048 10.4 / 12.4 / 13.5 / 13.5;
// flipped, 64 x 7168 -> 1536 16.5 / 14.0 / 11.8 / 11.2.
int pick_cluster(int64_t tiles, int64_t steps, double sums) {
  int best = 1;
  double least = static_cast<double>(steps);
  for (int s = 2; s <= 8 && s <= steps && tiles * s <= num_sms(); s *= 2) {
    const double cost = static_cast<double>(steps) / s + sums;
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

MxPlan plan_product(const MxProduct& g) {
  const int64_t R = g.R, C = g.C, K = g.K;
  MxPlan p{};
  const int64_t pairs = (R + 255) / 256 * ((C + 255) / 256);
  const int64_t tiles = (R + 127) / 128 * ((C + 127) / 128);
  p.flip = R <= 64;
  p.cluster = 1;
  // A pair takes four tiles' worth in the time that an SM takes one of its own
  // tiles (operands per product halved), so it is chosen where half of the pairs
  // have work and it pads to less than twice the tiles: 128 x 1536 -> 24576 took
  // 24.8 us in pairs, half of them empty.  Single / pairs (us, with the
  // quantiser): 75 pairs 3815 x 5664 -> 1248 39.6 / 27.4; 64 2048 x 4096 -> 2048
  // 15.7 / 14.0; 48 1536 x 7168 -> 2048 19.8 / 18.1; 40 1280 x 4096 -> 2048 14.5 /
  // 12.9, 1280 x 1536 -> 2048 9.4 / 9.7; 32 1024 x 7168 -> 2048 15.0 / 16.3.
  // A linear's two gradients go in one launch of single CTAs where neither fills
  // the pairs, so for them all pairs have to have work: 570 x 320 -> 8384 22.4 us
  // in one launch, 28.9 with one of them in 66 pairs.
  const int64_t least = g.after_tiles ? num_sms() / 2 : num_sms() / 4;
  p.pair = !p.flip && pairs >= least && pairs * 4 < tiles * 2;
  if (p.pair) {
    p.tiles = static_cast<int>(pairs);
    return p;
  }
  p.tiles = static_cast<int>(p.flip ? (C + 127) / 128 : tiles);
  p.cluster = pick_cluster(p.tiles, (K + 255) / 256, p.flip ? 6.0 : 13.0);
  return p;
}

MxJob job_of(const MxProduct& g, const MxPlan& p) {
  MxJob j{};
  j.m_codes = p.flip ? g.c_codes : g.r_codes;
  j.n_codes = p.flip ? g.r_codes : g.c_codes;
  j.tiles = p.tiles;
  j.a.m_sf = p.flip ? g.c_scales : g.r_scales;
  j.a.n_sf = p.flip ? g.r_scales : g.c_scales;
  j.a.out = g.out;
  j.a.ld_out = g.ld_out;
  j.a.M = static_cast<int>(p.flip ? g.C : g.R);
  j.a.N = static_cast<int>(p.flip ? g.R : g.C);
  j.a.K = static_cast<int>(g.K);
  j.a.out_f32 = g.out_f32;
  j.a.cluster = p.cluster;
  j.a.status = g.status;
  j.a.flags = g.flags;
  j.a.flag_count = g.flag_count;
  j.a.wait_limit_ns = wait_limit_ns();
  return j;
}

}  // namespace

cudaError_t launch_mx_product(const MxProduct& g, cudaStream_t stream) {
  if (g.R == 0 || g.C == 0) return cudaSuccess;
  const MxPlan p = plan_product(g);
  const MxJob j = job_of(g, p);
  if (p.pair) {
    // Six stages cover more of what a load waits for and of a tile's turn, worth
    // most where tiles are short or the SM's memory is all shared memory already;
    // five leave an SM's split of shared memory and cache where the rows' quantiser
    // runs well, so that the two overlap.  Six / five (us): 4096 x 1536 -> 24576
    // 63.3 / 65.7, the gradients of 8192 x 7168 -> 2048 134.7 / 137.2 with their
    // quantiser; 8192 x 2048 -> 7168 46.3 / 44.3, 8192 x 4096 -> 4096 49.6 / 46.6
    // (all with 8 rows staged at a time).
    const bool deep = g.K <= 7 * 256 || g.after_tiles;
    if (g.out_f32) return deep ? launch_pair<float, 6>(j, stream) : launch_pair<float, 5>(j, stream);
    return deep ? launch_pair<__nv_bfloat16, 6>(j, stream) : launch_pair<__nv_bfloat16, 5>(j, stream);
  }
  return p.flip ? launch_tiles<64, true>(&j, 1, stream) : launch_tiles<128, false>(&j, 1, stream);
}

cudaError_t launch_mx_products(const MxProduct& g, const MxProduct& h, cudaStream_t stream) {
  const MxPlan p = plan_product(g), q = plan_product(h);
  if (p.pair || p.flip || q.pair || q.flip || g.R == 0 || h.R == 0) {
    const cudaError_t e = launch_mx_product(g, stream);
    return e != cudaSuccess ? e : launch_mx_product(h, stream);
  }
  const MxJob jobs[2] = {job_of(g, p), job_of(h, q)};
  return launch_tiles<128, false>(jobs, 2, stream);
}

}  // namespace megamoe
