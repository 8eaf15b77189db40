// MXFP4 grouped products of the routed experts for large batches: a pair of
// CTAs on a tile of 256 routed rows x 256 weight rows, as in the dense product
// (mx_gemm.cu), over the persistent expert-major tile schedule of the grouped
// GEMMs.
//
//   gate and up:  the 256 weight rows are the gate and the up rows of the same
//                 128 features, one CTA's memory each; SiLU(gate) * up of a row
//                 is then in one thread, which quantises its blocks of 32
//                 features to MXFP4 (codes row-major, scales in the atom layout
//                 that the down product reads)
//   down:         256 output features; y in BFP16 by rows (one exponent word per
//                 32 columns of a row, all in one lane), through shared memory as
//                 128-byte rows by tensor map
//
// Experts' rows start at multiples of 128 (the caller pads so), so that a CTA's
// 128 rows are whole scale atoms and the rows of a stored box belong to one
// expert.  A tile of at most 128 rows leaves the second CTA without rows of its
// own: it loads its half of the weights and stores nothing.
//
// What bounds it: at some 250 rows an expert the weights from HBM.  48 experts of
// 7168 x 2048, 2003 tokens of 6 slots: gate and up 150 us for 0.81 GB (80 % of the
// measured copy rate, the MMAs busy for 76 %), down 100 us for 0.39 GB and y.  At
// 1024 rows what an SM takes in: 35 KB a K step (one CTA on 128 x 256 takes 51 KB
// for half the product), 600 to 700 cycles against the MMAs' 513.  Measured and
// not kept here: the accumulators with columns in common, the ordinary stores and
// the sixth stage of mx_gemm.cu (316 against 315 us for the layer), and tiles of
// at most 128 rows shared between the two CTAs (314.5 against 313).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "mxfp4.cuh"

namespace megamoe {

namespace {

struct PairMaps {
  CUtensorMap tok, tok_sf, w, w_sf, y;
};

struct PairArgs {
  const int32_t* offsets;
  const int32_t* padded_offsets;
  int E, N, K;  // N: weight rows of an expert
  uint8_t* h_codes;   // gate and up: [rows, N / 4]
  uint8_t* h_scales;  // atom layout of [rows, N / 2]
  uint16_t* y_exp;    // down: [rows, N / 32]
  uint32_t* status;
  uint64_t wait_limit_ns;
};

struct Cfg {
  static constexpr int THREADS = 320;  // producer, MMA issuer, 8 epilogue warps
  static constexpr int STAGES = 5;
  static constexpr int TILE = 128 * 128;  // a CTA's rows of either operand
  static constexpr int SF = 1024;
  static constexpr int OFF_W = TILE;
  static constexpr int OFF_SFT = 2 * TILE;
  static constexpr int OFF_SFW = OFF_SFT + SF;  // all 256 weight rows
  static constexpr int STAGE = OFF_SFW + 2 * SF;
  static constexpr int SF_COLS = 8 + 16;
  static constexpr int SF_COL0 = 256;  // two sets, taken in turn
  static constexpr int STG = 32 * 128;  // 32 rows x 128 bytes per epilogue warp (down)
  static constexpr int STG_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = STG_OFF + kEpiWarps * STG;
  static constexpr int TOFF_OFF = BAR_OFF + 256;
  static constexpr int SMEM = 1024 + TOFF_OFF + 4 * (MEGAMOE_MAX_EXPERTS + 1);
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(STAGE % 1024 == 0, "128-byte swizzle atoms");
};

// s_toff[e] = first tile of expert e (256 rows x one weight tile each),
// s_toff[E] = all tiles.  All threads.
__device__ void build_offsets(const int32_t* offsets, int E, int MT, int* s_toff, int* s_scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (E + Cfg::THREADS - 1) / Cfg::THREADS;
  const int e0 = min(E, tid * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    const int cnt = __ldcg(offsets + e + 1) - __ldcg(offsets + e);
    sum += cnt > 0 ? (cnt + 255) / 256 * MT : 0;
  }
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_scan[warp] = x;
  __syncthreads();
  int base = x - sum;
  for (int w = 0; w < warp; ++w) base += s_scan[w];
  for (int e = e0; e < e1; ++e) {
    const int cnt = __ldcg(offsets + e + 1) - __ldcg(offsets + e);
    s_toff[e] = base;
    base += cnt > 0 ? (cnt + 255) / 256 * MT : 0;
  }
  if (tid == Cfg::THREADS - 1) s_toff[E] = base;
  __syncthreads();
}

template <bool SILU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg::THREADS, 1)
    k_mx_experts_pair(const __grid_constant__ PairMaps maps, const PairArgs p) {
  using C = Cfg;
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
  int* s_toff = reinterpret_cast<int*>(smem + C::TOFF_OFF);
  __shared__ int s_scan[C::THREADS / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int MT = SILU ? p.N / 2 / 128 : p.N / 256;  // weight tiles of an expert
  const int KT = p.K / 256;

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.tok);
    prefetch_tensormap(&maps.tok_sf);
    prefetch_tensormap(&maps.w);
    prefetch_tensormap(&maps.w_sf);
    if (!SILU) prefetch_tensormap(&maps.y);
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
  // the routing was complete before the kernel ahead of this one started
  build_offsets(p.offsets, p.E, MT, s_toff, s_scan);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are there before either is arrived on
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();
  pdl_trigger();
  const int total = s_toff[p.E];
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;  // tiles of this pair

  if (warp == 0) {
    {
      // ------------------------------------------------------------ producer
      // (the whole warp, one lane of it issuing: elect_one)
      const bool leader = elect_one();
      const uint64_t pol_w_once = policy_evict_first(), pol_w_again = policy_evict_normal();
      const uint64_t pol_t = policy_evict_last();
      int stage = 0, issued = 0, e_lo = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first; ok && tile < total; tile += step) {
        const TileInfo ti = decode_tile(tile, s_toff, p.E, MT, e_lo);
        e_lo = ti.e;
        const int poff = __ldg(p.padded_offsets + ti.e);
        const int cnt = __ldg(p.offsets + ti.e + 1) - __ldg(p.offsets + ti.e);
        const int row0 = poff + ti.nt * 256 + rank * 128;
        const bool both = cnt - ti.nt * 256 > 128;  // the second CTA has rows
        const bool mine = rank == 0 || both;
        const uint32_t bytes = 2 * C::STAGE - (both ? 0 : C::TILE + C::SF);
        const uint64_t pol_w = ti.ntiles > 1 ? pol_w_again : pol_w_once;
        // this CTA's block of 128 weight rows at K step 0 (gate and up blocks
        // are neighbours), and the tile's two 128-row groups of scales: groups
        // mt of the expert's gate and up rows, or two neighbours
        const int sf_y = SILU ? ti.mt : ti.e * (p.N / 128) + 2 * ti.mt, sf_z = SILU ? 2 * ti.e : 0;
        const int blk = SILU ? (ti.e * MT + ti.mt) * KT * 2 + rank : (sf_y + rank) * KT;
        for (int kt = 0; kt < KT; ++kt) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          uint8_t* sb = smem + stage * C::STAGE;
          if (leader) {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], bytes);
            const uint32_t bar = cluster_address(&full[stage], 0);
            tma_load_2d_pair(sb + C::OFF_W, &maps.w, bar, 0, (blk + (SILU ? 2 : 1) * kt) * 128, pol_w);
            if (mine) {
              tma_load_2d_pair(sb, &maps.tok, bar, kt * 128, row0, pol_t);
              tma_load_2d_pair(sb + C::OFF_SFT, &maps.tok_sf, bar, kt * 256, row0 >> 7, pol_t);
            }
            tma_load_3d_pair(sb + C::OFF_SFW, &maps.w_sf, bar, kt * 256, sf_y, sf_z, pol_w);
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
      const uint64_t scales = sdesc_atom(smem_u32(smem) + C::OFF_SFT);
      int stage = 0, sets = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int tile = first; ok && tile < total; tile += step) {
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
              mma_mxf4_pair(tmem, sdesc_at(cd, 32 * c), sdesc_at(cd, C::OFF_W + 32 * c),
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
      __syncwarp();
      mbar_drain(drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int half = warp >= 6 ? 1 : 0;
    uint8_t* stg = smem + C::STG_OFF + (warp - 2) * C::STG;
    uint32_t acc_phase = 0;
    int e_lo = 0;
    bool bad = false;
    for (int tile = first; tile < total; tile += step) {
      const TileInfo ti = decode_tile(tile, s_toff, p.E, MT, e_lo);
      e_lo = ti.e;
      const int poff = __ldg(p.padded_offsets + ti.e);
      const int cnt = __ldg(p.offsets + ti.e + 1) - __ldg(p.offsets + ti.e);
      const int in_expert = ti.nt * 256 + rank * 128 + quarter * 32;  // this warp's first row
      const bool valid = in_expert + lane < cnt;
      const int64_t row0 = poff + in_expert;  // a multiple of 32
      if (!mbar_wait(acc_full, acc_phase, abort_flag, p.status, p.wait_limit_ns)) break;
      tc_fence_after();
      const uint32_t base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      uint32_t v[128];  // this lane's row: 64 gate and 64 up values, or 128 of y
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld_32x32b_x32(base + (SILU ? (c >> 1) * 128 + half * 64 + (c & 1) * 32
                                        : half * 128 + 32 * c),
                           v + 32 * c);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty, 0);
      acc_phase ^= 1u;
      if (in_expert >= cnt) continue;  // warp-uniform: none of its rows is the expert's
      if (SILU) {
        const int f = ti.mt * 128 + half * 64, I = p.N / 2;
        uint32_t bytes = 0;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float hv[32];
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float gv = __uint_as_float(v[32 * b + j]), uv = __uint_as_float(v[64 + 32 * b + j]);
            hv[j] = silu_mul(gv, uv);
            m = max(m, __float_as_uint(hv[j]) & 0x7fffffffu);
          }
          const uint32_t byte = mx_scale_byte(m);
          const float inv = mx_inverse(byte);
          uint32_t q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float e8[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e8[j] = hv[8 * i + j];
            q[i] = mx_codes8(e8, inv);
          }
          if (valid)
            *reinterpret_cast<uint4*>(p.h_codes + (row0 + lane) * (I / 2) + f / 2 + 16 * b) =
                make_uint4(q[0], q[1], q[2], q[3]);
          bytes |= byte << (8 * b);
          bad |= valid && byte == kMxNan;
        }
        if (valid)
          *reinterpret_cast<uint16_t*>(p.h_scales + mx_atom_offset(row0 + lane, f >> 5, mx_atoms(I))) =
              static_cast<uint16_t>(bytes);
      } else {
        // BFP16 by rows: this lane's row has four groups of 32 columns here.  The low
        // 16 bits of x + 1.5 * 2^23 + 2^15 are rint(x) + 32768 (x is exact, so the
        // fused sum rounds once, as bfp16_round_int does).
        const int c0 = ti.mt * 256 + half * 128;
        uint32_t w[64], words[2] = {0, 0};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j) m = max(m, v[32 * g + j] & 0x7fffffffu);
          uint32_t word = static_cast<uint32_t>(bfp16_exponent(m)) & 0xffu;
          if (m < 0x7f800000u || !valid) {
            const float sc = bfp16_pow2(-bfp16_row_exponent(word));
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[16 * g + j] = __byte_perm(
                  __float_as_uint(__fmaf_rn(__uint_as_float(v[32 * g + 2 * j]), sc, 12615680.f)),
                  __float_as_uint(__fmaf_rn(__uint_as_float(v[32 * g + 2 * j + 1]), sc, 12615680.f)),
                  0x5410);
          } else {  // Inf or NaN: the exponent of the others
            m = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const uint32_t b = v[32 * g + j] & 0x7fffffffu;
              m = b < 0x7f800000u ? max(m, b) : m;
            }
            word = bfp16_special_word(m);
            const float sc = bfp16_pow2(-bfp16_row_exponent(word));
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[16 * g + j] = bfp16_special_value(__uint_as_float(v[32 * g + 2 * j]), sc) |
                              bfp16_special_value(__uint_as_float(v[32 * g + 2 * j + 1]), sc) << 16;
          }
          words[g >> 1] |= word << (16 * (g & 1));
        }
        if (valid)
          *reinterpret_cast<uint2*>(p.y_exp + (row0 + lane) * (p.N / kRowGroup) + c0 / kRowGroup) =
              make_uint2(words[0], words[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // 64 columns
          if (lane == 0) bulk_store_wait_read();  // the chunk before has left
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)  // 16-byte piece j of the row, swizzled
            *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                make_uint4(w[32 * c + 4 * j], w[32 * c + 4 * j + 1], w[32 * c + 4 * j + 2],
                           w[32 * c + 4 * j + 3]);
          fence_async_shared();
          __syncwarp();
          if (lane == 0) tma_store_2d(&maps.y, stg, c0 + 64 * c, static_cast<int32_t>(row0));
        }
      }
    }
    if (bad) set_status(p.status, MEGAMOE_DEV_NONFINITE);
    if (!SILU && lane == 0) bulk_store_wait();
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

template <bool SILU>
cudaError_t launch_typed(const MxExperts& g, cudaStream_t stream) {
  PairMaps maps;
  const uint64_t rows = static_cast<uint64_t>(g.rows), K = g.K;
  const uint64_t groups = static_cast<uint64_t>(g.E) * (g.N / 128), KT = K / 256;
  const uint64_t sf_row = static_cast<uint64_t>(mx_atoms(g.K)) * 512;
  if (!make_codes_map(&maps.tok, g.act_codes, rows, K / 2, 128) ||
      !make_map(&maps.tok_sf, CU_TENSOR_MAP_DATA_TYPE_UINT32, g.act_scales, sf_row / 4,
                (rows + 127) / 128, sf_row, 256, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      // packed blocks of 128 rows x 128 bytes, swizzled already
      !make_map(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.w_codes, 128, groups * KT * 128, 128, 128,
                128, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      // [2 E][I / 128] groups of gate and up rows, two of the first; or all groups, two of them
      !make_map_3d(&maps.w_sf, g.w_scales, sf_row / 4, SILU ? g.N / 256 : groups,
                   SILU ? 2 * static_cast<uint64_t>(g.E) : 1, sf_row,
                   SILU ? sf_row * (g.N / 256) : sf_row * groups, 256, SILU ? 1 : 2, SILU ? 2 : 1))
    return cudaErrorInvalidValue;
  if (SILU) maps.y = maps.tok;  // not used
  else if (!make_map(&maps.y, CU_TENSOR_MAP_DATA_TYPE_UINT16, g.y, g.N, rows,
                     static_cast<uint64_t>(g.N) * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const PairArgs a{g.offsets,  g.padded_offsets, g.E,     g.N,      g.K,
                   g.h_codes,  g.h_scales,       reinterpret_cast<uint16_t*>(g.y_exp),
                   g.status,   wait_limit_ns()};
  auto kern = k_mx_experts_pair<SILU>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(num_sms() / 2 * 2), dim3(Cfg::THREADS), Cfg::SMEM, stream, maps, a);
}

}  // namespace

cudaError_t launch_mx_experts(const MxExperts& g, cudaStream_t stream) {
  if (g.rows == 0) return cudaSuccess;
  return g.y ? launch_typed<false>(g, stream) : launch_typed<true>(g, stream);
}

}  // namespace megamoe
