// Products of 16-bit operands grouped by expert, on tcgen05 tensor cores with
// fp32 accumulation: rows lie in the order of their experts, expert e's are
// [start_e, start_e + count_e), any count.
//
//   forward:      out[r, n]     = sum_k x[r, k] w[e, n, k]
//   grad of x:    grad_x[r, k]  = sum_n grad_out[r, n] w[e, n, k]
//   grad of w:    grad_w[e,n,k] = sum_r grad_out[r, n] x[r, k]
//
// A pair of CTAs (tcgen05.mma cta_group::2) works on a tile.  In the first two
// the weights are the MMA's M side (256 features) and the rows its N side: N is
// the tile's row count rounded up to 16, so an expert with one row pays for 16
// and one with 300 for two tiles of 160, where rows on M would pay for 512.
// The gradient of w sums over rows; its tile is 256 x 256 of one expert.
//
// Operands come by tensor map in the 128-byte swizzle, 64 elements of the
// summed dimension a stage.  Where that dimension is contiguous (x and w of the
// forward, grad_out of grad_x) boxes are K-major; w in grad_x and both operands
// of grad_w are read as they lie, MN-major (64 x 64 boxes, one after another).
//
// Ends.  Features and columns past the matrix read as zeros and are not
// stored.  Rows past an expert's last belong to the next one: as N columns they
// are computed and not stored; where they are summed over (grad_w) one warp of
// each CTA overwrites them with zeros in shared memory before the MMAs read
// them, in both operands, since 0 * Inf is not 0.
//
// Tensor memory holds two accumulators of 256 columns: a tile is read, rounded
// and stored under the next one's products.
//
// What bounds it, as measured.  Few rows an expert: the weights' bytes; 48 experts of
// 4096 x 7168 with 48 rows take 280 us for 1.88 GB (99 % of the copy rate), of 7168 x
// 2048 with 1, 64 and 256 rows each 208, 222 and 259 us (208, 217 and 242 of bytes).
// From there to some 500 rows what an SM takes in, 50 to 55 bytes a cycle: with 272
// rows each expert has two tiles of 144, whose stages of 28 KB take the 560 cycles of
// a full one, 340 us.  Many rows: the MMAs; 16384 rows of eight experts, 7168 x 2048,
// take 266 us forward and for grad_x (1.81 PFLOP/s, 95 % of a library's dense
// product) and 270 us for grad_w in bf16.  Few tiles: 5.8 us for one of 512 x 512,
// launch and the first loads; whole turns of the 76 pairs.
//
// Measured and not kept: tiles of 512 rows, which load the weights once for two parts
// (fewer stages fit: 293 against 340 us at 272 rows, 313 against 259 at 256, 468
// against 467 at 512, and nothing left of it with uneven experts); rows on M.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace megamoe {

namespace {

enum Mode { kForward, kGradX, kGradW };

struct GroupedMaps {
  CUtensorMap m, n;  // the MMA's M and N side
  CUtensorMap n8;    // forward, grad_x: the N side in boxes of 8 rows (n: of 32)
};

struct GroupedArgs {
  const int32_t* offsets;
  const int32_t* padded_offsets;
  int64_t rows;  // of the row matrices
  int E;
  int F;    // features on the M side (N, K or K)
  int G;    // grad_w: features on the N side (N)
  int sum;  // forward, grad_x: length of the sums (K or N)
  void* out;
  int64_t ld_out;
  uint32_t idesc;  // instruction descriptor without N
  int split;       // pairs that share a tile's sum (SPLIT)
  // grad_w right behind grad_x: it needs nothing of it, and that kernel has waited for
  // what both read before it let this one start.  So this one waits for it only at its
  // end, for the sake of the kernel that comes next (both gradients of 8 rows of eight
  // experts of 512 x 512 12.9 us one after the other, 9.2 so; of 4000 rows of 2048 x 2048
  // 80.6 and 73.8).
  bool late_wait;
  uint32_t* status;
  uint64_t wait_limit_ns;
};

struct Cfg {
  static constexpr int THREADS = 384;  // producer, MMA issuer, tail warp, idle; 8 epilogue warps
  // Where sums are added up in parts the epilogue's warps hold 128 each; the first four
  // then give up registers for them (without that some spill: uneven experts' grad_w
  // took 315 us, 300 with it).  A thread's of either (168 at launch):
  static constexpr int FEW_REGS = 64, MANY_REGS = 216;
  static constexpr int STAGES = 6;
  static constexpr int TILE = 128 * 128;  // a CTA's part of either operand
  static constexpr int STAGE = 2 * TILE;
  static constexpr int STG = 2048;  // staged output of an epilogue warp
  static constexpr int STG_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = STG_OFF + kEpiWarps * STG;
  static constexpr int RANGE_OFF = BAR_OFF + 256;  // experts' rows, first tiles
  static constexpr int TOFF_OFF = RANGE_OFF + 8 * MEGAMOE_MAX_EXPERTS;
  static constexpr int SMEM = 1024 + TOFF_OFF + 4 * (MEGAMOE_MAX_EXPERTS + 1);
  static_assert(SMEM <= 232448, "shared memory budget");
};

// kind::f16 over the pair: rows 0 .. 127 of A and D in rank 0's memory, 128 ..
// 255 in rank 1's, half of B's rows in each.
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand in the 128-byte swizzle: atoms of 64 elements x 8 steps of
// the summed dimension (1024 bytes), atoms along that dimension 1024 bytes
// apart, the next 64 elements 8 KB on.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;  // descriptor version
  d |= static_cast<uint64_t>(2) << 61;  // 128-byte swizzle
  return d;
}

// Rows of an expert, kept inside the matrix whatever the offsets say.
struct Range {
  int start, count;
};

// An expert's rows in tiles of equal size, a multiple of 16 up to 256.
__device__ __forceinline__ int tile_rows(int count) {
  const int tiles = (count + 255) / 256;
  return tiles ? ((count + tiles - 1) / tiles + 15) / 16 * 16 : 16;
}

// Experts e0 .. e1 - 1 that share a row with one before them have none.  All threads; its
// own function because code that a call jumps over costs it 0.3 us.
__device__ __noinline__ bool leave_out_shared(Range* s_range, int e0, int e1) {
  uint32_t out = 0;
  for (int e = e0; e < e1; ++e) {
    const Range r = s_range[e];
    for (int f = 0; f < e; ++f) {
      const Range q = s_range[f];
      if (min(r.start + r.count, q.start + q.count) > max(r.start, q.start)) out |= 1u << (e - e0);
    }
  }
  __syncthreads();
  for (int e = e0; e < e1; ++e)
    if (out >> (e - e0) & 1u) s_range[e].count = 0;
  return out != 0;
}

// Experts' rows, and s_toff[e] = first tile of expert e, s_toff[E] = all tiles
// (forward, grad_x).  All threads.  Tiles are at most grouped_tiles, and no two of them
// write one row: rows outside the matrix are left out, and so is an expert that shares a
// row with one before it.  Where experts follow each other, as they do but for broken or
// shuffled offsets, neighbours tell that none does.
__device__ void build_tables(const GroupedArgs& p, int MT, Range* s_range, int* s_toff,
                             int* s_scan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.E + Cfg::THREADS - 1) / Cfg::THREADS;
  const int e0 = min(p.E, tid * per), e1 = min(p.E, e0 + per);
  bool bad = false, back = false;  // (back: starts before its neighbour's end)
  int begin = 0, end = 0;          // of this thread's experts
  auto range = [&](int e) {
    const int64_t o0 = __ldcg(p.offsets + e), o1 = __ldcg(p.offsets + e + 1);
    const int64_t s = p.padded_offsets ? __ldcg(p.padded_offsets + e) : o0;
    const int64_t start = min(max(s, int64_t{0}), p.rows);
    const int64_t count = max(min(s + o1 - o0, p.rows) - start, int64_t{0});
    bad |= start != s || count != o1 - o0;
    return Range{static_cast<int>(start), static_cast<int>(count)};
  };
  Range before{0, 0};  // the warp before's last
  if (lane == 0 && e0 > 0 && e0 < p.E) before = range(e0 - 1);
  for (int e = e0; e < e1; ++e) {
    const Range r = range(e);
    s_range[e] = r;
    if (e == e0) begin = r.start;
    else back |= r.start < end;
    end = r.start + r.count;
  }
  const int left = __shfl_up_sync(0xffffffffu, end, 1);
  if (e0 < e1) back |= begin < (lane ? left : before.start + before.count);
  int sum, x;  // of this thread's tiles; with those of the warp's threads before it
  while (true) {
    sum = 0;
    for (int e = e0; e < e1; ++e) {
      const int count = s_range[e].count, rows = tile_rows(count);
      s_toff[e] = (count + rows - 1) / rows * MT;
      sum += s_toff[e];
    }
    x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    if (!__syncthreads_or(back)) break;
    bad |= leave_out_shared(s_range, e0, e1);
    back = false;
  }
  if (bad && blockIdx.x == 0) set_status(p.status, MEGAMOE_DEV_BAD_OFFSETS);
  int base = x - sum;
  for (int w = 0; w < warp; ++w) base += s_scan[w];
  for (int e = e0; e < e1; ++e) {
    const int t = s_toff[e];
    s_toff[e] = base;
    base += t;
  }
  if (tid == Cfg::THREADS - 1) s_toff[p.E] = base;
  __syncthreads();
}

// Four floats at the same place in CTA `rank` of the cluster.
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
__device__ __forceinline__ void store4(__half* p, float4 v) {
  const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

// A tile as every role sees it.
struct Tile {
  int e;
  int m0;     // first feature
  int n0;     // first row, or (grad_w) first feature of the N side
  int rows;   // rows: of the tile, or those that are summed over
  int start;  // grad_w: the expert's first row
  int n;      // the MMA's N
  int steps;  // stages of the sum
  bool again;  // the weights are read by other tiles, too
  // the first stage of a share of the sum
  __device__ int first(int share, int of) const { return of == 1 ? share * steps : share * steps / of; }
  // grad_w: a stage whose last sixteen rows are not all the expert's
  __device__ bool ragged_at(int i) const { return i == steps - 1 && (rows & 15) != 0; }
};
template <Mode MODE>
__device__ __forceinline__ Tile decode(const GroupedArgs& p, int q, const Range* s_range,
                                       const int* s_toff, int MT, int NT, int* e_lo) {
  Tile t;
  if (MODE == kGradW) {
    t.e = q / (MT * NT);
    const int local = q - t.e * MT * NT, mt = local / NT;
    const Range r = s_range[t.e];
    t.m0 = mt * 256;
    t.n0 = (local - mt * NT) * 256;
    t.start = r.start;
    t.rows = r.count;
    t.n = 256;
    t.steps = (r.count + 63) / 64;
    t.again = true;
  } else {
    const TileInfo ti = decode_tile(q, s_toff, p.E, MT, *e_lo);
    *e_lo = ti.e;
    const Range r = s_range[ti.e];
    const int per = tile_rows(r.count);
    t.e = ti.e;
    t.m0 = ti.mt * 256;
    t.n0 = r.start + ti.nt * per;
    t.start = r.start;
    t.rows = min(per, r.count - ti.nt * per);
    t.n = (t.rows + 15) / 16 * 16;
    t.steps = (p.sum + 63) / 64;
    t.again = ti.ntiles > 1;
  }
  return t;
}

__device__ __forceinline__ void store_rounded(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_rounded(float v, __half* p) { *p = __float2half_rn(v); }

// Sums in tensor memory drop what lies past their last bit, always towards zero: each
// addition of 16 terms up to one unit of 2^-23 of what has been added up (2^20 terms of
// one sign came out 0.7 % short).  So a sum is taken in parts, which the epilogue adds up
// in registers, rounding to nearest: of 512 terms for fp32 results (off by 5e-7 at any
// length), of 1024 for 16-bit ones.  Random sums of 7168 so round to another bf16 than the
// exact ones in 0.06 % of all cases (0.40 in one part, 0.11 in parts of 2048, 0.04 with
// fp32 products).
//
// What that costs (us, one part / parts): 48 experts of 4096 x 7168 with a row each 433 /
// 432, of 7168 x 2048 with 245 rows on average 294 / 295; 16384 rows of eight experts,
// 7168 x 2048, 260 / 263, their grad_w in bf16 288 / 296.  Sums of one part are taken
// without (100 rows of each of eight experts, 1000 -> 520, 9.3 / 9.6).
constexpr int kPart32 = 8, kPart16 = 16;  // stages

// SPLIT: a cluster of p.split pairs shares a tile's sum, and has one tile at most.
// FOLD: sums are taken in parts.
template <Mode MODE, typename O, bool SPLIT, bool FOLD>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    k_grouped_pair(const __grid_constant__ GroupedMaps maps, const GroupedArgs p) {
  using C = Cfg;
  constexpr int STAGES = C::STAGES;
  constexpr bool M_MN = MODE != kForward;  // the M side is read MN-major
  constexpr int SEG = !FOLD ? 1 << 30 : sizeof(O) == 4 ? kPart32 : kPart16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);  // rank 0's
  uint64_t* empty = full + STAGES;
  uint64_t* tail = empty + STAGES;  // grad_w: this CTA's copies of an expert's last stage
  uint64_t* acc_full = tail + STAGES;
  uint64_t* acc_empty = acc_full + 2;  // rank 0's: the epilogue warps of both
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  Range* s_range = reinterpret_cast<Range*>(smem + C::RANGE_OFF);
  int* s_toff = reinterpret_cast<int*>(smem + C::TOFF_OFF);
  __shared__ int s_scan[C::THREADS / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA in its pair, the pair's first CTA in the cluster, this pair's share
  const uint32_t in_cluster = cluster_rank(), head = SPLIT ? in_cluster & ~1u : 0u;
  const int rank = static_cast<int>(in_cluster & 1u);
  const int split = SPLIT ? p.split : 1, share = SPLIT ? static_cast<int>(in_cluster >> 1) : 0;
  const int MT = (p.F + 255) / 256, NT = MODE == kGradW ? (p.G + 255) / 256 : 1;

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.m);
    prefetch_tensormap(&maps.n);
    if (MODE != kGradW) prefetch_tensormap(&maps.n8);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 2);  // rank 0's producer twice, or both tail warps
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
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
  if (MODE != kGradW || !p.late_wait) pdl_wait();
  pdl_trigger();
  build_tables(p, MT, s_range, s_toff, s_scan);
  const int total = MODE == kGradW ? p.E * MT * NT : s_toff[p.E];
  const int step = gridDim.x / (2 * split), first = blockIdx.x / (2 * split);  // tiles of this pair

  if (warp < 4) {
    if (FOLD) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::FEW_REGS));
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      // (the whole warp, one lane of it issuing: elect_one)
      const bool leader = elect_one();
      const uint64_t pol_once = policy_evict_first(), pol_again = policy_evict_normal();
      int stage = 0, issued = 0, e_lo = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int q = first; ok && q < total; q += step) {
        const Tile t = decode<MODE>(p, q, s_range, s_toff, MT, NT, &e_lo);
        const int m0 = t.m0 + rank * 128;
        // forward, grad_x: a CTA has half of N
        const int half = t.n / 2, r0 = t.n0 + rank * half;
        const RowBoxes mine(t.rows - rank * half, half), other(t.rows - (1 - rank) * half, half);
        const uint64_t pol_m = t.again ? pol_again : pol_once;
        for (int i = t.first(share, split); i < t.first(share + 1, split); ++i) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          uint8_t* sm = smem + stage * C::STAGE;
          uint8_t* sn = sm + C::TILE;
          if (leader) {
            const bool ragged = MODE == kGradW && t.ragged_at(i);
            if (rank == 0 && !ragged) {
              mbar_arrive_expect_tx(&full[stage], 2 * C::TILE + (MODE == kGradW ? 2 * C::TILE
                                                                            : mine.bytes() + other.bytes()));
              mbar_arrive(&full[stage]);
            }
            if (MODE == kGradW) {
              const int r = t.start + i * 64, n0 = t.n0 + rank * 128;
              uint32_t bar = cluster_address(&full[stage], head);
              if (ragged) {
                mbar_arrive_expect_tx(&tail[stage], C::STAGE);
                bar = cluster_address(&tail[stage], head + rank);
              }
              tma_load_2d_pair(sm, &maps.m, bar, m0, r, pol_again);
              tma_load_2d_pair(sm + 8192, &maps.m, bar, m0 + 64, r, pol_again);
              tma_load_2d_pair(sn, &maps.n, bar, n0, r, pol_again);
              tma_load_2d_pair(sn + 8192, &maps.n, bar, n0 + 64, r, pol_again);
            } else {
              const uint32_t bar = cluster_address(&full[stage], head);
              if (M_MN) {
                tma_load_3d_pair(sm, &maps.m, bar, m0, i * 64, t.e, pol_m);
                tma_load_3d_pair(sm + 8192, &maps.m, bar, m0 + 64, i * 64, t.e, pol_m);
              } else {
                tma_load_3d_pair(sm, &maps.m, bar, i * 64, m0, t.e, pol_m);
              }
              for (int b = 0; b < mine.large; ++b)
                tma_load_2d_pair(sn + b * 4096, &maps.n, bar, i * 64, r0 + b * 32, pol_again);
              for (int b = 0; b < mine.small; ++b)
                tma_load_2d_pair(sn + b * 1024, &maps.n8, bar, i * 64, r0 + b * 8, pol_again);
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
      drain_pair_copies(full, STAGES, issued, rank, !ok);
      __syncwarp();
    } else if (warp == 1) {
      if (rank == 0) {
        // ---------------------------------------------------------- MMA issuer
        const bool leader = elect_one();
        const uint64_t dm = M_MN ? sdesc_mn(smem_u32(smem)) : sdesc_sw128(smem_u32(smem));
        const uint64_t dn = MODE == kGradW ? sdesc_mn(smem_u32(smem) + C::TILE)
                                           : sdesc_sw128(smem_u32(smem) + C::TILE);
        // 16 of the summed dimension: 32 bytes of a row, or 16 rows of 128 bytes
        constexpr uint32_t AM = M_MN ? 2048 : 32, AN = MODE == kGradW ? 2048 : 32;
        int stage = 0, parts = 0, e_lo = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int q = first; ok && q < total; q += step) {
          const Tile t = decode<MODE>(p, q, s_range, s_toff, MT, NT, &e_lo);
          const uint32_t idesc = p.idesc | static_cast<uint32_t>(t.n >> 3) << 17;
          uint32_t buf = 0;
          const int i0 = t.first(share, split), i1 = t.first(share + 1, split);
          for (int i = i0; i < i1; ++i) {
            const int at = (i - i0) % SEG;  // in its part
            if (at == 0) {
              buf = parts & 1;
              if (!mbar_wait(&acc_empty[buf], (parts >> 1 & 1) ^ 1u, abort_flag, p.status,
                             p.wait_limit_ns)) {
                ok = false;
                break;
              }
              ++parts;
            }
            if (!mbar_wait(&full[stage], phase, abort_flag, p.status, p.wait_limit_ns)) {
              ok = false;
              break;
            }
            if (MODE == kGradW && t.ragged_at(i)) fence_cluster();  // the tail warps' zeros
            tc_fence_after();
            const uint64_t cm = sdesc_at(dm, stage * C::STAGE), cn = sdesc_at(dn, stage * C::STAGE);
            // sixteens of the last stage that hold nothing are left out
            const int left = (MODE == kGradW ? t.rows : p.sum) - i * 64;
            if (leader) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (16 * c < left)
                  mma_f16_pair(tmem + buf * 256, sdesc_at(cm, AM * c), sdesc_at(cn, AN * c), idesc,
                               (at != 0 || c != 0) ? 1u : 0u);
              tc_commit_pair(&empty[stage], head);
              if (at == SEG - 1 || i == i1 - 1) tc_commit_pair(&acc_full[buf], head);
            }
            __syncwarp();
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // every MMA issued so far must finish before tensor memory is released
        if (leader) tc_commit_pair(drain, head);
        __syncwarp();
        mbar_drain(drain, 0);
      }
      __syncwarp();
    } else if (MODE == kGradW && warp == 2) {
      {
        // ---------------------------------------------------------- tail warp
        // in an expert's last stage the rows past its end become zeros, up to the
        // sixteen that are read; the other stages go from the copies to the MMAs
        int at = 0, e_lo = 0;
        uint32_t phases = 0;  // a bit for each stage's barrier
        for (int q = first; q < total; q += step) {
          const Tile t = decode<MODE>(p, q, s_range, s_toff, MT, NT, &e_lo);
          at = (at + t.steps) % STAGES;
          if (!t.ragged_at(t.steps - 1)) continue;
          const int stage = (at + STAGES - 1) % STAGES;
          if (!mbar_wait(&tail[stage], phases >> stage & 1u, abort_flag, p.status, p.wait_limit_ns)) break;
          phases ^= 1u << stage;
          uint8_t* sb = smem + stage * C::STAGE;
          const int left = t.rows - (t.steps - 1) * 64;
          const int end = (left + 15) / 16 * 16;  // rows of 128 bytes in each of four boxes
          for (int v = left * 8 + lane; v < end * 8; v += 32)
#pragma unroll
            for (int b = 0; b < 4; ++b)
              *reinterpret_cast<uint4*>(sb + b * 8192 + v * 16) = make_uint4(0, 0, 0, 0);
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(&full[stage], head);
          __syncwarp();
        }
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    if (FOLD) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::MANY_REGS));
    const int quarter = warp & 3;
    const int half = warp >= 8 ? 1 : 0;
    uint8_t* stg = smem + C::STG_OFF + (warp - 4) * C::STG;
    // A lane has a feature, a column is a row of the output.  The two warps of a
    // quarter take chunks of 32 columns in turn.
    O* out = static_cast<O*>(p.out);
    int parts = 0, e_lo = 0;
    bool ok = true;
    for (int q = first; ok && q < total; q += step) {
      const Tile t = decode<MODE>(p, q, s_range, s_toff, MT, NT, &e_lo);
      const int m = t.m0 + rank * 128 + quarter * 32;  // this warp's first feature
      // rows of the output: the tile's, or (grad_w) features of the other side
      const int rows = MODE == kGradW ? min(256, p.G - t.n0) : t.rows;
      const int chunks = (rows + 31) / 32;
      const int64_t row0 = (MODE == kGradW ? static_cast<int64_t>(t.e) * p.G : 0) + t.n0;
      O* at = out + row0 * p.ld_out + m;
      auto chunk_of = [&](int c) { return half + 2 * c; };
      auto let_go = [&](uint32_t buf) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(&acc_empty[buf], head);
      };
      float sum[FOLD ? 4 : 1][32];
      if (FOLD) {  // the parts, and the accumulator's back before anything is stored
#pragma unroll
        for (int c = 0; c < 4 * FOLD; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
        for (int i = t.first(share, split); i < t.first(share + 1, split); i += SEG, ++parts) {
          const uint32_t buf = parts & 1;
          if (!mbar_wait(&acc_full[buf], parts >> 1 & 1, abort_flag, p.status, p.wait_limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t base = tmem + buf * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (chunk_of(c) >= chunks) continue;
            uint32_t v[32];
            tmem_ld_32x32b_x32(base + 32 * chunk_of(c), v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[c * FOLD][j] += __uint_as_float(v[j]);
          }
          let_go(buf);
        }
      } else if (t.steps != 0) {
        ok = mbar_wait(&acc_full[parts & 1], parts >> 1 & 1, abort_flag, p.status, p.wait_limit_ns);
        tc_fence_after();
      }
      if (!ok) break;
      if constexpr (SPLIT) {
        // this pair's share of the sums, fp32 [rows][128 features], where the stages were
        float* to = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
        const uint32_t buf = parts & 1;
        const uint32_t base = tmem + buf * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (chunk_of(c) >= chunks) continue;
          float v[32];
          if constexpr (FOLD) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = sum[c][j];
          } else {
            uint32_t u[32];
            tmem_ld_32x32b_x32(base + 32 * chunk_of(c), u);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) to[(32 * chunk_of(c) + j) * 128] = v[j];
        }
        if (!FOLD) let_go(buf);
      } else if constexpr (sizeof(O) == 4) {
        // fp32: 32 features of a row are 128 bytes as they lie
        if (m + lane < p.F) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float* to = at + 32 * chunk_of(c) * p.ld_out + lane;
#pragma unroll
            for (int j = 0; j < 32; ++j, to += p.ld_out)
              if (32 * chunk_of(c) + j < rows) __stcs(to, sum[c][j]);
          }
        }
        __syncwarp();
      } else {
        // 16 bits: 64 bytes of 32 features of a row, through shared memory
        const uint32_t buf = parts & 1;
        const uint32_t base = tmem + buf * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
        const int piece = lane & 3;
        const bool in = m + piece * 8 < p.F;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (chunk_of(c) >= chunks) continue;
          float v[32];
          if constexpr (FOLD) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = sum[c][j];
          } else {
            uint32_t u[32] = {};
            if (t.steps != 0) {
              tmem_ld_32x32b_x32(base + 32 * chunk_of(c), u);
              tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
          }
          if (m >= p.F) continue;  // warp-uniform
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            store_rounded(v[j], reinterpret_cast<O*>(stg) + j * 32 + lane);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = j * 8 + (lane >> 2), row = 32 * chunk_of(c) + r;
            const uint4 x = *reinterpret_cast<const uint4*>(stg + r * 64 + piece * 16);
            if (in && row < rows) *reinterpret_cast<uint4*>(at + row * p.ld_out + piece * 8) = x;
          }
        }
        if (!FOLD && t.steps != 0) {
          let_go(buf);
          ++parts;
        }
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if constexpr (SPLIT) {
    // Each pair adds up its share of the tile's rows over the cluster, in the pairs'
    // order; a CTA its 128 features, a warp a row at a time.
    cluster_sync();  // all shares are there
    if (first < total) {
      int e_lo = 0;
      const Tile t = decode<MODE>(p, first, s_range, s_toff, MT, NT, &e_lo);
      const int m = t.m0 + rank * 128 + lane * 4;
      const int end = (share + 1) * t.rows / split;
      for (int r = share * t.rows / split + warp; r < end; r += C::THREADS / 32) {
        const float* from = reinterpret_cast<const float*>(smem) + r * 128 + lane * 4;
        float4 sum = load_cluster4(from, rank);
        for (int s = 1; s < split; ++s) {
          const float4 v = load_cluster4(from, 2 * s + rank);
          sum.x += v.x;
          sum.y += v.y;
          sum.z += v.z;
          sum.w += v.w;
        }
        if (m < p.F) store4(static_cast<O*>(p.out) + (t.n0 + static_cast<int64_t>(r)) * p.ld_out + m, sum);
      }
    }
  }
  // the first CTA's commits arrive on the other's barriers too: none is on its way after
  // the last
  if (warp == 1) mbar_drain(drain, 0);
  __syncwarp();
  cluster_sync();  // no CTA leaves while another still reaches into it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  if (MODE == kGradW && p.late_wait) pdl_wait();
}

template <Mode MODE, typename O, bool SPLIT, bool FOLD>
cudaError_t launch_typed(const GroupedMaps& maps, const GroupedArgs& a, int64_t tiles,
                         cudaStream_t stream) {
  auto kern = k_grouped_pair<MODE, O, SPLIT, FOLD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  if (FOLD) {
    // what the warps hold after giving up and taking registers is what they start with
    static std::atomic<bool> fits{false};
    cudaFuncAttributes f;
    if (!fits.load(std::memory_order_relaxed)) {
      if ((e = cudaFuncGetAttributes(&f, kern)) != cudaSuccess) return e;
      if (f.numRegs * Cfg::THREADS < 128 * Cfg::FEW_REGS + 256 * Cfg::MANY_REGS)
        return cudaErrorInvalidConfiguration;
      fits.store(true, std::memory_order_relaxed);
    }
  }
  const int64_t pairs = SPLIT ? tiles * a.split : std::min<int64_t>(std::max(num_sms() / 2, 1), tiles);
  return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(Cfg::THREADS), Cfg::SMEM,
                            SPLIT ? 2 * a.split : 2, stream, maps, a);
}

// Pairs that share a tile's sum, where the others would idle.  Clusters of 4, 6 and 8
// CTAs of which each fills an SM fit the GPU 36, 23 and 15 times; the exchange and the
// sums over the cluster cost about eight stages, and some five more for 256 rows.
// Whole / shared, us: 8 rows, one expert of 7168 -> 2048 (8 tiles) 29.7 / 15.2, -> 4096
// 29.8 / 18.6, -> 7168 (28 tiles) 30.1 / 24.3; 64 rows of 4096 -> 4096 19.4 / 14.7; 1000
// rows of 7168 -> 512 35.4 / 20.5; 64 rows of eight of 2048 -> 1024 12.2 / 11.8.
int share_sum(const GroupedArgs& a, int64_t tiles) {
  static constexpr int kMost[] = {0, 0, 34, 22, 14};  // tiles, by pairs
  const double steps = (a.sum + 63) / 64, rows = std::min(256.0, static_cast<double>(a.rows) / a.E);
  int best = 1;
  double least = steps;
  for (int s = 2; s <= 4; ++s) {
    const double cost = steps / s + 8 + rows / 50;
    if (tiles <= kMost[s] && cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

// In parts, unless a 16-bit result's sum (a pair's share of it) is one at most.
template <Mode MODE, typename O, bool SPLIT>
cudaError_t launch_parts(const GroupedMaps& maps, const GroupedArgs& a, int64_t tiles,
                         cudaStream_t stream) {
  if constexpr (sizeof(O) == 2) {
    const int64_t stages = ((MODE == kGradW ? a.rows : a.sum) + 63) / 64;
    if ((stages + a.split - 1) / a.split <= kPart16)
      return launch_typed<MODE, O, SPLIT, false>(maps, a, tiles, stream);
  }
  return launch_typed<MODE, O, SPLIT, true>(maps, a, tiles, stream);
}

template <Mode MODE, typename O>
cudaError_t launch_shared(const GroupedMaps& maps, GroupedArgs a, int64_t tiles, cudaStream_t stream) {
  a.split = 1;
  if constexpr (MODE != kGradW) {
    a.split = share_sum(a, tiles);
    if (a.split > 1) return launch_parts<MODE, O, true>(maps, a, tiles, stream);
  }
  return launch_parts<MODE, O, false>(maps, a, tiles, stream);
}

template <Mode MODE>
cudaError_t launch_mode(const GroupedMaps& maps, const GroupedArgs& a, int out_type, int64_t tiles,
                        cudaStream_t stream) {
  if constexpr (MODE != kGradX)
    if (out_type == MEGAMOE_TYPE_F32) return launch_shared<MODE, float>(maps, a, tiles, stream);
  if (out_type == MEGAMOE_TYPE_F16) return launch_shared<MODE, __half>(maps, a, tiles, stream);
  return launch_shared<MODE, __nv_bfloat16>(maps, a, tiles, stream);
}

// [E, N, K] weights, boxes of 64 x `rows`.
bool weight_map(CUtensorMap* map, const Grouped& g, uint32_t rows) {
  const uint64_t row = static_cast<uint64_t>(g.K) * 2;
  return make_map_3d(map, g.w, g.K, g.N, g.E, row, row * g.N, 64, rows, 1,
                     CU_TENSOR_MAP_DATA_TYPE_UINT16, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool rows_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t ld,
              uint32_t box) {
  return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, base, cols, rows,
                  static_cast<uint64_t>(ld) * 2, 64, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Instruction descriptor (kind::f16) without N: fp32 sums, M = 256, MN-major sides.
uint32_t idesc_f16(int type, bool m_mn, bool n_mn) {
  const uint32_t format = type == MEGAMOE_TYPE_BF16 ? 1u : 0u;
  return (1u << 4) | format << 7 | format << 10 | (m_mn ? 1u << 15 : 0u) | (n_mn ? 1u << 16 : 0u) |
         (256u >> 4) << 24;
}

GroupedArgs args_of(const Grouped& g) {
  GroupedArgs a{};
  a.offsets = g.offsets;
  a.padded_offsets = g.padded_offsets;
  a.rows = g.rows;
  a.E = g.E;
  a.status = g.status;
  a.wait_limit_ns = wait_limit_ns();
  return a;
}

}  // namespace

cudaError_t launch_grouped_forward(const Grouped& g, void* out, int out_type, int64_t ld_out,
                                   cudaStream_t stream) {
  if (g.rows == 0) return cudaSuccess;
  GroupedMaps maps;
  if (!weight_map(&maps.m, g, 128) || !rows_map(&maps.n, g.x, g.K, g.rows, g.ld_x, 32) ||
      !rows_map(&maps.n8, g.x, g.K, g.rows, g.ld_x, 8))
    return cudaErrorInvalidValue;
  GroupedArgs a = args_of(g);
  a.F = g.N;
  a.sum = g.K;
  a.out = out;
  a.ld_out = ld_out;
  a.idesc = idesc_f16(g.type, false, false);
  return launch_mode<kForward>(maps, a, out_type, grouped_tiles(g.rows, g.E, g.N), stream);
}

cudaError_t launch_grouped_grad_x(const Grouped& g, void* out, int64_t ld_out, cudaStream_t stream) {
  if (g.rows == 0) return cudaSuccess;
  GroupedMaps maps;
  if (!weight_map(&maps.m, g, 64) || !rows_map(&maps.n, g.grad, g.N, g.rows, g.ld_grad, 32) ||
      !rows_map(&maps.n8, g.grad, g.N, g.rows, g.ld_grad, 8))
    return cudaErrorInvalidValue;
  GroupedArgs a = args_of(g);
  a.F = g.K;
  a.sum = g.N;
  a.out = out;
  a.ld_out = ld_out;
  a.idesc = idesc_f16(g.type, true, false);
  const int64_t tiles = grouped_tiles(g.rows, g.E, g.K);
  return launch_mode<kGradX>(maps, a, g.type, tiles, stream);
}

cudaError_t launch_grouped_grad_w(const Grouped& g, void* out, int out_type, bool after_grad_x,
                                  cudaStream_t stream) {
  GroupedArgs a = args_of(g);
  a.late_wait = after_grad_x;
  a.F = g.K;
  a.G = g.N;
  a.out = out;
  a.ld_out = g.K;
  a.idesc = idesc_f16(g.type, true, true);
  if (g.rows == 0)  // nothing to add up
    return cudaMemsetAsync(out, 0, static_cast<size_t>(g.E) * g.N * g.K *
                                       (out_type == MEGAMOE_TYPE_F32 ? 4 : 2), stream);
  GroupedMaps maps;
  if (!rows_map(&maps.m, g.x, g.K, g.rows, g.ld_x, 64) ||
      !rows_map(&maps.n, g.grad, g.N, g.rows, g.ld_grad, 64))
    return cudaErrorInvalidValue;
  maps.n8 = maps.n;  // not used
  const int64_t tiles = static_cast<int64_t>(g.E) * ((g.N + 255) / 256) * ((g.K + 255) / 256);
  return launch_mode<kGradW>(maps, a, out_type, tiles, stream);
}

}  // namespace megamoe
