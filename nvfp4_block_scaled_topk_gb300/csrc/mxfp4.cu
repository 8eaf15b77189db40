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

// t / n, by 32-bit division whenever t fits.
__device__ __forceinline__ int64_t task_div(int64_t t, int n) {
  return (t >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(t) / static_cast<uint32_t>(n))
                        : t / n;
}

// Scale byte of the 32-element block that four neighbouring lanes share.
template <typename X>
__device__ __forceinline__ uint32_t block_byte(const Eight<X>& x) {
  uint32_t m = x.widest();
  m = Eight<X>::wider(m, __shfl_xor_sync(kAll, m, 1));
  m = Eight<X>::wider(m, __shfl_xor_sync(kAll, m, 2));
  return mx_scale_byte(Eight<X>::bits(m));
}

__device__ __forceinline__ int64_t scale_offset(int layout, int64_t row, int64_t b, int64_t K) {
  return layout == MEGAMOE_SCALES_MMA ? mx_atom_offset(row, b, mx_atoms(K)) : row * (K / 32) + b;
}

// Along rows.  Four lanes take a 32-element block, eight elements each, so a
// warp reads 256 consecutive elements (a K step) with 16-byte loads and writes
// 128 consecutive bytes of codes; the block's largest value is two shuffles.
// A warp task is four neighbouring steps of a row: their loads are in flight
// together, they share the address arithmetic, and each lane stores one of the
// 32 scale bytes (past the row's end zeros, in the atom layout).  8195 x 7168
// bf16 take 24.2 us (6.1 TB/s), 8192 x 7168 fp32 39.2 us (6.8 TB/s): near the
// copy's rate, with 70 % of the issue slots taken.
constexpr int kRowSteps = 4;

template <typename X>
__global__ void __launch_bounds__(256)
    k_mx_rows(const X* __restrict__ x, int64_t rows, int K, int64_t ld, uint8_t* __restrict__ codes,
              uint8_t* __restrict__ scales, int layout, uint32_t* status, uint32_t* flags) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int groups = (K + 256 * kRowSteps - 1) / (256 * kRowSteps);
  const int end = layout == MEGAMOE_SCALES_MMA ? static_cast<int>(mx_atoms(K)) * 4 : K / 32;
  const int64_t tasks = rows * groups;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  bool bad = false;
  for (int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
       w < tasks; w += warps) {
    const int64_t r = task_div(w, groups);
    const int col = static_cast<int>(w - r * groups) * (256 * kRowSteps) + 8 * lane;
    const X* from = x + r * ld + col;
    Eight<X> e[kRowSteps];
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
      if (col + 256 * i < K) e[i].load(from + 256 * i);
      else e[i].clear();
    }
    uint8_t* to = codes + (r * K + col) / 2;
    uint32_t mine = 0;  // the scale byte that this lane stores: of step lane % 4
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
      const uint32_t byte = block_byte(e[i]);
      if ((lane & 3) == i) mine = byte;
      float v[8];
      e[i].values(v);
      if (col + 256 * i < K)
        *reinterpret_cast<uint32_t*>(to + 128 * i) = mx_codes8(v, mx_inverse(byte));
    }
    // (a step past the end is all zeros: byte 0)
    const int b = (col >> 5) + 8 * (lane & 3);
    if (b < end) scales[scale_offset(layout, r, b, K)] = static_cast<uint8_t>(mine);
    bad |= mine == kMxNan;
  }
  report_nonfinite(bad, status, flags);
}

// Along columns: codes [K, R / 2] and scales of x^T, R = rows up to a multiple
// of 32 (elements past the last row count as zeros); on request the rows' own
// codes and scales from the same read of x.  A block walks over tiles of 256
// rows (fp32: 128) x 64 columns, the next one on its way into shared memory
// (16-byte asynchronous copies) while it encodes the present one.  Down the
// columns a thread takes 32 rows of two neighbouring columns into registers (a
// 2-byte type: one 32-bit word per row, the warp's words consecutive; fp32: one
// column), and their codes go out through shared memory as 128-byte (fp32: 64-byte)
// runs.  Instructions bound it (65 to 70 % of the issue slots), so a thread's
// copies and stores walk pointers and magnitudes and products go two an
// instruction.  8195 x 7168 bf16 along columns 30 to 31 us (4.8 TB/s), 16384 rows 57
// (5.2 TB/s), 8192 x 7168 fp32 42 (6.3 TB/s).  Six blocks of 128 threads an SM
// instead of three of 256, whose runs are 64 bytes long, are 1 to 4 % faster on bf16
// alone (8195 x 7168 29.8 us against 31.0 in a graph), 3 to 4 % slower on fp32, and
// leave a linear's gradients, which read the codes, as they are (8192 x 7168 -> 2048
// 124.3 against 124.5, 4096 x 2048 -> 7168 82.8 against 82.4).
constexpr int kTileCols = 64;
constexpr int kTileThreads = 256;
constexpr int kTileBytes = 128 * kTileThreads;  // of x in a tile, for every type
template <typename X>
constexpr int kTileRows = kTileBytes / kTileCols / static_cast<int>(sizeof(X));
constexpr int kTileCodes = kTileBytes / 4;  // bytes of column codes of a tile

// One row's word of a thread's columns: NC of them.
template <typename X>
struct Word {
  static constexpr int NC = 2;
  uint32_t u;
  __device__ __forceinline__ void load(const X* p) { u = *reinterpret_cast<const uint32_t*>(p); }
  // (the sign bits of what comes out are of no use)
  __device__ __forceinline__ void widen(Word v) { u = wider_pair<X>(u, v.u); }
  __device__ __forceinline__ float value(int c) const;
};
template <>
__device__ __forceinline__ float Word<__nv_bfloat16>::value(int c) const {
  return __uint_as_float(c ? u & 0xffff0000u : u << 16);
}
template <>
__device__ __forceinline__ float Word<__half>::value(int c) const {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(c ? u >> 16 : u)));
}
template <>
struct Word<float> {
  static constexpr int NC = 1;
  uint32_t u;
  __device__ __forceinline__ void load(const float* p) { u = *reinterpret_cast<const uint32_t*>(p); }
  // bit patterns of non-negative values order as the values do
  __device__ __forceinline__ void widen(Word v) { u = max(u, v.u & 0x7fffffffu); }
  __device__ __forceinline__ float value(int) const { return __uint_as_float(u); }
};

// Starts the copies of a tile (zeros outside the matrix).
template <typename X>
__device__ __forceinline__ void load_tile(const MxTile& job, int row_tile, int col_tile,
                                          uint8_t* buf) {
  constexpr int per = 16 / sizeof(X), vecs = kTileCols / per;
  constexpr int rise = kTileThreads / vecs;  // rows between a thread's copies
  const int64_t r0 = static_cast<int64_t>(row_tile) * kTileRows<X> + threadIdx.x / vecs;
  const int c0 = col_tile * kTileCols + threadIdx.x % vecs * per;
  const X* x = static_cast<const X*>(job.x);
  const X* from = x + r0 * job.ld + c0;
  const int64_t hop = rise * job.ld;
  const int64_t left = job.rows - r0;
  const int here = c0 >= job.K ? 0 : left > kTileRows<X> ? kTileRows<X> : static_cast<int>(left);
  const uint32_t to = smem_u32(buf + 16 * threadIdx.x);
#pragma unroll
  for (int i = 0; i < kTileBytes / 16 / kTileThreads; ++i) {
    const bool in = i * rise < here;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + 16 * kTileThreads * i),
                 "l"(in ? from : x), "r"(in ? 16 : 0)
                 : "memory");
    from += hop;
  }
}

template <typename X>
__device__ __forceinline__ bool encode_tile(const MxTile& job, int row_tile, int col_tile,
                                            const uint8_t* buf, uint8_t* s_codes) {
  using W = Word<X>;
  const X* tile = reinterpret_cast<const X*>(buf);  // [kTileRows][kTileCols]
  constexpr int R = kTileRows<X>, blocks = R / 32;
  constexpr int per = 16 / sizeof(X), vecs = kTileCols / per;
  const int K = job.K;
  const int64_t rows = job.rows, padded = (rows + 31) / 32 * 32;
  const int64_t r0 = static_cast<int64_t>(row_tile) * R;
  const int c0 = col_tile * kTileCols;
  bool bad = false;
  if (job.row_codes) {
    const int64_t atoms = mx_atoms(K);
#pragma unroll 2
    for (int i = 0; i < kTileBytes / 16 / kTileThreads; ++i) {
      const int t = threadIdx.x + kTileThreads * i;
      const int r = t / vecs, col = c0 + t % vecs * per;
      const X* e = tile + t * per;
      const uint4 q = *reinterpret_cast<const uint4*>(e);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      float e8[8] = {};
      W word, most;
      most.u = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        word.u = w[j];
        most.widen(word);
#pragma unroll
        for (int c = 0; c < W::NC; ++c) e8[W::NC * j + c] = word.value(c);
      }
      uint32_t m = __float_as_uint(most.value(0)) & 0x7fffffffu;
      if (W::NC == 2) m = max(m, __float_as_uint(most.value(1)) & 0x7fffffffu);
      // the lanes of a row's block of 32 are neighbours
#pragma unroll
      for (int o = 1; o < 32 / per; o <<= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
      const uint32_t byte = mx_scale_byte(m);
      const uint32_t code = mx_codes8(e8, mx_inverse(byte));
      if (r0 + r < rows) {
        if (col < K) {
          uint8_t* to = job.row_codes + ((r0 + r) * K + col) / 2;
          if (per == 8) *reinterpret_cast<uint32_t*>(to) = code;
          else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(code);
          bad |= byte == kMxNan;
        }
        // past the row's end, up to whole K steps: zeros (a zero block's byte)
        if ((col & 31) == 0 && col < atoms * 128)
          job.row_scales[mx_atom_offset(r0 + r, col >> 5, atoms)] = static_cast<uint8_t>(byte);
      }
    }
  }
  if (job.col_codes && c0 < K) {  // block-uniform
    // chunk q (16 bytes) of column c at q ^ (c / NC % 8): the chunks written
    // together (one block of 32 columns) and read together (the blocks of a
    // column) fall in different banks
    constexpr int lanes = kTileCols / W::NC;  // threads across the columns
    const int across = threadIdx.x % lanes, blk = threadIdx.x / lanes;
    const X* from = tile + blk * 32 * kTileCols + W::NC * across;
    W v[32], m;
    m.u = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v[i].load(from + i * kTileCols);
      m.widen(v[i]);
    }
    uint32_t bytes[W::NC];
#pragma unroll
    for (int c = 0; c < W::NC; ++c) {
      const uint32_t byte = mx_scale_byte(__float_as_uint(m.value(c)) & 0x7fffffffu);
      const float inv = mx_inverse(byte);
      uint32_t q[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float e8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e8[i] = v[8 * g + i].value(c);
        q[g] = mx_codes8(e8, inv);
      }
      const int col = W::NC * across + c;
      *reinterpret_cast<uint4*>(s_codes + col * (16 * blocks) +
                                ((blk ^ (across % blocks)) * 16)) = make_uint4(q[0], q[1], q[2], q[3]);
      bytes[c] = byte;
    }
    const int64_t block = r0 / 32 + blk;
    const bool atom = job.col_layout == MEGAMOE_SCALES_MMA;
    const bool stored = block * 32 < rows || (atom && block < mx_atoms(padded) * 4);
    // two neighbouring columns, of which the first is even: rows of one atom
    uint8_t* scale = job.col_scales + scale_offset(job.col_layout, c0 + W::NC * across, block, padded);
#pragma unroll
    for (int c = 0; c < W::NC; ++c) {
      if (c0 + W::NC * across + c < K && stored) {
        scale[c * (atom ? 16 : padded / 32)] = static_cast<uint8_t>(bytes[c]);
        bad |= bytes[c] == kMxNan;
      }
    }
    __syncthreads();
    constexpr int hop = kTileThreads / blocks;  // columns between a thread's chunks
    const int part = threadIdx.x % blocks, col0 = threadIdx.x / blocks;
    uint8_t* to = job.col_codes + (c0 + col0) * (padded / 2) + r0 / 2 + part * 16;
    const bool in = r0 + part * 32 < rows;
#pragma unroll
    for (int i = 0; i < kTileCols / hop; ++i) {
      const int col = col0 + hop * i;
      if (in && c0 + col < K)
        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(
            s_codes + col * (16 * blocks) + ((part ^ (col / W::NC % blocks)) * 16));
      to += hop * (padded / 2);
    }
  }
  return bad;
}

// Up to three matrices in one launch; tile t belongs to the last job whose
// first tile is not past t.  WIDE: one of them may be fp32.
template <bool WIDE>
__global__ void __launch_bounds__(kTileThreads, 768 / kTileThreads)
    k_mx_tiles(const __grid_constant__ MxTiles jobs) {
  extern __shared__ __align__(16) uint8_t s_raw[];  // two tiles, then a tile's column codes
  pdl_wait();
  pdl_trigger();
  auto with = [&](int tile, auto&& f) {  // f(job, row tile, column tile)
    int j = 0;
    while (j + 1 < jobs.count && tile >= jobs.job[j + 1].first) ++j;
    const MxTile& job = jobs.job[j];
    const int t = tile - job.first;
    f(job, t / job.col_tiles, t % job.col_tiles);
  };
  auto load = [&](int tile, uint8_t* buf) {
    with(tile, [&](const MxTile& job, int r, int c) {
      if (WIDE && job.type == MEGAMOE_TYPE_F32) load_tile<float>(job, r, c, buf);
      else load_tile<__half>(job, r, c, buf);  // any 2-byte type
    });
  };
  int turn = 0;
  bool bad = false;
  if (static_cast<int>(blockIdx.x) < jobs.tiles) load(blockIdx.x, s_raw);
  asm volatile("cp.async.commit_group;" ::: "memory");
  for (int tile = blockIdx.x; tile < jobs.tiles; tile += gridDim.x, turn ^= 1) {
    if (tile + static_cast<int>(gridDim.x) < jobs.tiles)
      load(tile + gridDim.x, s_raw + (turn ^ 1) * kTileBytes);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const uint8_t* buf = s_raw + turn * kTileBytes;
    uint8_t* s_codes = s_raw + 2 * kTileBytes;
    with(tile, [&](const MxTile& job, int r, int c) {
      if (WIDE && job.type == MEGAMOE_TYPE_F32) bad |= encode_tile<float>(job, r, c, buf, s_codes);
      else if (job.type == MEGAMOE_TYPE_F16) bad |= encode_tile<__half>(job, r, c, buf, s_codes);
      else bad |= encode_tile<__nv_bfloat16>(job, r, c, buf, s_codes);
    });
    __syncthreads();  // the tile and the codes are free again
  }
  report_nonfinite(bad, jobs.status, jobs.flags);
}

// Token rows into their routed rows: slot j of token t goes to row
// slot_dst[t k + j] (skipped when negative).  A row is encoded once.  A lane takes
// a whole block of 32 elements, so that a copy of 1024 elements is one 16-byte
// store of codes a lane and one word of scales for every four; d is a multiple
// of 256.  Bound by the k copies' stores and, per element, by the encoding: 2003
// tokens of 7168 into 12018 rows 14 us.
__global__ void __launch_bounds__(256)
    k_mx_routed(const __nv_bfloat16* __restrict__ x, int64_t T, int d,
                const int32_t* __restrict__ slot_dst, int k, int atoms, uint8_t* __restrict__ codes,
                uint8_t* __restrict__ scales, uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int blocks = d / 32, groups = (blocks + 31) / 32;
  const int64_t tasks = T * groups;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  bool bad = false;
  for (int64_t w = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
       w < tasks; w += warps) {
    const int64_t t = task_div(w, groups);
    const int b = static_cast<int>(w - t * groups) * 32 + lane;
    const bool in = b < blocks;  // by fours: blocks is a multiple of eight
    const int my_dst = lane < k ? __ldg(slot_dst + t * k + lane) : -1;
    Eight<__nv_bfloat16> e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (in) e[i].load(x + t * d + 32 * b + 8 * i);
      else e[i].clear();
    }
    uint32_t m = e[0].widest();
#pragma unroll
    for (int i = 1; i < 4; ++i) m = Eight<__nv_bfloat16>::wider(m, e[i].widest());
    const uint32_t byte = mx_scale_byte(Eight<__nv_bfloat16>::bits(m));
    const float inv = mx_inverse(byte);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
      e[i].values(v);
      c[i] = mx_codes8(v, inv);
    }
    bad |= byte == kMxNan;
    // lane 4 i: the scale bytes of blocks 4 i .. 4 i + 3
    uint32_t word = byte | (__shfl_down_sync(kAll, byte, 1) << 8);
    word |= __shfl_down_sync(kAll, word, 2) << 16;
    for (int j = 0; j < k; ++j) {
      const int64_t dst = __shfl_sync(kAll, my_dst, j);
      if (dst < 0 || !in) continue;
      *reinterpret_cast<uint4*>(codes + dst * (d / 2) + 16 * b) = make_uint4(c[0], c[1], c[2], c[3]);
      if ((lane & 3) == 0)
        *reinterpret_cast<uint32_t*>(scales + (atoms ? mx_atom_offset(dst, b, d / 128)
                                                     : dst * (d / 16) + mx_routed_offset(b))) = word;
    }
  }
  if (bad) set_status(status, MEGAMOE_DEV_NONFINITE);
}

// Two E2M1 codes (a byte, the even element low) -> two halves.
__device__ __forceinline__ uint32_t e2m1x2_halves(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 t, u;\n\tmov.b16 {t, u}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(r)
      : "h"(static_cast<uint16_t>(byte)));
  return r;
}

// Eight codes times a block's scale -> 16 bytes of bf16 (exact: bf16 holds
// every MXFP4 value).  The five exponent bits of a half moved to the place of
// bf16's eight are the value times 2^-112; two multiplications by powers of two
// bring it up and apply the scale.
__device__ __forceinline__ void store_values(__nv_bfloat16* p, uint32_t codes, uint32_t byte) {
  const __nv_bfloat162 up = __float2bfloat162_rn(__uint_as_float((127u + 112u) << 23));
  const __nv_bfloat162 s = __float2bfloat162_rn(mx_scale_value(byte));
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e2m1x2_halves(codes >> (8 * i) & 0xffu);
    const uint32_t b = (h & 0x80008000u) | ((h & 0x7fff7fffu) >> 3);
    const __nv_bfloat162 v = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), up), s);
    u[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store_values(float* p, uint32_t codes, uint32_t byte) {
  const float s = mx_scale_value(byte);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = e2m1x2_halves(codes >> (16 * i) & 0xffu);
    const uint32_t b = e2m1x2_halves(codes >> (16 * i + 8) & 0xffu);
    const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
    reinterpret_cast<float4*>(p)[i] = make_float4(fa.x * s, fa.y * s, fb.x * s, fb.y * s);
  }
}

// The values: four bytes of codes in, eight elements out per thread, four of
// them at once; no division where the rows of out follow each other.  Bound by
// HBM: 8195 x 7168 to bf16 24.8 us, 16384 rows 48.0 (6.3 TB/s).  Ordinary stores:
// what is read next are the values.  Stored to leave L2 first they took 21.7 and 50.7
// us by themselves, but with a pass over them after it 60.4 against 58.9 and 118
// against 115.6, and at 512 to 2048 rows 3 to 6 % more by themselves too.
template <typename O>
__global__ void __launch_bounds__(256)
    k_mx_values(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows,
                int K, O* __restrict__ out, int64_t ld) {
  pdl_wait();
  pdl_trigger();
  const int vecs = K / 8;
  const int64_t total = rows * vecs;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  constexpr int n = 4;
  for (int64_t i0 = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i0 < total;
       i0 += n * stride) {
    uint32_t c[n], s[n];
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const int64_t i = i0 + j * stride;
      if (i < total) {
        c[j] = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
        s[j] = __ldg(scales + (i >> 2));
      }
    }
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const int64_t i = i0 + j * stride;
      if (i >= total) break;
      int64_t at = i * 8;
      if (ld != K) {
        const int64_t r = task_div(i, vecs);
        at = r * ld + (i - r * vecs) * 8;
      }
      store_values(out + at, c[j], s[j]);
    }
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
cudaError_t quantize_rows(const MxQuant& q, cudaStream_t s, int* blocks) {
  const int64_t tasks = q.rows * ((q.K + 1023) / 1024);
  // enough blocks for every task at small sizes, several tasks a warp at large ones
  const unsigned n = blocks_for(tasks, 8);
  if (blocks) *blocks = static_cast<int>(n);
  return launch_pdl(k_mx_rows<X>, dim3(n), dim3(256), 0, s,
                    static_cast<const X*>(q.x), q.rows, q.K, q.ld, q.codes, q.scales, q.layout,
                    q.status, q.flags);
}

}  // namespace

cudaError_t launch_mx_tiles(MxTiles jobs, cudaStream_t s, int* blocks) {
  jobs.tiles = 0;
  bool wide = false;
  for (int j = 0; j < jobs.count; ++j) {
    MxTile& t = jobs.job[j];
    const int tall = t.type == MEGAMOE_TYPE_F32 ? kTileRows<float> : kTileRows<__half>;
    wide |= t.type == MEGAMOE_TYPE_F32;
    // a row's scales in the atom layout reach to whole K steps of 256
    const int64_t cols = t.row_codes ? mx_atoms(t.K) * 128 : t.K;
    t.col_tiles = static_cast<int>((cols + kTileCols - 1) / kTileCols);
    t.first = jobs.tiles;
    const bool steps = t.col_codes && t.col_layout == MEGAMOE_SCALES_MMA;  // and so do a column's
    const int64_t rows = t.rows == 0 ? 0 : steps ? mx_atoms(t.rows) * 128 : t.rows;
    const int64_t n = (rows + tall - 1) / tall * t.col_tiles;
    if (jobs.tiles + n >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
    jobs.tiles += static_cast<int>(n);
  }
  if (jobs.tiles == 0) return cudaSuccess;
  constexpr int smem = 2 * kTileBytes + kTileCodes;
  auto kern = wide ? k_mx_tiles<true> : k_mx_tiles<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // three blocks an SM by shared memory
  const int n = std::min(jobs.tiles, 768 / kTileThreads * num_sms());
  if (blocks) *blocks = n;
  return launch_pdl(kern, dim3(n), dim3(kTileThreads), smem, s, jobs);
}

int mx_flags_words() { return num_sms() * 16; }

cudaError_t launch_mx_quantize(const MxQuant& q, cudaStream_t s, int* blocks) {
  if (q.rows == 0) return cudaSuccess;
  if (q.transpose) {
    MxTiles jobs{};
    jobs.count = 1;
    jobs.job[0].x = q.x;
    jobs.job[0].type = q.type;
    jobs.job[0].rows = q.rows;
    jobs.job[0].ld = q.ld;
    jobs.job[0].K = q.K;
    jobs.job[0].col_codes = q.codes;
    jobs.job[0].col_scales = q.scales;
    jobs.job[0].col_layout = q.layout;
    jobs.status = q.status;
    jobs.flags = q.flags;
    return launch_mx_tiles(jobs, s, blocks);
  }
  switch (q.type) {
    case MEGAMOE_TYPE_BF16: return quantize_rows<__nv_bfloat16>(q, s, blocks);
    case MEGAMOE_TYPE_F16: return quantize_rows<__half>(q, s, blocks);
    default: return quantize_rows<float>(q, s, blocks);
  }
}

cudaError_t launch_mx_routed(const uint16_t* x, int64_t T, int d, const int32_t* slot_dst, int k,
                             bool atoms, uint8_t* codes, uint8_t* scales, uint32_t* status,
                             cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  return launch_pdl(k_mx_routed, dim3(blocks_for(T * ((d + 1023) / 1024), 8)), dim3(256), 0, s,
                    reinterpret_cast<const __nv_bfloat16*>(x), T, d, slot_dst, k, atoms ? 1 : 0, codes,
                    scales, status);
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
