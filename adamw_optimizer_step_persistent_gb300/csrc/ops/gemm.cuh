// The matrix product behind the loss and the weight gradients:
//   D[m, n] = sum_k A[m, k] B[n, k],  A and B 16-bit, D in fp32,
// handed to an epilogue tile by tile.
//
// A pair of CTAs (a cluster of two, one CTA per SM) computes a 256 x 256 tile
// (256 x fewer where that fills the last wave of tiles better) with
// tcgen05.mma.cta_group::2: each CTA keeps 128 rows of A and half the tile's
// rows of B per step of 64 in k, so a step moves 32 KB per SM where a CTA of
// its own would move 48 KB for 128 x 256.  Warps of a CTA: eight for the epilogue, one
// that issues the bulk copies, one that issues the tensor-core work (in the
// pair's first CTA).  The accumulators, two of 128 lanes x 256 columns, fill
// the tensor memory: a tile's epilogue runs under the next tile's products.
//
// Either operand may lie in memory with k contiguous ("k-major") or with its
// own index contiguous (A_MN, B_MN: what a product with a transposed matrix
// reads), so no operand is ever transposed in memory.  In shared memory a
// k-major operand is 128 rows of 128 bytes (64 k), the other kind two blocks
// of 64 rows of k, each 128 bytes (64 of its index); both with the 128-byte
// swizzle, which repeats every eight rows (1024 bytes).
#pragma once

#include "ops_device.cuh"
#include "ops_internal.h"

namespace fadam_ops {

constexpr int kTileM = 256, kTileN = 256, kTileK = 64;
constexpr int kStages = 6;
constexpr int kOperandBytes = 128 * kTileK * 2;  // one operand of one stage in one CTA
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpilogueWarps = 8;
constexpr int kGemmThreads = (kEpilogueWarps + 2) * 32;
constexpr int kPiece = 128;  // most columns of a tile that one epilogue warp takes
constexpr int kTmemColumns = 512;
constexpr int kStagingBytes = 4096;  // of one epilogue warp: 32 rows of 128 bytes

struct GemmBarriers {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint32_t tmem;
};
constexpr size_t kGemmSmem =
    1024 + size_t(kStages) * kStageBytes + kEpilogueWarps * kStagingBytes + sizeof(GemmBarriers);
static_assert(kGemmSmem <= 227 * 1024, "shared memory of one CTA");

// How the work is cut: tiles in groups of `group_m` rows of tiles, within a
// group one column of tiles after the other, so that CTA pairs that run at
// the same time share operands in L2; each tile's k steps in `splits` parts.
struct GemmShape {
  int64_t m, n;
  int32_t tile_n;  // a multiple of 32, at most kTileN
  int32_t m_tiles, n_tiles, group_m;
  int32_t k_steps, splits, steps_per_split;
  int64_t items;
  int* status;
};

// Into how many parts to cut k: one, unless the tiles leave most CTA pairs
// idle and each part keeps at least eight steps.
inline int choose_splits(int64_t m, int64_t n, int64_t k, int tile_n, int pairs) {
  const int64_t tiles = ceil_div(m, kTileM) * ceil_div(n, tile_n);
  const int64_t steps = ceil_div(k, kTileK);
  int64_t splits = pairs / tiles;
  if (splits > steps / 8) splits = steps / 8;
  return splits < 2 ? 1 : int(splits);
}

// The tile's columns.  What a step costs is what it loads (256 rows of A, the
// tile's of B), so a narrower tile pays only where it saves waves of tiles:
// 11008 x 4096 outputs of 8192 rows took 434 us in ten waves of 256 columns,
// 613 us in eleven of 224.  Narrower than 256 by 128 only where B's own index
// is contiguous (its boxes are 64 wide and start on 128 bytes).
inline int choose_tile_n(int64_t m, int64_t n, int64_t k, bool b_mn, bool split, int pairs) {
  int best = kTileN;
  int64_t least = 0;
  for (int t = kTileN; t >= (b_mn ? 128 : 64); t -= b_mn ? 128 : 32) {
    const int parts = split ? choose_splits(m, n, k, t, pairs) : 1;
    const int64_t waves = ceil_div(ceil_div(m, kTileM) * ceil_div(n, t) * parts, pairs);
    const int64_t cost = waves * (kTileM + t) * 64 / parts;
    if (t == kTileN || cost * 102 < least * 100) {
      best = t;
      least = cost;
    }
  }
  return best;
}

inline GemmShape gemm_shape(int64_t m, int64_t n, int64_t k, int tile_n, int splits, int* status) {
  GemmShape s{};
  s.m = m;
  s.n = n;
  s.tile_n = tile_n;
  s.m_tiles = int32_t(ceil_div(m, kTileM));
  s.n_tiles = int32_t(ceil_div(n, tile_n));
  s.group_m = 8;
  s.k_steps = int32_t(ceil_div(k, kTileK));
  s.steps_per_split = int32_t(ceil_div(s.k_steps, splits));
  s.splits = int32_t(ceil_div(s.k_steps, s.steps_per_split));
  s.items = int64_t(s.m_tiles) * s.n_tiles * s.splits;
  s.status = status;
  return s;
}

struct GemmItem {
  int m0, n0, split, step0, steps;
};

__device__ __forceinline__ GemmItem gemm_item(const GemmShape& s, int64_t item) {
  GemmItem it;
  const int64_t tile = item / s.splits;
  it.split = int(item - tile * s.splits);
  const int64_t per_group = int64_t(s.group_m) * s.n_tiles;
  const int group = int(tile / per_group);
  const int in_group = int(tile - group * per_group);
  const int rows = min(s.group_m, s.m_tiles - group * s.group_m);
  it.n0 = in_group / rows * s.tile_n;
  it.m0 = (group * s.group_m + in_group % rows) * kTileM;
  it.step0 = it.split * s.steps_per_split;
  it.steps = min(s.steps_per_split, s.k_steps - it.step0);
  return it;
}

// Shared-memory descriptor of an operand: address, distance between blocks of
// 64 of the operand's index (other-major only), 1024 bytes between groups of
// eight rows, 128-byte swizzle.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  const uint64_t lead = MN ? (64 * 128) >> 4 : 1;
  return uint64_t((addr & 0x3ffff) >> 4) | lead << 16 | uint64_t(1024 >> 4) << 32 |
         uint64_t(1) << 46 | uint64_t(2) << 61;
}

// One operand's share of one step: `rows` (at most 128) of its rows from
// `row`, 64 of k from `k`.  Returns the bytes that will arrive.
template <bool MN>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, int row, int rows,
                                             int k, uint32_t bar) {
  if (MN) {
    load_box_pair(dst, map, row, k, bar);
    if (rows > 64) load_box_pair(dst + kOperandBytes / 2, map, row + 64, k, bar);
  } else {
    load_box_pair(dst, map, k, row, bar);
  }
}
// Rows of the boxes that a map must have for it, and the bytes of its boxes.
inline int box_rows(bool mn, int rows) { return mn ? kTileK : rows; }
__host__ __device__ inline int operand_bytes(bool mn, int rows) {
  return (mn ? (rows + 63) / 64 * 64 : rows) * kTileK * 2;
}

// What an epilogue warp works on: rows row0 .. row0 + 31 (one to a lane) and
// `width` columns from `col` of the product, the part of k, the columns'
// address in tensor memory, its staging memory.
struct GemmPiece {
  int64_t row0, col;
  int width, split;
  uint32_t tmem;
  uint32_t acc_empty;  // the accumulator's barrier, in the pair's first CTA
  unsigned char* staging;

  // N (a multiple of 32) columns from column c of this lane's row.
  template <int N>
  __device__ __forceinline__ void load(int c, float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; i += 32) tmem_load32(tmem + c + i, v + i);
    tmem_wait<N>(v);
  }
  // The accumulator has been read.
  __device__ __forceinline__ void release() const {
    fence_before_sync();
    __syncwarp();
    if (threadIdx.x % 32 == 0) bar_arrive_cluster(acc_empty);
  }
};

// Hands 8 kPerUnit columns of a warp's rows, from column c of its piece, to
// `emit` row by row: each lane holds one row's columns (v), and the stores
// want consecutive lanes on consecutive columns, so they go through the warp's
// staging memory, 128 bytes of each row (their 16-byte words exchanged by row
// so that no bank is hit twice).  `pack(v + i)` makes 16 bytes of kPerUnit
// elements; emit(row, column, unit) gets every unit that starts inside the
// piece.
template <int kPerUnit, class Pack, class Emit>
__device__ __forceinline__ void emit_rows(const float (&v)[8 * kPerUnit], const GemmPiece& at, int c,
                                          int64_t rows, Pack pack, Emit emit) {
  const int lane = threadIdx.x % 32;
  uint4* staging = reinterpret_cast<uint4*>(at.staging);
#pragma unroll
  for (int u = 0; u < 8; ++u) staging[lane * 8 + (u ^ (lane & 7))] = pack(v + u * kPerUnit);
  __syncwarp();
  const int u = lane % 8, col = c + u * kPerUnit;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + lane / 8;
    const uint4 unit = staging[r * 8 + (u ^ (r & 7))];
    if (at.row0 + r < rows && col < at.width) emit(at.row0 + r, at.col + col, unit);
  }
  __syncwarp();
}

// Epi: operator()(const GemmPiece&) is called by whole warps, loads the piece,
// and calls release() once.  (Rows beyond m and columns from `width` on hold
// nothing of the product.)
template <class T, bool A_MN, bool B_MN, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ GemmShape shape, const __grid_constant__ Epi epi) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t tiles = (shared_addr(smem_raw) + 1023) & ~1023u;
  unsigned char* staging = smem_raw + (tiles - shared_addr(smem_raw)) + size_t(kStages) * kStageBytes;
  GemmBarriers* bars = reinterpret_cast<GemmBarriers*>(staging + kEpilogueWarps * kStagingBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const int64_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(shared_addr(&bars->full[i]), 1);
      bar_init(shared_addr(&bars->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(shared_addr(&bars->acc_full[i]), 1);
      bar_init(shared_addr(&bars->acc_empty[i]), 2 * kEpilogueWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kEpilogueWarps + 1) tmem_alloc_pair(shared_addr(&bars->tmem), kTmemColumns);
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  fence_after_sync();
  const uint32_t tmem = bars->tmem;

  if (warp == kEpilogueWarps) {
    if (lane == 0) {
      prefetch_map(&map_a);
      prefetch_map(&map_b);
      const int half = shape.tile_n / 2;
      const int step_bytes = 2 * (operand_bytes(A_MN, 128) + operand_bytes(B_MN, half));
      int64_t count = 0;  // steps issued
      bool ok = true;
      for (int64_t item = pair; ok && item < shape.items; item += pairs) {
        const GemmItem it = gemm_item(shape, item);
        for (int i = 0; ok && i < it.steps; ++i, ++count) {
          const int stage = int(count % kStages);
          const unsigned parity = unsigned(count / kStages) & 1;
          // a barrier that no phase has completed passes for the other parity
          ok = bar_wait(shared_addr(&bars->empty[stage]), parity ^ 1, shape.status);
          if (!ok) break;
          if (rank == 0) bar_expect(shared_addr(&bars->full[stage]), step_bytes);
          const uint32_t full = map_rank(shared_addr(&bars->full[stage]), 0);
          const uint32_t a = tiles + stage * kStageBytes, b = a + kOperandBytes;
          const int k = (it.step0 + i) * kTileK;
          load_operand<A_MN>(a, &map_a, it.m0 + int(rank) * 128, 128, k, full);
          load_operand<B_MN>(b, &map_b, it.n0 + int(rank) * half, half, k, full);
        }
      }
      // every stage's copies have landed and been used before the CTA ends
      for (int i = 0; i < kStages; ++i)
        if (int64_t at = count - 1 - i; at >= 0)
          bar_wait(shared_addr(&bars->empty[at % kStages]), unsigned(at / kStages) & 1, shape.status);
    }
  } else if (warp == kEpilogueWarps + 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t kType = T::code == FADAM_DT_BF16 ? 1 : 0;
      // fp32 result, operand types, which operands are not k-major, the tile
      const uint32_t idesc = 1u << 4 | kType << 7 | kType << 10 | uint32_t(A_MN) << 15 |
                             uint32_t(B_MN) << 16 | uint32_t(shape.tile_n / 8) << 17 |
                             uint32_t(kTileM / 16) << 24;
      // 16 of k further on: 32 bytes of a row, or 16 rows
      constexpr uint64_t a_step = A_MN ? (16 * 128) >> 4 : 32 >> 4;
      constexpr uint64_t b_step = B_MN ? (16 * 128) >> 4 : 32 >> 4;
      int64_t count = 0, tile = 0;
      bool ok = true;
      for (int64_t item = pair; ok && item < shape.items; item += pairs, ++tile) {
        const GemmItem it = gemm_item(shape, item);
        const int acc = int(tile & 1);
        ok = bar_wait(shared_addr(&bars->acc_empty[acc]), (unsigned(tile >> 1) & 1) ^ 1, shape.status);
        if (!ok) break;
        fence_after_sync();
        for (int i = 0; i < it.steps; ++i, ++count) {
          const int stage = int(count % kStages);
          ok = bar_wait(shared_addr(&bars->full[stage]), unsigned(count / kStages) & 1, shape.status);
          if (!ok) break;
          fence_after_sync();
          const uint32_t a = tiles + stage * kStageBytes;
          const uint64_t da = operand_desc<A_MN>(a), db = operand_desc<B_MN>(a + kOperandBytes);
#pragma unroll
          for (int k = 0; k < kTileK / 16; ++k)
            mma_pair(tmem + acc * kTileN, da + k * a_step, db + k * b_step, idesc, i > 0 || k > 0);
          commit_pair(shared_addr(&bars->empty[stage]));
        }
        commit_pair(shared_addr(&bars->acc_full[acc]));
      }
    }
  } else {
    const int quarter = warp % 4, half = warp / 4, half_n = shape.tile_n / 2;
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + half * half_n;
    GemmPiece at;
    at.staging = staging + warp * kStagingBytes;
    int64_t tile = 0;
    for (int64_t item = pair; item < shape.items; item += pairs, ++tile) {
      const GemmItem it = gemm_item(shape, item);
      const int acc = int(tile & 1);
      if (!bar_wait(shared_addr(&bars->acc_full[acc]), unsigned(tile >> 1) & 1, shape.status)) break;
      fence_after_sync();
      at.row0 = int64_t(it.m0) + rank * 128 + quarter * 32;
      at.col = int64_t(it.n0) + half * half_n;
      at.width = int(min(int64_t(half_n), shape.n - at.col));
      at.split = it.split;
      at.tmem = lanes + acc * kTileN;
      at.acc_empty = map_rank(shared_addr(&bars->acc_empty[acc]), 0);
      if (at.row0 < shape.m && at.width > 0)
        epi(at);
      else
        at.release();
    }
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == kEpilogueWarps + 1) tmem_free_pair(tmem, kTmemColumns);
}

// Launch over all SMs, a pair of CTAs per two SMs.
template <class T, bool A_MN, bool B_MN, class Epi>
fadam_status launch_gemm(const CUtensorMap& a, const CUtensorMap& b, const GemmShape& shape,
                         const Epi& epi, int sm_count, cudaStream_t stream) {
  auto* kernel = gemm_kernel<T, A_MN, B_MN, Epi>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(kGemmSmem));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  const int64_t pairs = shape.items < sm_count / 2 ? shape.items : sm_count / 2;
  kernel<<<unsigned(2 * pairs), kGemmThreads, kGemmSmem, stream>>>(a, b, shape, epi);
  const cudaError_t l = cudaGetLastError();
  return l == cudaSuccess ? FADAM_OK : cuda_fail(l, "matrix product launch");
}

}  // namespace fadam_ops
