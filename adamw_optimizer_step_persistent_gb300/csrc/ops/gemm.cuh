// The matrix product behind the loss and the weight gradients:
//   D[m, n] = sum_k A[m, k] B[n, k],  A and B 16-bit, D in fp32,
// handed to an epilogue tile by tile.
//
// A pair of CTAs (a cluster of two, one CTA per SM) computes a 256 x 256 tile
// (256 x fewer where that fills the last wave of tiles better) with
// tcgen05.mma.cta_group::2: each CTA keeps 128 rows of A and half the tile's
// rows of B per step of 64 in k, so a step moves 32 KB per SM where a CTA of
// its own would move 48 KB for 128 x 256.  Warps of a CTA: eight for the
// epilogue, one for each operand's bulk copies, one that issues the tensor-core
// work (in the pair's first CTA), one that is idle.  The accumulators, two of
// 128 lanes x 256 columns, fill the tensor memory: while one is filled, the
// epilogue's warps read the other.
//
// The tensor cores' fp32 additions truncate: each of the k / 16 of a sum loses
// half a unit of the sum so far on average, always towards zero.  Whole sums
// were off by 2.5e-4 of themselves over 40000 terms of one sign and by 5e-4 over
// 131072.  So they add only a chunk of some 1024 of k, and the epilogue's warps
// add the chunks in registers, rounded to nearest, under the next chunk's
// products.  Holding a whole piece there costs 1 to 2% (the weight gradient of
// 8192 x 4096 x 11008 420 us in place of 412), chunks of 16, 32 or all steps
// the same.
//
// Bound by the tensor cores, and they by the card's power: 2048 x 4096 x 32000
// in 285 to 300 us, 1.8 to 1.9 PFLOP/s, 4096 x 11008 x 8192 in 385.  A step of
// 64 in k takes about 550 cycles where the instructions alone take 512; a tile
// some 1500 more, which shows when k is short (1037 x 1000 x 50021: 16 steps to
// a tile, 60%).
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
constexpr int kLoadA = kEpilogueWarps, kLoadB = kLoadA + 1, kMultiply = kLoadA + 2;  // the other warps
constexpr int kGemmThreads = (kEpilogueWarps + 4) * 32;  // whole groups of four warps; one is idle
// Registers of a thread: 168 as launched (384 threads in 65536); the epilogue's
// warps, which hold 128 sums each, take over what the other four do without
// (with 224 and 56 the 16-bit instances spill 100 bytes).
constexpr int kLaunchRegisters = 168, kEpilogueRegisters = 232, kOtherRegisters = 40;
static_assert(2 * kEpilogueRegisters + kOtherRegisters == 3 * kLaunchRegisters, "no more than launched with");
static_assert(kEpilogueWarps == 8 && kLaunchRegisters * kGemmThreads <= 65536, "an SM's registers");
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

// How the work is cut.  Tiles go in groups of `group_m` rows of tiles, within
// a group one column of tiles after the other, so that CTA pairs that run at
// the same time share operands in L2.  The first `full` tiles are whole items;
// the rest are cut along k into `splits` items each, whose sums go to scratch
// memory and are joined by a second kernel.
struct GemmShape {
  int64_t m, n;
  int32_t tile_n;  // a multiple of 32, at most kTileN
  int32_t m_tiles, n_tiles, group_m;
  int32_t full, splits;
  int32_t k_steps, steps_per_split;
  int32_t items;
  int32_t a_box, b_box;  // rows of a k-major operand's box
  int32_t chunk;         // steps of k that the tensor cores add up
  int* status;
};

// A product's plan: the tile's columns, and how its tiles become items.
struct GemmPlan {
  int tile_n, full, splits;
  int64_t rest;  // tiles that are split
};

// Rows of a split tile's sums in scratch memory.
__host__ __device__ inline int64_t split_rows(int64_t m) { return m < kTileM ? m : kTileM; }
inline size_t split_bytes(int64_t m, const GemmPlan& p) {
  return p.splits > 1 ? size_t(p.rest) * p.splits * split_rows(m) * p.tile_n * sizeof(float) : 0;
}

// The plan with the least estimated time, in steps of a 256-column tile.  A
// step costs what it loads (256 rows of A, the tile's of B), so a narrower
// tile pays only where it saves waves of tiles: 11008 x 4096 outputs of 8192
// rows took 434 us in ten waves of 256 columns, 613 us in eleven of 224.  An
// item costs six steps more (the ring's fill, the epilogue's end), split sums
// their way through memory.  Where B's own index is contiguous its boxes are
// 64 wide and start on 128 bytes, so its tiles are 256 or 128.
inline GemmPlan plan_gemm(int64_t m, int64_t n, int64_t k, bool b_mn, bool may_split, int pairs) {
  GemmPlan best{};
  double least = 0;
  const int64_t steps = ceil_div(k, kTileK);
  for (int t = kTileN; t >= (b_mn ? 128 : 64); t -= b_mn ? 128 : 32) {
    const int64_t tiles = ceil_div(m, kTileM) * ceil_div(n, t);
    const double step = double(kTileM + t) / (2 * kTileM);
    // whole waves first; split the rest, or the rest and one wave
    for (int64_t full = tiles / pairs * pairs; full >= 0; full -= pairs) {
      const int64_t rest = tiles - full;
      for (int64_t s = 1; s <= (may_split && rest ? 32 : 1) && (s == 1 || steps / s >= 8); ++s) {
        const double sums = s > 1 ? double(rest) * s * split_rows(m) * t * 8 / 6.7e12 / 0.34e-6 + 12 : 0;
        const double cost = (full / pairs * (steps + 6) +
                             ceil_div(rest * s, pairs) * (ceil_div(steps, s) + 6)) * step + sums;
        // (filling the last wave also lowers the clock that the card's power allows:
        // less than 7% estimated came to nothing)
        if (least == 0 || cost < least * (s > 1 ? 0.93 : 0.98)) {
          least = cost;
          best = {t, int(s > 1 ? full : tiles), int(s), s > 1 ? rest : 0};
        }
      }
      if (full < pairs || tiles - full > pairs) break;
    }
  }
  return best;
}

inline GemmShape gemm_shape(int64_t m, int64_t n, int64_t k, const GemmPlan& plan, int* status) {
  GemmShape s{};
  s.m = m;
  s.n = n;
  s.tile_n = plan.tile_n;
  s.m_tiles = int32_t(ceil_div(m, kTileM));
  s.n_tiles = int32_t(ceil_div(n, plan.tile_n));
  s.group_m = 8;
  s.k_steps = int32_t(ceil_div(k, kTileK));
  const int32_t tiles = s.m_tiles * s.n_tiles;
  s.full = plan.splits > 1 && plan.full < tiles ? plan.full : tiles;
  s.steps_per_split = int32_t(ceil_div(s.k_steps, plan.splits));
  s.splits = int32_t(ceil_div(s.k_steps, s.steps_per_split));
  s.items = s.full + (tiles - s.full) * s.splits;
  s.a_box = m < 128 ? int32_t(round_up(m, 8)) : 128;
  s.b_box = plan.tile_n / 2;
  // 16 steps, or as many as make even chunks of about that (17 steps are one
  // chunk, not 16 and one)
  s.chunk = int32_t(ceil_div(s.steps_per_split, s.steps_per_split < 24 ? 1 : (s.steps_per_split + 8) / 16));
  s.status = status;
  return s;
}

struct GemmItem {
  int m0, n0, step0, steps;
  int slot;  // of a split tile's part: (tile - full) * splits + split; else -1
};

__device__ __forceinline__ void gemm_tile(const GemmShape& s, unsigned tile, int& m0, int& n0) {
  const unsigned per_group = unsigned(s.group_m) * unsigned(s.n_tiles);
  const unsigned group = tile / per_group, in_group = tile - group * per_group;
  const unsigned rows = min(unsigned(s.group_m), unsigned(s.m_tiles) - group * s.group_m);
  const unsigned col = in_group / rows;
  n0 = int(col) * s.tile_n;
  m0 = int(group * s.group_m + in_group - col * rows) * kTileM;
}
// The steps of an item alone, for the thread that needs no more.
__device__ __forceinline__ int gemm_steps(const GemmShape& s, int item, int& step0) {
  if (item < s.full) {
    step0 = 0;
    return s.k_steps;
  }
  step0 = int(unsigned(item - s.full) % unsigned(s.splits)) * s.steps_per_split;
  return min(s.steps_per_split, s.k_steps - step0);
}
__device__ __forceinline__ GemmItem gemm_item(const GemmShape& s, int item) {
  GemmItem it;
  it.steps = gemm_steps(s, item, it.step0);
  it.slot = item < s.full ? -1 : item - s.full;
  gemm_tile(s, item < s.full ? item : s.full + unsigned(item - s.full) / unsigned(s.splits), it.m0, it.n0);
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

// One operand's share of one step, for one CTA: its rows from `row`, 64 of k
// from `k`, in one box of `box` rows (or up to two of 64 columns where its own
// index is contiguous).  Boxes that lie wholly outside the matrix's `limit`
// rows are left out: what their place holds reaches only results that are not
// stored.
template <bool MN>
__device__ __forceinline__ int operand_boxes(int row, int box, int64_t limit) {
  if (row >= limit) return 0;
  return MN && box > 64 && row + 64 < limit ? 2 : 1;
}
template <bool MN>
__device__ __forceinline__ int box_bytes(int box) { return (MN ? 64 : box) * kTileK * 2; }
template <bool MN>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, int row, int boxes,
                                             int k, uint32_t bar) {
  if (boxes > 0) load_box_pair(dst, map, MN ? row : k, MN ? k : row, bar);
  if (MN && boxes > 1) load_box_pair(dst + kOperandBytes / 2, map, row + 64, k, bar);
}
// Rows of the boxes of an operand's map.
inline int box_rows(bool mn, int box) { return mn ? kTileK : box; }

// The thread that loads one operand: its boxes of every step of this CTA's
// items into the ring.  The pair's first CTA counts what arrives in both.
template <bool MN>
__device__ __forceinline__ void load_loop(const GemmShape& shape, const CUtensorMap* map,
                                          GemmBarriers* bars, uint32_t to, bool is_a, int box,
                                          uint32_t rank) {
  prefetch_map(map);
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int apart = is_a ? 128 : shape.tile_n / 2;  // from the first CTA's rows to the second's
  const int64_t limit = is_a ? shape.m : shape.n;
  int stage = 0;
  unsigned parity = 1;  // a barrier that no phase has completed passes for parity 1
  int64_t count = 0;    // steps issued
  bool ok = true;
  for (int item = pair; ok && item < shape.items; item += pairs) {
    const GemmItem it = gemm_item(shape, item);
    const int first = is_a ? it.m0 : it.n0, row = first + int(rank) * apart;
    const int boxes = operand_boxes<MN>(row, box, limit);
    const int bytes = (operand_boxes<MN>(first, box, limit) +
                       operand_boxes<MN>(first + apart, box, limit)) * box_bytes<MN>(box);
    int k = it.step0 * kTileK;
    for (int i = 0; i < it.steps; ++i, ++count, k += kTileK) {
      ok = bar_wait(shared_addr(&bars->empty[stage]), parity, shape.status);
      if (!ok) break;
      const uint32_t full = shared_addr(&bars->full[stage]);
      if (rank == 0) bar_expect(full, bytes);
      load_operand<MN>(to + stage * kStageBytes, map, row, boxes, k, map_rank(full, 0));
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1;
      }
    }
  }
  // every stage's copies have landed and been used before the CTA ends
  for (int i = 0; i < kStages; ++i)
    if (int64_t at = count - 1 - i; at >= 0)
      bar_wait(shared_addr(&bars->empty[at % kStages]), unsigned(at / kStages) & 1, shape.status);
}

// What an epilogue warp works on: rows row0 .. row0 + 31 (one to a lane) and
// `width` columns from `col` of the product, the columns' address in tensor
// memory, its staging memory.
struct GemmPiece {
  int64_t row0, col;
  int width;
  int slot;            // of a split tile's part, or -1
  int tile_row, tile_col;  // row0 and col within the tile
  uint32_t tmem;
  uint32_t acc_empty;  // the accumulator's barrier, in the pair's first CTA
  uint32_t staging;    // shared address

  // The columns from column c of this lane's row, those below `columns`.
  template <int N>
  __device__ __forceinline__ void load(int c, int columns, float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; i += 32)
      if (c + i < columns) tmem_load32(tmem + c + i, v + i);
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
// piece, by its row and column there.
template <int kPerUnit, class Pack, class Emit>
__device__ __forceinline__ void emit_rows(const float (&v)[8 * kPerUnit], const GemmPiece& at, int c,
                                          int64_t rows, Pack pack, Emit emit) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int u = 0; u < 8; ++u)
    store_shared(at.staging + (lane * 8 + (u ^ (lane & 7))) * 16, pack(v + u * kPerUnit));
  __syncwarp();
  const int u = lane % 8, col = c + u * kPerUnit;
  uint4 unit[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + lane / 8;
    unit[i] = load_shared(at.staging + (r * 8 + (u ^ (r & 7))) * 16);
  }
  __syncwarp();
  if (col >= at.width) return;
  const int left = int(min(int64_t(32), rows - at.row0));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + lane / 8;
    if (r < left) emit(r, col, unit[i]);
  }
}

// Epi: begin() is called by one thread of the launch at its start.
// operator()(const GemmPiece&, float (&)[kPiece]) is called by whole warps with
// a piece's sums, a lane's row each.  (Rows beyond m and columns from `width` on
// hold nothing of the product.)
template <class T, bool A_MN, bool B_MN, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ GemmShape shape, const __grid_constant__ Epi epi) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t tiles = (shared_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t staging = tiles + kStages * kStageBytes;
  GemmBarriers* bars = reinterpret_cast<GemmBarriers*>(
      smem_raw + (staging + kEpilogueWarps * kStagingBytes - shared_addr(smem_raw)));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(shared_addr(&bars->full[i]), 2);  // what A's and B's loads expect
      bar_init(shared_addr(&bars->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(shared_addr(&bars->acc_full[i]), 1);
      bar_init(shared_addr(&bars->acc_empty[i]), 2 * kEpilogueWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMultiply) tmem_alloc_pair(shared_addr(&bars->tmem), kTmemColumns);
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  fence_after_sync();
  const uint32_t tmem = bars->tmem;
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) epi.begin();

  if (warp >= kEpilogueWarps) {
    keep_registers<kOtherRegisters>();
    if (warp == kLoadA) {
      if (lane == 0) load_loop<A_MN>(shape, &map_a, bars, tiles, true, A_MN ? 128 : shape.a_box, rank);
    } else if (warp == kLoadB) {
      if (lane == 0) load_loop<B_MN>(shape, &map_b, bars, tiles + kOperandBytes, false, shape.b_box, rank);
    } else if (warp == kMultiply) {
      if (rank == 0 && lane == 0) {
        constexpr uint32_t kType = T::code == FADAM_DT_BF16 ? 1 : 0;
        // fp32 result, operand types, which operands are not k-major, the tile
        const uint32_t idesc = 1u << 4 | kType << 7 | kType << 10 | uint32_t(A_MN) << 15 |
                               uint32_t(B_MN) << 16 | uint32_t(shape.tile_n / 8) << 17 |
                               uint32_t(kTileM / 16) << 24;
        // 16 of k further on: 32 bytes of a row, or 16 rows
        constexpr uint64_t a_step = A_MN ? (16 * 128) >> 4 : 32 >> 4;
        constexpr uint64_t b_step = B_MN ? (16 * 128) >> 4 : 32 >> 4;
        int stage = 0, tile = 0;
        unsigned parity = 0;
        bool ok = true;
        for (int item = pair; ok && item < shape.items; item += pairs, ++tile) {
          int step0;
          const int steps = gemm_steps(shape, item, step0);
          int acc = 0, left = 0;  // left: steps of the accumulator's chunk
          for (int i = 0; i < steps; ++i, --left) {
            const bool fresh = left == 0;
            if (fresh) {  // the next accumulator
              if (i > 0) {
                commit_pair(shared_addr(&bars->acc_full[acc]));
                ++tile;
              }
              left = shape.chunk;
              acc = tile & 1;
              ok = bar_wait(shared_addr(&bars->acc_empty[acc]), (unsigned(tile >> 1) & 1) ^ 1, shape.status);
              if (!ok) break;
              fence_after_sync();
            }
            ok = bar_wait(shared_addr(&bars->full[stage]), parity, shape.status);
            if (!ok) break;
            fence_after_sync();
            const uint32_t a = tiles + stage * kStageBytes;
            const uint64_t da = operand_desc<A_MN>(a), db = operand_desc<B_MN>(a + kOperandBytes);
#pragma unroll
            for (int k = 0; k < kTileK / 16; ++k)
              mma_pair(tmem + acc * kTileN, da + k * a_step, db + k * b_step, idesc, !fresh || k > 0);
            commit_pair(shared_addr(&bars->empty[stage]));
            if (++stage == kStages) {
              stage = 0;
              parity ^= 1;
            }
          }
          if (!ok) break;
          commit_pair(shared_addr(&bars->acc_full[acc]));
        }
      }
    }
  } else {
    take_registers<kEpilogueRegisters>();
    const int quarter = warp % 4, half = warp / 4, half_n = shape.tile_n / 2;
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + half * half_n;
    GemmPiece at;
    at.staging = staging + warp * kStagingBytes;
    at.tile_row = int(rank) * 128 + quarter * 32;
    at.tile_col = half * half_n;
    int tile = 0;
    bool ok = true;
    for (int item = pair; ok && item < shape.items; item += pairs) {
      const GemmItem it = gemm_item(shape, item);
      at.row0 = int64_t(it.m0) + at.tile_row;
      at.col = int64_t(it.n0) + at.tile_col;
      at.width = int(min(int64_t(half_n), shape.n - at.col));
      at.slot = it.slot;
      const bool here = at.row0 < shape.m && at.width > 0;
      const auto next_acc = [&] {
        const int acc = tile & 1;
        ok = bar_wait(shared_addr(&bars->acc_full[acc]), unsigned(tile >> 1) & 1, shape.status);
        ++tile;
        fence_after_sync();
        at.tmem = lanes + acc * kTileN;
        at.acc_empty = map_rank(shared_addr(&bars->acc_empty[acc]), 0);
        return ok;
      };
      float v[kPiece];
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[i] = 0.0f;
      next_acc();
      if (here && ok) at.load(0, half_n, v);
      at.release();
      for (int c = shape.chunk; c < it.steps && ok && next_acc(); c += shape.chunk) {
        if (here) {
#pragma unroll
          for (int g = 0; g < kPiece; g += 32)
            if (g < half_n) {
              float t[32];
              at.load(g, half_n, t);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[g + i] += t[i];
            }
        }
        at.release();
      }
      if (here && ok) epi(at, v);
    }
  }
  __syncwarp();
  chain_next();
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == kMultiply) tmem_free_pair(tmem, kTmemColumns);
}

// Launch over all SMs, a pair of CTAs per two SMs.
template <class T, bool A_MN, bool B_MN, class Epi>
fadam_status launch_gemm(const CUtensorMap& a, const CUtensorMap& b, const GemmShape& shape,
                         const Epi& epi, int sm_count, cudaStream_t stream) {
  auto* kernel = gemm_kernel<T, A_MN, B_MN, Epi>;
  // a kernel built with fewer would wait for its share of registers for ever
  static const int registers = [&] {
    cudaFuncAttributes f{};
    return cudaFuncGetAttributes(&f, kernel) == cudaSuccess ? f.numRegs : -1;
  }();
  if (registers != kLaunchRegisters)
    return fail(FADAM_ECUDA, "the matrix product was built with %d registers a thread, not %d", registers,
                kLaunchRegisters);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(kGemmSmem));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  const int pairs = shape.items < sm_count / 2 ? shape.items : sm_count / 2;
  return launch_chained("matrix product launch", kernel, 2 * pairs, kGemmThreads, kGemmSmem, stream, a,
                        b, shape, epi);
}

}  // namespace fadam_ops
