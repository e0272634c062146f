// The epilogue that scales a product and writes it out, and the join of the
// parts of a product whose k was split.
#pragma once

#include <type_traits>

#include "gemm.cuh"

namespace fadam_ops {

// How a product becomes an output: out = round(scale * (sum + added)), and
// zero in rows that `targets` marks as ignored.
struct StoreArgs {
  void* out;
  int64_t ld;            // elements from one row of out to the next
  int64_t m, n;
  const float* scale;    // device scalar, NULL for 1
  float constant;        // another factor
  float* carry;          // fp32 [m, scratch_ld(n)]: products summed over several launches
  int32_t read_carry;    // the sum starts from carry
  int32_t write_carry;   // the sum goes back to carry, not to out
  int32_t accumulate;    // out's old value is added to the scaled sum
  const int64_t* targets;
  int64_t ignore_index;
  bool wide;             // 16-byte stores to out are aligned

  __device__ __forceinline__ float factor() const {
    return constant * (scale ? __ldg(scale) : 1.0f);
  }
  __device__ __forceinline__ bool masked(int64_t row) const {
    return targets && targets[row] == ignore_index;
  }
};

inline bool wide_stores(const void* out, int64_t ld, int size) {
  return !misaligned(out, 16) && ld * size % 16 == 0;
}

// Scratch rows of sums: fp32, padded so that every row starts on 16 bytes.
__host__ __device__ inline int64_t scratch_ld(int64_t n) { return (n + 3) / 4 * 4; }

template <class Out>
struct StoreEpilogue {
  StoreArgs s;
  float* parts;  // fp32 [slots, split_rows(m), tile_n]: sums of split tiles, joined by join_kernel
  int tile_n;

  static constexpr bool kChunked = false;
  __device__ __forceinline__ void begin() const {}
  __device__ __forceinline__ void operator()(const GemmPiece& at) const {
    const int64_t row = at.row0 + threadIdx.x % 32;
    const bool sums = at.slot >= 0 || s.write_carry;
    const bool zero = !sums && row < s.m && s.masked(row);
    const float f = sums ? 1.0f : s.factor();
    if (sizeof(Out) == 2 && !sums && !s.read_carry && !s.accumulate) {
      Out* out = static_cast<Out*>(s.out) + at.row0 * s.ld + at.col;
#pragma unroll 1
      for (int c = 0; c < at.width; c += 64) {
        float v[64];
        at.load(c, v);
        if (c + 64 >= at.width) at.release();
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = zero ? 0.0f : v[i] * f;
        if (s.wide && s.n % 8 == 0)
          emit_rows<8>(
              v, at, c, s.m,
              [](const float* p) {
                return make_uint4(pack2<Half>(p[0], p[1]), pack2<Half>(p[2], p[3]),
                                  pack2<Half>(p[4], p[5]), pack2<Half>(p[6], p[7]));
              },
              [&](int r, int col, uint4 u) { *reinterpret_cast<uint4*>(out + r * s.ld + col) = u; });
        else
          store_elements(v, at, c);
      }
      return;
    }
    float* part = at.slot < 0 ? nullptr
                              : parts + at.slot * split_rows(s.m) * tile_n + int64_t(at.tile_row) * tile_n +
                                    at.tile_col;
#pragma unroll 1
    for (int c = 0; c < at.width; c += 32) {
      float v[32];
      at.load(c, v);
      if (c + 32 >= at.width) at.release();
      if (zero)
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
      emit_rows<4>(
          v, at, c, s.m,
          [](const float* p) {
            return make_uint4(__float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]),
                              __float_as_uint(p[3]));
          },
          [&](int r, int col, uint4 u) {
            if (part)
              *reinterpret_cast<uint4*>(part + r * tile_n + col) = u;
            else
              finish4(at.row0 + r, at.col + col,
                      make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                  __uint_as_float(u.w)), f);
          });
    }
  }

  // Four columns of a whole sum: add what is carried; carry on, or scale, add
  // what is there, round, store.
  __device__ __forceinline__ void finish4(int64_t row, int64_t col, float4 v, float f) const {
    if (s.read_carry || s.write_carry) {
      float4* carry = reinterpret_cast<float4*>(s.carry + row * scratch_ld(s.n) + col);
      if (s.read_carry) {
        const float4 o = *carry;
        v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
      }
      if (s.write_carry) {
        *carry = v;
        return;
      }
    }
    const float e[4] = {v.x, v.y, v.z, v.w};
    Out* out = static_cast<Out*>(s.out) + row * s.ld + col;
    const int left = int(min(int64_t(4), s.n - col));
    if (s.wide && left == 4) {
      if constexpr (sizeof(Out) == 4) {
        float4* to = reinterpret_cast<float4*>(out);
        const float4 o = s.accumulate ? *to : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        *to = make_float4(e[0] * f + o.x, e[1] * f + o.y, e[2] * f + o.z, e[3] * f + o.w);
      } else {
        uint2* to = reinterpret_cast<uint2*>(out);
        float2 a = make_float2(0.0f, 0.0f), b = a;
        if (s.accumulate) {
          const uint2 old = *to;
          a = unpack2<Out>(old.x);
          b = unpack2<Out>(old.y);
        }
        *to = make_uint2(pack2<Out>(e[0] * f + a.x, e[1] * f + a.y),
                         pack2<Out>(e[2] * f + b.x, e[3] * f + b.y));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) out[i] = from_float<Out>(e[i] * f + (s.accumulate ? to_float(out[i]) : 0.0f));
    }
  }

  // 64 columns of 16-bit rows that do not start on 16 bytes: through the
  // staging memory, then a row at a time, element by element.
  using Half = typename std::conditional<sizeof(Out) == 2, Out, __half>::type;
  __device__ __forceinline__ void store_elements(const float (&v)[64], const GemmPiece& at, int c) const {
    const int lane = threadIdx.x % 32;
    // unit u of row r at unit 8 r + (u ^ r % 8): 16-byte stores without a bank hit twice
#pragma unroll
    for (int u = 0; u < 8; ++u)
      store_shared(at.staging + (lane * 8 + (u ^ (lane & 7))) * 16,
                   make_uint4(pack2<Half>(v[8 * u], v[8 * u + 1]), pack2<Half>(v[8 * u + 2], v[8 * u + 3]),
                              pack2<Half>(v[8 * u + 4], v[8 * u + 5]), pack2<Half>(v[8 * u + 6], v[8 * u + 7])));
    __syncwarp();
    uint16_t* out = reinterpret_cast<uint16_t*>(s.out) + at.row0 * s.ld + at.col + c + lane;
    const int rows = int(min(int64_t(32), s.m - at.row0)), left = at.width - c - lane;
#pragma unroll 8
    for (int r = 0; r < rows; ++r, out += s.ld) {
      const uint32_t row = at.staging + r * 128 + lane % 8 * 2;
      if (left > 0) out[0] = load_shared_u16(row + ((lane / 8) ^ (r & 7)) * 16);
      if (left > 32) out[32] = load_shared_u16(row + ((4 + lane / 8) ^ (r & 7)) * 16);
    }
    __syncwarp();
  }
};

// The split tiles' parts added up in their order and finished.
template <class Out>
__global__ void __launch_bounds__(256)
    join_kernel(const __grid_constant__ StoreEpilogue<Out> e, const __grid_constant__ GemmShape shape) {
  chain_wait();
  chain_next();
  const StoreArgs& s = e.s;
  const int64_t rows = split_rows(s.m), per_part = rows * e.tile_n;
  const int per_row = e.tile_n / 4;
  const int tiles = shape.m_tiles * shape.n_tiles - shape.full;
  const float f = s.factor();
  const unsigned per_tile = unsigned(rows) * unsigned(per_row);
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < int64_t(tiles) * per_tile;
       i += int64_t(gridDim.x) * 256) {
    const int tile = int(i / per_tile);
    const unsigned at = unsigned(i - int64_t(tile) * per_tile);
    const int r = int(at / unsigned(per_row)), c = int(at - unsigned(r) * per_row) * 4;
    int m0, n0;
    gemm_tile(shape, unsigned(shape.full + tile), m0, n0);
    const int64_t row = int64_t(m0) + r, col = int64_t(n0) + c;
    if (row >= s.m || col >= s.n) continue;
    const float* p = e.parts + int64_t(tile) * shape.splits * per_part + r * e.tile_n + c;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int k = 0; k < shape.splits; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(p + k * per_part);
      sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
    }
    if (s.masked(row)) sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    e.finish4(row, col, sum, f);
  }
}

// A product with the storing epilogue; `parts` has the plan's split_bytes.
template <class T, bool A_MN, bool B_MN, class Out>
fadam_status store_product(const CUtensorMap& a, const CUtensorMap& b, const GemmShape& shape,
                           const StoreArgs& args, float* parts, int sm_count, cudaStream_t stream) {
  using E = typename Out::type;
  const StoreEpilogue<E> epi{args, parts, shape.tile_n};
  const fadam_status st = launch_gemm<T, A_MN, B_MN>(a, b, shape, epi, sm_count, stream);
  const int64_t split = int64_t(shape.m_tiles) * shape.n_tiles - shape.full;
  if (st || split == 0) return st;
  const int64_t blocks = ceil_div(split * split_rows(args.m) * (shape.tile_n / 4), 256);
  return launch_chained("join launch", join_kernel<E>, blocks < 4096 ? blocks : 4096, 256, 0, stream, epi,
                        shape);
}

}  // namespace fadam_ops
