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

  __device__ __forceinline__ void begin() const {}
  __device__ __forceinline__ void operator()(const GemmPiece& at, float (&v)[kPiece]) const {
    const int64_t row = at.row0 + threadIdx.x % 32;
    const bool sums = at.slot >= 0 || s.write_carry;
    const bool zero = !sums && row < s.m && s.masked(row);
    const float f = sums ? 1.0f : s.factor();
    if (sizeof(Out) == 2 && !sums && !s.read_carry) {
      Out* out = static_cast<Out*>(s.out) + at.row0 * s.ld + at.col;
#pragma unroll
      for (int c = 0; c < kPiece; c += 64) {
        if (c >= at.width) break;
        float (&e)[64] = reinterpret_cast<float (&)[64]>(v[c]);
        if (s.accumulate) {
          if constexpr (sizeof(Out) == 2) add_rows(e, at, c, zero ? 0.0f : f);
          continue;
        }
#pragma unroll
        for (int i = 0; i < 64; ++i) e[i] = zero ? 0.0f : e[i] * f;
        if (s.wide && s.n % 8 == 0)
          emit_rows<8>(
              e, at, c, s.m,
              [](const float* p) {
                return make_uint4(pack2<Half>(p[0], p[1]), pack2<Half>(p[2], p[3]),
                                  pack2<Half>(p[4], p[5]), pack2<Half>(p[6], p[7]));
              },
              [&](int r, int col, uint4 u) { *reinterpret_cast<uint4*>(out + r * s.ld + col) = u; });
        else
          store_elements(e, at, c);
      }
      return;
    }
    float* part = at.slot < 0 ? nullptr
                              : parts + at.slot * split_rows(s.m) * tile_n + int64_t(at.tile_row) * tile_n +
                                    at.tile_col;
#pragma unroll
    for (int c = 0; c < kPiece; c += 32) {
      if (c >= at.width) break;
      float (&e)[32] = reinterpret_cast<float (&)[32]>(v[c]);
      if (zero)
#pragma unroll
        for (int i = 0; i < 32; ++i) e[i] = 0.0f;
      finish_rows(e, at, c, f, part);
    }
  }

  // 32 columns of a warp's sums, from column c of its piece: into the split
  // tile's part, or added to what is carried and carried on, or scaled, added
  // to what is there, rounded and stored.  Through the staging memory as in
  // emit_rows.  All old values are on their way before the first is used and
  // before the first store, which might alias the next load: eight round trips
  // to memory for a tile in place of 32.
  __device__ __forceinline__ void finish_rows(const float (&v)[32], const GemmPiece& at, int c, float f,
                                              float* part) const {
    const int lane = threadIdx.x % 32, u = lane % 8, r0 = lane / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      store_shared(at.staging + (lane * 8 + (i ^ (lane & 7))) * 16,
                   make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                              __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
    __syncwarp();
    const auto staged = [&](int i) {  // the unit of row 4 i + r0
      const int r = i * 4 + r0;
      return at.staging + (r * 8 + (u ^ (r & 7))) * 16;
    };
    const int left = c + u * 4 < at.width ? int(min(int64_t(32), s.m - at.row0)) : 0;
    const int64_t row = at.row0 + r0, col = at.col + c + u * 4;
    if (part) {
      part += r0 * tile_n + c + u * 4;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * 4 + r0 < left) *reinterpret_cast<uint4*>(part + i * 4 * tile_n) = load_shared(staged(i));
    } else {
      const int64_t carry_ld = scratch_ld(s.n);
      float4* carry = reinterpret_cast<float4*>(s.carry + row * carry_ld + col);
      float4 old[8];
      if (s.read_carry) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 4 + r0 < left) old[i] = carry[i * carry_ld];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 4 + r0 < left) {
            const float4 sum = add4(as_float4(load_shared(staged(i))), old[i]);
            store_shared(staged(i), make_uint4(__float_as_uint(sum.x), __float_as_uint(sum.y),
                                               __float_as_uint(sum.z), __float_as_uint(sum.w)));
          }
      }
      if (s.write_carry) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 4 + r0 < left) carry[i * carry_ld] = as_float4(load_shared(staged(i)));
      } else {
        Out* out = static_cast<Out*>(s.out) + row * s.ld + col;
        const int columns = int(min(int64_t(4), s.n - col));
#pragma unroll
        for (int i = 0; i < 8; ++i)
          old[i] = s.accumulate && i * 4 + r0 < left ? load4(out + i * 4 * s.ld, columns)
                                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 4 + r0 < left)
            store4(out + i * 4 * s.ld, fma4(as_float4(load_shared(staged(i))), f, old[i]), columns);
      }
    }
    __syncwarp();
  }

  // 64 columns of a warp's sums, scaled, added to 16-bit rows: 16 rows at a time
  // through the staging memory, so that eight lanes have a whole line of a row.
  __device__ __forceinline__ void add_rows(const float (&v)[64], const GemmPiece& at, int c, float f) const {
    const int lane = threadIdx.x % 32, u = lane % 8, r0 = lane / 8;
    const int columns = min(8, at.width - c - u * 8), left = int(min(int64_t(32), s.m - at.row0));
    Out* out = static_cast<Out*>(s.out) + (at.row0 + r0) * s.ld + at.col + c + u * 8;
#pragma unroll 1
    for (int half = 0; half < 2; ++half, out += 16 * s.ld) {
      // unit i of a row (four columns): even ones first, exchanged by row
      if (lane / 16 == half)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          store_shared(at.staging + (lane % 16 * 16 + ((i % 2 * 8 + i / 2) ^ (lane & 7))) * 16,
                       make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                  __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
      __syncwarp();
      uint4 old[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (columns > 0 && half * 16 + i * 4 + r0 < left) old[i] = load8(out + i * 4 * s.ld, columns);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (columns > 0 && half * 16 + i * 4 + r0 < left) {
          const int r = i * 4 + r0;
          const uint32_t row = at.staging + r * 256;
          const float2 w0 = unpack2<Out>(old[i].x), w1 = unpack2<Out>(old[i].y);
          const float2 w2 = unpack2<Out>(old[i].z), w3 = unpack2<Out>(old[i].w);
          const float4 a = fma4(as_float4(load_shared(row + (u ^ (r & 7)) * 16)), f,
                                make_float4(w0.x, w0.y, w1.x, w1.y));
          const float4 b = fma4(as_float4(load_shared(row + ((8 + u) ^ (r & 7)) * 16)), f,
                                make_float4(w2.x, w2.y, w3.x, w3.y));
          store8(out + i * 4 * s.ld, a, b, columns);
        }
      __syncwarp();
    }
  }
  __device__ __forceinline__ uint4 load8(const Out* at, int columns) const {
    if (s.wide && columns == 8) return *reinterpret_cast<const uint4*>(at);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < columns) w[i / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(at)[i]) << (i % 2 * 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store8(Out* at, float4 a, float4 b, int columns) const {
    if (s.wide && columns == 8) {
      *reinterpret_cast<uint4*>(at) = make_uint4(pack2<Out>(a.x, a.y), pack2<Out>(a.z, a.w),
                                                 pack2<Out>(b.x, b.y), pack2<Out>(b.z, b.w));
    } else {
      store4(at, a, min(4, columns));
      store4(at + 4, b, columns - 4);
    }
  }

  // finish_rows for four columns of a whole sum.
  __device__ __forceinline__ void finish4(int64_t row, int64_t col, float4 v, float f) const {
    float4* carry = reinterpret_cast<float4*>(s.carry + row * scratch_ld(s.n) + col);
    if (s.read_carry) v = add4(v, *carry);
    if (s.write_carry) {
      *carry = v;
      return;
    }
    Out* out = static_cast<Out*>(s.out) + row * s.ld + col;
    const int columns = int(min(int64_t(4), s.n - col));
    const float4 old = s.accumulate ? load4(out, columns) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    store4(out, fma4(v, f, old), columns);
  }

  static __device__ __forceinline__ float4 as_float4(uint4 u) {
    return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
  }
  static __device__ __forceinline__ float4 fma4(float4 a, float f, float4 b) {
    return make_float4(fmaf(a.x, f, b.x), fmaf(a.y, f, b.y), fmaf(a.z, f, b.z), fmaf(a.w, f, b.w));
  }
  // Up to four neighbouring elements of out.
  __device__ __forceinline__ float4 load4(const Out* at, int columns) const {
    if (s.wide && columns == 4) {
      if constexpr (sizeof(Out) == 4) {
        return *reinterpret_cast<const float4*>(at);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(at);
        const float2 a = unpack2<Out>(u.x), b = unpack2<Out>(u.y);
        return make_float4(a.x, a.y, b.x, b.y);
      }
    }
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = i < columns ? to_float(at[i]) : 0.0f;
    return make_float4(e[0], e[1], e[2], e[3]);
  }
  __device__ __forceinline__ void store4(Out* at, float4 v, int columns) const {
    if (s.wide && columns == 4) {
      if constexpr (sizeof(Out) == 4)
        *reinterpret_cast<float4*>(at) = v;
      else
        *reinterpret_cast<uint2*>(at) = make_uint2(pack2<Out>(v.x, v.y), pack2<Out>(v.z, v.w));
    } else {
      const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < columns) at[i] = from_float<Out>(e[i]);
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
