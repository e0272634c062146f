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
  float* parts;  // fp32 [splits, m, scratch_ld(n)] when k is split: joined by join_kernel

  __device__ __forceinline__ void operator()(const GemmPiece& at) const {
    const int64_t row = at.row0 + threadIdx.x % 32;
    const bool sums = parts || s.write_carry;
    const bool zero = !sums && row < s.m && s.masked(row);
    const float f = sums ? 1.0f : s.factor();
    if (sizeof(Out) == 2 && !sums && !s.read_carry && !s.accumulate) {
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
              [&](int64_t r, int64_t col, uint4 u) {
                *reinterpret_cast<uint4*>(static_cast<Out*>(s.out) + r * s.ld + col) = u;
              });
        else
          store_elements(v, at, c);
      }
      return;
    }
    const int64_t ld = scratch_ld(s.n);
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
          [&](int64_t r, int64_t col, uint4 u) {
            if (parts) {
              *reinterpret_cast<uint4*>(parts + (at.split * s.m + r) * ld + col) = u;
              return;
            }
            float4 sum = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                                     __uint_as_float(u.w));
            float4* carry = reinterpret_cast<float4*>(s.carry + r * ld + col);
            if (s.read_carry) {
              const float4 o = *carry;
              sum = make_float4(sum.x + o.x, sum.y + o.y, sum.z + o.z, sum.w + o.w);
            }
            if (s.write_carry)
              *carry = sum;
            else
              put4(r, col, sum, f);
          });
    }
  }

  // Four columns: scale, add what is there, round, store.
  __device__ __forceinline__ void put4(int64_t row, int64_t col, float4 v, float f) const {
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
    uint32_t* staging = reinterpret_cast<uint32_t*>(at.staging);
    // pair p of row r at word 32 r + (p ^ r): no two lanes on one bank
#pragma unroll
    for (int p = 0; p < 32; ++p) staging[lane * 32 + (p ^ lane)] = pack2<Half>(v[2 * p], v[2 * p + 1]);
    __syncwarp();
    uint16_t* out = reinterpret_cast<uint16_t*>(s.out) + at.row0 * s.ld + at.col + c + lane;
    const int rows = int(min(int64_t(32), s.m - at.row0)), left = at.width - c - lane;
#pragma unroll 8
    for (int r = 0; r < rows; ++r, out += s.ld) {
      const uint32_t a = staging[r * 32 + ((lane / 2) ^ r)], b = staging[r * 32 + ((16 + lane / 2) ^ r)];
      if (left > 0) out[0] = uint16_t(lane % 2 ? a >> 16 : a);
      if (left > 32) out[32] = uint16_t(lane % 2 ? b >> 16 : b);
    }
    __syncwarp();
  }
};

// out = round(scale * sum over the parts), in the parts' order.
template <class Out>
__global__ void __launch_bounds__(256) join_kernel(const float* parts, int splits, StoreEpilogue<Out> e) {
  const StoreArgs& s = e.s;
  const int64_t ld = scratch_ld(s.n), per_row = ld / 4, total = s.m * per_row;
  const float f = s.factor();
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t row = i / per_row;
    const float4* p = reinterpret_cast<const float4*>(parts) + i;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
      const float4 v = p[k * total];
      sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
    }
    if (s.masked(row)) sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    e.put4(row, (i - row * per_row) * 4, sum, f);
  }
}

// A product with the storing epilogue, k split when `parts` is not NULL.
template <class T, bool A_MN, bool B_MN, class Out>
fadam_status store_product(const CUtensorMap& a, const CUtensorMap& b, const GemmShape& shape,
                           const StoreArgs& args, float* parts, int sm_count, cudaStream_t stream) {
  using E = typename Out::type;
  float* where = shape.splits > 1 ? parts : nullptr;
  const fadam_status st =
      launch_gemm<T, A_MN, B_MN>(a, b, shape, StoreEpilogue<E>{args, where}, sm_count, stream);
  if (st || !where) return st;
  const int64_t blocks = ceil_div(args.m * scratch_ld(args.n) / 4, 256);
  join_kernel<E><<<unsigned(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(
      where, shape.splits, StoreEpilogue<E>{args, nullptr});
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FADAM_OK : cuda_fail(e, "join launch");
}

}  // namespace fadam_ops
