// The epilogue that scales a product and writes it out, and the join of the
// parts of a product whose k was split.
#pragma once

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
  float* carry;          // fp32 [m, n]: products summed over several launches
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

// Eight consecutive columns of one row, `v` scaled already.
template <class Out>
__device__ __forceinline__ void store8(Out* out, const float* v, bool accumulate) {
  float r[8];
  if (accumulate) {
    float old[8];
    if (sizeof(Out) == 4) {
      *reinterpret_cast<float4*>(old) = *reinterpret_cast<const float4*>(out);
      *reinterpret_cast<float4*>(old + 4) = *reinterpret_cast<const float4*>(out + 4);
    } else {
      const uint4 raw = *reinterpret_cast<const uint4*>(out);
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Out* p = reinterpret_cast<const Out*>(&w[i]);
        old[2 * i] = to_float(p[0]);
        old[2 * i + 1] = to_float(p[1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i] + old[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i];
  }
  if constexpr (sizeof(Out) == 4) {
    *reinterpret_cast<float4*>(out) = make_float4(r[0], r[1], r[2], r[3]);
    *reinterpret_cast<float4*>(out + 4) = make_float4(r[4], r[5], r[6], r[7]);
  } else {
    *reinterpret_cast<uint4*>(out) = make_uint4(pack2<Out>(r[0], r[1]), pack2<Out>(r[2], r[3]),
                                                pack2<Out>(r[4], r[5]), pack2<Out>(r[6], r[7]));
  }
}

template <class Out>
struct StoreEpilogue {
  StoreArgs s;
  float* parts;  // fp32 [splits, m, n] when k is split: joined by join_kernel

  __device__ __forceinline__ void operator()(float (&v)[kPiece], int64_t row, int64_t col,
                                             int split) const {
    if (row >= s.m || col >= s.n) return;
    const int width = int(min(int64_t(kPiece), s.n - col));
    if (parts) {
      put(parts + (split * s.m + row) * s.n + col, v, width);
      return;
    }
    if (s.read_carry) {
      const float* c = s.carry + row * s.n + col;
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
        if (i < width) v[i] += c[i];
    }
    if (s.write_carry) {
      put(s.carry + row * s.n + col, v, width);
      return;
    }
    const float f = s.factor();
    const bool zero = s.masked(row);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] = zero ? 0.0f : v[i] * f;
    Out* out = static_cast<Out*>(s.out) + row * s.ld + col;
    if (s.wide && width == kPiece) {
#pragma unroll
      for (int i = 0; i < kPiece; i += 8) store8<Out>(out + i, v + i, s.accumulate);
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
        if (i < width) out[i] = from_float<Out>(s.accumulate ? v[i] + to_float(out[i]) : v[i]);
    }
  }

  // fp32 scratch rows: 16-byte stores where the row's start allows them
  static __device__ __forceinline__ void put(float* to, const float (&v)[kPiece], int width) {
    if (width == kPiece && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < kPiece; i += 4)
        *reinterpret_cast<float4*>(to + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
        if (i < width) to[i] = v[i];
    }
  }
};

// out = round(scale * sum over the parts), in the parts' order.
template <class Out>
__global__ void __launch_bounds__(256) join_kernel(const float* parts, int splits, StoreArgs s) {
  const int64_t total = s.m * s.n;
  const float f = s.factor();
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    float sum = 0.0f;
    for (int p = 0; p < splits; ++p) sum += parts[p * total + i];
    const int64_t row = i / s.n, col = i - row * s.n;
    Out* out = static_cast<Out*>(s.out) + row * s.ld + col;
    if (s.read_carry) sum += s.carry[i];
    if (s.write_carry) {
      s.carry[i] = sum;
      continue;
    }
    sum = s.masked(row) ? 0.0f : sum * f;
    *out = from_float<Out>(s.accumulate ? sum + to_float(*out) : sum);
  }
}

// A product with the storing epilogue, k split when `parts` is not NULL.
template <class T, bool A_MN, bool B_MN, class Out>
fadam_status store_product(const CUtensorMap& a, const CUtensorMap& b, const GemmShape& shape,
                           const StoreArgs& args, float* parts, int sm_count, cudaStream_t stream) {
  float* where = shape.splits > 1 ? parts : nullptr;
  const fadam_status st = launch_gemm<T, A_MN, B_MN>(
      a, b, shape, StoreEpilogue<typename Out::type>{args, where}, sm_count, stream);
  if (st || !where) return st;
  const int64_t blocks = ceil_div(args.m * args.n, 256);
  join_kernel<typename Out::type><<<unsigned(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(
      where, shape.splits, args);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FADAM_OK : cuda_fail(e, "join launch");
}

// Into how many parts to cut k: one, unless the tiles leave most CTA pairs
// idle and each part keeps at least eight steps.
inline int choose_splits(int64_t m, int64_t n, int64_t k, int pairs) {
  const int64_t tiles = ceil_div(m, kTileM) * ceil_div(n, kTileN);
  const int64_t steps = ceil_div(k, kTileK);
  int64_t splits = pairs / tiles;
  if (splits > steps / 8) splits = steps / 8;
  return splits < 2 ? 1 : int(splits);
}

}  // namespace fadam_ops
