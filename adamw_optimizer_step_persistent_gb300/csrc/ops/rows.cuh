// Rows of activations, eight elements to a thread at a time: loads and stores
// of any of the three types, and the 8-bit codes of a group.
#pragma once

#include "ops_device.cuh"

namespace fadam_ops {

constexpr int kGroup = FADAM_CHECKPOINT8_GROUP;
constexpr int kLanesPerGroup = kGroup / 8;  // threads that hold one group
// A group whose largest magnitude is below this is kept as zeros: its 127 / a
// could be infinite.
constexpr float kTinyGroup = 7.888609052210118e-31f;  // 2^-100

// Elements [col, col + 8) of a row of `width`, zeros beyond it.  `wide`: the
// row starts on 16 bytes and width is a multiple of 8.
template <class E>
__device__ __forceinline__ void load8(const E* row, int col, int width, bool wide, float (&v)[8]) {
  if (wide) {
    if (col >= width) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    } else if constexpr (sizeof(E) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(row + col);
      const float4 b = *reinterpret_cast<const float4*>(row + col + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 raw = *reinterpret_cast<const uint4*>(row + col);
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = unpack2<E>(w[i]);
        v[2 * i] = p.x;
        v[2 * i + 1] = p.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < width ? to_float(row[col + i]) : 0.0f;
  }
}

template <class E>
__device__ __forceinline__ void store_row8(E* row, int col, int width, bool wide, const float (&v)[8]) {
  if (wide) {
    if (col >= width) return;
    if constexpr (sizeof(E) == 4) {
      *reinterpret_cast<float4*>(row + col) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(row + col + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(row + col) = make_uint4(pack2<E>(v[0], v[1]), pack2<E>(v[2], v[3]),
                                                        pack2<E>(v[4], v[5]), pack2<E>(v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < width) row[col + i] = from_float<E>(v[i]);
  }
}

// Parameters may be fp32 under 16-bit activations.
template <class E>
__device__ __forceinline__ void load_param8(const void* p, int64_t offset, bool f32, int col,
                                            int width, bool wide, float (&v)[8]) {
  if (f32)
    load8<float>(static_cast<const float*>(p) + offset, col, width, wide, v);
  else
    load8<E>(static_cast<const E*>(p) + offset, col, width, wide, v);
}

// Keeps a thread's eight elements, with the 15 other threads of the half warp
// that hold the rest of the group: every lane of the warp must call it.
// Lanes beyond the row hold zeros.  Column col + i has code i; the group's
// first lane writes the scale.
__device__ __forceinline__ void keep8(const float (&v)[8], int8_t* codes, float* scales, int col,
                                      int width, bool wide) {
  // the largest magnitude by its bits: a NaN's are above an infinity's
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
  for (int i = kLanesPerGroup / 2; i; i /= 2) top = max(top, __shfl_xor_sync(~0u, top, i));
  if (col >= width) return;
  const float a = __uint_as_float(top);
  const bool finite = top < 0x7f800000u, tiny = finite && a < kTinyGroup;
  const float inverse = tiny || !finite ? 0.0f : __fdiv_rn(127.0f, a);
  if (col % kGroup == 0)
    scales[col / kGroup] = tiny ? 0.0f : finite ? __fdiv_rn(a, 127.0f) : __uint_as_float(0x7fffffffu);
  uint32_t word[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int code = finite ? __float2int_rn(__fmul_rn(v[i], inverse)) : 0;
    word[i / 4] |= (uint32_t(code) & 0xffu) << (i % 4 * 8);
  }
  if (wide) {
    *reinterpret_cast<uint2*>(codes + col) = make_uint2(word[0], word[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < width) codes[col + i] = int8_t(word[i / 4] >> (i % 4 * 8) & 0xffu);
  }
}

// Eight kept elements.
__device__ __forceinline__ void kept8(const int8_t* codes, const float* scales, int col, int width,
                                      bool wide, float (&v)[8]) {
  if (col >= width) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    return;
  }
  const float scale = scales[col / kGroup];
  if (wide) {
    const uint2 raw = *reinterpret_cast<const uint2*>(codes + col);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = i < 4 ? raw.x : raw.y;
      v[i] = float(int(w << (24 - i % 4 * 8)) >> 24) * scale;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < width ? float(codes[col + i]) * scale : 0.0f;
  }
}

}  // namespace fadam_ops
