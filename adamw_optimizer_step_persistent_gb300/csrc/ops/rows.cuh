// Rows of activations in registers: vectors of eight elements, as four pairs
// of floats (the packed fp32 instructions take two elements each), loads and
// stores of any of the three types, and the 8-bit codes of a group.
#pragma once

#include "ops_device.cuh"

namespace fadam_ops {

constexpr int kGroup = FADAM_CHECKPOINT8_GROUP;
// A group whose largest magnitude is below this is kept as zeros: its 127 / a
// could be infinite.
constexpr float kTinyGroup = 7.888609052210118e-31f;  // 2^-100

// ---- pairs ------------------------------------------------------------------------

using Pair = unsigned long long;

__device__ __forceinline__ Pair make_pair(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split(Pair p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair both(float a) { return make_pair(a, a); }
__device__ __forceinline__ float sum2(Pair p) {
  const float2 v = split(p);
  return v.x + v.y;
}

// ---- vectors ----------------------------------------------------------------------

// Eight elements as they lie in memory.
template <class E>
struct Raw {
  uint32_t w[2 * sizeof(E)];
};

template <class E>
__device__ __forceinline__ Raw<E> load_raw(const E* p) {
  Raw<E> r;
#pragma unroll
  for (int i = 0; i < int(sizeof(E)) / 2; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(p)[i];
    r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
  }
  return r;
}
template <class E>
__device__ __forceinline__ void store_raw(E* p, const Raw<E>& r) {
#pragma unroll
  for (int i = 0; i < int(sizeof(E)) / 2; ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
}

template <class E>
__device__ __forceinline__ void widen(const Raw<E>& r, Pair (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 4) {
      v[i] = make_pair(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    } else {
      const float2 p = unpack2<E>(r.w[i]);
      v[i] = make_pair(p.x, p.y);
    }
  }
}
template <class E>
__device__ __forceinline__ Raw<E> narrow(const Pair (&v)[4]) {
  Raw<E> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = split(v[i]);
    if constexpr (sizeof(E) == 4) {
      r.w[2 * i] = __float_as_uint(p.x);
      r.w[2 * i + 1] = __float_as_uint(p.y);
    } else {
      r.w[i] = pack2<E>(p.x, p.y);
    }
  }
  return r;
}

// Where a thread's NV vectors of eight elements lie in a row.  kWide, rows of
// whole aligned vectors: a vector's elements next to each other, consecutive
// threads' vectors too.  Else a warp has NV * 256 consecutive elements and its
// lanes take them in turn, so that element-wise accesses coalesce and differ
// by constants.
template <int NV, bool kWide>
struct Columns {
  int threads, tid, width;
  int lone0, left;  // the first element of a row that is not wide, and how far it is from the end
  __device__ __forceinline__ Columns(int threads, int tid, int width)
      : threads(threads), tid(tid), width(width), lone0(tid / 32 * NV * 256 + tid % 32),
        left(width - lone0) {}
  __device__ __forceinline__ int first(int j) const { return (j * threads + tid) * 8; }
  __device__ __forceinline__ int lone(int j, int i) const { return lone0 + (j * 8 + i) * 32; }
  __device__ __forceinline__ bool valid(int j, int i) const { return (j * 8 + i) * 32 < left; }
};

template <class E>
__device__ __forceinline__ Raw<E> zero_raw() {
  Raw<E> r;
#pragma unroll
  for (int i = 0; i < int(2 * sizeof(E)); ++i) r.w[i] = 0;
  return r;
}

// Vector j of a row, zeros beyond its end.
template <class E, int NV, bool kWide>
__device__ __forceinline__ Raw<E> load_vector(const E* row, const Columns<NV, kWide>& c, int j) {
  Raw<E> r = zero_raw<E>();
  if constexpr (kWide) {
    if (c.first(j) < c.width) r = load_raw(row + c.first(j));
  } else {
    const E* at = row + c.lone0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c.valid(j, i)) {
        if constexpr (sizeof(E) == 4)
          r.w[i] = __float_as_uint(at[(j * 8 + i) * 32]);
        else
          r.w[i / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(at)[(j * 8 + i) * 32]) << (i % 2 * 16);
      }
  }
  return r;
}
template <class E, int NV, bool kWide>
__device__ __forceinline__ void store_vector(E* row, const Columns<NV, kWide>& c, int j, const Raw<E>& r) {
  if constexpr (kWide) {
    if (c.first(j) < c.width) store_raw(row + c.first(j), r);
  } else {
    E* at = row + c.lone0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c.valid(j, i)) {
        if constexpr (sizeof(E) == 4)
          at[(j * 8 + i) * 32] = __uint_as_float(r.w[i]);
        else
          reinterpret_cast<uint16_t*>(at)[(j * 8 + i) * 32] = uint16_t(r.w[i / 2] >> (i % 2 * 16));
      }
  }
}
template <class E, class C>
__device__ __forceinline__ void load_pairs(const E* row, const C& c, int j, Pair (&v)[4]) {
  widen<E>(load_vector(row, c, j), v);
}
template <class E, class C>
__device__ __forceinline__ void store_pairs(E* row, const C& c, int j, const Pair (&v)[4]) {
  store_vector(row, c, j, narrow<E>(v));
}

// Parameters may be fp32 under 16-bit activations.
template <class E, class C>
__device__ __forceinline__ void load_param(const void* p, int64_t offset, bool f32, const C& c, int j,
                                           Pair (&v)[4]) {
  if (f32)
    load_pairs(static_cast<const float*>(p) + offset, c, j, v);
  else
    load_pairs(static_cast<const E*>(p) + offset, c, j, v);
}

// ---- 8-bit codes ----------------------------------------------------------------------

// The bits of the largest magnitude; a NaN's are above an infinity's.
template <class E>
__device__ __forceinline__ uint32_t top_bits(const Raw<E>& r) {
  uint32_t top = 0;
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, r.w[i] & 0x7fffffffu);
    return top;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, r.w[i] & 0x7fff7fffu);
    return max(top >> 16, top & 0xffffu);
  }
}
template <class E>
__device__ __forceinline__ float from_bits(uint32_t bits) {
  if constexpr (sizeof(E) == 4) return __uint_as_float(bits);
  else return unpack2<E>(bits).x;
}

// A group's scale, and what its elements are multiplied by (0 in a group of
// zeros or one that is not finite).  The scale is rounded towards zero: 127
// times it is then never above a, which may be the type's largest value.
struct Scaling {
  float scale, inverse;
};
// a / 127 rounded towards zero: a times the float below 1/127 is at most that
// and two units short of it; the exact remainder's sign tells whether the next
// float still fits.
__device__ __forceinline__ float over_127(float a) {
  float q = __fmul_rz(a, 0x1.020408p-7f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float next = __uint_as_float(__float_as_uint(q) + 1);
    q = __fmaf_rn(-127.0f, next, a) >= 0.0f ? next : q;
  }
  return q;
}
__device__ __forceinline__ Scaling scaling(float a) {
  const bool finite = a < INFINITY, tiny = a < kTinyGroup;
  const float safe = tiny || !finite ? 1.0f : a;
  return {finite ? tiny ? 0.0f : over_127(safe) : __uint_as_float(0x7fffffffu),
          tiny || !finite ? 0.0f : __fdiv_rn(127.0f, safe)};
}

// Eight codes.  x * inverse, rounded, + 1.5 * 2^23 rounds the product to an
// integer (nearest even) whose low byte is the code; |code| <= 127 because
// inverse is 127 / a rounded once.  (What is not finite is multiplied by 0:
// its codes mean nothing beside a NaN scale.)  The products are not packed: a
// packed multiply and the add that follows were contracted (one code in 10^5,
// next to a tie, then differed from that of the two operations).
template <class E>
__device__ __forceinline__ uint2 code8(const Raw<E>& r, float inverse) {
  Pair v[4];
  widen<E>(r, v);
  uint32_t bits[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 e = split(v[i]);
    const float2 p = split(add2(make_pair(__fmul_rn(e.x, inverse), __fmul_rn(e.y, inverse)), both(12582912.0f)));
    bits[2 * i] = __float_as_uint(p.x);
    bits[2 * i + 1] = __float_as_uint(p.y);
  }
  uint32_t word[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    word[i] = __byte_perm(__byte_perm(bits[4 * i], bits[4 * i + 1], 0x0040),
                          __byte_perm(bits[4 * i + 2], bits[4 * i + 3], 0x0040), 0x5410);
  return make_uint2(word[0], word[1]);
}

// Vectors of N rows (or N vectors of one row) in 8 bits; half a warp holds a
// group of each.  group_top() gives every lane the bits of its group's largest
// magnitude and share_scaling() shares the N groups' divisions out over their
// lanes; every lane of the warp calls both, lanes beyond the row with zeros.
// N is a power of two, at most 16; lane n of a group has the n-th one's scaling.
template <class E>
__device__ __forceinline__ uint32_t group_top(const Raw<E>& r) {
  uint32_t top = top_bits(r);
#pragma unroll
  for (int i = 8; i; i /= 2) top = max(top, __shfl_xor_sync(~0u, top, i));
  return top;
}
template <int N>
__device__ __forceinline__ Scaling share_scaling(const float (&top)[N]) {
  // top[lane % N], by the lane's bits (an index would put the array in memory)
  float mine[N];
#pragma unroll
  for (int n = 0; n < N; ++n) mine[n] = top[n];
#pragma unroll
  for (int bit = 1; bit < N; bit *= 2)
#pragma unroll
    for (int n = 0; n < N; n += 2 * bit) mine[n] = threadIdx.x & bit ? mine[n + bit] : mine[n];
  return scaling(mine[0]);
}
template <class E>
__device__ __forceinline__ void keep_vector(const Raw<E>& r, const Scaling& shared, int n, int8_t* codes,
                                            float* scale, bool valid, bool group_valid) {
  const float inverse = __shfl_sync(~0u, shared.inverse, n, 16);
  if (valid) *reinterpret_cast<uint2*>(codes) = code8(r, inverse);
  if (threadIdx.x % 16 == n && group_valid) *scale = shared.scale;
}

// A warp keeps one group [col0, col0 + 128) of a row, element by element.
template <class E>
__device__ __forceinline__ void keep_group(const E* row, int col0, int width, int8_t* codes,
                                           float* scales) {
  const int lane = threadIdx.x % 32;
  float v[kGroup / 32];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kGroup / 32; ++i) {
    const int col = col0 + i * 32 + lane;
    v[i] = col < width ? to_float(row[col]) : 0.0f;
    top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  }
#pragma unroll
  for (int i = 16; i; i /= 2) top = max(top, __shfl_xor_sync(~0u, top, i));
  const Scaling s = scaling(__uint_as_float(top));
  if (lane == 0) scales[col0 / kGroup] = s.scale;
#pragma unroll
  for (int i = 0; i < kGroup / 32; ++i) {
    const int col = col0 + i * 32 + lane;
    const uint32_t bits = __float_as_uint(__fadd_rn(__fmul_rn(v[i], s.inverse), 12582912.0f));
    if (col < width) codes[col] = int8_t(bits & 0xffu);
  }
}

// Eight codes times `factor`.  A code's byte with its sign bit flipped, in the
// low mantissa bits of 2^23, is 2^23 + 128 + code exactly: cheaper than eight
// integer conversions.
__device__ __forceinline__ void codes_pairs(uint2 raw, float factor, Pair (&v)[4]) {
  raw.x ^= 0x80808080u;
  raw.y ^= 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? raw.x : raw.y;
    const Pair p = make_pair(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540 + i % 2 * 2)),
                             __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7541 + i % 2 * 2)));
    v[i] = mul2(add2(p, both(-8388736.0f)), both(factor));
  }
}

// Vector j of a kept row times `factor`; `scale` is that of the vector's group
// when the row is wide.
template <int NV, bool kWide>
__device__ __forceinline__ void load_kept(const int8_t* codes, const float* scales, float scale,
                                          float factor, const Columns<NV, kWide>& c, int j, Pair (&v)[4]) {
  if constexpr (kWide) {
    uint2 raw = make_uint2(0, 0);
    if (c.first(j) < c.width) raw = *reinterpret_cast<const uint2*>(codes + c.first(j));
    codes_pairs(raw, scale * factor, v);
  } else {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      e[i] = c.valid(j, i) ? float(codes[c.lone0 + (j * 8 + i) * 32]) *
                                 (scales[c.lone(j, i) / kGroup] * factor)
                           : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_pair(e[2 * i], e[2 * i + 1]);
  }
}

}  // namespace fadam_ops
