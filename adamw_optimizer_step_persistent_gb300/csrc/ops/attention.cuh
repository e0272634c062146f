// Device helpers of attention: tensor-core and tensor-memory instructions of a
// single CTA, boxes of a head's rows, scores and masks.
#pragma once

#include <atomic>

#include "attention_internal.h"
#include "ops_device.cuh"
#include "rows.cuh"

namespace fadam_ops {

// Sixteen warps hold scores, four more multiply and load.  A thread's registers
// are 96 as launched (640 threads in 65536); the sixteen take over what the
// four do without.
constexpr int kScoreWarps = 16, kAttentionThreads = (kScoreWarps + 4) * 32;
constexpr int kMultiply = kScoreWarps, kLoad = kMultiply + 1, kMultiply2 = kMultiply + 2, kIdle = kMultiply + 3;
constexpr int kLaunchRegisters = 96, kScoreRegisters = 104, kOtherRegisters = 64;
static_assert(4 * kScoreRegisters + kOtherRegisters == 5 * kLaunchRegisters, "no more than launched with");
static_assert(kLaunchRegisters * kAttentionThreads <= 65536, "an SM's registers");
// A kernel built with fewer would wait for its share of registers for ever.  (Asked
// once a process; a question that failed, for lack of memory, say, is asked again.)
template <auto kKernel>
fadam_status launched_with(const char* what) {
  static std::atomic<bool> right{false};
  if (right.load(std::memory_order_relaxed)) return FADAM_OK;
  cudaFuncAttributes f{};
  const cudaError_t e = cudaFuncGetAttributes(&f, kKernel);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
  if (f.numRegs != kLaunchRegisters)
    return fail(FADAM_ECUDA, "%s was built with %d registers a thread, not %d", what, f.numRegs, kLaunchRegisters);
  right.store(true, std::memory_order_relaxed);
  return FADAM_OK;
}

constexpr int kBoxBytes = kRows * kChunk * 2;  // 128 rows of 128 bytes, 128-byte swizzle

// A place in a ring of N and the parity of its barrier's phase.  (Kept from turn
// to turn: a quotient and a remainder a turn cost the multiplying warps, whose
// instructions wait among those of twenty warps, some 300 cycles.)
template <int N>
struct Place {
  int at = 0;
  unsigned parity = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      parity ^= 1;
    }
  }
};

// A wait of a whole warp: all lanes have one answer, also when it gives up, so that
// they meet at the next instruction that takes all of them.
__device__ __forceinline__ bool warp_wait(uint32_t bar, unsigned parity, int* status) {
  if (__all_sync(~0u, bar_try(bar, parity))) return true;
  const unsigned long long t0 = now_ns();
  while (!__all_sync(~0u, bar_try(bar, parity)))
    if (__any_sync(~0u, now_ns() - t0 > kWaitNs)) {
      atomicExch(status, FADAM_ETIMEOUT);
      return false;
    }
  return true;
}

// ---- copies -----------------------------------------------------------------------------

__device__ __forceinline__ void load_head_box(uint32_t dst, const CUtensorMap* map, int x, int head,
                                              int token, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(head), "r"(token), "r"(bar)
      : "memory");
}
// 128 tokens of one head, C blocks of 64 elements.
template <int C>
__device__ __forceinline__ void load_head(uint32_t dst, const CUtensorMap* map, int head, int token,
                                          uint32_t bar) {
#pragma unroll
  for (int c = 0; c < C; ++c) load_head_box(dst + c * kBoxBytes, map, c * kChunk, head, token, bar);
}
__device__ __forceinline__ void store_head_box(const CUtensorMap* map, int x, int head, int token,
                                               uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(x), "r"(head), "r"(token), "r"(src)
               : "memory");
}
// Waits until this thread's stores have read shared memory (they are written
// by the time that the kernel ends).
__device__ __forceinline__ void wait_stores() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}
// What this thread wrote to shared memory is there for bulk copies and tensor cores.
__device__ __forceinline__ void fence_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// A barrier of a group of warps; and one that says whether any thread's `x` holds.
__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool group_any(int id, int threads, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(uint32_t(x))
      : "memory");
  return any != 0;
}

// ---- tensor cores ----------------------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t dst_shared, int columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_shared),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, int columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

// One lane of a whole warp, always the same one.  (The compiler knows it for
// one: tensor-core instructions behind it take their operands from uniform
// registers as they are; behind lane == 0 each cost 85 to 130 cycles.)
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// A value that is the same in all lanes, so that the compiler knows it.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(~0u, x, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(~0u, x, 0); }

// D (+)= A B, both 16-bit in shared memory.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}
// The same with A in tensor memory: a lane to a row, two elements to a column.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}
// Arrive at `bar` once the tensor-core work issued so far by this thread is done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

// 32 columns of this warp's 32 lanes, stored once tmem_stored() returns.
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A tile's block as the operand whose k runs along its rows' elements (k-major:
// scores), or along the rows themselves (MN: products with v, k, q, grad_out,
// blocks of 64 elements one box apart).
template <bool MN>
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  const uint64_t lead = MN ? kBoxBytes >> 4 : 1;
  return uint64_t((addr & 0x3ffff) >> 4) | lead << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
         uint64_t(2) << 61;
}
template <class T, bool B_MN>
__device__ __forceinline__ uint32_t instruction(int n) {
  constexpr uint32_t kType = T::code == FADAM_DT_BF16 ? 1 : 0;
  return 1u << 4 | kType << 7 | kType << 10 | uint32_t(B_MN) << 16 | uint32_t(n / 8) << 17 |
         uint32_t(kRows / 16) << 24;
}

// D[128, 128] = A B^T over `steps` 16s of a head's elements.  `half` is called
// half way through.
struct Nothing {
  __device__ __forceinline__ void operator()() const {}
};
template <class T, int C, class Half = Nothing>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b, int steps, Half half = Half()) {
  const uint64_t da = tile_desc<false>(a), db = tile_desc<false>(b);
  const uint32_t idesc = instruction<T, false>(kRows);
#pragma unroll
  for (int k = 0; k < C * kChunk / 16; ++k) {
    const uint64_t at = (k / 4) * (kBoxBytes >> 4) + (k % 4) * 2;  // 16 elements on: 32 bytes, or the next box
    if (k < steps) mma(d, da + at, db + at, idesc, k > 0);
    if (k == C * kChunk / 32 - 1) half();
  }
}

// D[128, n] (+)= A B over the tile's 128 rows, A in tensor memory: kEach
// elements (half as many columns) in a place, the places `apart`.
template <class T, int kEach>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, int apart, uint32_t b, int n, bool add) {
  const uint64_t db = tile_desc<true>(b);
  const uint32_t idesc = instruction<T, true>(n);
#pragma unroll
  for (int k = 0; k < kRows / 16; ++k)  // 16 rows on: 2048 bytes, 8 columns
    mma_tmem(d, a + k * 16 / kEach * apart + k * 16 % kEach / 2, db + k * (2048 >> 4), idesc, add || k > 0);
}

// Rows of a tile (its first one is token `at`) that lie outside all documents
// become zero, so that 0 times what padding holds is 0.  By a whole warp,
// between the copy's arrival and the product over the tile's rows.
template <int C>
__device__ __forceinline__ void clean_rows(uint32_t tile, int at, const AttentionArgs& g) {
  const int from = __ldg(g.documents) - at, to = __ldg(g.documents + g.n_documents) - at;
  if (from <= 0 && to >= kRows) return;
  for (int r = threadIdx.x % 32; r < kRows; r += 32)
    if (r < from || r >= to)
#pragma unroll
      for (int i = 0; i < 8 * C; ++i)
        store_shared(tile + (i / 8) * kBoxBytes + r * 128 + (i % 8) * 16, make_uint4(0, 0, 0, 0));
  fence_shared();
  __syncwarp();
}

// N elements of a lane's row, from element c of the head, rounded into a tile:
// `place` is the row's in its first block.
template <class E, int N>
__device__ __forceinline__ void store_units(uint32_t place, int c, const float (&o)[N]) {
#pragma unroll
  for (int u = 0; u < N / 8; ++u) {
    const int unit = c % kChunk / 8 + u;
    store_shared(place + c / kChunk * kBoxBytes + ((unit ^ (threadIdx.x & 7)) * 16),
                 make_uint4(pack2<E>(o[8 * u], o[8 * u + 1]), pack2<E>(o[8 * u + 2], o[8 * u + 3]),
                            pack2<E>(o[8 * u + 4], o[8 * u + 5]), pack2<E>(o[8 * u + 6], o[8 * u + 7])));
  }
}

// 32 floats of shared memory, the same for all lanes.
__device__ __forceinline__ void load_pairs(uint32_t at, Pair (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 u = load_shared(at + i * 16);
    v[2 * i] = make_pair(__uint_as_float(u.x), __uint_as_float(u.y));
    v[2 * i + 1] = make_pair(__uint_as_float(u.z), __uint_as_float(u.w));
  }
}

// ---- masks -----------------------------------------------------------------------------

// The spans of token i of the document [a, b) with a prefix of p tokens.
__host__ __device__ __forceinline__ Spans spans_in(int i, int a, int b, int p, bool causal) {
  Spans s{a, b, a, b};
  if (causal) {
    s.key_hi = i + 1 > a + p ? i + 1 : a + p;
    s.query_lo = i < a + p ? a : i;
  }
  return s;
}
__device__ __forceinline__ Spans spans_of(const AttentionArgs& g, int i) {
  if (g.spans) {
    const int4 v = __ldg(reinterpret_cast<const int4*>(g.spans) + i);
    return Spans{v.x, v.y, v.z, v.w};
  }
  const int d = i / g.sequence, a = d * g.sequence;
  const int p = g.prefix ? min(max(__ldg(g.prefix + d), 0), g.sequence) : 0;
  return spans_in(i, a, a + g.sequence, p, g.causal);
}

// Where in `peaks` a token's document has its place; whether it is in one.
struct Entry {
  int at;
  bool lives;
};
__device__ __forceinline__ Entry entry_of(const AttentionArgs& g, int i) {
  if (i >= g.tokens) return Entry{0, false};
  if (!g.spans) return Entry{i / g.sequence, true};
  const int2 keys = __ldg(reinterpret_cast<const int2*>(g.spans + i));
  return Entry{keys.x, keys.x < keys.y};
}

// What a tile's 128 rows need of the other side, from the spans of its rows
// that see anything: any of it lies in [lo, hi), all rows see [all_lo, all_hi).
struct Reach {
  int lo, hi, all_lo, all_hi;
  __device__ __forceinline__ int first() const { return lo / kRows; }
  __device__ __forceinline__ int last() const { return hi > lo ? (hi + kRows - 1) / kRows : lo / kRows; }
};
constexpr int kNever = 0x7fffff80;  // a multiple of 128
// One warp's part of it; rows that do not exist (`here` false) ask for nothing.
__device__ __forceinline__ Reach reach_of(int lo, int hi, bool here) {
  const bool sees = here && lo < hi;
  Reach r;
  r.lo = __reduce_min_sync(~0u, sees ? lo : kNever);
  r.hi = __reduce_max_sync(~0u, sees ? hi : 0);
  r.all_lo = __reduce_max_sync(~0u, here ? lo : 0);
  r.all_hi = __reduce_min_sync(~0u, here ? hi : kNever);
  return r;
}
__device__ __forceinline__ Reach join(const Reach& a, const Reach& b) {
  return Reach{min(a.lo, b.lo), max(a.hi, b.hi), max(a.all_lo, b.all_lo), min(a.all_hi, b.all_hi)};
}
__device__ __forceinline__ Reach uniform(const Reach& r) {
  return Reach{uniform(r.lo), uniform(r.hi), uniform(r.all_lo), uniform(r.all_hi)};
}

// ---- scores ------------------------------------------------------------------------------

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inverse_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Scores in units of log 2, from products q . k.
struct Scores {
  float mul;         // scale log2 e
  float cap;         // cap log2 e; 0: none
  float inverse;     // 1 / cap: scores to multiples of the cap
  float slope;       // slope log2 e; 0: none
  const float2 (&series)[4];
  __device__ __forceinline__ Scores(const AttentionArgs& g, int head) : series(g.series) {
    mul = g.scale * kLog2e;
    cap = g.softcap * kLog2e;
    inverse = g.softcap > 0.0f ? g.scale / g.softcap : 0.0f;
    slope = g.slopes ? __ldg(g.slopes + head) * kLog2e : 0.0f;
  }
  // Products become capped scores, cap tanh(s / cap).  Those up to a quarter of the
  // cap by tanh's Taylor series to the seventh power (off by 9e-8 of the cap there):
  // six multiplications for two scores.  (In powers of the product itself they are
  // five, but the factors of a wide cap's higher powers are then below fp32's
  // numbers.)  Those beyond it by 1 - 2 / (exp(2 y) + 1),
  // whose exponential and reciprocal take three times the time of the softmax's own
  // exponential, and which a warp without any leaves out.  Each score's form is its
  // own: what lies beside it, seen or not, changes no bit of it.  (4096 packed
  // tokens, 32 heads of 128, in a graph: with a cap of 50, which no score comes near, forward 61 us
  // and backward 158; with one of 2, where every warp has scores beyond, 95 and 202,
  // and 68 and 171 as long as these warps took the second form for all of theirs.)
  template <int N>
  __device__ __forceinline__ void capped(float (&s)[N]) const {
    float far[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < N; c += 4)
#pragma unroll
      for (int k = 0; k < 2; ++k) far[k] = fmaxf(fmaxf(far[k], fabsf(s[c + k])), fabsf(s[c + 2 + k]));
    if (__any_sync(~0u, fmaxf(far[0], far[1]) * inverse > 0.25f)) {
      // (two passes in place: both forms of a score at a time would not fit the registers)
      unsigned done[N / 32] = {};
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (fabsf(s[c]) * inverse > 0.25f) {
          const float e = exp2_fast(s[c] * (2.0f * kLog2e * inverse));
          s[c] = fmaf(-2.0f * cap, inverse_fast(e + 1.0f), cap);
          done[c / 32] |= 1u << c % 32;
        }
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const float x = s[c], y = x * inverse, u = y * y;
        const float near = x * fmaf(u, fmaf(u, fmaf(u, series[3].x, series[2].x), series[1].x), series[0].x);
        if (!(done[c / 32] >> c % 32 & 1)) s[c] = near;
      }
      return;
    }
    Pair of[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) of[i] = make_pair(series[i].x, series[i].y);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const Pair x = make_pair(s[c], s[c + 1]), y = mul2(x, both(inverse)), u = mul2(y, y);
      const float2 v = split(mul2(x, fma2(u, fma2(u, fma2(u, of[3], of[2]), of[1]), of[0])));
      s[c] = v.x;
      s[c + 1] = v.y;
    }
  }
  // A bias by distance; `apart`: the first column's place less the row's.
  template <int N>
  __device__ __forceinline__ void lowered(float (&s)[N], float apart) const {
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] = fmaf(-slope, fabsf(apart + float(c)), s[c]);
  }
  // Products become scores, but for a factor that is returned.  (Without kCap there
  // is none.)
  template <bool kCap, int N>
  __device__ __forceinline__ float finish(float (&s)[N], float apart) const {
    if (kCap && cap != 0.0f) {
      capped(s);
    } else if (slope != 0.0f) {
#pragma unroll
      for (int c = 0; c < N; ++c) s[c] *= mul;
    } else {
      return mul;
    }
    if (slope != 0.0f) lowered(s, apart);
    return 1.0f;
  }
};

}  // namespace fadam_ops
