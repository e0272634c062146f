// The norms around a block: post-norm, gate, residual scale, add, pre-norm,
// forward and backward (formulas at fadam_block_norm and below).  Bound by
// memory: both directions read and write every row once.
//
// CTAs stay and take runs of rows, so that the parameters are read once (and,
// backward, the sums over rows of their gradients stay with the thread that
// owns the columns).  A row is spread over the CTA, 16 columns to a thread
// (32 beyond 8192).  Where rows are whole aligned words, a few threads copy the
// coming rows' tensors into a ring of stages in shared memory with bulk
// copies, so that the loads in flight do not depend on how many warps the
// registers allow; elsewhere, and when each CTA has one row only, threads load
// their own columns.  The barrier of a row's reduction also says that its
// stage has been read.  Up to 4096 columns two and more CTAs share an SM, which
// hides their reductions' latency in one another.  Backward, 16384 x 4096 in
// bf16 from checkpoints: 121 us, 5.3 TB/s; forward, 8192 x 4096 with both
// checkpoints: 66 us, 5.1 TB/s.  What is left over memory is the issue of some
// 40 instructions an element (half the slots) by the 16 warps that 128
// registers a thread leave an SM, and a row's two or one reductions.
//
// Backward, with hh = h_out r2, fh = f r1 and, for a row,
//   g = grad_x_out pre_weight
//   e = grad_h_out + r2 (g - hh mean(g hh))                (= grad_h)
//   t = alpha gate post_weight e
//   grad_f = r1 (t - fh mean(t fh))                        (or t, no post-norm)
// the second mean would wait for the first; instead one reduction gives
//   S1 = sum g hh,  S2 = sum a fh (grad_h_out + r2 g),  S3 = sum a fh hh
// with a = alpha gate post_weight, and sum t fh = S2 - S3 r2 S1 / width.
// The parameters' gradients need two sums per column,
//   Q = sum e fh (over rows of one gate),  P = sum grad_x_out hh:
// grad_gate = alpha post_weight Q, grad_post_weight = sum over gates of
// alpha gate Q, grad_pre_weight = P.  The CTAs' sums go to the workspace and a
// second kernel adds them in a fixed order.
#pragma once

#include "block_norm_internal.h"
#include "rows.cuh"

namespace fadam_ops {
namespace {

// How a row reaches the registers: through the ring, or loaded by each thread,
// whole vectors or element by element.
constexpr int kRing = 0, kVectors = 1, kElements = 2;

struct Run {
  int gate, begin, end;
};
__device__ __forceinline__ Run norm_run(const NormRuns& r, int run) {
  const int gate = int(unsigned(run) / unsigned(r.slices)), slice = run - gate * r.slices;
  const int first = gate * r.rows_per_gate;
  return {gate, first + int(int64_t(r.rows_per_gate) * slice / r.slices),
          first + int(int64_t(r.rows_per_gate) * (slice + 1) / r.slices)};
}

// The ring.  The first lanes of the CTA's first warps feed it, each its share
// of the row's tensors (one thread for all of them would hold up its warp, and
// with it every row's barrier): the CTA's rows in order, `stages` of them ahead
// of the one that is worked on.
struct Ring {
  const RingArgs& args;
  const NormRuns& runs;
  uint64_t* full;          // [stages] barriers
  uint32_t stages;         // shared address of the stages
  int run, row, end;       // feeding threads: the next row to copy
  int next, stage;         // stage it goes to; stage that is worked on
  unsigned parity;         // of the latter's barrier
  bool ok;                 // no wait has given up (the warps stay together either way)

  __device__ __forceinline__ Ring(const RingArgs& a, const NormRuns& r, uint64_t* bars, void* memory)
      : args(a), runs(r), full(bars), stages(shared_addr(memory)), run(blockIdx.x), next(0), stage(0),
        parity(0), ok(true) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < args.stages; ++i) bar_init(shared_addr(full + i), 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    const Run first = norm_run(runs, run);
    row = first.begin;
    end = first.end;
    if (feeds())
      for (int i = 0; i < args.stages; ++i) feed();
  }

  __device__ __forceinline__ bool feeds() const {
    return threadIdx.x % 32 == 0 && int(threadIdx.x) / 32 < args.sources;
  }

  __device__ __forceinline__ void feed() {
    if (row == end) {
      if (run + int(gridDim.x) >= runs.runs) return;
      run += gridDim.x;
      const Run r = norm_run(runs, run);
      row = r.begin;
      end = r.end;
    }
    const uint32_t bar = shared_addr(full + next);
    const uint32_t to = stages + next * args.bytes;
    // (a copy may land before what is expected is known: the phase waits for the arrival)
    if (threadIdx.x == 0) bar_expect(bar, args.bytes);
    for (int i = threadIdx.x / 32; i < args.sources; i += blockDim.x / 32) {
      const RingSource& s = args.source[i];
      load_bytes(to + s.offset, static_cast<const char*>(s.base) + row * s.stride, s.bytes, bar);
    }
    ++row;
    next = next + 1 == args.stages ? 0 : next + 1;
  }

  // Waits for the next row; returns its offset in the stages.
  __device__ __forceinline__ int wait() {
    if (ok) ok = bar_wait(shared_addr(full + stage), parity, args.status);
    return stage * args.bytes;
  }
  // Every thread has read the row (the caller has passed a barrier since).
  __device__ __forceinline__ void release() {
    if (feeds() && ok) feed();
    if (++stage == args.stages) {
      stage = 0;
      parity ^= 1;
    }
  }
  // After a wait that gave up: the copies still in flight get time to land.
  __device__ __forceinline__ void drain() {
    if (ok || threadIdx.x != 0) return;
    for (int i = 0; i < args.stages; ++i) {
      bar_wait(shared_addr(full + stage), parity, args.status);
      if (++stage == args.stages) {
        stage = 0;
        parity ^= 1;
      }
    }
  }
};

// Sums one value, or four, over the CTA's first `threads` threads; each of
// them gets the sums.  `shared` holds 4 * kMaxWarps floats and is free again
// after their next barrier.  Four: in two steps every lane gives away half of
// its values and takes the other half of its neighbour's, so that the four
// sums take 6 shuffles and not 20; lane i then has value i / 8.
__device__ __forceinline__ void sync_rows(int threads) {
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}
__device__ __forceinline__ float block_sum(float v, float* shared, int threads) {
#pragma unroll
  for (int i = 16; i; i /= 2) v += __shfl_xor_sync(~0u, v, i);
  const int lane = threadIdx.x % 32, warps = threads / 32;
  if (lane == 0) shared[threadIdx.x / 32] = v;
  sync_rows(threads);
  v = lane % kMaxWarps < warps ? shared[lane % kMaxWarps] : 0.0f;
#pragma unroll
  for (int i = kMaxWarps / 2; i; i /= 2) v += __shfl_xor_sync(~0u, v, i);
  return v;
}
__device__ __forceinline__ void block_sums(float (&v)[4], float* shared, int threads) {
  const int lane = threadIdx.x % 32, warps = threads / 32;
  const bool high = lane & 16, odd = lane & 8;
  float a = high ? v[2] : v[0], b = high ? v[3] : v[1];
  a += __shfl_xor_sync(~0u, high ? v[0] : v[2], 16);
  b += __shfl_xor_sync(~0u, high ? v[1] : v[3], 16);
  float s = odd ? b : a;
  s += __shfl_xor_sync(~0u, odd ? a : b, 8);
#pragma unroll
  for (int i = 4; i; i /= 2) s += __shfl_xor_sync(~0u, s, i);
  // lane 8 n has value n of this warp
  if (lane % 8 == 0) shared[lane / 8 * kMaxWarps + threadIdx.x / 32] = s;
  sync_rows(threads);
  const int w = lane % 8;
  const float* from = shared + lane / 8 * kMaxWarps;
  s = (w < warps ? from[w] : 0.0f) + (w + 8 < warps ? from[w + 8] : 0.0f);
#pragma unroll
  for (int i = 4; i; i /= 2) s += __shfl_xor_sync(~0u, s, i);
#pragma unroll
  for (int n = 0; n < 4; ++n) v[n] = __shfl_sync(~0u, s, 8 * n);
}

// ---- forward -------------------------------------------------------------------------

// A row's f and h_out kept in 8 bits, from registers where the vectors lie
// next to each other.
template <class F, class H, int NV>
__device__ __forceinline__ void keep_row(const NormArgs& a, int64_t row, const Columns<NV, true>& c,
                                         const Raw<F> (&f)[NV], const Raw<H> (&h)[NV]) {
  const int64_t at = row * c.width, group_at = row * ((c.width + kGroup - 1) / kGroup);
  float top[2 * NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    top[j] = a.f_codes ? from_bits<F>(group_top(f[j])) : 0.0f;
    top[NV + j] = a.h_codes ? from_bits<H>(group_top(h[j])) : 0.0f;
  }
  const Scaling shared = share_scaling<2 * NV>(top);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = c.first(j), group = col / kGroup;
    const bool valid = col < c.width, group_valid = group * kGroup < c.width;
    if (a.f_codes)
      keep_vector(f[j], shared, j, a.f_codes + at + col, a.f_scales + group_at + group, valid, group_valid);
    if (a.h_codes)
      keep_vector(h[j], shared, NV + j, a.h_codes + at + col, a.h_scales + group_at + group, valid,
                  group_valid);
  }
}
// Else from memory (h_out once the CTA has written it), a warp to a group.
template <class E, int NV>
__device__ __forceinline__ void keep_row(const E* row, int64_t index, int8_t* codes, float* scales,
                                         const Columns<NV, false>& c) {
  const int groups = (c.width + kGroup - 1) / kGroup;
  for (int g = c.tid / 32; g < groups; g += c.threads / 32)
    keep_group(row, g * kGroup, c.width, codes + index * c.width, scales + index * groups);
}

template <class F, class H, int NV, int MODE>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    norm_forward_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float shared[2][4 * kMaxWarps];
  __shared__ __align__(8) uint64_t bars[kMaxNormStages];
  extern __shared__ __align__(128) unsigned char dynamic[];
  constexpr bool kWide = MODE != kElements;
  const Columns<NV, kWide> c(a.threads, int(threadIdx.x), a.width);
  const int width = a.width;
  const float inv_width = 1.0f / float(width);
  chain_wait();
  // (a ring of no stages when rows are loaded directly)
  Ring ring(a.ring, a.runs, bars, dynamic);
  Pair pre[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_param<F>(a.pre, 0, a.params_f32, c, j, pre[j]);

  for (int u = blockIdx.x; u < a.runs.runs; u += gridDim.x) {
    const Run run = norm_run(a.runs, u);
    Pair scale[NV][4];  // alpha gate post_weight
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) scale[j][i] = both(a.alpha);
      Pair v[4];
      if (a.gate) {
        load_param<F>(a.gate, int64_t(run.gate) * width, a.params_f32, c, j, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) scale[j][i] = mul2(scale[j][i], v[i]);
      }
      if (a.post) {
        load_param<F>(a.post, 0, a.params_f32, c, j, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) scale[j][i] = mul2(scale[j][i], v[i]);
      }
    }
    for (int at_row = run.begin; at_row < run.end; ++at_row) {
      const int64_t row = at_row;
      Raw<F> f_raw[NV];
      Pair h[NV][4];
      if (MODE == kRing) {
        const unsigned char* at = dynamic + ring.wait();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          f_raw[j] = load_vector(reinterpret_cast<const F*>(at), c, j);
          load_pairs(reinterpret_cast<const H*>(at + a.ring.source[1].offset), c, j, h[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          f_raw[j] = load_vector(static_cast<const F*>(a.f) + row * a.f_stride, c, j);
          load_pairs(static_cast<const H*>(a.h) + row * a.h_stride, c, j, h[j]);
        }
      }
      float r1 = 1.0f;
      if (a.post) {
        Pair s = both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          Pair f[4];
          widen<F>(f_raw[j], f);
#pragma unroll
          for (int i = 0; i < 4; ++i) s = fma2(f[i], f[i], s);
        }
        r1 = rsqrtf(block_sum(sum2(s), shared[0], c.threads) * inv_width + a.eps);
        if (c.tid == 0) a.r1[row] = r1;
      }
      Pair s = both(0.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Pair f[4];
        widen<F>(f_raw[j], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[j][i] = fma2(mul2(f[i], both(r1)), scale[j][i], h[j][i]);
          s = fma2(h[j][i], h[j][i], s);
        }
      }
      const float r2 = rsqrtf(block_sum(sum2(s), shared[1], c.threads) * inv_width + a.eps);
      if (c.tid == 0) a.r2[row] = r2;
      if (MODE == kRing) ring.release();
      Raw<H> out[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        out[j] = narrow<H>(h[j]);
        store_vector(static_cast<H*>(a.h_out) + row * width, c, j, out[j]);
        Pair x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = mul2(mul2(h[j][i], both(r2)), pre[j][i]);
        store_pairs(static_cast<F*>(a.x_out) + row * width, c, j, x);
      }
      if (a.f_codes || a.h_codes) {
        if constexpr (kWide) {
          keep_row<F, H, NV>(a, row, c, f_raw, out);
        } else {
          __threadfence_block();
          sync_rows(c.threads);
          if (a.f_codes)
            keep_row(static_cast<const F*>(a.f) + row * a.f_stride, row, a.f_codes, a.f_scales, c);
          if (a.h_codes) keep_row(static_cast<const H*>(a.h_out) + row * width, row, a.h_codes, a.h_scales, c);
        }
      }
      if (!a.post) sync_rows(c.threads);  // one buffer's barrier guards the other's reuse
    }
  }
  chain_next();
  if (MODE == kRing) ring.drain();
}

// ---- backward --------------------------------------------------------------------------

// Where the column sums and the parameters live follows the registers there
// are: the parameters in shared memory, the sums in registers (shared memory
// for NV 4, where pre_weight no longer fits and is read again for every row).
template <class F, class H, int NV, int MODE>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    norm_backward_kernel(const __grid_constant__ NormGradArgs a) {
  constexpr bool kSharedSums = NV > 2, kPreAgain = NV > 2;
  __shared__ float shared[2][4 * kMaxWarps];
  __shared__ __align__(8) uint64_t bars[kMaxNormStages];
  extern __shared__ __align__(128) unsigned char dynamic[];
  constexpr bool kWide = MODE != kElements;
  const Columns<NV, kWide> c(a.threads, int(threadIdx.x), a.width);
  const int width = a.width, groups = (width + kGroup - 1) / kGroup, threads = a.threads, tid = c.tid;
  const float inv_width = 1.0f / float(width);
  // [vector][pair / 2][thread][2]
  Pair* params = reinterpret_cast<Pair*>(dynamic + (MODE == kRing ? a.ring.stages * a.ring.bytes : 0));
  Pair* sums = params + (kPreAgain ? 1 : 2) * NV * 4 * threads;
  chain_wait();
  Ring ring(a.ring, a.runs, bars, dynamic);
  constexpr int NS = kSharedSums ? 1 : NV;
  Pair q_reg[NS][4], p_reg[NS][4], pre_again[4];
  // column sums: Q of the current run, and P
  auto q = [&](int j, int i) -> Pair& {
    if constexpr (kSharedSums) return sums[((j * 2 + i / 2) * threads + tid) * 2 + i % 2]; else return q_reg[j][i];
  };
  auto p = [&](int j, int i) -> Pair& {
    if constexpr (kSharedSums) return sums[(((NV + j) * 2 + i / 2) * threads + tid) * 2 + i % 2]; else return p_reg[j][i];
  };
  // parameters: a = alpha gate post_weight of the current gate, and pre_weight
  auto scale = [&](int j, int i) -> Pair& { return params[((j * 2 + i / 2) * threads + tid) * 2 + i % 2]; };
  auto pre = [&](int j, int i) -> Pair& {
    if constexpr (kPreAgain) return pre_again[i]; else return params[(((NV + j) * 2 + i / 2) * threads + tid) * 2 + i % 2];
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    Pair v[4];
    load_param<F>(a.pre, 0, a.params_f32, c, j, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p(j, i) = both(0.0f);
      pre(j, i) = v[i];
    }
  }

  int turn = 0;
  for (int u = blockIdx.x; u < a.runs.runs; u += gridDim.x) {
    const Run run = norm_run(a.runs, u);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Pair s[4], v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = both(a.alpha);
      if (a.gate) {
        load_param<F>(a.gate, int64_t(run.gate) * width, a.params_f32, c, j, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = mul2(s[i], v[i]);
      }
      if (a.post) {
        load_param<F>(a.post, 0, a.params_f32, c, j, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = mul2(s[i], v[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        scale(j, i) = s[i];
        q(j, i) = both(0.0f);
      }
    }

    // what a row needs beside its vectors, read one row ahead
    float r1_next, r2_next, f_scale[NV], h_scale[NV];
    auto fetch = [&](int64_t row) {
      r1_next = a.r1 ? __ldg(a.r1 + row) : 1.0f;
      r2_next = __ldg(a.r2 + row);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int group = min(c.first(j), width - 1) / kGroup;
        f_scale[j] = kWide && a.f_codes ? __ldg(a.f_scales + row * groups + group) : 0.0f;
        h_scale[j] = kWide && a.h_codes ? __ldg(a.h_scales + row * groups + group) : 0.0f;
      }
    };
    fetch(run.begin);

    for (int at_row = run.begin; at_row < run.end; ++at_row, turn ^= 1) {
      const int64_t row = at_row;
      const float r1 = r1_next, r2 = r2_next;
      Pair fh[NV][4], hh[NV][4], eg[NV][4];
      Pair s1 = both(0.0f), s2 = s1, s3 = s1;
      const unsigned char* at = dynamic + (MODE == kRing ? ring.wait() : 0);
      const int to_f = a.ring.source[1].offset, to_h = a.ring.source[2].offset,
                to_gh = a.ring.source[3].offset;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Pair gx[4];
        if (MODE == kRing) {
          load_pairs(reinterpret_cast<const F*>(at), c, j, gx);
          if (a.f_codes)
            load_kept(reinterpret_cast<const int8_t*>(at + to_f), nullptr, f_scale[j], r1, c, j, fh[j]);
          else
            load_pairs(reinterpret_cast<const F*>(at + to_f), c, j, fh[j]);
          if (a.h_codes)
            load_kept(reinterpret_cast<const int8_t*>(at + to_h), nullptr, h_scale[j], r2, c, j, hh[j]);
          else
            load_pairs(reinterpret_cast<const H*>(at + to_h), c, j, hh[j]);
          if (a.gh) load_pairs(reinterpret_cast<const H*>(at + to_gh), c, j, eg[j]);
        } else {
          load_pairs(static_cast<const F*>(a.gx) + row * a.gx_stride, c, j, gx);
          if (a.f_codes)
            load_kept(a.f_codes + row * width, a.f_scales + row * groups, f_scale[j], r1, c, j, fh[j]);
          else
            load_pairs(static_cast<const F*>(a.f) + row * a.f_stride, c, j, fh[j]);
          if (a.h_codes)
            load_kept(a.h_codes + row * width, a.h_scales + row * groups, h_scale[j], r2, c, j, hh[j]);
          else
            load_pairs(static_cast<const H*>(a.h) + row * a.h_stride, c, j, hh[j]);
          if (a.gh) load_pairs(static_cast<const H*>(a.gh) + row * a.gh_stride, c, j, eg[j]);
        }
        if (!a.gh)
#pragma unroll
          for (int i = 0; i < 4; ++i) eg[j][i] = both(0.0f);
        if (!a.f_codes)
#pragma unroll
          for (int i = 0; i < 4; ++i) fh[j][i] = mul2(fh[j][i], both(r1));
        if (!a.h_codes)
#pragma unroll
          for (int i = 0; i < 4; ++i) hh[j][i] = mul2(hh[j][i], both(r2));
        if constexpr (kPreAgain) load_param<F>(a.pre, 0, a.params_f32, c, j, pre_again);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p(j, i) = fma2(gx[i], hh[j][i], p(j, i));
          const Pair g = mul2(gx[i], pre(j, i));
          s1 = fma2(g, hh[j][i], s1);
          eg[j][i] = fma2(both(r2), g, eg[j][i]);
          const Pair af = mul2(scale(j, i), fh[j][i]);
          s2 = fma2(af, eg[j][i], s2);
          s3 = fma2(af, hh[j][i], s3);
        }
      }
      if (at_row + 1 < run.end) fetch(at_row + 1);
      float s[4] = {sum2(s1), sum2(s2), sum2(s3), 0.0f};
      block_sums(s, shared[turn], threads);
      if (MODE == kRing) ring.release();
      const float mean = s[0] * inv_width;
      const Pair c1 = both(-r2 * mean);
      const Pair c2 = both(a.post ? -r1 * ((s[1] - s[2] * r2 * mean) * inv_width) : 0.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Pair df[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Pair e = fma2(hh[j][i], c1, eg[j][i]);
          q(j, i) = fma2(e, fh[j][i], q(j, i));
          df[i] = fma2(mul2(scale(j, i), e), both(r1), mul2(fh[j][i], c2));
          eg[j][i] = e;
        }
        store_pairs(static_cast<H*>(a.dh) + row * width, c, j, eg[j]);
        store_pairs(static_cast<F*>(a.df) + row * width, c, j, df);
      }
    }

    // this run's share of the gate's and the post-norm's gradients
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Pair v[4], g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = g[i] = both(1.0f);
      if (a.post) load_param<F>(a.post, 0, a.params_f32, c, j, v);
      if (a.gate) load_param<F>(a.gate, int64_t(run.gate) * width, a.params_f32, c, j, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Pair sum = mul2(both(a.alpha), q(j, i));
        g[i] = mul2(g[i], sum);
        v[i] = mul2(v[i], sum);
      }
      if (a.post_parts) {  // summed over this CTA's runs
        float* part = a.post_parts + int64_t(blockIdx.x) * width;
        if (u != int(blockIdx.x)) {
          Pair old[4];
          load_pairs(part, c, j, old);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = add2(g[i], old[i]);
        }
        store_pairs(part, c, j, g);
      }
      if (a.gate_parts) {
        store_pairs(a.gate_parts + int64_t(u) * width, c, j, v);
      } else if (a.gate_out) {
        if (a.params_f32)
          store_pairs(static_cast<float*>(a.gate_out) + int64_t(run.gate) * width, c, j, v);
        else
          store_pairs(static_cast<F*>(a.gate_out) + int64_t(run.gate) * width, c, j, v);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    Pair v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p(j, i);
    store_pairs(a.pre_parts + int64_t(blockIdx.x) * width, c, j, v);
  }
  chain_next();
  if (MODE == kRing) ring.drain();
}

// ---- launches ------------------------------------------------------------------------------

template <class Args>
fadam_status launch_norm(void (*kernel)(Args), const Args& a, int threads, size_t smem,
                         cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  // Beyond 48 KB, static arrays included, it has to be asked for: always as much as
  // any launch takes, because the limit is the kernel's, and one that another
  // thread lowered before this launch would refuse it.
  if (smem > 40 * 1024)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kNormSharedBytes));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  return launch_chained("block norm launch", kernel, a.runs.ctas, threads, smem, stream, a);
}

// Whether rows go through the ring, and with how many stages: rows of whole
// aligned words, more than one to a CTA, two stages at least.
inline bool plan_ring(RingArgs& ring, const NormRuns& runs, bool wide, int threads,
                      size_t other_bytes) {
  ring.bytes = 0;
  for (int i = 0; i < ring.sources; ++i) {
    RingSource& s = ring.source[i];
    s.offset = ring.bytes;
    ring.bytes += s.bytes;
    wide = wide && !misaligned(s.base, 16) && s.stride % 16 == 0 && s.bytes % 16 == 0;
  }
  const size_t share = kNormSharedBytes / norm_ctas_per_sm(threads);
  if (!wide || int64_t(runs.gates) * runs.rows_per_gate <= runs.ctas || share < other_bytes) return false;
  const size_t fit = (share - other_bytes) / ring.bytes;
  ring.stages = int(fit < kMaxNormStages ? fit : kMaxNormStages);
  return ring.stages >= 2;
}

template <class F, class H, int NV>
fadam_status forward(const NormArgs& a, int mode, size_t smem, cudaStream_t stream) {
  return launch_norm<const NormArgs>(mode == kRing      ? norm_forward_kernel<F, H, NV, kRing>
                                     : mode == kVectors ? norm_forward_kernel<F, H, NV, kVectors>
                                                        : norm_forward_kernel<F, H, NV, kElements>,
                                     a, a.threads, smem, stream);
}

template <class F, class H>
fadam_status norm_forward(NormArgs a, cudaStream_t stream) {
  const RowShape r = row_shape(a.width);
  a.threads = r.threads;
  a.ring.sources = 2;
  a.ring.source[0] = {a.f, a.f_stride * int64_t(sizeof(F)), a.width * int(sizeof(F))};
  a.ring.source[1] = {a.h, a.h_stride * int64_t(sizeof(H)), a.width * int(sizeof(H))};
  int mode = kRing;
  if (!plan_ring(a.ring, a.runs, a.wide, r.threads, 0)) {
    a.ring.stages = 0;
    mode = a.wide ? kVectors : kElements;
  }
  const size_t smem = size_t(a.ring.stages) * a.ring.bytes;
  return r.nv == 2 ? forward<F, H, 2>(a, mode, smem, stream) : forward<F, H, 4>(a, mode, smem, stream);
}

template <class F, class H>
fadam_status norm_backward(NormGradArgs a, cudaStream_t stream) {
  const RowShape r = row_shape(a.width);
  a.threads = r.threads;
  const int f = int(sizeof(F)), h = int(sizeof(H));
  a.ring.sources = a.gh ? 4 : 3;
  a.ring.source[0] = {a.gx, a.gx_stride * f, a.width * f};
  a.ring.source[1] = a.f_codes ? RingSource{a.f_codes, a.width, a.width}
                               : RingSource{a.f, a.f_stride * f, a.width * f};
  a.ring.source[2] = a.h_codes ? RingSource{a.h_codes, a.width, a.width}
                               : RingSource{a.h, a.h_stride * h, a.width * h};
  a.ring.source[3] = {a.gh, a.gh_stride * h, a.width * h};
  const size_t array = size_t(r.nv) * 8 * r.threads * sizeof(float);
  int mode = kRing;
  if (r.nv > 2 || !plan_ring(a.ring, a.runs, a.wide, r.threads, 2 * array)) {
    a.ring.stages = 0;
    mode = a.wide ? kVectors : kElements;
  }
  const size_t smem = size_t(a.ring.stages) * a.ring.bytes + (r.nv == 2 ? 2 : 3) * array;
  if (r.nv > 2)
    return launch_norm<const NormGradArgs>(mode == kVectors ? norm_backward_kernel<F, H, 4, kVectors>
                                                            : norm_backward_kernel<F, H, 4, kElements>,
                                           a, r.threads, smem, stream);
  return launch_norm<const NormGradArgs>(mode == kRing      ? norm_backward_kernel<F, H, 2, kRing>
                                         : mode == kVectors ? norm_backward_kernel<F, H, 2, kVectors>
                                                            : norm_backward_kernel<F, H, 2, kElements>,
                                         a, r.threads, smem, stream);
}

}  // namespace
}  // namespace fadam_ops
