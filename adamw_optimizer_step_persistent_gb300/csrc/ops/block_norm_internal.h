// What the host side of the block norms (block_norm.cu) and their kernels, one
// translation unit for each block dtype, share.
#pragma once

#include "ops_internal.h"

namespace fadam_ops {

constexpr int kMaxWarps = 16;  // of a CTA: at 128 registers a thread, an SM's worth
constexpr int kMaxNormStages = 8;
// Shared memory of an SM that its CTAs' rings and parameters share; no CTA takes more.
constexpr size_t kNormSharedBytes = 216 * 1024;

// The tensors that a row's stage in shared memory holds, one after the other.
struct RingSource {
  const void* base;
  int64_t stride;  // bytes from one row to the next
  int bytes;       // of one row
  int offset;      // in the stage
};
struct RingArgs {
  RingSource source[4];
  int sources, bytes, stages;
  int* status;
};

// Rows are taken in runs that share one row of the gate: run u holds slice
// u % slices of the rows of gate u / slices.
struct NormRuns {
  int gates, rows_per_gate;
  int slices, ctas, runs;
};

struct NormArgs {
  const void *f, *h, *post, *pre, *gate;
  void *h_out, *x_out;
  float *r1, *r2;
  int8_t *f_codes, *h_codes;
  float *f_scales, *h_scales;
  int64_t f_stride, h_stride;
  NormRuns runs;
  RingArgs ring;
  int width, threads;
  float alpha, eps;
  bool params_f32, wide;
};

struct NormGradArgs {
  const void *gh, *gx, *f, *h;
  const int8_t *f_codes, *h_codes;
  const float *f_scales, *h_scales;
  const float *r1, *r2;
  const void *post, *pre, *gate;
  void *df, *dh;
  float* gate_parts;   // [runs, width], or NULL
  void* gate_out;      // [gates, width] in place of gate_parts, when there is one slice
  float* post_parts;   // [CTAs, width], or NULL
  float* pre_parts;    // [CTAs, width]
  int64_t gh_stride, gx_stride, f_stride, h_stride;
  NormRuns runs;
  RingArgs ring;
  int width, threads;
  float alpha;
  bool params_f32, wide;
};

// Threads and vectors of eight columns per thread for a row: whole warps, two
// vectors a thread (four beyond 512 threads).
struct RowShape {
  int threads, nv;
};
inline RowShape row_shape(int64_t width) {
  const int64_t vectors = ceil_div(width, 8);
  const int nv = vectors <= 2 * kMaxWarps * 32 ? 2 : 4;
  return {int(round_up(ceil_div(vectors, nv), 32)), nv};
}

// CTAs that an SM's registers hold at once.
inline int norm_ctas_per_sm(int threads) {
  const int fit = kMaxWarps * 32 / threads;
  return fit < 8 ? fit : 8;
}

// Every CTA that fits gets a run, and a gate's rows are cut into as many as
// that takes.  (Giving each at least four rows, to read the parameters and
// write the sums less often, took 13.3 us in place of 9.0 for 512 x 512.)
inline NormRuns norm_runs(int64_t rows, int64_t gates, int64_t width, int sm_count) {
  const int64_t most = int64_t(sm_count) * norm_ctas_per_sm(row_shape(width).threads);
  int64_t slices = most / gates;
  if (slices > rows / gates) slices = rows / gates;
  if (slices < 1) slices = 1;
  const int64_t runs = gates * slices;
  return {int(gates), int(rows / gates), int(slices), int(runs < most ? runs : most), int(runs)};
}

// The kernels' launches, by block dtype and whether the residual stream is fp32.
fadam_status norm_forward_bf16(const NormArgs& a, bool residual_f32, cudaStream_t stream);
fadam_status norm_forward_f16(const NormArgs& a, bool residual_f32, cudaStream_t stream);
fadam_status norm_forward_f32(const NormArgs& a, cudaStream_t stream);
fadam_status norm_backward_bf16(const NormGradArgs& a, bool residual_f32, cudaStream_t stream);
fadam_status norm_backward_f16(const NormGradArgs& a, bool residual_f32, cudaStream_t stream);
fadam_status norm_backward_f32(const NormGradArgs& a, cudaStream_t stream);

}  // namespace fadam_ops
