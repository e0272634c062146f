// What the host side of the block norms (block_norm.cu) and their kernels, one
// translation unit for each block dtype, share.
#pragma once

#include "ops_internal.h"

namespace fadam_ops {

constexpr int kMaxWarps = 16;  // of a CTA

struct NormArgs {
  const void *f, *h, *post, *pre, *gate;
  void *h_out, *x_out;
  float *r1, *r2;
  int8_t *f_codes, *h_codes;
  float *f_scales, *h_scales;
  int64_t rows, f_stride, h_stride, rows_per_gate;
  int width;
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
  float* gate_parts;   // [gates, slices, width], or NULL
  void* gate_out;      // [gates, width] in place of gate_parts, when there is one slice
  float* post_parts;   // [CTAs, width], or NULL
  float* pre_parts;    // [CTAs, width]
  int64_t rows, gates, rows_per_gate;
  int64_t gh_stride, gx_stride, f_stride, h_stride;
  int width, slices, ctas;
  float alpha;
  bool params_f32, wide;
};

// Threads and vectors per thread for a row: whole warps, at most 512 threads,
// as few vectors as that allows (1, 2 or 4).
struct RowShape {
  int threads, nv;
};
inline RowShape row_shape(int64_t width) {
  const int64_t vectors = ceil_div(width, 8);
  const int nv = vectors <= 512 ? 1 : vectors <= 1024 ? 2 : 4;
  return {int(round_up(ceil_div(vectors, nv), 32)), nv};
}

// The kernels' launches, by block dtype and whether the residual stream is fp32.
fadam_status norm_forward_bf16(const NormArgs& a, bool residual_f32, cudaStream_t stream);
fadam_status norm_forward_f16(const NormArgs& a, bool residual_f32, cudaStream_t stream);
fadam_status norm_forward_f32(const NormArgs& a, cudaStream_t stream);
fadam_status norm_backward_bf16(const NormGradArgs& a, bool residual_f32, cudaStream_t stream);
fadam_status norm_backward_f16(const NormGradArgs& a, bool residual_f32, cudaStream_t stream);
fadam_status norm_backward_f32(const NormGradArgs& a, cudaStream_t stream);

}  // namespace fadam_ops
