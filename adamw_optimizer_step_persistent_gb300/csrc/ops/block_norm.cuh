// The norms around a block: post-norm, gate, residual scale, add, pre-norm,
// forward and backward (formulas at fadam_block_norm and below).  Bound by
// memory: both directions read and write every row once.
//
// Forward: one CTA per row, the row in registers.  Backward: CTAs stay and
// take runs of rows, because the parameters' gradients are sums over rows: a
// thread owns its columns and keeps their sums in registers (in shared memory
// for the widest rows); the CTAs' sums go to the workspace and a second kernel
// adds them in a fixed order.
//
// Backward, with hh = h_out r2, fh = f r1 and, for a row,
//   g = grad_x_out pre_weight
//   e = grad_h_out + r2 (g - hh mean(g hh))                (= grad_h)
//   t = alpha gate post_weight e
//   grad_f = r1 (t - fh mean(t fh))                        (or t, no post-norm)
// the second mean would wait for the first; instead one reduction gives
//   S1 = sum g hh,  S2 = sum a fh (grad_h_out + r2 g),  S3 = sum a fh hh r2
// with a = alpha gate post_weight, and sum t fh = S2 - S3 S1 / width.
// The parameters' gradients need two sums per column,
//   Q = sum e fh (over rows of one gate),  P = sum grad_x_out hh:
// grad_gate = alpha post_weight Q, grad_post_weight = sum over gates of
// alpha gate Q, grad_pre_weight = P.
#pragma once

#include "block_norm_internal.h"
#include "rows.cuh"

namespace fadam_ops {
namespace {

// Sums N values over the block; every thread gets them.  `shared` holds
// N * kMaxWarps floats and is free again after the block's next barrier.
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float* shared) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 16; i; i /= 2) v[n] += __shfl_xor_sync(~0u, v[n], i);
  const int warp = threadIdx.x / 32, warps = blockDim.x / 32;
  if (threadIdx.x % 32 == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) shared[n * kMaxWarps + warp] = v[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = 0.0f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += shared[n * kMaxWarps + w];
}

template <class F, class H, int NV>
__global__ void __launch_bounds__(kMaxWarps * 32) norm_forward_kernel(const NormArgs a) {
  __shared__ float shared[2][kMaxWarps];
  const int64_t row = blockIdx.x;
  const int width = a.width;
  float f[NV][8], h[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * blockDim.x + threadIdx.x) * 8;
    load8<F>(static_cast<const F*>(a.f) + row * a.f_stride, col, width, a.wide, f[j]);
    load8<H>(static_cast<const H*>(a.h) + row * a.h_stride, col, width, a.wide, h[j]);
  }
  if (a.f_codes) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      keep8(f[j], a.f_codes + row * width, a.f_scales + row * ((width + kGroup - 1) / kGroup),
            (j * blockDim.x + threadIdx.x) * 8, width, a.wide);
  }
  if (a.post) {
    float sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] += f[j][i] * f[j][i];
    block_sums(sum, shared[0]);
    const float r1 = rsqrtf(sum[0] / float(width) + a.eps);
    if (threadIdx.x == 0) a.r1[row] = r1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[8];
      load_param8<F>(a.post, 0, a.params_f32, (j * blockDim.x + threadIdx.x) * 8, width, a.wide, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j][i] *= r1 * w[i];
    }
  }
  float sum[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (a.gate) {
      float w[8];
      load_param8<F>(a.gate, row / a.rows_per_gate * width, a.params_f32,
                     (j * blockDim.x + threadIdx.x) * 8, width, a.wide, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j][i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[j][i] += a.alpha * f[j][i];
      sum[0] += h[j][i] * h[j][i];
    }
  }
  block_sums(sum, shared[1]);
  const float r2 = rsqrtf(sum[0] / float(width) + a.eps);
  if (threadIdx.x == 0) a.r2[row] = r2;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * blockDim.x + threadIdx.x) * 8;
    float w[8], x[8];
    load_param8<F>(a.pre, 0, a.params_f32, col, width, a.wide, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = h[j][i] * r2 * w[i];
    store_row8<H>(static_cast<H*>(a.h_out) + row * width, col, width, a.wide, h[j]);
    store_row8<F>(static_cast<F*>(a.x_out) + row * width, col, width, a.wide, x);
    if (a.h_codes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = to_float(from_float<H>(h[j][i]));
      keep8(h[j], a.h_codes + row * width, a.h_scales + row * ((width + kGroup - 1) / kGroup), col,
            width, a.wide);
    }
  }
}

// SHARED: the column sums live in shared memory ([3][threads * NV * 8] floats).
template <class F, class H, int NV, bool SHARED>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) norm_backward_kernel(const NormGradArgs a) {
  __shared__ float shared[2][3 * kMaxWarps];
  extern __shared__ float sums[];
  const int width = a.width, groups = (width + kGroup - 1) / kGroup;
  const int tid = threadIdx.x;
  const float inv_width = 1.0f / float(width);
  constexpr int N = SHARED ? 1 : NV;
  float q_reg[N][8], p_reg[N][8], w_reg[N][8];
  // column sums: Q of the current gate, P, and grad_post_weight's
  auto q = [&](int j, int i) -> float& {
    if constexpr (SHARED) return sums[(j * 8 + i) * blockDim.x + tid]; else return q_reg[j][i];
  };
  auto p = [&](int j, int i) -> float& {
    if constexpr (SHARED) return sums[((NV + j) * 8 + i) * blockDim.x + tid]; else return p_reg[j][i];
  };
  auto w = [&](int j, int i) -> float& {
    if constexpr (SHARED) return sums[((2 * NV + j) * 8 + i) * blockDim.x + tid]; else return w_reg[j][i];
  };
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) p(j, i) = w(j, i) = 0.0f;

  int turn = 0;
  for (int64_t unit = blockIdx.x; unit < a.gates * a.slices; unit += gridDim.x) {
    const int64_t gate = unit / a.slices, slice = unit - gate * a.slices;
    const int64_t begin = gate * a.rows_per_gate + a.rows_per_gate * slice / a.slices;
    const int64_t end = gate * a.rows_per_gate + a.rows_per_gate * (slice + 1) / a.slices;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) q(j, i) = 0.0f;

    for (int64_t row = begin; row < end; ++row, turn ^= 1) {
      const float r1 = a.r1 ? a.r1[row] : 1.0f, r2 = a.r2[row];
      // e's two parts and what they multiply, kept from the sums to the outputs
      float fh[NV][8], hh[NV][8], eg[NV][8];
      float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * blockDim.x + tid) * 8;
        float gx[8], pre[8], scale[8];
        if (a.gh) {
          load8<H>(static_cast<const H*>(a.gh) + row * a.gh_stride, col, width, a.wide, eg[j]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) eg[j][i] = 0.0f;
        }
        load8<F>(static_cast<const F*>(a.gx) + row * a.gx_stride, col, width, a.wide, gx);
        if (a.f)
          load8<F>(static_cast<const F*>(a.f) + row * a.f_stride, col, width, a.wide, fh[j]);
        else
          kept8(a.f_codes + row * width, a.f_scales + row * groups, col, width, a.wide, fh[j]);
        if (a.h)
          load8<H>(static_cast<const H*>(a.h) + row * a.h_stride, col, width, a.wide, hh[j]);
        else
          kept8(a.h_codes + row * width, a.h_scales + row * groups, col, width, a.wide, hh[j]);
        load_param8<F>(a.pre, 0, a.params_f32, col, width, a.wide, pre);
#pragma unroll
        for (int i = 0; i < 8; ++i) scale[i] = a.alpha;
        if (a.post) {
          float v[8];
          load_param8<F>(a.post, 0, a.params_f32, col, width, a.wide, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) scale[i] *= v[i];
        }
        if (a.gate) {
          float v[8];
          load_param8<F>(a.gate, gate * width, a.params_f32, col, width, a.wide, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) scale[i] *= v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          fh[j][i] *= r1;
          hh[j][i] *= r2;
          p(j, i) += gx[i] * hh[j][i];
          const float g = gx[i] * pre[i];
          s[0] += g * hh[j][i];
          eg[j][i] += r2 * g;
          s[1] += scale[i] * fh[j][i] * eg[j][i];
          s[2] += scale[i] * fh[j][i] * (hh[j][i] * r2);
        }
      }
      block_sums(s, shared[turn]);
      const float c1 = r2 * (s[0] * inv_width);
      const float c2 = a.post ? (s[1] - s[2] * (s[0] * inv_width)) * inv_width : 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int col = (j * blockDim.x + tid) * 8;
        float scale[8], df[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) scale[i] = a.alpha;
        if (a.post) {
          float v[8];
          load_param8<F>(a.post, 0, a.params_f32, col, width, a.wide, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) scale[i] *= v[i];
        }
        if (a.gate) {
          float v[8];
          load_param8<F>(a.gate, gate * width, a.params_f32, col, width, a.wide, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) scale[i] *= v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = eg[j][i] - hh[j][i] * c1;
          q(j, i) += e * fh[j][i];
          df[i] = r1 * (scale[i] * e - fh[j][i] * c2);
          eg[j][i] = e;
        }
        store_row8<H>(static_cast<H*>(a.dh) + row * width, col, width, a.wide, eg[j]);
        store_row8<F>(static_cast<F*>(a.df) + row * width, col, width, a.wide, df);
      }
    }

    // this run's share of the gate's and the post-norm's gradients
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * blockDim.x + tid) * 8;
      float post[8], g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) post[i] = g[i] = 1.0f;
      if (a.post) load_param8<F>(a.post, 0, a.params_f32, col, width, a.wide, post);
      if (a.gate) load_param8<F>(a.gate, gate * width, a.params_f32, col, width, a.wide, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float sum = a.alpha * q(j, i);
        w(j, i) += g[i] * sum;
        if (a.gate_parts && col + i < width) a.gate_parts[unit * width + col + i] = post[i] * sum;
        q(j, i) = post[i] * sum;
      }
      if (a.gate_out) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = q(j, i);
        if (a.params_f32)
          store_row8<float>(static_cast<float*>(a.gate_out) + gate * width, col, width, a.wide, v);
        else
          store_row8<F>(static_cast<F*>(a.gate_out) + gate * width, col, width, a.wide, v);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * blockDim.x + tid) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < width) {
        a.pre_parts[int64_t(blockIdx.x) * width + col + i] = p(j, i);
        if (a.post_parts) a.post_parts[int64_t(blockIdx.x) * width + col + i] = w(j, i);
      }
  }
}

template <class F, class H>
fadam_status norm_forward(const NormArgs& a, cudaStream_t stream) {
  const RowShape r = row_shape(a.width);
  auto* kernel = r.nv == 1 ? norm_forward_kernel<F, H, 1>
                 : r.nv == 2 ? norm_forward_kernel<F, H, 2> : norm_forward_kernel<F, H, 4>;
  kernel<<<unsigned(a.rows), r.threads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FADAM_OK : cuda_fail(e, "block norm forward launch");
}

template <class F, class H>
fadam_status norm_backward(const NormGradArgs& a, cudaStream_t stream) {
  const RowShape r = row_shape(a.width);
  auto* kernel = r.nv == 1 ? norm_backward_kernel<F, H, 1, false>
                 : r.nv == 2 ? norm_backward_kernel<F, H, 2, false>
                             : norm_backward_kernel<F, H, 4, true>;
  const size_t smem = r.nv == 4 ? size_t(3) * 4 * 8 * r.threads * sizeof(float) : 0;
  if (smem) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  }
  kernel<<<unsigned(a.ctas), r.threads, smem, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FADAM_OK : cuda_fail(e, "block norm backward launch");
}

}  // namespace
}  // namespace fadam_ops
