// Host side of the block norms, and the kernel that adds up the CTAs' sums of
// the parameters' gradients.
#include "block_norm_internal.h"
#include "ops_device.cuh"

namespace fadam_ops {
namespace {

// out[o, c] = sum over `parts` of in[o, part, c]: 32 columns to a CTA, each
// warp every 32nd part, then the warps' sums, in a fixed order.
struct SumArgs {
  const float* in;
  void* out;
  int64_t outer;
  int parts, width, dtype;
};
struct SumJobs {
  SumArgs job[3];
};
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) column_sums_kernel(const __grid_constant__ SumJobs jobs, int blocks) {
  __shared__ float shared[kSumWarps][33];
  chain_wait();
  chain_next();
  const SumArgs& a = jobs.job[blockIdx.x / unsigned(blocks)];
  if (!a.out) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t blocks_per_row = (a.width + 31) / 32;
  for (int64_t b = blockIdx.x % unsigned(blocks); b < a.outer * blocks_per_row; b += blocks) {
    const int64_t o = b / blocks_per_row;
    const int col = int(b - o * blocks_per_row) * 32 + lane;
    float sum = 0.0f;
    if (col < a.width) {
      const float* in = a.in + o * a.parts * a.width + col;
#pragma unroll 8
      for (int p = warp; p < a.parts; p += kSumWarps) sum += in[int64_t(p) * a.width];
    }
    __syncthreads();
    shared[warp][lane] = sum;
    __syncthreads();
    // each warp adds up one column
    sum = shared[lane][warp];
#pragma unroll
    for (int i = 16; i; i /= 2) sum += __shfl_xor_sync(~0u, sum, i);
    const int to = int(b - o * blocks_per_row) * 32 + warp;
    if (lane == 0 && to < a.width) {
      const int64_t at = o * a.width + to;
      if (a.dtype == FADAM_DT_F32)
        static_cast<float*>(a.out)[at] = sum;
      else if (a.dtype == FADAM_DT_BF16)
        static_cast<__nv_bfloat16*>(a.out)[at] = from_float<__nv_bfloat16>(sum);
      else
        static_cast<__half*>(a.out)[at] = from_float<__half>(sum);
    }
  }
}

struct Plan {
  NormRuns runs;
  float *gate_parts, *post_parts, *pre_parts;
  size_t bytes;
};

Plan plan_backward(const fadam_block_norm_grad& d, char* base, int sm_count) {
  Plan p{};
  Carver c{base};
  p.runs = norm_runs(d.rows, d.gate_rows, d.width, sm_count);
  const size_t part = sizeof(float) * p.runs.ctas * d.width;
  p.pre_parts = static_cast<float*>(c.take(part));
  if (d.post_weight) p.post_parts = static_cast<float*>(c.take(part));
  if (d.gate && p.runs.slices > 1)
    p.gate_parts = static_cast<float*>(c.take(sizeof(float) * int64_t(p.runs.runs) * d.width));
  p.bytes = c.used;
  return p;
}

fadam_status check_sizes(int64_t rows, int64_t width, int64_t gate_rows, bool gate, int32_t block,
                         int32_t residual, int32_t param, float alpha) {
  if (elem_size(block) == 0) return fail(FADAM_EDTYPE, "block dtype %d is not fp32, bf16 or fp16", block);
  if (residual != block && residual != FADAM_DT_F32)
    return fail(FADAM_EDTYPE, "residual dtype %d is neither fp32 nor the block's %d", residual, block);
  if (param != block && param != FADAM_DT_F32)
    return fail(FADAM_EDTYPE, "param dtype %d is neither fp32 nor the block's %d", param, block);
  if (rows < 0 || width < 1) return fail(FADAM_EINVAL, "%lld rows of width %lld", (long long)rows,
                                         (long long)width);
  if (width > FADAM_BLOCK_NORM_MAX_WIDTH)
    return fail(FADAM_ELIMIT, "width %lld beyond %d", (long long)width, FADAM_BLOCK_NORM_MAX_WIDTH);
  if (rows > int64_t(1) << 30) return fail(FADAM_ELIMIT, "rows beyond 2^30");
  if (gate_rows < 1 || rows % gate_rows || (!gate && gate_rows != 1))
    return fail(FADAM_EINVAL, "%lld gate rows for %lld rows", (long long)gate_rows, (long long)rows);
  if (alpha - alpha != 0.0f) return fail(FADAM_EINVAL, "residual_scale is not finite");
  return FADAM_OK;
}

fadam_status check(const fadam_block_norm* d) {
  if (!d) return fail(FADAM_EINVAL, "the descriptor is NULL");
  const fadam_status st = check_sizes(d->rows, d->width, d->gate_rows, d->gate, d->block_dtype,
                                      d->residual_dtype, d->param_dtype, d->residual_scale);
  if (st) return st;
  if (!(d->eps >= 0.0f) || d->eps - d->eps != 0.0f)
    return fail(FADAM_EINVAL, "eps %g is not finite and >= 0", d->eps);
  if (d->f_stride < d->width || d->h_stride < d->width)
    return fail(FADAM_EINVAL, "a row stride is below the width %lld", (long long)d->width);
  if (!d->pre_weight || (d->rows > 0 && (!d->f || !d->h || !d->h_out || !d->x_out || !d->rstd_pre)))
    return fail(FADAM_EINVAL, "f, h, pre_weight, h_out, x_out and rstd_pre must be non-NULL");
  if (d->rows > 0 && !d->post_weight != !d->rstd_post)
    return fail(FADAM_EINVAL, "post_weight and rstd_post go together");
  if (d->rows > 0 && (!d->f_kept.codes != !d->f_kept.scales || !d->h_kept.codes != !d->h_kept.scales))
    return fail(FADAM_EINVAL, "a checkpoint needs both codes and scales");
  const int b = elem_size(d->block_dtype), h = elem_size(d->residual_dtype),
            w = elem_size(d->param_dtype);
  if (misaligned(d->f, b) || misaligned(d->x_out, b) || misaligned(d->h, h) ||
      misaligned(d->h_out, h) || misaligned(d->post_weight, w) || misaligned(d->pre_weight, w) ||
      misaligned(d->gate, w) || misaligned(d->rstd_post, 4) || misaligned(d->rstd_pre, 4) ||
      misaligned(d->f_kept.scales, 4) || misaligned(d->h_kept.scales, 4))
    return fail(FADAM_EALIGN, "a pointer is not aligned to its element size");
  return FADAM_OK;
}

fadam_status check(const fadam_block_norm_grad* d) {
  if (!d) return fail(FADAM_EINVAL, "the descriptor is NULL");
  const fadam_status st = check_sizes(d->rows, d->width, d->gate_rows, d->gate, d->block_dtype,
                                      d->residual_dtype, d->param_dtype, d->residual_scale);
  if (st) return st;
  if ((d->grad_h_out && d->grad_h_out_stride < d->width) || d->grad_x_out_stride < d->width ||
      (d->f && d->f_stride < d->width) || (d->h_out && d->h_out_stride < d->width))
    return fail(FADAM_EINVAL, "a row stride is below the width %lld", (long long)d->width);
  if (!d->pre_weight || !d->grad_pre_weight || !d->post_weight != !d->grad_post_weight ||
      !d->gate != !d->grad_gate)
    return fail(FADAM_EINVAL, "every parameter, and only those, needs a gradient");
  if (d->rows > 0) {
    if (!d->grad_x_out || !d->rstd_pre || !d->grad_f || !d->grad_h)
      return fail(FADAM_EINVAL, "grad_x_out, rstd_pre, grad_f and grad_h must be non-NULL");
    if (!d->post_weight != !d->rstd_post)
      return fail(FADAM_EINVAL, "post_weight and rstd_post go together");
    if ((!d->f && (!d->f_kept.codes || !d->f_kept.scales)) ||
        (!d->h_out && (!d->h_kept.codes || !d->h_kept.scales)))
      return fail(FADAM_EINVAL, "f and h_out must be given, or their checkpoints");
  }
  const int b = elem_size(d->block_dtype), h = elem_size(d->residual_dtype),
            w = elem_size(d->param_dtype);
  if (misaligned(d->f, b) || misaligned(d->grad_x_out, b) || misaligned(d->grad_f, b) ||
      misaligned(d->h_out, h) || misaligned(d->grad_h_out, h) || misaligned(d->grad_h, h) ||
      misaligned(d->post_weight, w) || misaligned(d->pre_weight, w) || misaligned(d->gate, w) ||
      misaligned(d->grad_post_weight, w) || misaligned(d->grad_pre_weight, w) ||
      misaligned(d->grad_gate, w) || misaligned(d->rstd_post, 4) || misaligned(d->rstd_pre, 4) ||
      misaligned(d->f_kept.scales, 4) || misaligned(d->h_kept.scales, 4))
    return fail(FADAM_EALIGN, "a pointer is not aligned to its element size");
  return FADAM_OK;
}

// Whether a matrix's rows all start on 16 bytes.
bool wide_rows(const void* p, int64_t stride, int size) {
  return !misaligned(p, 16) && stride * size % 16 == 0;
}

}  // namespace
}  // namespace fadam_ops

using namespace fadam_ops;

extern "C" fadam_status fadam_block_norm_forward(const fadam_block_norm* desc, fadam_stream stream_) {
  clear_error();
  fadam_status st = check(desc);
  if (st || desc->rows == 0) return st;
  const fadam_block_norm& d = *desc;
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int b = elem_size(d.block_dtype), h = elem_size(d.residual_dtype);
  NormArgs a{};
  a.f = d.f;
  a.h = d.h;
  a.post = d.post_weight;
  a.pre = d.pre_weight;
  a.gate = d.gate;
  a.h_out = d.h_out;
  a.x_out = d.x_out;
  a.r1 = d.rstd_post;
  a.r2 = d.rstd_pre;
  a.f_codes = d.f_kept.codes;
  a.f_scales = d.f_kept.scales;
  a.h_codes = d.h_kept.codes;
  a.h_scales = d.h_kept.scales;
  a.f_stride = d.f_stride;
  a.h_stride = d.h_stride;
  a.runs = norm_runs(d.rows, d.gate_rows, d.width, dev.sm_count);
  a.ring.status = dev.status;
  a.width = int(d.width);
  a.alpha = d.residual_scale;
  a.eps = d.eps;
  a.params_f32 = d.param_dtype == FADAM_DT_F32;
  a.wide = d.width % 8 == 0 && wide_rows(d.f, d.f_stride, b) && wide_rows(d.h, d.h_stride, h) &&
           !misaligned(d.h_out, 16) && !misaligned(d.x_out, 16) && !misaligned(d.post_weight, 16) &&
           !misaligned(d.pre_weight, 16) && !misaligned(d.gate, 16) &&
           !misaligned(d.f_kept.codes, 8) && !misaligned(d.h_kept.codes, 8);
  const bool f32 = d.residual_dtype == FADAM_DT_F32;
  if (d.block_dtype == FADAM_DT_BF16) return norm_forward_bf16(a, f32, stream);
  if (d.block_dtype == FADAM_DT_F16) return norm_forward_f16(a, f32, stream);
  return norm_forward_f32(a, stream);
}

extern "C" fadam_status fadam_block_norm_backward_workspace(const fadam_block_norm_grad* desc,
                                                            size_t* bytes) {
  clear_error();
  if (!bytes) return fail(FADAM_EINVAL, "bytes is NULL");
  fadam_status st = check(desc);
  if (st) return st;
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  *bytes = desc->rows == 0 ? 0 : plan_backward(*desc, nullptr, dev.sm_count).bytes;
  return FADAM_OK;
}

extern "C" fadam_status fadam_block_norm_backward(const fadam_block_norm_grad* desc, void* workspace,
                                                  size_t bytes, fadam_stream stream_) {
  clear_error();
  fadam_status st = check(desc);
  if (st) return st;
  const fadam_block_norm_grad& d = *desc;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int b = elem_size(d.block_dtype), h = elem_size(d.residual_dtype),
            w = elem_size(d.param_dtype);
  if (d.rows == 0) {
    cudaError_t e = cudaMemsetAsync(d.grad_pre_weight, 0, d.width * w, stream);
    if (e == cudaSuccess && d.grad_post_weight)
      e = cudaMemsetAsync(d.grad_post_weight, 0, d.width * w, stream);
    if (e == cudaSuccess && d.grad_gate)
      e = cudaMemsetAsync(d.grad_gate, 0, d.gate_rows * d.width * w, stream);
    return e == cudaSuccess ? FADAM_OK : cuda_fail(e, "cudaMemsetAsync");
  }
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  const Plan p = plan_backward(d, static_cast<char*>(workspace), dev.sm_count);
  if (!workspace || bytes < p.bytes)
    return fail(FADAM_EINVAL, "the workspace has %zu bytes, %zu are needed",
                workspace ? bytes : size_t(0), p.bytes);
  if (misaligned(workspace, 256)) return fail(FADAM_EALIGN, "the workspace is not 256-byte aligned");
  NormGradArgs a{};
  a.gh = d.grad_h_out;
  a.gx = d.grad_x_out;
  a.f = d.f;
  a.h = d.h_out;
  a.f_codes = d.f_kept.codes;
  a.f_scales = d.f_kept.scales;
  a.h_codes = d.h_kept.codes;
  a.h_scales = d.h_kept.scales;
  a.r1 = d.rstd_post;
  a.r2 = d.rstd_pre;
  a.post = d.post_weight;
  a.pre = d.pre_weight;
  a.gate = d.gate;
  a.df = d.grad_f;
  a.dh = d.grad_h;
  a.gate_parts = p.gate_parts;
  a.gate_out = p.gate_parts ? nullptr : d.grad_gate;
  a.post_parts = p.post_parts;
  a.pre_parts = p.pre_parts;
  a.gh_stride = d.grad_h_out_stride;
  a.gx_stride = d.grad_x_out_stride;
  a.f_stride = d.f_stride;
  a.h_stride = d.h_out_stride;
  a.width = int(d.width);
  a.runs = p.runs;
  a.ring.status = dev.status;
  a.alpha = d.residual_scale;
  a.params_f32 = d.param_dtype == FADAM_DT_F32;
  a.wide = d.width % 8 == 0 && (!d.grad_h_out || wide_rows(d.grad_h_out, d.grad_h_out_stride, h)) &&
           wide_rows(d.grad_x_out, d.grad_x_out_stride, b) &&
           (!d.f || wide_rows(d.f, d.f_stride, b)) &&
           (!d.h_out || wide_rows(d.h_out, d.h_out_stride, h)) && !misaligned(d.f_kept.codes, 8) &&
           !misaligned(d.h_kept.codes, 8) && !misaligned(d.post_weight, 16) &&
           !misaligned(d.pre_weight, 16) && !misaligned(d.gate, 16) && !misaligned(d.grad_f, 16) &&
           !misaligned(d.grad_h, 16) && !misaligned(d.grad_gate, 16);
  const bool f32 = d.residual_dtype == FADAM_DT_F32;
  st = d.block_dtype == FADAM_DT_BF16  ? norm_backward_bf16(a, f32, stream)
       : d.block_dtype == FADAM_DT_F16 ? norm_backward_f16(a, f32, stream)
                                       : norm_backward_f32(a, stream);
  if (st) return st;
  SumJobs jobs{};
  const int width = int(d.width);
  jobs.job[0] = {p.pre_parts, d.grad_pre_weight, 1, p.runs.ctas, width, d.param_dtype};
  if (p.post_parts) jobs.job[1] = {p.post_parts, d.grad_post_weight, 1, p.runs.ctas, width, d.param_dtype};
  if (p.gate_parts)
    jobs.job[2] = {p.gate_parts, d.grad_gate, d.gate_rows, p.runs.slices, width, d.param_dtype};
  const int64_t blocks = (p.gate_parts ? d.gate_rows : 1) * ceil_div(d.width, 32);
  const int grid = int(blocks < 4096 ? blocks : 4096);
  return launch_chained("column sums launch", column_sums_kernel, 3 * grid, kSumWarps * 32, 0, stream, jobs,
                        grid);
}
