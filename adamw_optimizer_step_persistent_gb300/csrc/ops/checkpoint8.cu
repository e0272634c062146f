// Activations kept in 8 bits: groups of 128 of a row with one fp32 scale, and
// the weight gradient of a linear layer from its input's checkpoint.
//
// Packing and restoring are one pass over memory: a thread takes vectors of
// eight elements (16 bytes in, 8 bytes out for 16-bit activations) of
// consecutive rows, half a warp a group, whose largest magnitude it finds
// with four shuffles.
#include "gemm_store.cuh"
#include "rows.cuh"

namespace fadam_ops {
namespace {

constexpr int kThreads = 256;

// A CTA takes `threads` vectors of eight columns (a chunk of a row, or all of
// it) of R rows, one vector of each row per thread: R independent loads.
struct ChunkGrid {
  int threads, chunks, unroll;
  unsigned ctas;
};
// Four rows to a thread where that still leaves every SM eight CTAs of work,
// else one: 8192 x 11008 in bf16 are packed in 43.4 us (6.3 TB/s) and restored
// in 40.6 (6.7 TB/s) with four rows, 63.8 and 51.7 us with one.
ChunkGrid chunk_grid(int64_t rows, int64_t width) {
  ChunkGrid g;
  const int64_t vectors = ceil_div(width, 8);
  g.threads = int(vectors < kThreads ? round_up(vectors, 32) : kThreads);
  g.chunks = int(ceil_div(vectors, g.threads));
  g.unroll = ceil_div(rows, 4) * g.chunks >= 152 * 8 ? 4 : 1;
  g.ctas = unsigned(ceil_div(rows, g.unroll) * g.chunks);
  return g;
}

// Rows of whole aligned vectors.
template <class E, int R>
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const E* x, int64_t rows, int width, int64_t x_stride, int8_t* codes, float* scales,
                int chunks) {
  chain_wait();
  chain_next();
  const unsigned block = blockIdx.x / unsigned(chunks);
  const int col = int((blockIdx.x - block * chunks) * blockDim.x + threadIdx.x) * 8;
  const int64_t row0 = int64_t(block) * R;
  const int groups = (width + kGroup - 1) / kGroup;
  const int left = int(min(rows - row0, int64_t(R)));
  x += row0 * x_stride + col;
  codes += row0 * width + col;
  scales += row0 * groups + col / kGroup;
  const bool group_here = col / kGroup * kGroup < width;
  Raw<E> v[R];
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = r < left && col < width ? load_raw(x + r * x_stride) : zero_raw<E>();
  float top[R];
#pragma unroll
  for (int r = 0; r < R; ++r) top[r] = from_bits<E>(group_top(v[r]));
  const Scaling shared = share_scaling<R>(top);
#pragma unroll
  for (int r = 0; r < R; ++r)
    keep_vector(v[r], shared, r, codes + r * int64_t(width), scales + r * groups, r < left && col < width,
                r < left && group_here);
}

// What a checkpoint is divided by, and its product multiplied by, so that fp16
// can hold the largest element: a power of two, 1 where it can without.
struct Range {
  unsigned peak;  // bits of the largest finite scale
  float undo;     // written by restore_*_kernel
};
__global__ void __launch_bounds__(kThreads) peak_kernel(const float* scales, int64_t n, Range* range) {
  chain_wait();
  chain_next();
  unsigned top = 0;
  const int64_t step = int64_t(gridDim.x) * kThreads;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += step) {
    const float s = fabsf(scales[i]);
    if (s < INFINITY) top = max(top, __float_as_uint(s));
  }
  top = __reduce_max_sync(~0u, top);
  if (threadIdx.x % 32 == 0) atomicMax(&range->peak, top);
}
// 2^-e with 127 peak 2^-e below 2^15, at most 1.  (The first thread leaves 2^e.)
__device__ __forceinline__ float fit_range(Range* range) {
  const float peak = __uint_as_float(range->peak);
  const int e = peak < 256.0f ? 0 : ilogbf(peak) - 7;
  if (blockIdx.x == 0 && threadIdx.x == 0) range->undo = ldexpf(1.0f, e);
  return ldexpf(1.0f, -e);
}

template <class E, int R, bool kFit>
__global__ void __launch_bounds__(kThreads)
    restore_kernel(const int8_t* codes, const float* scales, int64_t rows, int width, E* x,
                   int64_t x_stride, int chunks, Range* range) {
  chain_wait();
  chain_next();
  const float fit = kFit ? fit_range(range) : 1.0f;
  const unsigned block = blockIdx.x / unsigned(chunks);
  const int col = int((blockIdx.x - block * chunks) * blockDim.x + threadIdx.x) * 8;
  if (col >= width) return;
  const int64_t row0 = int64_t(block) * R;
  const int groups = (width + kGroup - 1) / kGroup;
  const int left = int(min(rows - row0, int64_t(R)));
  x += row0 * x_stride + col;
  codes += row0 * width + col;
  scales += row0 * groups + col / kGroup;
  uint2 raw[R];
  float scale[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (r < left) {
      raw[r] = __ldg(reinterpret_cast<const uint2*>(codes + r * int64_t(width)));
      scale[r] = __ldg(scales + r * groups);
    }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (r < left) {
      Pair v[4];
      codes_pairs(raw[r], kFit ? scale[r] * fit : scale[r], v);
      store_raw(x + r * x_stride, narrow<E>(v));
    }
}

// Any rows: a warp to a group.
template <class E>
__global__ void __launch_bounds__(kThreads)
    pack_any_kernel(const E* x, int64_t rows, int width, int64_t x_stride, int8_t* codes, float* scales) {
  chain_wait();
  chain_next();
  const int groups = (width + kGroup - 1) / kGroup;
  const int64_t warps = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < rows * groups; i += warps) {
    const int64_t row = i / groups;
    keep_group(x + row * x_stride, int(i - row * groups) * kGroup, width, codes + row * width,
               scales + row * groups);
  }
}

template <class E, bool kFit>
__global__ void __launch_bounds__(kThreads)
    restore_any_kernel(const int8_t* codes, const float* scales, int64_t rows, int width, E* x,
                       int64_t x_stride, Range* range) {
  chain_wait();
  chain_next();
  const float fit = kFit ? fit_range(range) : 1.0f;
  const int groups = (width + kGroup - 1) / kGroup;
  const int64_t warps = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < rows * groups; i += warps) {
    const int64_t row = i / groups;
    const int group = int(i - row * groups);
    const float scale = kFit ? scales[i] * fit : scales[i];
#pragma unroll
    for (int k = 0; k < kGroup / 32; ++k) {
      const int col = group * kGroup + k * 32 + threadIdx.x % 32;
      if (col < width) x[row * x_stride + col] = from_float<E>(float(codes[row * width + col]) * scale);
    }
  }
}

unsigned any_grid(int64_t rows, int64_t width) {
  const int64_t ctas = ceil_div(rows * ceil_div(width, kGroup), kThreads / 32);
  return unsigned(ctas < 152 * 16 ? ctas : 152 * 16);
}

template <class E>
fadam_status pack(const void* x, int64_t rows, int64_t width, int64_t stride,
                  const fadam_checkpoint8& out, cudaStream_t stream) {
  const bool wide = width % 8 == 0 && !misaligned(x, 16) && stride * sizeof(E) % 16 == 0 &&
                    !misaligned(out.codes, 8);
  const char* what = "checkpoint8 pack launch";
  const E* from = static_cast<const E*>(x);
  if (!wide)
    return launch_chained(what, pack_any_kernel<E>, any_grid(rows, width), kThreads, 0, stream, from, rows,
                          int(width), stride, out.codes, out.scales);
  const ChunkGrid g = chunk_grid(rows, width);
  return launch_chained(what, g.unroll == 4 ? pack_kernel<E, 4> : pack_kernel<E, 1>, g.ctas, g.threads, 0,
                        stream, from, rows, int(width), stride, out.codes, out.scales, g.chunks);
}

template <class E, bool kFit = false>
fadam_status restore(const fadam_checkpoint8& in, int64_t rows, int64_t width, void* x,
                     int64_t stride, cudaStream_t stream, Range* range = nullptr) {
  const bool wide = width % 8 == 0 && !misaligned(x, 16) && stride * sizeof(E) % 16 == 0 &&
                    !misaligned(in.codes, 8);
  const char* what = "checkpoint8 restore launch";
  E* to = static_cast<E*>(x);
  const int8_t* codes = in.codes;
  const float* scales = in.scales;
  if (!wide)
    return launch_chained(what, restore_any_kernel<E, kFit>, any_grid(rows, width), kThreads, 0, stream,
                          codes, scales, rows, int(width), to, stride, range);
  const ChunkGrid g = chunk_grid(rows, width);
  return launch_chained(what, g.unroll == 4 ? restore_kernel<E, 4, kFit> : restore_kernel<E, 1, kFit>,
                        g.ctas, g.threads, 0, stream, codes, scales, rows, int(width), to, stride, g.chunks,
                        range);
}

fadam_status check_matrix(const void* x, int64_t rows, int64_t width, int64_t stride, int32_t dtype,
                          const fadam_checkpoint8* kept) {
  if (elem_size(dtype) == 0) return fail(FADAM_EDTYPE, "dtype %d is not fp32, bf16 or fp16", dtype);
  if (rows < 0 || width < 1) return fail(FADAM_EINVAL, "%lld rows of width %lld", (long long)rows,
                                         (long long)width);
  if (rows > int64_t(1) << 30 || width > int64_t(1) << 30)
    return fail(FADAM_ELIMIT, "rows or width beyond 2^30");
  if (stride < width) return fail(FADAM_EINVAL, "stride %lld is below the width %lld",
                                  (long long)stride, (long long)width);
  if (!kept) return fail(FADAM_EINVAL, "the checkpoint is NULL");
  if (rows > 0 && (!x || !kept->codes || !kept->scales))
    return fail(FADAM_EINVAL, "x, codes and scales must be non-NULL");
  if (misaligned(x, elem_size(dtype)) || misaligned(kept->scales, 4))
    return fail(FADAM_EALIGN, "a pointer is not aligned to its element size");
  return FADAM_OK;
}

// ---- the weight gradient -----------------------------------------------------------

struct Layout {
  GemmPlan plan;
  int64_t x_ld, dy_ld;
  void* x;        // the restored checkpoint
  void* dy_rows;  // an aligned copy of dy, where its own rows are not
  Range* range;   // where X may be beyond fp16's range
  float* parts;
  size_t bytes;
};

Layout layout(const fadam_wgrad& d, char* base, int sm_count) {
  Layout l{};
  Carver c{base};
  l.plan = plan_gemm(d.n, d.width, d.rows, true, true, sm_count / 2);
  l.x_ld = round_up(d.width, 8);
  l.dy_ld = d.dy_stride;
  l.x = c.take(2 * d.rows * l.x_ld);
  if (!bulk_readable(d.dy, d.dy_stride)) {
    l.dy_ld = round_up(d.n, 8);
    l.dy_rows = c.take(2 * d.rows * l.dy_ld);
  }
  if (d.dtype == FADAM_DT_F16 && (d.flags & FADAM_WGRAD_WIDE_X))
    l.range = static_cast<Range*>(c.take(sizeof(Range)));
  if (const size_t parts = split_bytes(d.n, l.plan)) l.parts = static_cast<float*>(c.take(parts));
  l.bytes = c.used;
  return l;
}

template <class E>
__global__ void __launch_bounds__(kThreads)
    align_kernel(const E* from, int64_t from_ld, E* to, int64_t to_ld, int64_t rows, int64_t width) {
  chain_wait();
  chain_next();
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (int64_t i = threadIdx.x; i < width; i += kThreads) to[row * to_ld + i] = from[row * from_ld + i];
}

template <class T, class Out>
fadam_status run(const fadam_wgrad& d, const Layout& l, const DeviceFacts& dev, cudaStream_t stream) {
  using E = typename T::type;
  fadam_status st;
  const void* dy = d.dy;
  if (l.dy_rows) {
    if ((st = launch_chained("row copy launch", align_kernel<E>, d.rows < 8192 ? d.rows : 8192, kThreads, 0,
                             stream, static_cast<const E*>(d.dy), d.dy_stride,
                             static_cast<E*>(l.dy_rows), l.dy_ld, d.rows, d.n)))
      return st;
    dy = l.dy_rows;
  }
  if constexpr (T::code == FADAM_DT_F16) {
    if (d.flags & FADAM_WGRAD_WIDE_X) {
      const cudaError_t e = cudaMemsetAsync(l.range, 0, sizeof(Range), stream);
      if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
      const int64_t scales = d.rows * ceil_div(d.width, kGroup), ctas = ceil_div(scales, 8 * kThreads);
      if ((st = launch_chained("peak launch", peak_kernel, ctas < 8 * dev.sm_count ? ctas : 8 * dev.sm_count,
                               kThreads, 0, stream, static_cast<const float*>(d.x.scales), scales, l.range)))
        return st;
      st = restore<E, true>(d.x, d.rows, d.width, l.x, l.x_ld, stream, l.range);
    } else {
      st = restore<E>(d.x, d.rows, d.width, l.x, l.x_ld, stream);
    }
  } else {
    st = restore<E>(d.x, d.rows, d.width, l.x, l.x_ld, stream);
  }
  if (st) return st;
  CUtensorMap a, b;
  if ((st = matrix_map(&a, dy, d.rows, d.n, l.dy_ld, box_rows(true, 0)))) return st;
  if ((st = matrix_map(&b, l.x, d.rows, d.width, l.x_ld, box_rows(true, 0)))) return st;
  StoreArgs s{};
  s.out = d.out;
  s.ld = d.out_stride;
  s.m = d.n;
  s.n = d.width;
  s.constant = 1.0f;
  if (l.range) s.scale = &l.range->undo;
  s.accumulate = (d.flags & FADAM_WGRAD_ACCUMULATE) != 0;
  s.wide = wide_stores(d.out, d.out_stride, sizeof(typename Out::type));
  const GemmShape shape = gemm_shape(d.n, d.width, d.rows, l.plan, dev.status);
  return store_product<T, true, true, Out>(a, b, shape, s, l.parts, dev.sm_count, stream);
}

fadam_status check(const fadam_wgrad* d) {
  if (!d) return fail(FADAM_EINVAL, "the descriptor is NULL");
  if (!is_16bit(d->dtype)) return fail(FADAM_EDTYPE, "dtype %d is not bf16 or fp16", d->dtype);
  if (d->out_dtype != d->dtype && d->out_dtype != FADAM_DT_F32)
    return fail(FADAM_EDTYPE, "out dtype %d is neither fp32 nor dy's %d", d->out_dtype, d->dtype);
  if (d->flags & ~(FADAM_WGRAD_ACCUMULATE | FADAM_WGRAD_WIDE_X))
    return fail(FADAM_EINVAL, "unknown flag bits 0x%x", d->flags);
  const fadam_status st = check_matrix(d->dy, d->rows, d->n, d->dy_stride, d->dtype, &d->x);
  if (st) return st;
  if (d->width < 1 || d->out_stride < d->width)
    return fail(FADAM_EINVAL, "width %lld, out stride %lld", (long long)d->width,
                (long long)d->out_stride);
  if (d->width > int64_t(1) << 30) return fail(FADAM_ELIMIT, "width beyond 2^30");
  if (!d->out) return fail(FADAM_EINVAL, "out is NULL");
  if (misaligned(d->out, elem_size(d->out_dtype)))
    return fail(FADAM_EALIGN, "a pointer is not aligned to its element size");
  return FADAM_OK;
}

}  // namespace
}  // namespace fadam_ops

using namespace fadam_ops;

extern "C" fadam_status fadam_checkpoint8_pack(const void* x, int64_t rows, int64_t width,
                                               int64_t x_stride, int32_t dtype,
                                               const fadam_checkpoint8* out, fadam_stream stream_) {
  clear_error();
  const fadam_status st = check_matrix(x, rows, width, x_stride, dtype, out);
  if (st || rows == 0) return st;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (dtype == FADAM_DT_BF16) return pack<__nv_bfloat16>(x, rows, width, x_stride, *out, stream);
  if (dtype == FADAM_DT_F16) return pack<__half>(x, rows, width, x_stride, *out, stream);
  return pack<float>(x, rows, width, x_stride, *out, stream);
}

extern "C" fadam_status fadam_checkpoint8_restore(const fadam_checkpoint8* in, int64_t rows,
                                                  int64_t width, void* x, int64_t x_stride,
                                                  int32_t dtype, fadam_stream stream_) {
  clear_error();
  const fadam_status st = check_matrix(x, rows, width, x_stride, dtype, in);
  if (st || rows == 0) return st;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (dtype == FADAM_DT_BF16) return restore<__nv_bfloat16>(*in, rows, width, x, x_stride, stream);
  if (dtype == FADAM_DT_F16) return restore<__half>(*in, rows, width, x, x_stride, stream);
  return restore<float>(*in, rows, width, x, x_stride, stream);
}

extern "C" fadam_status fadam_checkpoint8_wgrad_workspace(const fadam_wgrad* desc, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(FADAM_EINVAL, "bytes is NULL");
  fadam_status st = check(desc);
  if (st) return st;
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  *bytes = desc->rows == 0 ? 0 : layout(*desc, nullptr, dev.sm_count).bytes;
  return FADAM_OK;
}

extern "C" fadam_status fadam_checkpoint8_wgrad(const fadam_wgrad* desc, void* workspace,
                                                size_t bytes, fadam_stream stream_) {
  clear_error();
  fadam_status st = check(desc);
  if (st) return st;
  const fadam_wgrad& d = *desc;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (d.rows == 0) {
    if (d.flags & FADAM_WGRAD_ACCUMULATE) return FADAM_OK;
    const int size = elem_size(d.out_dtype);
    const cudaError_t e =
        cudaMemset2DAsync(d.out, d.out_stride * size, 0, d.width * size, d.n, stream);
    return e == cudaSuccess ? FADAM_OK : cuda_fail(e, "cudaMemset2DAsync");
  }
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  const Layout l = layout(d, static_cast<char*>(workspace), dev.sm_count);
  if (!workspace || bytes < l.bytes)
    return fail(FADAM_EINVAL, "the workspace has %zu bytes, %zu are needed",
                workspace ? bytes : size_t(0), l.bytes);
  if (misaligned(workspace, 256)) return fail(FADAM_EALIGN, "the workspace is not 256-byte aligned");
  const bool wide = d.out_dtype == FADAM_DT_F32;
  if (d.dtype == FADAM_DT_BF16)
    return wide ? run<BF16, F32>(d, l, dev, stream) : run<BF16, BF16>(d, l, dev, stream);
  return wide ? run<F16, F32>(d, l, dev, stream) : run<F16, F16>(d, l, dev, stream);
}
