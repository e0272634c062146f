// Attention: argument checks, workspaces, tensor maps, and the small kernels
// beside the tensor-core ones.
#include "attention.cuh"

namespace fadam_ops {
namespace {

constexpr int kThreads = 256;

// ---- spans of documents ------------------------------------------------------------------

// A thread to a token: its document by bisection, and what that makes it see.
// A token outside all documents (or offsets that decrease) sees nothing.
__global__ void __launch_bounds__(kThreads)
    spans_kernel(const int32_t* documents, int64_t n, const int32_t* prefix, int tokens, bool causal,
                 Spans* spans) {
  chain_wait();
  chain_next();
  const int i = int(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= tokens) return;
  int64_t lo = 0, hi = n + 1;  // the last offset that is not beyond i lies in [lo - 1, hi - 1]
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (__ldg(documents + mid) <= i) lo = mid + 1;
    else hi = mid;
  }
  Spans s{};
  const int64_t d = lo - 1;
  if (d >= 0 && d < n) {
    const int a = max(__ldg(documents + d), 0), b = min(__ldg(documents + d + 1), tokens);
    if (a <= i && i < b) {
      const int p = prefix ? min(max(__ldg(prefix + d), 0), b - a) : 0;
      s = spans_in(i, a, b, p, causal);
    }
  }
  spans[i] = s;
}

// ---- the rows' lse and delta for the backward pass -------------------------------------------

// What is added to a row's scores, -lse in units of log 2 and the lift of p's
// exponent, and to its grad_out . v: -delta = -grad_out . out, 16 lanes to a
// row.  Rows that see nothing, and those up to a whole tile, get -infinity: p
// is 0.
constexpr int kStatRows = 64;  // tokens of a CTA, of one head: 16 at a time
template <class E, bool kPeak>
__global__ void __launch_bounds__(kThreads)
    stats_kernel(const E* out, int64_t out_ld, int64_t out_head_ld, const E* grad, int64_t grad_ld,
                 int64_t grad_head_ld, const float* lse,
                 int tokens, int heads, int width, int pitch, float lift, float* stats, unsigned* peak) {
  chain_wait();
  chain_next();
  const int head = int(blockIdx.x % unsigned(heads)), token0 = int(blockIdx.x / unsigned(heads)) * kStatRows;
  const int group = threadIdx.x / 16, lane = threadIdx.x % 16;
  constexpr int kTurns = kStatRows / 16;
  Raw<E> a[kTurns], b[kTurns];
  float l[kTurns];
#pragma unroll
  for (int r = 0; r < kTurns; ++r) {
    const int t = token0 + r * 16 + group;
    a[r] = zero_raw<E>();
    b[r] = zero_raw<E>();
    l[r] = t < tokens ? lse[int64_t(t) * heads + head] : -INFINITY;
    if (l[r] != -INFINITY && lane * 8 < width) {
      a[r] = load_raw(out + t * out_ld + head * out_head_ld + lane * 8);
      b[r] = load_raw(grad + t * grad_ld + head * grad_head_ld + lane * 8);
    }
  }
  float top = 0.0f;
#pragma unroll
  for (int r = 0; r < kTurns; ++r) {
    Pair x[4], y[4];
    widen(a[r], x);
    widen(b[r], y);
    Pair sum = mul2(x[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sum = fma2(x[i], y[i], sum);
    float delta = sum2(sum);
#pragma unroll
    for (int d = 8; d > 0; d /= 2) delta += __shfl_xor_sync(~0u, delta, d);
    if (kPeak) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = split(y[i]);
        // (a NaN counts as an infinity: the gradients are not finite anyway)
        top = fmaxf(top, v.x == v.x ? fabsf(v.x) : INFINITY);
        top = fmaxf(top, v.y == v.y ? fabsf(v.y) : INFINITY);
      }
    }
    const int t = token0 + r * 16 + group;
    if (lane == 0 && t < pitch) {
      stats[int64_t(head) * pitch + t] = l[r] == -INFINITY ? -INFINITY : lift - l[r] * kLog2e;
      stats[int64_t(heads + head) * pitch + t] = -delta;
    }
  }
  if (kPeak) {
    const unsigned bits = __reduce_max_sync(~0u, __float_as_uint(top));
    if (threadIdx.x % 32 == 0 && bits) atomicMax(peak, bits);
  }
}

// grad_k and grad_v from their sums by splits of the query heads, in order.
template <class E>
__global__ void __launch_bounds__(kThreads)
    join_kernel(const float* parts, int splits, int64_t n, E* grad_v, E* grad_k) {
  chain_wait();
  chain_next();
  const int64_t eights = n / 8, i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= 2 * eights) return;
  const bool key = i >= eights;
  const int64_t at = (key ? i - eights : i) * 8;
  Pair sum[4] = {};
  for (int s = 0; s < splits; ++s) {
    Pair v[4];
    widen(load_raw(parts + (int64_t(s) * 2 + key) * n + at), v);
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = add2(sum[k], v[k]);
  }
  store_raw((key ? grad_k : grad_v) + at, narrow<E>(sum));
}

bool finite(float x) { return x - x == 0.0f; }

fadam_status check_rows(const char* name, const void* p, int64_t stride, int64_t head_stride,
                        const fadam_attention& d, int heads) {
  if (d.tokens > 0 && !p) return fail(FADAM_EINVAL, "%s is NULL", name);
  if (misaligned(p, 16)) return fail(FADAM_EALIGN, "%s is not aligned to 16 bytes", name);
  if ((d.tokens > 1 && stride % 8) || (heads > 1 && head_stride % 8))
    return fail(FADAM_EALIGN, "%s has strides %lld and %lld, not multiples of 8 elements", name,
                (long long)stride, (long long)head_stride);
  // heads within a token, or tokens within a head
  const bool inner = heads == 1 || head_stride >= d.width;
  const bool outer = d.tokens <= 1 || stride >= d.width;
  const int64_t most = int64_t(1) << 38;
  if (!inner || !outer || stride > most || head_stride > most)
    return fail(FADAM_EINVAL, "%s has strides %lld and %lld with heads of %d", name, (long long)stride,
                (long long)head_stride, d.width);
  return FADAM_OK;
}

fadam_status check(const fadam_attention* d) {
  if (!d) return fail(FADAM_EINVAL, "the descriptor is NULL");
  if (!is_16bit(d->dtype)) return fail(FADAM_EDTYPE, "dtype %d is not bf16 or fp16", d->dtype);
  if (d->flags & ~FADAM_ATTENTION_CAUSAL || d->reserved)
    return fail(FADAM_EINVAL, "unknown flag bits 0x%x, reserved %u", d->flags, d->reserved);
  if (d->tokens < 0 || d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads || d->width < 8 ||
      d->width % 8)
    return fail(FADAM_EINVAL, "%lld tokens, %d heads over %d, width %d (a multiple of 8)",
                (long long)d->tokens, d->heads, d->kv_heads, d->width);
  if (d->tokens > int64_t(1) << 24 || d->heads > 1 << 14 || d->width > FADAM_ATTENTION_MAX_WIDTH)
    return fail(FADAM_ELIMIT, "%lld tokens (2^24), %d heads (2^14), width %d (%d)", (long long)d->tokens,
                d->heads, d->width, FADAM_ATTENTION_MAX_WIDTH);
  if (!d->documents && (d->sequence < 1 || d->tokens % d->sequence))
    return fail(FADAM_EINVAL, "%lld tokens are not whole sequences of %lld", (long long)d->tokens,
                (long long)d->sequence);
  if (d->documents && (d->n_documents < 0 || d->n_documents > int64_t(1) << 30))
    return fail(FADAM_EINVAL, "%lld documents", (long long)d->n_documents);
  if (!(d->scale > 0.0f) || !finite(d->scale)) return fail(FADAM_EINVAL, "scale is not finite and above 0");
  if (!(d->softcap >= 0.0f) || !finite(d->softcap)) return fail(FADAM_EINVAL, "softcap is not finite and at least 0");
  if (d->softcap > 0.0f && !finite(d->scale / d->softcap))
    return fail(FADAM_EINVAL, "scale %g over softcap %g is not finite", d->scale, d->softcap);
  fadam_status st;
  if ((st = check_rows("q", d->q, d->q_stride, d->q_head_stride, *d, d->heads)) ||
      (st = check_rows("k", d->k, d->k_stride, d->k_head_stride, *d, d->kv_heads)) ||
      (st = check_rows("v", d->v, d->v_stride, d->v_head_stride, *d, d->kv_heads)))
    return st;
  if (d->tokens > 0 && (!d->out || !d->lse)) return fail(FADAM_EINVAL, "out and lse must be non-NULL");
  if (misaligned(d->out, 16) || misaligned(d->lse, 4) || misaligned(d->slopes, 4) ||
      misaligned(d->documents, 4) || misaligned(d->prefix, 4))
    return fail(FADAM_EALIGN, "out is not aligned to 16 bytes, or lse, slopes, documents or prefix to 4");
  return FADAM_OK;
}

fadam_status check(const fadam_attention_grad* d) {
  if (!d) return fail(FADAM_EINVAL, "the descriptor is NULL");
  fadam_status st;
  if ((st = check(&d->forward)) ||
      (st = check_rows("out", d->forward.out, d->out_stride, d->out_head_stride, d->forward, d->forward.heads)) ||
      (st = check_rows("grad_out", d->grad_out, d->grad_out_stride, d->grad_out_head_stride, d->forward,
                       d->forward.heads)))
    return st;
  if (d->forward.tokens > 0 && (!d->grad_q || !d->grad_k || !d->grad_v))
    return fail(FADAM_EINVAL, "grad_q, grad_k and grad_v must be non-NULL");
  if (misaligned(d->grad_q, 16) || misaligned(d->grad_k, 16) || misaligned(d->grad_v, 16))
    return fail(FADAM_EALIGN, "a gradient is not aligned to 16 bytes");
  return FADAM_OK;
}

struct Layout {
  Spans* spans;
  float* stats;
  unsigned* peak;
  float* parts;
  int splits;
  size_t bytes;
};
Layout layout(const fadam_attention& d, char* base) {
  Layout l{};
  Carver c{base};
  if (d.documents) l.spans = static_cast<Spans*>(c.take(sizeof(Spans) * d.tokens));
  l.bytes = c.used;
  return l;
}

// Over how many CTAs the query heads that share a key head are split, for
// grad_k and grad_v: as few as give two CTAs to an SM.  (Under a causal mask
// the first keys' CTA does twice the average's work.)
int splits_of(const fadam_attention& d, int sm_count) {
  const int group = d.heads / d.kv_heads;
  const int64_t ctas = ceil_div(d.tokens, kRows) * d.kv_heads;
  for (int s = 1; s < group; ++s)
    if (group % s == 0 && ctas * s >= 2 * sm_count) return s;
  return group;
}
Layout layout(const fadam_attention_grad& desc, char* base, int sm_count) {
  const fadam_attention& d = desc.forward;
  Layout l{};
  Carver c{base};
  if (d.documents) l.spans = static_cast<Spans*>(c.take(sizeof(Spans) * d.tokens));
  l.stats = static_cast<float*>(c.take(sizeof(float) * 2 * d.heads * round_up(d.tokens, kRows)));
  l.peak = static_cast<unsigned*>(c.take(sizeof(unsigned)));
  l.splits = splits_of(d, sm_count);
  if (l.splits > 1)
    l.parts = static_cast<float*>(c.take(sizeof(float) * 2 * l.splits * d.tokens * d.kv_heads * d.width));
  l.bytes = c.used;
  return l;
}

AttentionArgs arguments(const fadam_attention& d, const Spans* spans, const DeviceFacts& dev) {
  AttentionArgs g{};
  g.tokens = int(d.tokens);
  g.sequence = d.documents ? 0 : int(d.sequence);
  g.heads = d.heads;
  g.group = d.heads / d.kv_heads;
  g.width = d.width;
  g.tiles = int(ceil_div(d.tokens, kRows));
  g.causal = (d.flags & FADAM_ATTENTION_CAUSAL) != 0;
  g.scale = d.scale;
  g.softcap = d.softcap;
  g.slopes = d.slopes;
  g.spans = spans;
  g.prefix = d.documents ? nullptr : d.prefix;
  g.documents = d.documents;
  g.n_documents = d.n_documents;
  g.lse = d.lse;
  g.status = dev.status;
  return g;
}

fadam_status find_spans(const fadam_attention& d, Spans* spans, cudaStream_t stream) {
  if (!d.documents) return FADAM_OK;
  return launch_chained("document spans launch", spans_kernel, ceil_div(d.tokens, kThreads), kThreads, 0,
                        stream, d.documents, d.n_documents, d.prefix, int(d.tokens),
                        (d.flags & FADAM_ATTENTION_CAUSAL) != 0, spans);
}

fadam_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need && (!workspace || bytes < need))
    return fail(FADAM_EINVAL, "the workspace has %zu bytes, %zu are needed", workspace ? bytes : size_t(0), need);
  if (misaligned(workspace, 256)) return fail(FADAM_EALIGN, "the workspace is not 256-byte aligned");
  return FADAM_OK;
}

template <class T>
fadam_status backward(const fadam_attention_grad& desc, const Layout& l, const BackwardMaps& maps,
                      const DeviceFacts& dev, cudaStream_t stream) {
  using E = typename T::type;
  constexpr bool kPeak = T::code == FADAM_DT_F16;
  const fadam_attention& d = desc.forward;
  AttentionArgs g = arguments(d, l.spans, dev);
  g.stats = l.stats;
  g.peak = l.peak;
  g.parts = l.parts;
  g.splits = l.splits;
  if (kPeak) {
    const cudaError_t e = cudaMemsetAsync(l.peak, 0, sizeof(unsigned), stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  }
  fadam_status st;
  if ((st = find_spans(d, l.spans, stream))) return st;
  const int pitch = g.tiles * kRows;
  if ((st = launch_chained("attention stats launch", stats_kernel<E, kPeak>,
                           int64_t(pitch / kStatRows) * d.heads, kThreads, 0, stream,
                           static_cast<const E*>(d.out), desc.out_stride, desc.out_head_stride,
                           static_cast<const E*>(desc.grad_out),
                           desc.grad_out_stride, desc.grad_out_head_stride,
                           static_cast<const float*>(d.lse), int(d.tokens), int(d.heads), int(d.width), pitch,
                           kPeak ? 10.0f : 0.0f, l.stats, l.peak)))
    return st;
  st = kPeak ? attention_backward_f16(maps, g, stream) : attention_backward_bf16(maps, g, stream);
  if (st || l.splits == 1) return st;
  const int64_t n = d.tokens * d.kv_heads * d.width;
  return launch_chained("attention join launch", join_kernel<E>, ceil_div(2 * n / 8, kThreads), kThreads, 0,
                        stream, static_cast<const float*>(l.parts), l.splits, n, static_cast<E*>(desc.grad_v),
                        static_cast<E*>(desc.grad_k));
}

}  // namespace
}  // namespace fadam_ops

using namespace fadam_ops;

extern "C" fadam_status fadam_attention_workspace(const fadam_attention* desc, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(FADAM_EINVAL, "bytes is NULL");
  const fadam_status st = check(desc);
  if (st) return st;
  *bytes = desc->tokens == 0 ? 0 : layout(*desc, nullptr).bytes;
  return FADAM_OK;
}

extern "C" fadam_status fadam_attention_run(const fadam_attention* desc, void* workspace, size_t bytes,
                                            fadam_stream stream_) {
  clear_error();
  fadam_status st = check(desc);
  if (st || desc->tokens == 0) return st;
  const fadam_attention& d = *desc;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  const Layout l = layout(d, static_cast<char*>(workspace));
  if ((st = check_workspace(workspace, bytes, l.bytes))) return st;
  ForwardMaps maps;
  if ((st = head_map(&maps.q, d.q, d.tokens, d.heads, d.width, d.q_stride, d.q_head_stride)) ||
      (st = head_map(&maps.k, d.k, d.tokens, d.kv_heads, d.width, d.k_stride, d.k_head_stride)) ||
      (st = head_map(&maps.v, d.v, d.tokens, d.kv_heads, d.width, d.v_stride, d.v_head_stride)) ||
      (st = head_map(&maps.out, d.out, d.tokens, d.heads, d.width, int64_t(d.heads) * d.width, d.width)))
    return st;
  if ((st = find_spans(d, l.spans, stream))) return st;
  const AttentionArgs g = arguments(d, l.spans, dev);
  return d.dtype == FADAM_DT_BF16 ? attention_forward_bf16(maps, g, stream)
                                  : attention_forward_f16(maps, g, stream);
}

extern "C" fadam_status fadam_attention_backward_workspace(const fadam_attention_grad* desc, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(FADAM_EINVAL, "bytes is NULL");
  fadam_status st = check(desc);
  if (st) return st;
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  *bytes = desc->forward.tokens == 0 ? 0 : layout(*desc, nullptr, dev.sm_count).bytes;
  return FADAM_OK;
}

extern "C" fadam_status fadam_attention_backward(const fadam_attention_grad* desc, void* workspace,
                                                 size_t bytes, fadam_stream stream_) {
  clear_error();
  fadam_status st = check(desc);
  if (st || desc->forward.tokens == 0) return st;
  const fadam_attention& d = desc->forward;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  const Layout l = layout(*desc, static_cast<char*>(workspace), dev.sm_count);
  if ((st = check_workspace(workspace, bytes, l.bytes))) return st;
  BackwardMaps maps;
  const int64_t q_ld = int64_t(d.heads) * d.width, k_ld = int64_t(d.kv_heads) * d.width;
  if ((st = head_map(&maps.q, d.q, d.tokens, d.heads, d.width, d.q_stride, d.q_head_stride)) ||
      (st = head_map(&maps.k, d.k, d.tokens, d.kv_heads, d.width, d.k_stride, d.k_head_stride)) ||
      (st = head_map(&maps.v, d.v, d.tokens, d.kv_heads, d.width, d.v_stride, d.v_head_stride)) ||
      (st = head_map(&maps.grad_out, desc->grad_out, d.tokens, d.heads, d.width, desc->grad_out_stride,
                     desc->grad_out_head_stride)) ||
      (st = head_map(&maps.grad_q, desc->grad_q, d.tokens, d.heads, d.width, q_ld, d.width)) ||
      (st = head_map(&maps.grad_k, desc->grad_k, d.tokens, d.kv_heads, d.width, k_ld, d.width)) ||
      (st = head_map(&maps.grad_v, desc->grad_v, d.tokens, d.kv_heads, d.width, k_ld, d.width)))
    return st;
  return d.dtype == FADAM_DT_BF16 ? backward<BF16>(*desc, l, maps, dev, stream)
                                  : backward<F16>(*desc, l, maps, dev, stream);
}
