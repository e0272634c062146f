// Attention: argument checks, workspaces, tensor maps, and the small kernels
// beside the tensor-core ones.
#include "attention.cuh"

namespace fadam_ops {
namespace {

constexpr int kThreads = 256;

// ---- plans: the spans of documents, and the order of the tiles -----------------------------------

constexpr int kNearOffsets = 4096;  // most that are kept in shared memory
struct PlanArgs {
  const int32_t* documents;
  const int32_t* prefix;
  int64_t n_documents;
  int tokens, sequence;
  bool causal;
  Spans* spans;        // [tokens], written where there are documents
  int* order;          // of `tiles` of `rows` queries, or NULL: not asked for
  int rows, tiles;
};

// What token i sees: by its document, found by bisection, or its sequence.  A
// token outside all documents (or with offsets that decrease) sees nothing.
// `offsets` are the documents', in shared memory where they fit.
__device__ __forceinline__ Spans find_spans(const PlanArgs& p, const int32_t* offsets, int i) {
  int64_t d;
  int a, b;
  if (p.documents) {
    int64_t lo = 0, hi = p.n_documents + 1;  // the last offset that is not beyond i lies in [lo - 1, hi - 1]
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (offsets[mid] <= i) lo = mid + 1;
      else hi = mid;
    }
    d = lo - 1;
    if (d < 0 || d >= p.n_documents) return Spans{};
    a = max(offsets[d], 0);
    b = min(offsets[d + 1], p.tokens);
    if (i < a || i >= b) return Spans{};
  } else {
    d = i / p.sequence;
    a = int(d) * p.sequence;
    b = a + p.sequence;
  }
  return spans_in(i, a, b, p.prefix ? min(max(__ldg(p.prefix + d), 0), b - a) : 0, p.causal);
}

// One block: the tiles sorted by how many tiles of keys their first and last
// rows reach (256 classes of length), longest first, so that no long one is left
// for the end.  (Equal ones in any order: it decides nothing but who is first.)
__device__ __forceinline__ void sort_tiles(const PlanArgs& p, const int32_t* offsets) {
  constexpr int kBuckets = 256;
  __shared__ int count[kBuckets];
  int lo = 0, hi = p.tokens;
  if (p.documents) {
    lo = min(max(offsets[0], 0), p.tokens);
    hi = min(max(offsets[p.n_documents], 0), p.tokens);
  }
  int shift = 0;
  while ((p.tokens / kRows) >> shift >= kBuckets) ++shift;
  const auto bucket = [&](int tile) {
    const int first = max(tile * p.rows, lo), last = min((tile + 1) * p.rows, hi) - 1;
    int work = 0;
    if (first <= last) {
      const Spans a = find_spans(p, offsets, first), b = find_spans(p, offsets, last);
      work = b.key_hi - a.key_lo;
    }
    return kBuckets - 1 - min(max(work / kRows >> shift, 0), kBuckets - 1);
  };
  for (int i = threadIdx.x; i < kBuckets; i += kThreads) count[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.tiles; i += kThreads) atomicAdd(&count[bucket(i)], 1);
  __syncthreads();
  if (threadIdx.x < 32) {
    int sum = 0;
    for (int i = 0; i < kBuckets; i += 32) {
      const int n = count[i + threadIdx.x];
      int upto = n;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int other = __shfl_up_sync(~0u, upto, d);
        if (int(threadIdx.x) >= d) upto += other;
      }
      count[i + threadIdx.x] = sum + upto - n;
      sum += __shfl_sync(~0u, upto, 31);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.tiles; i += kThreads) p.order[atomicAdd(&count[bucket(i)], 1)] = i;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanArgs p) {
  chain_wait();
  chain_next();
  // the offsets, next to the threads that bisect them (each step in global memory
  // would wait for L2)
  __shared__ int32_t near[kNearOffsets];
  const int32_t* offsets = p.documents;
  if (offsets && p.n_documents < kNearOffsets) {
    for (int i = threadIdx.x; i <= p.n_documents; i += kThreads) near[i] = offsets[i];
    __syncthreads();
    offsets = near;
  }
  // (the order first: it takes longest)
  const int block = int(blockIdx.x) - (p.order != nullptr);
  if (block < 0) return sort_tiles(p, offsets);
  const int i = block * kThreads + threadIdx.x;
  if (i < p.tokens) p.spans[i] = find_spans(p, offsets, i);
}

// ---- the rows' lse and delta for the backward pass -------------------------------------------

// What is added to a row's scores, -lse in units of log 2 and the lift of p's
// exponent, and to its grad_out . v: -delta = -grad_out . out, 16 lanes to a
// row.  Rows that see nothing, and those up to a whole tile, get -infinity: p
// is 0.  (Their lse is -infinity, but so is that of a row that sees keys whose
// scores all are: its gradients are NaN.)  For fp16 (kPeak) also the row's largest
// |grad_out|, and the documents' peaks (their largest finite ones: atomics of a
// maximum, whose order changes nothing); blocks behind those of the rows take the
// sums of v's magnitudes.
constexpr int kStatRows = 64;  // tokens of a CTA, of one head: 16 at a time
template <class E>
struct StatRows {
  const E* base;
  int64_t ld, head_ld;
  __device__ __forceinline__ Raw<E> load(int token, int head, int col) const {
    return load_raw(base + token * ld + head * head_ld + col);
  }
};

// A row's peak, counted with its CTA's first document's, or at its own place.
__device__ __forceinline__ void count_peak(unsigned* shared, int base, unsigned* peaks, int entry, float x) {
  if (!(x > 0.0f && x < INFINITY)) return;
  atomicMax(entry == base ? shared : peaks + entry, __float_as_uint(x));
}

template <class E, bool kPeak>
__global__ void __launch_bounds__(kThreads)
    stats_kernel(const StatRows<E> out, const StatRows<E> grad, const StatRows<E> values, float lift,
                 const __grid_constant__ AttentionArgs g) {
  chain_wait();
  chain_next();
  __shared__ unsigned shared[2];
  const unsigned row_blocks = unsigned(g.tiles) * (kRows / kStatRows) * g.heads;
  const bool of_v = kPeak && blockIdx.x >= row_blocks;
  const int kv_heads = g.heads / g.group, heads = of_v ? kv_heads : g.heads;
  const unsigned block = of_v ? blockIdx.x - row_blocks : blockIdx.x;
  const int head = int(block % unsigned(heads)), token0 = int(block / unsigned(heads)) * kStatRows;
  const int group = threadIdx.x / 16, lane = threadIdx.x % 16, width = g.width;
  constexpr int kTurns = kStatRows / 16;
  int base = 0;
  unsigned* peaks = nullptr;
  const int64_t apart = int64_t(kv_heads) * g.entries;
  if constexpr (kPeak) {
    if (threadIdx.x < 2) shared[threadIdx.x] = 0;
    base = entry_of(g, token0).at;
    peaks = g.peaks + int64_t(of_v ? head : head / g.group) * g.entries;
    __syncthreads();
  }
  Raw<E> a[kTurns], b[kTurns];
  if (kPeak && of_v) {
    Entry entry[kTurns];
#pragma unroll
    for (int r = 0; r < kTurns; ++r) {
      const int t = token0 + r * 16 + group;
      entry[r] = entry_of(g, t);
      a[r] = zero_raw<E>();
      if (entry[r].lives && lane * 8 < width) a[r] = values.load(t, head, lane * 8);
    }
#pragma unroll
    for (int r = 0; r < kTurns; ++r) {
      Pair x[4];
      widen(a[r], x);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = split(x[i]);
        sum += fabsf(v.x) < INFINITY ? fabsf(v.x) : 0.0f;
        sum += fabsf(v.y) < INFINITY ? fabsf(v.y) : 0.0f;
      }
#pragma unroll
      for (int d = 8; d > 0; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
      if (lane == 0 && entry[r].lives) count_peak(&shared[0], base, peaks + 2 * apart, entry[r].at, sum);
    }
    __syncthreads();
    if (threadIdx.x == 0 && shared[0]) atomicMax(peaks + 2 * apart + base, shared[0]);
    return;
  }
  float l[kTurns];
  int entry[kTurns];
  bool lives[kTurns];
#pragma unroll
  for (int r = 0; r < kTurns; ++r) {
    const int t = token0 + r * 16 + group;
    const Entry e = entry_of(g, t);
    entry[r] = e.at;
    a[r] = zero_raw<E>();
    b[r] = zero_raw<E>();
    lives[r] = e.lives;
    l[r] = e.lives ? g.lse[int64_t(t) * heads + head] : 0.0f;
    if (e.lives && lane * 8 < width) {
      a[r] = out.load(t, head, lane * 8);
      b[r] = grad.load(t, head, lane * 8);
    }
  }
  const int64_t pitch = int64_t(g.tiles) * kRows;
#pragma unroll
  for (int r = 0; r < kTurns; ++r) {
    Pair x[4], y[4];
    widen(a[r], x);
    widen(b[r], y);
    Pair sum = mul2(x[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sum = fma2(x[i], y[i], sum);
    float delta = sum2(sum), top = 0.0f;
#pragma unroll
    for (int d = 8; d > 0; d /= 2) delta += __shfl_xor_sync(~0u, delta, d);
    if (kPeak) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = split(y[i]);
        top = fmaxf(top, fabsf(v.x) < INFINITY ? fabsf(v.x) : 0.0f);
        top = fmaxf(top, fabsf(v.y) < INFINITY ? fabsf(v.y) : 0.0f);
      }
#pragma unroll
      for (int d = 8; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    }
    const int t = token0 + r * 16 + group;
    if (lane == 0) {  // (there is a place for every row of a tile)
      g.stats[head * pitch + t] = lives[r] ? lift - l[r] * kLog2e : -INFINITY;
      g.stats[(int64_t(heads) + head) * pitch + t] = -delta;
      if constexpr (kPeak) {
        g.stats[(2 * int64_t(heads) + head) * pitch + t] = top;
        if (lives[r]) {
          count_peak(&shared[0], base, peaks, entry[r], top);
          count_peak(&shared[1], base, peaks + apart, entry[r], fabsf(delta));
        }
      }
    }
  }
  if constexpr (kPeak) {
    __syncthreads();
    if (threadIdx.x < 2 && shared[threadIdx.x]) atomicMax(peaks + threadIdx.x * apart + base, shared[threadIdx.x]);
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
  if (ceil_div(d->tokens, kRows) * d->heads > int64_t(1) << 30)
    return fail(FADAM_ELIMIT, "%lld tokens of %d heads", (long long)d->tokens, d->heads);
  if (!d->documents && (d->sequence < 1 || d->tokens % d->sequence))
    return fail(FADAM_EINVAL, "%lld tokens are not whole sequences of %lld", (long long)d->tokens,
                (long long)d->sequence);
  if (d->documents && (d->n_documents < 0 || d->n_documents > int64_t(1) << 30))
    return fail(FADAM_EINVAL, "%lld documents", (long long)d->n_documents);
  if (!(d->scale > 0.0f) || !finite(d->scale)) return fail(FADAM_EINVAL, "scale is not finite and above 0");
  if (!(d->softcap >= 0.0f) || !finite(d->softcap)) return fail(FADAM_EINVAL, "softcap is not finite and at least 0");
  if (d->softcap > 0.0f) {
    // (the square of the cap in fp32, and no cap that has nothing to do with the scores)
    const double y = double(d->scale) / d->softcap;
    if (d->softcap < 1e-15f || d->softcap > 1e15f || d->softcap * y * y * y * y * y * y * y > 1e37)
      return fail(FADAM_EINVAL, "softcap %g with scale %g", d->softcap, d->scale);
  }
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
  int* order;  // forward: of what a CTA takes
  float* stats;
  unsigned* peaks;
  int entries;
  float* parts;
  int splits;
  size_t bytes;
};
bool several(const fadam_attention& d) { return d.documents || d.tokens > d.sequence; }
// Whether the forward pass takes its tiles in order of their work, longest first,
// rather than from the last one back (which is that order for one sequence): for
// several sequences whose CTAs come to some SMs twice, so that a long one at the
// end shows.  With up to one CTA to an SM all start at once and the order's launch
// is lost: 3 of 400 with 16 heads (80 CTAs) take 13.7 us sorted and 11.6 as they
// come, 5 of 777 with 8 (128) 20.7 and 18.6, 4 documents in 1500 tokens (144) 18.7
// and 17.5.  Up to two: 5 of 777 with 12 heads (192) 24.4 and 27.3, over 4 key
// heads 26.1 and 29.5, 11 documents in 4096 tokens (192, 256) 22.5 and 23.8, 26.4
// and 32.9, 4 of 1024 (256) 28.3 and 29.3, 3 of 700 (288) 29.3 both; but 2 of 1024
// (256) 25.8 and 23.4.  Beyond, sequences that take turns in L2 cost more than the
// order gives: 4 of 600 (320) 28.4 and 27.6, 3 of 1000 (384) 41.5 and 39.3, 4 of
// 1024 (512) 48.2 and 46.7, 8 of 2048 (1024) 141 and 137, 11 documents in 4096
// tokens (512) 56.5 and 53.2, though 13 in 16384 (1024) 159 and 164.
bool ordered(const fadam_attention& d, int sm_count) {
  const int64_t ctas = ceil_div(d.tokens, 2 * kRows) * d.heads;
  return several(d) && ctas > sm_count && ctas <= 2 * int64_t(sm_count);
}
// (The order has its place whether or not it is asked for: how large a workspace
// is depends on no device.)
Layout layout(const fadam_attention& d, char* base) {
  Layout l{};
  Carver c{base};
  if (d.documents) l.spans = static_cast<Spans*>(c.take(sizeof(Spans) * d.tokens));
  if (several(d)) l.order = static_cast<int*>(c.take(sizeof(int) * ceil_div(d.tokens, kRows)));
  l.bytes = c.used;
  return l;
}

// Over how many CTAs the query heads that share a key head are split, for
// grad_k and grad_v: where there are fewer CTAs than SMs, and one that all
// queries see would take more than eight turns.
int splits_of(const fadam_attention& d, int sm_count) {
  const int group = d.heads / d.kv_heads;
  const int64_t tiles = ceil_div(d.tokens, kRows);
  if (group * tiles <= 8) return 1;
  for (int s = 1; s < group; ++s)
    if (group % s == 0 && tiles * d.kv_heads * s >= sm_count) return s;
  return group;
}
size_t peaks_bytes(const fadam_attention& d, const Layout& l) {
  return sizeof(unsigned) * 3 * d.kv_heads * l.entries;
}
Layout layout(const fadam_attention_grad& desc, char* base, int sm_count) {
  const fadam_attention& d = desc.forward;
  const int64_t tiles = ceil_div(d.tokens, kRows);
  Layout l{};
  Carver c{base};
  if (d.documents) l.spans = static_cast<Spans*>(c.take(sizeof(Spans) * d.tokens));
  const bool f16 = d.dtype == FADAM_DT_F16;
  l.stats = static_cast<float*>(c.take(sizeof(float) * (f16 ? 3 : 2) * d.heads * tiles * kRows));
  l.entries = int(d.documents ? d.tokens : d.tokens / d.sequence);
  if (f16) l.peaks = static_cast<unsigned*>(c.take(peaks_bytes(d, l)));
  l.splits = splits_of(d, sm_count);
  if (l.splits > 1)
    l.parts = static_cast<float*>(c.take(sizeof(float) * 2 * l.splits * d.tokens * d.kv_heads * d.width));
  l.bytes = c.used;
  return l;
}

AttentionArgs arguments(const fadam_attention& d, const Layout& l, const DeviceFacts& dev) {
  AttentionArgs g{};
  g.tokens = int(d.tokens);
  g.sequence = d.documents ? 0 : int(d.sequence);
  g.heads = d.heads;
  g.group = d.heads / d.kv_heads;
  g.width = d.width;
  g.tiles = int(ceil_div(d.tokens, kRows));
  g.causal = (d.flags & FADAM_ATTENTION_CAUSAL) != 0;
  g.pair_heads = g.group % 2 == 0;
  g.scale = d.scale;
  g.softcap = d.softcap;
  if (d.softcap > 0.0f) {
    // cap tanh(y), y = x scale / cap: x scale tanh(y) / y by tanh's Taylor series
    const double taylor[4] = {1.0, -1.0 / 3.0, 2.0 / 15.0, -17.0 / 315.0};
    for (int i = 0; i < 4; ++i)
      g.series[i].x = g.series[i].y = float(double(d.scale) * 1.4426950408889634 * taylor[i]);
  }
  g.slopes = d.slopes;
  g.spans = l.spans;
  g.order = l.order;
  g.prefix = d.documents ? nullptr : d.prefix;
  g.documents = d.documents;
  g.n_documents = d.n_documents;
  g.lse = d.lse;
  g.status = dev.status;
  return g;
}

fadam_status plan(const fadam_attention& d, const Layout& l, cudaStream_t stream) {
  if (!l.spans && !l.order) return FADAM_OK;
  PlanArgs p{};
  p.documents = d.documents;
  p.prefix = d.prefix;
  p.n_documents = d.n_documents;
  p.tokens = int(d.tokens);
  p.sequence = d.documents ? 0 : int(d.sequence);
  p.causal = (d.flags & FADAM_ATTENTION_CAUSAL) != 0;
  p.spans = l.spans;
  p.order = l.order;
  p.rows = d.heads / d.kv_heads % 2 ? 2 * kRows : kRows;  // (an odd group: 256 rows of one head to a CTA)
  p.tiles = int(ceil_div(d.tokens, p.rows));
  const int64_t span_blocks = l.spans ? ceil_div(d.tokens, kThreads) : 0;
  return launch_chained("attention plan launch", plan_kernel, (p.order != nullptr) + span_blocks, kThreads, 0,
                        stream, p);
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
  AttentionArgs g = arguments(d, l, dev);
  g.stats = l.stats;
  g.peaks = l.peaks;
  g.entries = l.entries;
  g.parts = l.parts;
  g.splits = l.splits;
  if (kPeak) {
    const cudaError_t e = cudaMemsetAsync(l.peaks, 0, peaks_bytes(d, l), stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  }
  fadam_status st;
  if ((st = plan(d, l, stream))) return st;
  const StatRows<E> out{static_cast<const E*>(d.out), desc.out_stride, desc.out_head_stride};
  const StatRows<E> grad{static_cast<const E*>(desc.grad_out), desc.grad_out_stride, desc.grad_out_head_stride};
  const StatRows<E> values{static_cast<const E*>(d.v), d.v_stride, d.v_head_stride};
  const int64_t blocks = int64_t(g.tiles) * (kRows / kStatRows) * (d.heads + (kPeak ? d.kv_heads : 0));
  if ((st = launch_chained("attention stats launch", stats_kernel<E, kPeak>, blocks, kThreads, 0, stream, out,
                           grad, values, kPeak ? 10.0f : 0.0f, g)))
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
  Layout l = layout(d, static_cast<char*>(workspace));
  if ((st = check_workspace(workspace, bytes, l.bytes))) return st;
  if (!ordered(d, dev.sm_count)) l.order = nullptr;
  ForwardMaps maps;
  if ((st = head_map(&maps.q, d.q, d.tokens, d.heads, d.width, d.q_stride, d.q_head_stride)) ||
      (st = head_map(&maps.k, d.k, d.tokens, d.kv_heads, d.width, d.k_stride, d.k_head_stride)) ||
      (st = head_map(&maps.v, d.v, d.tokens, d.kv_heads, d.width, d.v_stride, d.v_head_stride)) ||
      (st = head_map(&maps.out, d.out, d.tokens, d.heads, d.width, int64_t(d.heads) * d.width, d.width)))
    return st;
  if ((st = plan(d, l, stream))) return st;
  const AttentionArgs g = arguments(d, l, dev);
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
