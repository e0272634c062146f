// The token embedding and its weight's gradient.
//
// Forward is one pass: a thread takes a vector of eight columns of several
// rows.  The gradient is a sum over each token's rows: the rows are sorted by
// token first (stable, so that every sum has one order), then the sorted list
// is cut into equal pieces whose sums do not depend on how often a token
// occurs, and what pieces' ends cut is joined by the last piece that has a part
// of it.  (That one adds a token's parts in turn: 16384 rows of 4096 in bf16 that
// are all one token are added into fp32 in 135 us, rows of a token each in 116;
// 2^20 rows of 512 in 3738 and 946.)  Rows of no token are zeroed by the sort, which knows them.  (By other
// CTAs of the sums' launch it took longer, 37 us for 50021 x 1000 in place of 29:
// the sums are a chain of loads, each of which then waits behind the zeros.)
#include "fadam_seq.h"
#include "ops_internal.h"
#include "rows.cuh"

namespace fadam_ops {
namespace {

constexpr int kThreads = 256;   // of a CTA that streams rows: 2048 columns
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kRange = 1024;    // most tokens of the vocabulary that one CTA sorts by
constexpr int kLongest = 64;    // most rows of a piece
constexpr int kZeroBytes = 16384;  // of a row zeroed by one bulk copy
// GB300's.  (What depends on it, and with it a sum's groups and the size of the
// workspace, depends on no device that is asked.)
constexpr int kSms = 152;

// Eight elements in one access: 16 bytes, or 32 for fp32 (two of 16 would each
// touch half of every 32-byte sector).
template <class E>
__device__ __forceinline__ Raw<E> load_eight(const E* p) {
  if constexpr (sizeof(E) == 4) {
    Raw<E> r;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]),
                   "=r"(r.w[6]), "=r"(r.w[7])
                 : "l"(p)
                 : "memory");
    return r;
  } else {
    return load_raw(p);
  }
}
template <class E>
__device__ __forceinline__ void store_eight(E* p, const Raw<E>& r) {
  if constexpr (sizeof(E) == 4)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0]),
                 "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
                 : "memory");
  else
    store_raw(p, r);
}
// Whether rows of these can be accessed so.
bool eights(const void* p, int64_t stride, int64_t width, int size) {
  return width % 8 == 0 && !misaligned(p, 8 * size) && stride % 8 == 0;
}

// A thread's eight columns of a row: one aligned vector, or (rows that are not
// whole vectors) every blockDim-th element, so that a warp's accesses coalesce.
template <bool kWide>
struct Eight {
  int col, step, width;
  __device__ __forceinline__ Eight(int part, int width) : width(width) {
    const int first = part * int(blockDim.x) * 8;
    col = kWide ? first + int(threadIdx.x) * 8 : first + int(threadIdx.x);
    step = kWide ? 1 : int(blockDim.x);
  }
  __device__ __forceinline__ bool any() const { return col < width; }
  __device__ __forceinline__ bool has(int i) const { return kWide || col + i * step < width; }

  template <class E>
  __device__ __forceinline__ void load(const E* row, Raw<E>& r) const {
    if constexpr (kWide) {
      r = load_eight(row + col);
    } else {
      E e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = has(i) ? row[col + i * step] : from_float<E>(0.0f);
      memcpy(&r, e, sizeof r);
    }
  }
  template <class E>
  __device__ __forceinline__ void store(E* row, const Raw<E>& r) const {
    if constexpr (kWide) {
      store_eight(row + col, r);
    } else {
      E e[8];
      memcpy(e, &r, sizeof r);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (has(i)) row[col + i * step] = e[i];
    }
  }
};

// How rows are cut into column parts of at most 2048.
struct Parts {
  int threads, count;
};
Parts parts_of(int64_t width) {
  Parts p;
  const int64_t eights = ceil_div(width, 8);
  p.threads = int(eights < kThreads ? round_up(eights, 32) : kThreads);
  p.count = int(ceil_div(eights, p.threads));
  return p;
}

// ---- forward -----------------------------------------------------------------------

// 8192 rows of 4096 from bf16 into fp32: 27 us, 6.1 TB/s.
template <class E, class Out, bool kWide, int R>
__global__ void __launch_bounds__(kThreads)
    gather_kernel(const int64_t* tokens, const E* weight, int64_t ld, Out* out, int64_t out_ld,
                  int64_t rows, int width, int64_t vocab, int64_t padding, bool padded, float scale,
                  int parts) {
  chain_wait();
  chain_next();
  const unsigned block = blockIdx.x / unsigned(parts);
  const Eight<kWide> at(int(blockIdx.x - block * parts), width);
  if (!at.any()) return;
  const int64_t row0 = int64_t(block) * R;
  int64_t token[R];
  Raw<E> raw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) token[r] = row0 + r < rows ? __ldg(tokens + row0 + r) : -1;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    raw[r] = zero_raw<E>();
    if (token[r] >= 0 && token[r] < vocab) at.load(weight + token[r] * ld, raw[r]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (row0 + r >= rows) return;
    // what is neither padding nor in the vocabulary becomes NaN
    const float bad = token[r] >= 0 && token[r] < vocab ? 0.0f : NAN;
    const float keep = padded && token[r] == padding ? 0.0f : 1.0f;
    Pair v[4];
    widen(raw[r], v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = split(v[i]);
      v[i] = keep == 0.0f ? make_pair(0.0f, 0.0f)
             : bad == 0.0f ? make_pair(p.x * scale, p.y * scale)
                           : make_pair(bad, bad);
    }
    at.store(out + (row0 + r) * out_ld, narrow<Out>(v));
  }
}

// ---- sorting rows by token -----------------------------------------------------------

struct SortArgs {
  const int64_t* tokens;
  int32_t rows;
  int64_t vocab, padding;
  bool padded;
  int32_t range;     // tokens of the vocabulary that a CTA takes
  int32_t* order;    // [rows] rows sorted by token, those of one token ascending
  int32_t* starts;   // [vocab + 1] where a token's rows begin in it
  int32_t* arrived;  // [marks] set to zero
  int32_t marks;
};

// Each CTA takes a range of the vocabulary and reads all tokens twice: first it
// counts its own (for each of its warps, which have consecutive runs of rows)
// and those below its range, which says where its part of the order begins;
// then it places them.  Nothing is exchanged between CTAs, and the order is
// stable: within a warp's 32 rows a row comes behind those of its token in
// lower lanes.  Of T rows every CTA reads 16 T bytes, from L2 mostly: there is one
// to an SM for vocabularies up to 1024 tokens an SM, and one for each 1024 tokens
// beyond.  A sort by digits would take three launches or more (1037 rows over
// 50021: some 8000 cycles).
// At the end (unless kKeep) rows of no token are zeroed, by bulk copies where
// they allow it: 131072 x 4096 in fp32 from 16384 rows 320 us, 6.1 TB/s.
template <class Out, bool kWide, bool kKeep>
__global__ void __launch_bounds__(kSortThreads)
    sort_kernel(const SortArgs a, Out* out, int64_t out_ld, int width) {
  // kZeroBytes of zeros where rows are written, then counts [kSortWarps][range]
  extern __shared__ __align__(16) unsigned char sort_smem[];
  constexpr int kZeros = kKeep || !kWide ? 0 : kZeroBytes;
  int* counts = reinterpret_cast<int*>(sort_smem + kZeros);
  __shared__ int warp_sum[kSortWarps];
  __shared__ bool unused[kKeep ? 1 : kRange];
  __shared__ int below;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t low = int64_t(blockIdx.x) * a.range;
  const int mine = int(min(int64_t(a.range), a.vocab - low));
  for (int i = threadIdx.x; i < kSortWarps * a.range; i += kSortThreads) counts[i] = 0;
  if (kZeros) {
    for (int i = threadIdx.x; i < kZeros / 16; i += kSortThreads)
      reinterpret_cast<uint4*>(sort_smem)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (threadIdx.x == 0) below = 0;
  __syncthreads();
  chain_wait();
  chain_next();

  for (int64_t i = int64_t(blockIdx.x) * kSortThreads + threadIdx.x; i < a.marks; i += int64_t(gridDim.x) * kSortThreads)
    a.arrived[i] = 0;
  // rows of a warp: whole groups of 32
  const int per_warp = int((int64_t(a.rows) + kSortThreads - 1) / kSortThreads) * 32;
  const int first = warp * per_warp;
  const int last = int(min(int64_t(a.rows), int64_t(first) + per_warp));
  int* own = counts + warp * a.range;
  // the row's token within the range; -1 below it, -2 elsewhere
  const auto place = [&](int row) {
    if (row >= last) return -2;
    const int64_t t = __ldg(a.tokens + row);
    if (t < 0 || t >= a.vocab || (a.padded && t == a.padding)) return -2;
    return t < low ? -1 : t < low + mine ? int(t - low) : -2;
  };
  constexpr int kAhead = 8;  // loads in flight
  int fewer = 0;
  for (int row = first; row < last; row += 32 * kAhead) {
    int at[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) at[k] = place(row + 32 * k + lane);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      fewer += at[k] == -1;
      if (!__any_sync(~0u, at[k] >= 0)) continue;
      const unsigned peers = __match_any_sync(~0u, at[k]);
      if (at[k] >= 0 && lane == __ffs(peers) - 1) own[at[k]] += __popc(peers);
      __syncwarp();
    }
  }
  fewer = __reduce_add_sync(~0u, fewer);
  if (lane == 0 && fewer) atomicAdd(&below, fewer);
  __syncthreads();

  // a thread to a token: where its rows begin, then each warp's share of them
  const int v = threadIdx.x, used = per_warp ? (a.rows + per_warp - 1) / per_warp : 0;
  int count = 0;
  if (v < mine)
#pragma unroll 8
    for (int w = 0; w < used; ++w) count += counts[w * a.range + v];
  int sum = count;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int n = __shfl_up_sync(~0u, sum, d);
    if (lane >= d) sum += n;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  int base = below;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  const int start = base + sum - count;
  if (v < mine) {
    int next = start;
    for (int w0 = 0; w0 < used; w0 += 8) {
      int n[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) n[w] = w0 + w < used ? counts[(w0 + w) * a.range + v] : 0;
#pragma unroll
      for (int w = 0; w < 8; ++w)
        if (w0 + w < used) {
          counts[(w0 + w) * a.range + v] = next;
          next += n[w];
        }
    }
    if (!kKeep) unused[v] = count == 0;
    a.starts[low + v] = start;
    if (low + v == a.vocab - 1) a.starts[a.vocab] = start + count;
  }
  __syncthreads();

  for (int row = first; row < last; row += 32 * kAhead) {
    int at[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) at[k] = place(row + 32 * k + lane);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (!__any_sync(~0u, at[k] >= 0)) continue;
      const unsigned peers = __match_any_sync(~0u, at[k]);
      if (at[k] >= 0) a.order[own[at[k]] + __popc(peers & ((1u << lane) - 1))] = row + 32 * k + lane;
      __syncwarp();
      if (at[k] >= 0 && lane == __ffs(peers) - 1) own[at[k]] += __popc(peers);
      __syncwarp();
    }
  }

  if constexpr (!kKeep) {
    for (int r = warp; r < mine; r += kSortWarps) {
      if (!unused[r]) continue;
      Out* row = out + (low + r) * out_ld;
      if constexpr (kWide) {
        // bulk copies of zeros, by a lane of its own each
        const int64_t bytes = int64_t(width) * sizeof(Out);
        for (int64_t c = int64_t(lane) * kZeroBytes; c < bytes; c += 32 * kZeroBytes)
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                           reinterpret_cast<unsigned char*>(row) + c),
                       "r"(shared_addr(sort_smem)), "r"(int(min(int64_t(kZeroBytes), bytes - c)))
                       : "memory");
      } else {
        for (int c = lane; c < width; c += 32) row[c] = from_float<Out>(0.0f);
      }
    }
    if (kWide) asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
  }
}

// ---- sums over the sorted rows ----------------------------------------------------------

struct SumArgs {
  const int64_t* tokens;
  const int32_t* order;
  const int32_t* starts;
  int64_t vocab;
  int32_t width, parts, piece;   // piece: sorted rows of a CTA
  int64_t grad_ld, out_ld, carry_ld;
  float* carry;    // [pieces][2][carry_ld]: sums that a piece's begin and end cut
  int32_t* arrived;  // [pieces][parts]: of a token whose rows begin in the piece and end in another, the
                     // pieces that have left their part
  float scale;
};

// The scaled sum of a token's rows, written or added.
template <class Out, bool kWide, bool kKeep>
__device__ __forceinline__ void put(const Eight<kWide>& at, Out* row, const float (&sum)[8], float scale) {
  Pair v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_pair(sum[2 * i] * scale, sum[2 * i + 1] * scale);
  if constexpr (kKeep) {
    Raw<Out> old;
    Pair o[4];
    at.load(row, old);
    widen(old, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], o[i]);
  }
  at.store(row, narrow<Out>(v));
}

// The sum of the token `id`, whose rows are cut by pieces: the last of them to
// leave its part (in `carry`) adds all parts, in order.
template <class Out, bool kWide, bool kKeep>
__device__ __forceinline__ void join_parts(const SumArgs& a, const Eight<kWide>& at, int64_t id, unsigned part,
                                           int carry_col, Out* out) {
  __shared__ int before;
  const int begin = a.starts[id], end = a.starts[id + 1];
  const int first = begin / a.piece, last = (end - 1) / a.piece;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) before = atomicAdd(&a.arrived[int64_t(first) * a.parts + part], 1);
  __syncthreads();
  const bool mine = before == last - first;
  __syncthreads();  // (a CTA may come here twice)
  if (!mine || !at.any()) return;
  __threadfence();
  const float* carry = a.carry + carry_col;
  // a token that begins where its piece does has left its part as one that was cut there
  float sum[8] = {};
  constexpr int kAhead = 4;  // loads in flight
  for (int p = first; p <= last; p += kAhead) {
    Raw<float> raw[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      raw[k] = p + k > last ? zero_raw<float>()
                            : load_eight(carry + (int64_t(p + k) * 2 + (p + k == first && begin % a.piece)) * a.carry_ld);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] += __uint_as_float(raw[k].w[c]);
  }
  put<Out, kWide, kKeep>(at, out + id * a.out_ld, sum, a.scale);
}

// A piece's rows, several loads in flight; a token's sum is written when its
// first and its last row are in the piece, else its part is left for
// join_parts: in the piece's first place when the token's rows begin before the
// piece or with it, else in the second.  16384 rows of 4096 in bf16 into fp32:
// 45 us, 4.4 TB/s of what is read and written.
template <class E, class Out, bool kWide, bool kKeep>
__global__ void __launch_bounds__(kThreads, kWide ? 4 : 2)
    sum_kernel(const SumArgs a, const E* grad, Out* out) {
  __shared__ int rows[kLongest];
  __shared__ int ids[kLongest];
  chain_wait();
  // (No chain_next(): the next call's sort, placed while this runs, at times
  // stood where this one's CTAs were needed: 35 us a call of 50021 x 1000 in
  // place of 26.)
  const unsigned piece = blockIdx.x / unsigned(a.parts), part = blockIdx.x - piece * a.parts;
  const Eight<kWide> at(int(part), a.width);
  const int n = a.starts[a.vocab];  // rows that count
  const int begin = int(piece) * a.piece;
  const int many = min(a.piece, n - begin);
  if (many <= 0) return;
  for (int i = threadIdx.x; i < many; i += blockDim.x) {
    rows[i] = a.order[begin + i];
    ids[i] = int(a.tokens[rows[i]]);
  }
  __syncthreads();
  const int head = ids[0], tail = ids[many - 1];
  const bool cut_begin = a.starts[head] < begin, cut_end = a.starts[tail + 1] > begin + many;
  const int carry_col = Eight<true>(int(part), a.width).col;  // a thread's eight sums lie together
  float* carry = a.carry + int64_t(piece) * 2 * a.carry_ld + carry_col;
  const auto keep = [&](int place, const float(&sum)[8]) {
    Raw<float> raw;
#pragma unroll
    for (int c = 0; c < 8; ++c) raw.w[c] = __float_as_uint(sum[c]);
    store_eight(carry + place * a.carry_ld, raw);
  };

  if (at.any()) {
    float sum[8] = {};
    int id = head;
    constexpr int kAhead = kWide ? 4 : 2;
    for (int i = 0; i < many; i += kAhead) {
      Raw<E> raw[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i + k < many) at.load(grad + rows[i + k] * a.grad_ld, raw[k]);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i + k >= many) break;
        if (ids[i + k] != id) {
          if (cut_begin && id == head) keep(0, sum);
          else put<Out, kWide, kKeep>(at, out + id * a.out_ld, sum, a.scale);
          id = ids[i + k];
#pragma unroll
          for (int c = 0; c < 8; ++c) sum[c] = 0.0f;
        }
        Pair v[4];
        widen(raw[k], v);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 p = split(v[c]);
          sum[2 * c] += p.x;
          sum[2 * c + 1] += p.y;
        }
      }
    }
    if (cut_end || (cut_begin && tail == head)) keep(tail == head ? 0 : 1, sum);
    else put<Out, kWide, kKeep>(at, out + tail * a.out_ld, sum, a.scale);
  }
  if (cut_begin || (cut_end && tail == head)) join_parts<Out, kWide, kKeep>(a, at, head, part, carry_col, out);
  if (cut_end && tail != head) join_parts<Out, kWide, kKeep>(a, at, tail, part, carry_col, out);
}

// ---- host ----------------------------------------------------------------------------

template <class E, class Out>
fadam_status forward(const fadam_embed& d, cudaStream_t stream) {
  const bool wide = eights(d.weight, d.weight_stride, d.width, sizeof(E)) &&
                    eights(d.out, d.out_stride, d.width, sizeof(Out));
  const Parts p = parts_of(d.width);
  // four rows to a thread where that leaves every SM four CTAs
  const bool many = ceil_div(d.rows, 4) * p.count >= kSms * 4;
  auto* kernel = wide ? (many ? gather_kernel<E, Out, true, 4> : gather_kernel<E, Out, true, 1>)
                      : (many ? gather_kernel<E, Out, false, 4> : gather_kernel<E, Out, false, 1>);
  return launch_chained("embedding launch", kernel, ceil_div(d.rows, many ? 4 : 1) * p.count, p.threads, 0,
                        stream, d.tokens, static_cast<const E*>(d.weight), d.weight_stride,
                        static_cast<Out*>(d.out), d.out_stride, d.rows, int(d.width), d.vocab,
                        d.padding_index, (d.flags & FADAM_EMBED_PADDING) != 0, d.scale, p.count);
}

struct Layout {
  int32_t* order;
  int32_t* starts;
  float* carry;
  int32_t* arrived;
  int32_t piece;
  int64_t pieces, carry_ld;
  size_t bytes;
};

Layout layout(const fadam_embed_grad& d, char* base) {
  Layout l{};
  Carver c{base};
  const Parts p = parts_of(d.width);
  // pieces as long as leave every SM eight CTAs, 4 to 64 rows
  const int64_t per = d.rows * p.count / (kSms * 8);
  l.piece = int32_t(per < 4 ? 4 : per > kLongest ? kLongest : per);
  l.pieces = ceil_div(d.rows, l.piece);
  l.carry_ld = int64_t(p.count) * p.threads * 8;
  l.order = static_cast<int32_t*>(c.take(4 * d.rows));
  l.starts = static_cast<int32_t*>(c.take(4 * (d.vocab + 1)));
  l.carry = static_cast<float*>(c.take(4 * 2 * l.pieces * l.carry_ld));
  l.arrived = static_cast<int32_t*>(c.take(4 * l.pieces * p.count));
  l.bytes = c.used;
  return l;
}

template <class E, class Out, bool kWide, bool kKeep>
fadam_status gradient(const fadam_embed_grad& d, const Layout& l, const DeviceFacts& dev,
                      cudaStream_t stream) {
  Out* out = static_cast<Out*>(d.out);
  SortArgs s{};
  s.tokens = d.tokens;
  s.rows = int32_t(d.rows);
  s.vocab = d.vocab;
  s.padding = d.padding_index;
  s.padded = (d.flags & FADAM_EMBED_PADDING) != 0;
  const int64_t even = ceil_div(d.vocab, dev.sm_count);
  s.range = int32_t(even < kRange ? even : kRange);
  s.order = l.order;
  s.starts = l.starts;
  const Parts p = parts_of(d.width);
  s.arrived = l.arrived;
  s.marks = int32_t(l.pieces * p.count);
  auto* sort = sort_kernel<Out, kWide, kKeep>;
  constexpr int kZeros = kKeep || !kWide ? 0 : kZeroBytes;
  const cudaError_t e = cudaFuncSetAttribute(sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kZeros + kSortWarps * kRange * 4);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  const fadam_status st =
      launch_chained("token sort launch", sort, ceil_div(d.vocab, s.range), kSortThreads,
                     kZeros + size_t(kSortWarps) * s.range * 4, stream, s, static_cast<Out*>(d.out), d.out_stride,
                     int(d.width));
  if (st) return st;
  SumArgs a{};
  a.tokens = d.tokens;
  a.order = l.order;
  a.starts = l.starts;
  a.vocab = d.vocab;
  a.width = int32_t(d.width);
  a.parts = p.count;
  a.piece = l.piece;
  a.grad_ld = d.grad_stride;
  a.out_ld = d.out_stride;
  a.carry_ld = l.carry_ld;
  a.carry = l.carry;
  a.arrived = l.arrived;
  a.scale = d.scale;
  return launch_chained("embedding sums launch", sum_kernel<E, Out, kWide, kKeep>, l.pieces * p.count, p.threads, 0,
                        stream, a, static_cast<const E*>(d.grad), out);
}

template <class E, class Out>
fadam_status gradient(const fadam_embed_grad& d, const Layout& l, const DeviceFacts& dev,
                      cudaStream_t stream) {
  const bool wide = eights(d.grad, d.grad_stride, d.width, sizeof(E)) &&
                    eights(d.out, d.out_stride, d.width, sizeof(Out));
  const bool keep = (d.flags & FADAM_EMBED_ACCUMULATE) != 0;
  if (wide)
    return keep ? gradient<E, Out, true, true>(d, l, dev, stream)
                : gradient<E, Out, true, false>(d, l, dev, stream);
  return keep ? gradient<E, Out, false, true>(d, l, dev, stream)
              : gradient<E, Out, false, false>(d, l, dev, stream);
}

bool finite(float x) { return x - x == 0.0f; }

// What both directions' descriptors have in common.
fadam_status check_common(int64_t rows, int64_t width, int64_t vocab, float scale) {
  if (rows < 0 || width < 1 || vocab < 1)
    return fail(FADAM_EINVAL, "%lld rows of width %lld over a vocabulary of %lld", (long long)rows,
                (long long)width, (long long)vocab);
  const int64_t most = int64_t(1) << 30;
  if (rows > most || width > most || vocab > most)
    return fail(FADAM_ELIMIT, "rows, width or vocab beyond 2^30");
  if (!finite(scale)) return fail(FADAM_EINVAL, "scale is not finite");
  return FADAM_OK;
}

fadam_status check(const fadam_embed* d) {
  if (!d) return fail(FADAM_EINVAL, "the descriptor is NULL");
  if (!elem_size(d->weight_dtype)) return fail(FADAM_EDTYPE, "dtype %d is not fp32, bf16 or fp16", d->weight_dtype);
  if (d->out_dtype != d->weight_dtype && d->out_dtype != FADAM_DT_F32)
    return fail(FADAM_EDTYPE, "out dtype %d is neither fp32 nor the weight's %d", d->out_dtype, d->weight_dtype);
  if (d->flags & ~FADAM_EMBED_PADDING) return fail(FADAM_EINVAL, "unknown flag bits 0x%x", d->flags);
  if (const fadam_status st = check_common(d->rows, d->width, d->vocab, d->scale)) return st;
  if (d->weight_stride < d->width || d->out_stride < d->width)
    return fail(FADAM_EINVAL, "a row stride is below the width %lld", (long long)d->width);
  if (!d->weight || (d->rows > 0 && (!d->tokens || !d->out)))
    return fail(FADAM_EINVAL, "tokens, weight and out must be non-NULL");
  if (misaligned(d->tokens, 8) || misaligned(d->weight, elem_size(d->weight_dtype)) ||
      misaligned(d->out, elem_size(d->out_dtype)))
    return fail(FADAM_EALIGN, "a pointer is not aligned to its element size");
  return FADAM_OK;
}

fadam_status check(const fadam_embed_grad* d) {
  if (!d) return fail(FADAM_EINVAL, "the descriptor is NULL");
  if (!elem_size(d->grad_dtype)) return fail(FADAM_EDTYPE, "dtype %d is not fp32, bf16 or fp16", d->grad_dtype);
  if (!elem_size(d->out_dtype) || (d->out_dtype != d->grad_dtype && d->out_dtype != FADAM_DT_F32 &&
                                   d->grad_dtype != FADAM_DT_F32))
    return fail(FADAM_EDTYPE, "out dtype %d with gradients of %d", d->out_dtype, d->grad_dtype);
  if (d->flags & ~(FADAM_EMBED_PADDING | FADAM_EMBED_ACCUMULATE))
    return fail(FADAM_EINVAL, "unknown flag bits 0x%x", d->flags);
  if (const fadam_status st = check_common(d->rows, d->width, d->vocab, d->scale)) return st;
  if (d->grad_stride < d->width || d->out_stride < d->width)
    return fail(FADAM_EINVAL, "a row stride is below the width %lld", (long long)d->width);
  if (!d->out || (d->rows > 0 && (!d->tokens || !d->grad)))
    return fail(FADAM_EINVAL, "tokens, grad and out must be non-NULL");
  if (misaligned(d->tokens, 8) || misaligned(d->grad, elem_size(d->grad_dtype)) ||
      misaligned(d->out, elem_size(d->out_dtype)))
    return fail(FADAM_EALIGN, "a pointer is not aligned to its element size");
  return FADAM_OK;
}

}  // namespace
}  // namespace fadam_ops

using namespace fadam_ops;

extern "C" fadam_status fadam_embed_forward(const fadam_embed* desc, fadam_stream stream_) {
  clear_error();
  const fadam_status st = check(desc);
  if (st || desc->rows == 0) return st;
  const fadam_embed& d = *desc;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const bool wide = d.out_dtype == FADAM_DT_F32;
  if (d.weight_dtype == FADAM_DT_BF16)
    return wide ? forward<__nv_bfloat16, float>(d, stream) : forward<__nv_bfloat16, __nv_bfloat16>(d, stream);
  if (d.weight_dtype == FADAM_DT_F16)
    return wide ? forward<__half, float>(d, stream) : forward<__half, __half>(d, stream);
  return forward<float, float>(d, stream);
}

extern "C" fadam_status fadam_embed_grad_workspace(const fadam_embed_grad* desc, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(FADAM_EINVAL, "bytes is NULL");
  const fadam_status st = check(desc);
  if (st) return st;
  *bytes = desc->rows == 0 ? 0 : layout(*desc, nullptr).bytes;
  return FADAM_OK;
}

extern "C" fadam_status fadam_embed_grad_run(const fadam_embed_grad* desc, void* workspace, size_t bytes,
                                             fadam_stream stream_) {
  clear_error();
  fadam_status st = check(desc);
  if (st) return st;
  const fadam_embed_grad& d = *desc;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (d.rows == 0) {
    if (d.flags & FADAM_EMBED_ACCUMULATE) return FADAM_OK;
    const int size = elem_size(d.out_dtype);
    const cudaError_t e = cudaMemset2DAsync(d.out, d.out_stride * size, 0, d.width * size, d.vocab, stream);
    return e == cudaSuccess ? FADAM_OK : cuda_fail(e, "cudaMemset2DAsync");
  }
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  const Layout l = layout(d, static_cast<char*>(workspace));
  if (!workspace || bytes < l.bytes)
    return fail(FADAM_EINVAL, "the workspace has %zu bytes, %zu are needed",
                workspace ? bytes : size_t(0), l.bytes);
  if (misaligned(workspace, 256)) return fail(FADAM_EALIGN, "the workspace is not 256-byte aligned");
  if (d.grad_dtype == FADAM_DT_BF16)
    return d.out_dtype == FADAM_DT_F32 ? gradient<__nv_bfloat16, float>(d, l, dev, stream)
                                       : gradient<__nv_bfloat16, __nv_bfloat16>(d, l, dev, stream);
  if (d.grad_dtype == FADAM_DT_F16)
    return d.out_dtype == FADAM_DT_F32 ? gradient<__half, float>(d, l, dev, stream)
                                       : gradient<__half, __half>(d, l, dev, stream);
  if (d.out_dtype == FADAM_DT_BF16) return gradient<float, __nv_bfloat16>(d, l, dev, stream);
  if (d.out_dtype == FADAM_DT_F16) return gradient<float, __half>(d, l, dev, stream);
  return gradient<float, float>(d, l, dev, stream);
}
