// Softmax cross entropy of x W^T over a large vocabulary, with its gradients.
//
//   z = x W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,y(t)
//   dz_tv = s (exp(z_tv - lse_t) - [v = y(t)]),  dx = dz W,  dW = dz^T x
//
// Three products on the tensor cores (gemm.cuh).  The first never writes a
// logit: a piece of (most often) 128 of a row's logits is reduced in registers to its
// maximum and its sum of exponentials, and (for the gradients) its
// exponentials relative to that maximum are kept in 16 bits.  Then a row's
// pieces are joined to its largest logit and its sum of exponentials, the kept
// ones are turned into dz in place, and two more products give dx and dW:
// 6 T V D operations where a second computation of the logits would make it 8.
// The kept exponentials are those of a chunk of rows, so the scratch memory is
// bounded however many rows there are.
//
// Roundings to 16 bits: the exponentials are kept in fp16 whatever the
// inputs' type (they are in [0, 1]; 2^-11 relative down to 6e-5 of the piece's
// largest, 3e-8 of that largest absolute below), dz once more in the inputs'
// type, because the tensor cores take it from there.  fp16 dz is held times
// 2^15 (|dz| <= 1 before s), so that this second rounding leaves a probability
// of 1e-8 all its bits; the first does so only where its piece's largest is not
// far above it: beside a logit that dominates the piece, a probability 10^8
// times smaller is 0.
// Everything else (products' sums, maxima, sums, lse, loss) is fp32; the
// factor s is applied to the fp32 sums.
#include "gemm_store.cuh"

namespace fadam_ops {
namespace {

struct Control {
  unsigned int finished;  // blocks of the current lse launch (the first product sets it to 0)
  float scale;            // loss_scale / (rows that count, if the mean is taken)
};

// What the first product's epilogue needs to reduce the logits.
struct LogitEpilogue {
  int64_t rows, pieces;
  int piece;         // columns of a piece
  const int64_t* targets;
  float2* stats;     // [rows, pieces]: maximum and sum of exponentials
  float* target_z;   // [rows]
  __half* kept;      // [rows, pitch] or NULL
  int64_t pitch;
  Control* control;

  __device__ __forceinline__ void begin() const { control->finished = 0; }
  __device__ __forceinline__ void operator()(const GemmPiece& p, float (&v)[kPiece]) const {
    const int64_t row = p.row0 + threadIdx.x % 32;
    const int64_t at = row < rows ? targets[row] - p.col : -1;
    if (at >= 0 && at < p.width) {
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) z = i == at ? v[i] : z;
      target_z[row] = z;
    }
    if (p.width < kPiece) {  // beyond the vocabulary (or the piece): as if the logit were -inf
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
        if (i >= p.width) v[i] = -INFINITY;
    }
    float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 4; i < kPiece; ++i) m[i % 4] = fmaxf(m[i % 4], v[i]);
    const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    const float base = top == -INFINITY ? 0.0f : top;  // nothing above -inf: all terms are 0
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      v[i] = exp2_fast((v[i] - base) * 1.4426950408889634f);
      sum[i % 4] += v[i];
    }
    if (row < rows)
      stats[row * pieces + p.col / piece] = make_float2(top, (sum[0] + sum[1]) + (sum[2] + sum[3]));
    if (kept) {
#pragma unroll
      for (int c = 0; c < kPiece; c += 64) {
        if (c >= p.width) break;
        float (&e)[64] = reinterpret_cast<float (&)[64]>(v[c]);
        emit_rows<8>(
            e, p, c, rows,
            [](const float* e) {
              return make_uint4(pack2<__half>(e[0], e[1]), pack2<__half>(e[2], e[3]),
                                pack2<__half>(e[4], e[5]), pack2<__half>(e[6], e[7]));
            },
            [&](int r, int col, uint4 u) {
              *reinterpret_cast<uint4*>(kept + (p.row0 + r) * pitch + p.col + col) = u;
            });
      }
    }
  }

  // 2^x for x <= 0; what is below 2^-126 is 0 (its share of a sum that is at
  // least 1 is below every rounding).
  static __device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
  }
};

struct RowArgs {
  int64_t rows, vocab, pieces, pitch, width, x_ld, kept_x_ld;
  int piece;                     // columns of a piece, a multiple of 16
  int64_t first_row, all_rows;   // of this chunk, and of the whole call
  const float2* stats;
  const float* target_z;
  float2* joined;                // [rows]: the row's largest logit, and its sum of exponentials
  const int64_t* targets;        // of the whole call
  int64_t ignore_index;
  float loss_scale;
  int mean;
  float* loss;
  float* row_loss;
  float* lse;
  void* dz;                      // [rows, pitch]: exponentials in, dz out
  const void* x;                 // [rows, width]
  void* kept_x;                  // x with ignored rows zero, or NULL
  float dz_scale;
  int segments;
  Control* control;
};

constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 2;  // vectors of eight per thread, and as many in flight

// A warp per row: lse and loss from the row's pieces.  The last block adds up
// the losses, in a fixed order, and counts the rows that count.
__global__ void __launch_bounds__(kRowThreads) lse_kernel(const __grid_constant__ RowArgs a) {
  __shared__ double sums[kRowThreads / 32];
  __shared__ int64_t counts[kRowThreads / 32];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid % 32;
  const int64_t row = int64_t(blockIdx.x) * (kRowThreads / 32) + tid / 32;
  chain_wait();
  chain_next();
  if (row < a.rows) {
    const float2* st = a.stats + row * a.pieces;
    // eight pieces to a lane at a time, all on their way at once
    float top = -INFINITY;
    for (int64_t i = lane; i < a.pieces; i += 8 * 32) {
      float t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) t[u] = i + u * 32 < a.pieces ? st[i + u * 32].x : -INFINITY;
#pragma unroll
      for (int u = 0; u < 8; ++u) top = fmaxf(top, t[u]);
    }
#pragma unroll
    for (int i = 16; i; i /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, i));
    const float base = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (int64_t i = lane; i < a.pieces; i += 8 * 32) {
      float2 p[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        p[u] = i + u * 32 < a.pieces ? st[i + u * 32] : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += p[u].y * expf(p[u].x - base);  // (a piece of -inf alone: 0 * 0)
    }
#pragma unroll
    for (int i = 16; i; i /= 2) sum += __shfl_xor_sync(~0u, sum, i);
    if (lane == 0) {
      const int64_t target = a.targets[a.first_row + row];
      a.joined[row] = make_float2(base, sum);
      const float log_sum = logf(sum);
      a.lse[a.first_row + row] = base + log_sum;
      // not lse - z: lse is rounded to a unit of its own size (10^-3 at 12800), which
      // can be more than a confident row's whole loss; dz has base and sum for the
      // same reason.  A target outside the vocabulary shows as NaN in both.
      a.row_loss[a.first_row + row] = target == a.ignore_index                ? 0.0f
                                      : target >= 0 && target < a.vocab ? (base - a.target_z[row]) + log_sum
                                                                              : NAN;
      __threadfence();
    }
  }
  __syncthreads();
  if (tid == 0) last = atomicAdd(&a.control->finished, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  // the losses of the rows so far (of all of them in the last chunk), and how
  // many rows of the whole call count
  __threadfence();
  double loss = 0.0;
  int64_t count = 0;
  for (int64_t i = tid; i < a.all_rows; i += 8 * kRowThreads) {
    float l[8];
    int64_t t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t at = i + u * kRowThreads;
      l[u] = at < a.first_row + a.rows ? __ldcg(a.row_loss + at) : 0.0f;
      t[u] = at < a.all_rows ? a.targets[at] : a.ignore_index;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      loss += l[u];
      count += t[u] != a.ignore_index;
    }
  }
#pragma unroll
  for (int i = 16; i; i /= 2) {
    loss += __shfl_xor_sync(~0u, loss, i);
    count += __shfl_xor_sync(~0u, count, i);
  }
  if (lane == 0) {
    sums[tid / 32] = loss;
    counts[tid / 32] = count;
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kRowThreads / 32; ++i) {
      loss += sums[i];
      count += counts[i];
    }
    const double share = a.mean ? 1.0 / double(count > 0 ? count : 1) : 1.0;
    *a.loss = float(loss * share);
    a.control->scale = float(a.loss_scale * share);
  }
}

// dz in place of the kept exponentials, and the row of x that dW's product
// reads (a row that is ignored must not reach dW even where x is not finite:
// 0 * inf is NaN).  A block per row, or `segments` of them, each with a share
// of the row.  Bound by memory, 2 bytes in and out for each exponential: 8192
// rows of 131072 take 718 us (6.0 TB/s) with two vectors of a thread in flight,
// 765 us with four.
template <class T>
__global__ void __launch_bounds__(kRowThreads) dz_kernel(const __grid_constant__ RowArgs a) {
  using E = typename T::type;
  // the last rows first: the product before has left them in L2, and the one
  // after begins with the first
  const unsigned block = gridDim.x - 1 - blockIdx.x;
  const int64_t row = block / unsigned(a.segments);
  const int segment = int(block % unsigned(a.segments));
  const int tid = threadIdx.x;
  const float2* st = a.stats + row * a.pieces;
  const int all_vectors = int((a.vocab + 7) / 8);
  const int begin = int(int64_t(all_vectors) * segment / a.segments);
  const int vectors = int(int64_t(all_vectors) * (segment + 1) / a.segments);  // the segment's end
  uint4* dz = reinterpret_cast<uint4*>(static_cast<__half*>(a.dz) + row * a.pitch);

  chain_wait();
  chain_next();
  const int64_t target = a.targets[a.first_row + row];
  const bool ignored = target == a.ignore_index;
  const bool valid = target >= 0 && target < a.vocab;
  if (ignored) {
    for (int c = begin + tid; c < vectors; c += kRowThreads) dz[c] = make_uint4(0, 0, 0, 0);
  } else {
    uint4 raw[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u)
      if (begin + tid + u * kRowThreads < vectors) raw[u] = dz[begin + tid + u * kRowThreads];
    const float2 joined = a.joined[row];
    const float scale = valid ? a.dz_scale / joined.y : NAN;
    const int target_vector = valid ? int(target / 8) : -1;
    // vector c lies in piece c / per_piece; both advance with c
    const int per_piece = a.piece / 8;
    const int step = kRowThreads / per_piece, step_rest = kRowThreads % per_piece;
    int piece = (begin + tid) / per_piece, rest = (begin + tid) % per_piece;
    for (int first = begin + tid; first < vectors; first += kRowUnroll * kRowThreads) {
      uint4 now[kRowUnroll];
#pragma unroll
      for (int u = 0; u < kRowUnroll; ++u) {
        now[u] = raw[u];
        const int ahead = first + (kRowUnroll + u) * kRowThreads;
        if (ahead < vectors) raw[u] = dz[ahead];
      }
#pragma unroll
      for (int u = 0; u < kRowUnroll; ++u) {
        const int c = first + u * kRowThreads;
        if (c < vectors) {
          const float f = scale * exp2f((st[piece].x - joined.x) * 1.4426950408889634f);
          const uint32_t w[4] = {now[u].x, now[u].y, now[u].z, now[u].w};
          uint32_t out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 e = unpack2<__half>(w[i]);
            out[i] = pack2<E>(e.x * f, e.y * f);
          }
          dz[c] = make_uint4(out[0], out[1], out[2], out[3]);
          if (c == target_vector) {  // this thread has the target
            const uint32_t pair = target & 4 ? (target & 2 ? w[3] : w[2]) : (target & 2 ? w[1] : w[0]);
            const float2 e = unpack2<__half>(pair);
            reinterpret_cast<E*>(dz)[target] = from_float<E>((target & 1 ? e.y : e.x) * f - a.dz_scale);
          }
        }
        piece += step;
        rest += step_rest;
        if (rest >= per_piece) {
          rest -= per_piece;
          ++piece;
        }
      }
    }
  }
  if (a.kept_x && segment == 0) {
    const E* from = static_cast<const E*>(a.x) + row * a.x_ld;
    E* to = static_cast<E*>(a.kept_x) + row * a.kept_x_ld;
    const int whole = int(a.width / 8);
    for (int i = tid; i < whole; i += kRowThreads)
      reinterpret_cast<uint4*>(to)[i] =
          ignored ? make_uint4(0, 0, 0, 0) : reinterpret_cast<const uint4*>(from)[i];
    if (tid < a.width % 8)
      to[whole * 8 + tid] = ignored ? from_float<E>(0.0f) : from[whole * 8 + tid];
  }
}

// Rows copied to where bulk copies can read them (16-byte aligned rows).
template <class E>
__global__ void __launch_bounds__(256) align_rows_kernel(const E* from, int64_t from_ld, E* to,
                                                         int64_t to_ld, int64_t rows, int64_t width) {
  chain_wait();
  chain_next();
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (int64_t i = threadIdx.x; i < width; i += 256) to[row * to_ld + i] = from[row * from_ld + i];
}

// ---- host ------------------------------------------------------------------------

struct Layout {
  int64_t chunk, chunks, pieces, pitch, width_ld;
  GemmPlan logits, dx, dw;
  Control* control;
  float2* stats;
  float* target_z;
  float2* joined;
  void* kept;
  void* kept_x;
  void* x_rows;   // aligned copies, where the caller's rows are not
  void* w_rows;
  float* parts;
  float* carry;
  size_t bytes;
};

// Rows of one chunk: as many as keep the exponentials within 4 GiB (the loss
// alone: the pieces' maxima and sums within 1 GiB), in whole tiles.  (One chunk
// of 8192 rows x 131072 entries is 2 GiB; a second chunk costs dW's fp32 sum
// one more trip through memory.)
int64_t chunk_rows(const fadam_xent& d) {
  const bool grads = d.grad_x || d.grad_w;
  if (grads && d.chunk_rows > 0) return d.chunk_rows < d.rows ? d.chunk_rows : d.rows;
  const int64_t fit = grads ? (int64_t(4) << 30) / (round_up(d.vocab, 64) * 2)
                            : (int64_t(1) << 30) / (ceil_div(d.vocab, 32) * int64_t(sizeof(float2)));
  const int64_t whole = fit / kTileM * kTileM;
  const int64_t chunk = whole < kTileM ? kTileM : whole;
  return chunk < d.rows ? chunk : d.rows;
}

Layout layout(const fadam_xent& d, char* base, int sm_count) {
  Layout l{};
  Carver c{base};
  const bool grads = d.grad_x || d.grad_w;
  l.chunk = chunk_rows(d);
  l.chunks = ceil_div(d.rows, l.chunk);
  const int pairs = sm_count / 2;
  l.logits = plan_gemm(l.chunk, d.vocab, d.width, false, false, pairs);
  l.dx = plan_gemm(l.chunk, d.width, d.vocab, true, true, pairs);
  l.dw = plan_gemm(d.vocab, d.width, l.chunk, true, true, pairs);
  l.pieces = ceil_div(d.vocab, l.logits.tile_n / 2);
  l.pitch = round_up(d.vocab, 64);
  l.width_ld = round_up(d.width, 8);
  l.control = static_cast<Control*>(c.take(sizeof(Control)));
  l.stats = static_cast<float2*>(c.take(sizeof(float2) * l.chunk * l.pieces));
  l.target_z = static_cast<float*>(c.take(sizeof(float) * l.chunk));
  l.joined = static_cast<float2*>(c.take(sizeof(float2) * l.chunk));
  if (grads) l.kept = c.take(2 * l.chunk * l.pitch);
  if (d.grad_w) l.kept_x = c.take(2 * l.chunk * l.width_ld);
  if (!bulk_readable(d.x, d.x_stride)) l.x_rows = c.take(2 * d.rows * l.width_ld);
  if (!bulk_readable(d.w, d.w_stride)) l.w_rows = c.take(2 * d.vocab * l.width_ld);
  size_t parts = d.grad_x ? split_bytes(l.chunk, l.dx) : 0;
  if (d.grad_w && split_bytes(d.vocab, l.dw) > parts) parts = split_bytes(d.vocab, l.dw);
  if (parts) l.parts = static_cast<float*>(c.take(parts));
  if (d.grad_w && l.chunks > 1) l.carry = static_cast<float*>(c.take(4 * d.vocab * scratch_ld(d.width)));
  l.bytes = c.used;
  return l;
}

template <class T>
fadam_status align_rows(const void* from, int64_t from_ld, void* to, int64_t to_ld, int64_t rows,
                        int64_t width, cudaStream_t stream) {
  using E = typename T::type;
  return launch_chained("row copy launch", align_rows_kernel<E>, rows < 8192 ? rows : 8192, 256, 0, stream,
                        static_cast<const E*>(from), from_ld, static_cast<E*>(to), to_ld, rows, width);
}

template <class T, class OutW>
fadam_status run(const fadam_xent& d, const Layout& l, const DeviceFacts& dev, cudaStream_t stream) {
  using E = typename T::type;
  const bool grads = d.grad_x || d.grad_w;
  const E* x = static_cast<const E*>(d.x);
  const E* w = static_cast<const E*>(d.w);
  int64_t x_ld = d.x_stride, w_ld = d.w_stride;
  fadam_status st;
  if (l.x_rows) {
    if ((st = align_rows<T>(d.x, d.x_stride, l.x_rows, l.width_ld, d.rows, d.width, stream))) return st;
    x = static_cast<const E*>(l.x_rows);
    x_ld = l.width_ld;
  }
  if (l.w_rows) {
    if ((st = align_rows<T>(d.w, d.w_stride, l.w_rows, l.width_ld, d.vocab, d.width, stream))) return st;
    w = static_cast<const E*>(l.w_rows);
    w_ld = l.width_ld;
  }
  CUtensorMap w_k, w_mn;
  if ((st = matrix_map(&w_k, w, d.vocab, d.width, w_ld, box_rows(false, l.logits.tile_n / 2)))) return st;
  if ((st = matrix_map(&w_mn, w, d.vocab, d.width, w_ld, box_rows(true, 0)))) return st;
  // fp16 dz is held times 2^15
  const float dz_scale = T::code == FADAM_DT_F16 ? 32768.0f : 1.0f;

  for (int64_t first = 0; first < d.rows; first += l.chunk) {
    const int64_t rows = d.rows - first < l.chunk ? d.rows - first : l.chunk;
    const bool last_chunk = first + rows == d.rows;
    CUtensorMap map;
    GemmShape shape = gemm_shape(rows, d.vocab, d.width, l.logits, dev.status);
    // Over 4096 of k, lse is off by 1.5e-6 of itself with one chunk, 3.5e-7 with
    // chunks of 16 steps, 6e-8 with four.  One row of tiles waits for memory and
    // four cost it nothing; 2048 x 32000 logits take 277, 278 and 306 us.
    shape.chunk = shape.m_tiles == 1 ? 4 : 16;
    if ((st = matrix_map(&map, x + first * x_ld, rows, d.width, x_ld, box_rows(false, shape.a_box))))
      return st;
    LogitEpilogue epi{rows, l.pieces, l.logits.tile_n / 2, d.targets + first, l.stats, l.target_z,
                      static_cast<__half*>(l.kept), l.pitch, l.control};
    if ((st = launch_gemm<T, false, false>(map, w_k, shape, epi, dev.sm_count, stream))) return st;

    RowArgs r{};
    r.rows = rows;
    r.vocab = d.vocab;
    r.pieces = l.pieces;
    r.piece = l.logits.tile_n / 2;
    r.pitch = l.pitch;
    r.width = d.width;
    r.x_ld = x_ld;
    r.kept_x_ld = l.width_ld;
    r.first_row = first;
    r.all_rows = d.rows;
    r.stats = l.stats;
    r.target_z = l.target_z;
    r.joined = l.joined;
    r.targets = d.targets;
    r.ignore_index = d.ignore_index;
    r.loss_scale = d.loss_scale;
    r.mean = (d.flags & FADAM_XENT_MEAN) != 0;
    r.loss = d.loss;
    r.row_loss = d.row_loss;
    r.lse = d.lse;
    r.dz = l.kept;
    r.x = x + first * x_ld;
    r.kept_x = l.kept_x;
    r.dz_scale = dz_scale;
    r.control = l.control;
    if ((st = launch_chained("lse launch", lse_kernel, ceil_div(rows, kRowThreads / 32), kRowThreads, 0,
                             stream, r)))
      return st;
    if (!grads) continue;
    // eight blocks to an SM at least, each with 1024 vectors or more
    const int64_t most = ceil_div(d.vocab, 8 * 1024), few = ceil_div(8 * dev.sm_count, rows);
    r.segments = int(few < most ? few : most);
    if ((st = launch_chained("dz launch", dz_kernel<T>, rows * r.segments, kRowThreads, 0, stream, r)))
      return st;

    if (d.grad_x) {
      shape = gemm_shape(rows, d.width, d.vocab, l.dx, dev.status);
      if ((st = matrix_map(&map, l.kept, rows, d.vocab, l.pitch, box_rows(false, shape.a_box)))) return st;
      StoreArgs s{};
      s.out = static_cast<E*>(d.grad_x) + first * d.grad_x_stride;
      s.ld = d.grad_x_stride;
      s.m = rows;
      s.n = d.width;
      s.scale = &l.control->scale;
      s.constant = 1.0f / dz_scale;
      s.targets = d.targets + first;
      s.ignore_index = d.ignore_index;
      s.wide = wide_stores(s.out, s.ld, 2);
      if ((st = store_product<T, false, true, T>(map, w_mn, shape, s, l.parts, dev.sm_count, stream)))
        return st;
    }
    if (d.grad_w) {
      CUtensorMap x_mn;
      if ((st = matrix_map(&map, l.kept, rows, d.vocab, l.pitch, box_rows(true, 0)))) return st;
      if ((st = matrix_map(&x_mn, l.kept_x, rows, d.width, l.width_ld, box_rows(true, 0)))) return st;
      StoreArgs s{};
      s.out = d.grad_w;
      s.ld = d.grad_w_stride;
      s.m = d.vocab;
      s.n = d.width;
      s.scale = &l.control->scale;
      s.constant = 1.0f / dz_scale;
      s.carry = l.carry;
      s.read_carry = first > 0;
      s.write_carry = !last_chunk;
      s.accumulate = (d.flags & FADAM_XENT_ACCUMULATE) != 0;
      s.wide = wide_stores(s.out, s.ld, sizeof(typename OutW::type));
      shape = gemm_shape(d.vocab, d.width, rows, l.dw, dev.status);
      if ((st = store_product<T, true, true, OutW>(map, x_mn, shape, s, l.parts, dev.sm_count, stream)))
        return st;
    }
  }
  return FADAM_OK;
}

fadam_status check(const fadam_xent* d) {
  if (!d) return fail(FADAM_EINVAL, "the descriptor is NULL");
  if (!is_16bit(d->dtype)) return fail(FADAM_EDTYPE, "dtype %d is not bf16 or fp16", d->dtype);
  if (d->grad_w && d->grad_w_dtype != d->dtype && d->grad_w_dtype != FADAM_DT_F32)
    return fail(FADAM_EDTYPE, "grad_w dtype %d is neither fp32 nor the inputs' %d", d->grad_w_dtype,
                d->dtype);
  if (d->flags & ~(FADAM_XENT_MEAN | FADAM_XENT_ACCUMULATE))
    return fail(FADAM_EINVAL, "unknown flag bits 0x%x", d->flags);
  if (d->rows < 0 || d->width < 1 || d->vocab < 1 || d->chunk_rows < 0)
    return fail(FADAM_EINVAL, "%lld rows of width %lld over a vocabulary of %lld, chunk %lld",
                (long long)d->rows, (long long)d->width, (long long)d->vocab,
                (long long)d->chunk_rows);
  const int64_t most = int64_t(1) << 30;
  if (d->rows > most || d->width > most || d->vocab > most)
    return fail(FADAM_ELIMIT, "rows, width or vocab beyond 2^30");
  if (d->x_stride < d->width || d->w_stride < d->width ||
      (d->grad_x && d->grad_x_stride < d->width) || (d->grad_w && d->grad_w_stride < d->width))
    return fail(FADAM_EINVAL, "a row stride is below the width %lld", (long long)d->width);
  if (!d->loss || !d->w || (d->rows > 0 && (!d->x || !d->targets || !d->row_loss || !d->lse)))
    return fail(FADAM_EINVAL, "x, w, targets, loss, row_loss and lse must be non-NULL");
  if (misaligned(d->x, 2) || misaligned(d->w, 2) || misaligned(d->grad_x, 2) ||
      misaligned(d->grad_w, elem_size(d->grad_w ? d->grad_w_dtype : d->dtype)) ||
      misaligned(d->targets, 8) || misaligned(d->loss, 4) || misaligned(d->row_loss, 4) ||
      misaligned(d->lse, 4))
    return fail(FADAM_EALIGN, "a pointer is not aligned to its element size");
  if (!(d->loss_scale == d->loss_scale) || d->loss_scale - d->loss_scale != 0.0f)
    return fail(FADAM_EINVAL, "loss_scale is not finite");
  return FADAM_OK;
}

}  // namespace
}  // namespace fadam_ops

using namespace fadam_ops;

extern "C" fadam_status fadam_xent_workspace(const fadam_xent* desc, size_t* bytes) {
  clear_error();
  if (!bytes) return fail(FADAM_EINVAL, "bytes is NULL");
  fadam_status st = check(desc);
  if (st) return st;
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  *bytes = desc->rows == 0 ? 0 : layout(*desc, nullptr, dev.sm_count).bytes;
  return FADAM_OK;
}

extern "C" fadam_status fadam_xent_run(const fadam_xent* desc, void* workspace, size_t bytes,
                                       fadam_stream stream_) {
  clear_error();
  fadam_status st = check(desc);
  if (st) return st;
  const fadam_xent& d = *desc;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (d.rows == 0) {  // nothing to learn from: no loss, and no gradient unless one is there
    cudaError_t e = cudaMemsetAsync(d.loss, 0, sizeof(float), stream);
    if (e == cudaSuccess && d.grad_w && !(d.flags & FADAM_XENT_ACCUMULATE))
      e = cudaMemset2DAsync(d.grad_w, d.grad_w_stride * elem_size(d.grad_w_dtype), 0,
                            d.width * elem_size(d.grad_w_dtype), d.vocab, stream);
    return e == cudaSuccess ? FADAM_OK : cuda_fail(e, "cudaMemsetAsync");
  }
  DeviceFacts dev;
  if ((st = device_facts(&dev))) return st;
  const Layout l = layout(d, static_cast<char*>(workspace), dev.sm_count);
  if (!workspace || bytes < l.bytes)
    return fail(FADAM_EINVAL, "the workspace has %zu bytes, %zu are needed",
                workspace ? bytes : size_t(0), l.bytes);
  if (misaligned(workspace, 256)) return fail(FADAM_EALIGN, "the workspace is not 256-byte aligned");
  const bool wide_w = d.grad_w && d.grad_w_dtype == FADAM_DT_F32;
  if (d.dtype == FADAM_DT_BF16)
    return wide_w ? run<BF16, F32>(d, l, dev, stream) : run<BF16, BF16>(d, l, dev, stream);
  return wide_w ? run<F16, F32>(d, l, dev, stream) : run<F16, F16>(d, l, dev, stream);
}
