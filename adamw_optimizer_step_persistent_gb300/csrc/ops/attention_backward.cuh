// Attention, backward: with p = exp(s - lse) and
//   ds = p (grad_out . v - delta) ds/d(q . k),  delta = grad_out . out,
//   grad_v_j = sum_i p_ij grad_out_i,  grad_k_j = sum_i ds_ij q_i,
//   grad_q_i = sum_j ds_ij k_j.
//
// Two kinds of CTAs, each of which keeps one side in shared memory, walks over the
// other and sums in tensor memory, so that every sum has one order and nothing
// is added to memory: one takes 128 keys and walks over the queries that see
// them, of all query heads that share the key head (four products a tile: the
// transposed scores, grad_out . v, grad_v, grad_k); one takes 128 queries
// (three products).  Computing the scores twice costs seven products in place
// of five, where grad_q summed in memory would cost fp32 additions to it from
// every tile, in the order in which they arrive.
//
// Both are pipelined in the same way: sixteen warps turn scores into p and p
// into ds (four lanes to a row, 32 columns each) while the tensor cores do the
// products of the tile before and the scores of the next one.  p and ds go back
// to tensor memory in 16 bits, as the A operand of their products.
// Tiles are taken as they come: keys from the first one on, queries from the last
// one back, which is by their work where there is one sequence, and neighbours
// find what they share in L2 where there are several.  (By their work, 8
// sequences of 2048 with 16 heads took 487 us in place of 433, 5 of 777 with 12
// heads of 64 61.4 in place of 59.6, 4 of 1024 130.2 and 130.6.)
// (A warp may be a turn ahead of another one when it has written ds, which is
// why that has a barrier for even and one for odd turns.)
//
// Bound by the tensor cores: a turn of keys takes 2600 cycles, its products alone
// 2236; one of queries 2000, alone 1700 to 1940.  8192 causal tokens, 32 heads of
// 128, bf16: 1210 to 1250 us in a graph (26 of them the statistics), 1.1 PFLOP/s of
// the five products that a pass cannot do without, 1.6 of the seven; 1333 to 1360
// back to back, at the card's power limit.
#pragma once

#include "attention.cuh"

namespace fadam_ops {

// Tiles in flight of what a kernel walks over: X is needed by the scores and by
// the product with ds, Y by grad_out . v (and the product with p).
constexpr int kRingX = 3, kRingY = 2;
// fp16: p is held times 2^10 (the smallest normal number is 2^-14), ds times a
// power of two for each row, a query's where grad_q is summed, a key's where
// grad_k is: see ds_exponent().
template <class T>
constexpr int kLiftBits = T::code == FADAM_DT_F16 ? 10 : 0;

struct BackwardBarriers {
  uint64_t own_full, done;
  uint64_t x_full[kRingX], x_empty[kRingX], y_full[kRingY], y_empty[kRingY];
  uint64_t scores, dots;        // tensor cores: S, grad_out . v are there
  uint64_t scores_read, dots_read, weights;          // warps: S and dots read, p written
  uint64_t slopes[2];                                // ds written, of even and odd turns
  Reach reach[4];
  uint32_t tmem;
};
struct BackwardExtra {
  float lse[kRingY][kRows];     // with Y: read for p, before Y is done with
  float delta[kRingX][kRows];   // with X
  int8_t exponent[kRows];       // of the rows' ds, for the end
  BackwardBarriers bars;
};
template <int C>
constexpr size_t kBackwardSmem = (2 + kRingX + kRingY) * C * size_t(kBoxBytes) + sizeof(BackwardExtra);
static_assert(kBackwardSmem<2> <= 227 * 1024, "shared memory of one CTA");
constexpr int kColumnsS = 0, kColumnsDots = kRows, kColumnsA = 2 * kRows, kColumnsB = 3 * kRows;

// A bound of a row's ds: |p (go . v - delta)| is at most go's largest magnitude
// times the sum of v's, and |delta|.  Of the key `token` of a key head by what
// its document holds, so that one of small gradients keeps its bits beside one of
// large ones; of the query `token` of a head by its own grad_out and delta.
template <class T>
__device__ __forceinline__ float key_bound(const AttentionArgs& g, int kv, int token) {
  if constexpr (T::code != FADAM_DT_F16) return 0.0f;
  const int64_t kv_heads = g.heads / g.group, apart = kv_heads * g.entries;
  const unsigned* at = g.peaks + int64_t(kv) * g.entries + entry_of(g, token).at;
  return fmaf(__uint_as_float(at[0]), __uint_as_float(at[2 * apart]), __uint_as_float(at[apart]));
}
template <class T>
__device__ __forceinline__ float query_bound(const AttentionArgs& g, int head, int token) {
  if constexpr (T::code != FADAM_DT_F16) return 0.0f;
  const int64_t kv_heads = g.heads / g.group, pitch = int64_t(g.tiles) * kRows;
  const unsigned v = g.peaks[(2 * kv_heads + head / g.group) * g.entries + entry_of(g, token).at];
  const float delta = fabsf(g.stats[(g.heads + head) * pitch + token]);
  return fmaf(g.stats[(2 * int64_t(g.heads) + head) * pitch + token], __uint_as_float(v),
              delta < INFINITY ? delta : 0.0f);
}
// The exponent of a power of two that brings the bound to [2^14, 2^15): no ds is
// then infinite in fp16, whatever v holds, and one of 2^-28 of the bound is
// still a normal number.  (A bound is 0 or between 2^-48 and 2^42.)
__device__ __forceinline__ int ds_exponent(float bound) {
  return bound > 0.0f ? 14 + 127 - int(__float_as_uint(bound) >> 23) : 0;
}
__device__ __forceinline__ float power_of_two(int exponent) { return __uint_as_float(unsigned(127 + exponent) << 23); }

template <class T, int C>
struct Backward {
  static constexpr int kTile = C * kBoxBytes;
  uint32_t own0, own1, x, y;   // shared addresses of the tiles
  BackwardExtra* extra;
  BackwardBarriers* bars;

  // Sets up barriers and tensor memory, for one or two multiplying warps (which
  // both have to be done with an X).  False when shared memory does not
  // start on 1024 bytes, as the swizzle needs.
  __device__ __forceinline__ bool begin(unsigned char* smem, const AttentionArgs& g, int multiplying) {
    own0 = shared_addr(smem);
    if (own0 & 1023) {
      if (threadIdx.x == 0) atomicExch(g.status, FADAM_ECUDA);
      return false;
    }
    own1 = own0 + kTile;
    x = own1 + kTile;
    y = x + kRingX * kTile;
    extra = reinterpret_cast<BackwardExtra*>(smem + (2 + kRingX + kRingY) * kTile);
    bars = &extra->bars;
    if (threadIdx.x == kLoad * 32) {
      bar_init(shared_addr(&bars->own_full), 1);
      bar_init(shared_addr(&bars->done), multiplying);
      for (int i = 0; i < kRingX; ++i) {
        bar_init(shared_addr(&bars->x_full[i]), 1);
        bar_init(shared_addr(&bars->x_empty[i]), multiplying);
      }
      for (int i = 0; i < kRingY; ++i) {
        bar_init(shared_addr(&bars->y_full[i]), 1);
        bar_init(shared_addr(&bars->y_empty[i]), 1);
      }
      bar_init(shared_addr(&bars->scores), 1);
      bar_init(shared_addr(&bars->dots), 1);
      bar_init(shared_addr(&bars->scores_read), kScoreWarps);
      bar_init(shared_addr(&bars->dots_read), kScoreWarps);
      bar_init(shared_addr(&bars->weights), kScoreWarps);
      bar_init(shared_addr(&bars->slopes[0]), kScoreWarps);
      bar_init(shared_addr(&bars->slopes[1]), kScoreWarps);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x / 32 == kMultiply) tmem_alloc(shared_addr(&bars->tmem), 512);
    return true;
  }

  // What a row's ds (2^10 of it, fp16) is multiplied by, and its sums at the end.
  // (The four lanes of a row write the same: each reads what it wrote itself.)
  // Of a row that is `alone`, whose weights are 1 whatever its scores, the sums are 0
  // but for what grad_out . v and delta differ by in their roundings.
  static constexpr int kAlone = -128;
  __device__ __forceinline__ float keep_factor(int row, float bound, bool alone) const {
    const int exponent = T::code == FADAM_DT_F16 ? ds_exponent(bound) : 0;
    extra->exponent[row] = int8_t(alone ? kAlone : exponent);
    return T::code == FADAM_DT_F16 ? power_of_two(exponent - kLiftBits<T>) : 1.0f;
  }
  __device__ __forceinline__ float inverse_factor(int row) const {
    const int exponent = extra->exponent[row];
    return exponent == kAlone ? 0.0f : power_of_two(-exponent);
  }

  // What the 128 rows of the CTA need: rows are dealt to the first four warps.
  __device__ __forceinline__ Reach meet(int lo, int hi, bool here) const {
    const int warp = threadIdx.x / 32;
    if (warp < 4) {
      const Reach r = reach_of(lo, hi, here);
      if (threadIdx.x % 32 == 0) bars->reach[warp] = r;
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    return uniform(join(join(bars->reach[0], bars->reach[1]), join(bars->reach[2], bars->reach[3])));
  }

  __device__ __forceinline__ uint32_t x_at(int at) const { return x + at * kTile; }
  __device__ __forceinline__ uint32_t y_at(int at) const { return y + at * kTile; }
  __device__ __forceinline__ bool wait_x(const Place<kRingX>& p, int* status) const {
    return warp_wait(shared_addr(&bars->x_full[p.at]), p.parity, status);
  }
  __device__ __forceinline__ bool wait_y(const Place<kRingY>& p, int* status) const {
    return warp_wait(shared_addr(&bars->y_full[p.at]), p.parity, status);
  }

  // The loading thread: the CTA's own two tiles, while the others find out what
  // they need, then X and Y of n turns in turn.  load_x(dst, slot, bar).
  __device__ __forceinline__ void load_own(const CUtensorMap* map0, const CUtensorMap* map1, int head,
                                           int token) const {
    if (threadIdx.x != kLoad * 32) return;
    const uint32_t bar = shared_addr(&bars->own_full);
    bar_expect(bar, 2 * kTile);
    load_head<C>(own0, map0, head, token, bar);
    load_head<C>(own1, map1, head, token, bar);
  }
  template <class X, class Y>
  __device__ __forceinline__ void load_loop(int n, int x_extra, int y_extra, int* status, X load_x,
                                            Y load_y) const {
    bool ok = true;
    Place<kRingX> px;  // an empty place passes for the parity before the first phase's
    Place<kRingY> py;
    for (int i = 0; i < n; ++i, px.next(), py.next()) {
      ok = bar_wait(shared_addr(&bars->x_empty[px.at]), px.parity ^ 1, status);
      if (!ok) break;
      uint32_t bar = shared_addr(&bars->x_full[px.at]);
      bar_expect(bar, kTile + x_extra);
      load_x(x_at(px.at), px.at, bar);
      ok = bar_wait(shared_addr(&bars->y_empty[py.at]), py.parity ^ 1, status);
      if (!ok) break;
      bar = shared_addr(&bars->y_full[py.at]);
      bar_expect(bar, kTile + y_extra);
      load_y(y_at(py.at), py.at, bar);
    }
    // every copy has landed and been used when the CTA ends
    bar_wait(shared_addr(&bars->own_full), 0, status);
    for (int i = 0; i < kRingX; ++i, px.next())
      bar_wait(shared_addr(&bars->x_empty[px.at]), px.parity ^ 1, status);
    for (int i = 0; i < kRingY; ++i, py.next())
      bar_wait(shared_addr(&bars->y_empty[py.at]), py.parity ^ 1, status);
  }
};

// Which of 32 columns a lane's row does not see: those below lo, where a row
// of the tile is cut there, and those from hi on.
struct Cut {
  bool below, above;
  int lo, hi;
  __device__ __forceinline__ Cut(const Reach& r, int tile, int column, int span_lo, int span_hi)
      : below(r.all_lo > tile), above(r.all_hi < tile + kRows), lo(span_lo - column), hi(span_hi - column) {}
  // (one side at a time: most tiles that need a mask are cut on one)
  __device__ __forceinline__ void set(float (&v)[32], float to) const {
    if (below)
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = c >= lo ? v[c] : to;
    if (above)
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = c < hi ? v[c] : to;
  }
};

// 32 columns of scores of a lane's row, but for a factor `mul`, become p (times
// 2^lift), in 16 bits, and p times ds/d(q . k) in place: with a cap 1 - tanh^2,
// from the capped scores, without their bias by distance (kBias).
template <class E, bool kCap, bool kBias, class Lse>
__device__ __forceinline__ void weights_of(float (&s)[32], uint32_t (&p)[16], const Scores& f, float mul,
                                           float apart, Lse lse) {
  const Pair mul_pair = both(mul), less = both(kCap ? -1.0f / (f.cap * f.cap) : 0.0f);
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    const Pair z = make_pair(s[c], s[c + 1]);
    const float2 e = split(fma2(z, mul_pair, lse(c)));
    Pair w = make_pair(exp2_fast(e.x), exp2_fast(e.y));
    float2 v = split(w);
    p[c / 2] = pack2<E>(v.x, v.y);
    if constexpr (kCap) {
      Pair capped = z;
      if constexpr (kBias)
        capped = make_pair(fmaf(f.slope, fabsf(apart + float(c)), s[c]),
                           fmaf(f.slope, fabsf(apart + float(c + 1)), s[c + 1]));
      w = mul2(w, fma2(mul2(capped, capped), less, both(1.0f)));
      v = split(w);
    }
    s[c] = v.x;
    s[c + 1] = v.y;
  }
}
// From products q . k.  lse(c): what is added to columns c and c + 1; `apart`:
// the first column's place less the row's.  (What is not seen becomes p = 0, and
// any value in place.)
template <class E, class Lse>
__device__ __forceinline__ void weights(float (&s)[32], uint32_t (&p)[16], const Scores& f, float apart,
                                        const Cut& cut, Lse lse) {
  const float mul = f.finish<true>(s, apart);
  cut.set(s, -INFINITY);
  if (f.cap == 0.0f) weights_of<E, false, false>(s, p, f, mul, apart, lse);
  else if (f.slope == 0.0f) weights_of<E, true, false>(s, p, f, mul, apart, lse);
  else weights_of<E, true, true>(s, p, f, mul, apart, lse);
}

// 32 columns of ds: p (at s) times (grad_out . v - delta), `delta(c)` added to
// columns c and c + 1; fp16 times the row's `factor`.  What is not seen is set to 0.
template <class T, class Delta>
__device__ __forceinline__ void slopes_of(float (&s)[32], const float (&d)[32], uint32_t (&p)[16], float factor,
                                          const Cut& cut, Delta delta) {
  const Pair factor_pair = both(factor);
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    Pair e = mul2(make_pair(s[c], s[c + 1]), add2(make_pair(d[c], d[c + 1]), delta(c)));
    if constexpr (T::code == FADAM_DT_F16) e = mul2(e, factor_pair);
    const float2 v = split(e);
    s[c] = v.x;
    s[c + 1] = v.y;
  }
  cut.set(s, 0.0f);
#pragma unroll
  for (int c = 0; c < 32; c += 2) p[c / 2] = pack2<typename T::type>(s[c], s[c + 1]);
}

// ---- grad_k and grad_v: 128 keys, a walk over queries --------------------------------------

template <class T, int C>
__device__ __forceinline__ void keys_cta(unsigned char* smem, const BackwardMaps& maps, const AttentionArgs& g,
                                         unsigned item) {
  using E = typename T::type;
  Backward<T, C> b;
  if (!b.begin(smem, g, 1)) return;
  const int warp = uniform(int(threadIdx.x / 32)), lane = threadIdx.x % 32;
  BackwardBarriers* bars = b.bars;
  int* status = g.status;
  chain_wait();

  const unsigned kv_heads = unsigned(g.heads / g.group), columns = kv_heads * g.splits;
  const int tile = int(item / columns);
  const int rest = int(item % columns);
  const int kv = rest / g.splits, split = rest % g.splits;
  const int share = g.group / g.splits, head0 = kv * g.group + split * share;
  const int key0 = tile * kRows;
  const int row = threadIdx.x % kRows;  // of the first sixteen warps: a lane's key
  Spans span{};
  if (warp < kScoreWarps && key0 + row < g.tokens) span = spans_of(g, key0 + row);
  float bound = 0.0f;
  if (warp < kScoreWarps) bound = key_bound<T>(g, kv, key0 + row);  // (on its way while the CTA meets)
  // a document of one token
  const bool alone = span.query_hi - span.query_lo == 1 && span.key_hi - span.key_lo == 1;
  b.load_own(&maps.k, &maps.v, kv, key0);
  const Reach reach = b.meet(span.query_lo, span.query_hi, key0 + row < g.tokens);
  const uint32_t tmem = uniform(bars->tmem);
  const int first = reach.first(), turns = reach.last() - first, n = turns * share;

  if (warp >= kScoreWarps) keep_registers<kOtherRegisters>();
  if (warp == kIdle) {
  } else if (warp == kLoad) {
    if (lane == 0) {
      const int64_t pitch = int64_t(g.tiles) * kRows;
      const float* lse = g.stats;
      const float* delta = g.stats + pitch * g.heads;
      int head = head0, at = first;  // of the turn: a tile of queries
      b.load_loop(
          n, kRows * 4, kRows * 4, status,
          [&](uint32_t dst, int slot, uint32_t bar) {
            load_head<C>(dst, &maps.q, head, at * kRows, bar);
            load_bytes(shared_addr(b.extra->delta[slot]), delta + head * pitch + at * kRows, kRows * 4, bar);
          },
          [&](uint32_t dst, int slot, uint32_t bar) {
            load_head<C>(dst, &maps.grad_out, head, at * kRows, bar);
            load_bytes(shared_addr(b.extra->lse[slot]), lse + head * pitch + at * kRows, kRows * 4, bar);
            if (++at == first + turns) {
              at = first;
              ++head;
            }
          });
    }
  } else if (warp == kMultiply) {
    // One warp: while the scores' warps work on ds(i), grad_v and the scores of
    // i + 1 are computed, then, while they work on p(i + 1), grad_k and
    // grad_out . v.  (Two warps, one for each pair of products, ran them at the
    // same time, and p(i + 1) waited for both: 3600 cycles a turn.)
    if (n > 0) {
      const int steps = (g.width + 15) / 16, width = steps * 16;
      const uint32_t bar_weights = shared_addr(&bars->weights);
      const auto scores = [&](int at) {
        mma_scores<T, C>(tmem + kColumnsS, b.own0, b.x_at(at), steps);
        commit(shared_addr(&bars->scores));
      };
      const auto dots = [&](int at) {
        mma_scores<T, C>(tmem + kColumnsDots, b.own1, b.y_at(at), steps);
        commit(shared_addr(&bars->dots));
      };
      Place<kRingX> x, next_x;
      Place<kRingY> y, next_y;
      int query = first;  // the tile of next_x and next_y
      const auto clean = [&](uint32_t at) {
        if (g.documents) clean_rows<C>(at, query * kRows, g);
      };
      bool ok = warp_wait(shared_addr(&bars->own_full), 0, status) && b.wait_x(x, status) && b.wait_y(y, status);
      if (ok) {
        clean(b.x_at(0));
        clean(b.y_at(0));
        fence_after_sync();
        if (elect_one()) {
          scores(0);
          dots(0);
        }
      }
      for (int i = 0; ok && i < n; ++i) {
        const bool more = i + 1 < n;
        next_x.next();
        next_y.next();
        if (++query == first + turns) query = first;
        if (more) {
          ok = b.wait_x(next_x, status);
          if (ok) clean(b.x_at(next_x.at));
        }
        ok = ok && warp_wait(bar_weights, unsigned(i) & 1, status);
        if (!ok) break;
        fence_after_sync();
        if (elect_one()) {
          mma_rows<T, 32>(tmem + kColumnsA, tmem + kColumnsS, 32, b.y_at(y.at), width, i > 0);
          commit(shared_addr(&bars->y_empty[y.at]));
          if (more) scores(next_x.at);
        }
        ok = warp_wait(shared_addr(&bars->slopes[i & 1]), unsigned(i / 2) & 1, status);
        if (!ok) break;
        fence_after_sync();
        if (elect_one()) {
          mma_rows<T, 32>(tmem + kColumnsB, tmem + kColumnsDots, 32, b.x_at(x.at), width, i > 0);
          commit(shared_addr(&bars->x_empty[x.at]));
        }
        if (more) {
          // (not before grad_k's product: Y's place was given back only a turn ago)
          ok = b.wait_y(next_y, status);
          if (!ok) break;
          clean(b.y_at(next_y.at));
          fence_after_sync();
          if (elect_one()) dots(next_y.at);
        }
        x = next_x;
        y = next_y;
      }
      if (ok && elect_one()) commit(shared_addr(&bars->done));
    }
  } else if (warp < kScoreWarps) {
    take_registers<kScoreRegisters>();
    const int part = warp / 4, quarter = warp % 4;  // part: of the columns
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t at_s = lanes + kColumnsS + part * 32, at_dots = lanes + kColumnsDots + part * 32;
    const uint32_t bar_scores = shared_addr(&bars->scores), bar_dots = shared_addr(&bars->dots);
    const uint32_t bar_weights = shared_addr(&bars->weights);
    const float factor = b.keep_factor(row, bound, alone);
    bool ok = true;
    Place<kRingX> x;
    Place<kRingY> y;
    for (int h = 0, i = 0; h < share && ok; ++h) {
      const Scores f(g, head0 + h);
      for (int turn = 0; turn < turns; ++turn, ++i, x.next(), y.next()) {
        const int tile_at = (first + turn) * kRows, at = tile_at + part * 32;  // the first column's query
        const Cut cut(reach, tile_at, at, span.query_lo, span.query_hi);
        float s[32];
        uint32_t p[16];
        Pair of[16];  // the columns' lse, then their delta: read before the tensor cores are waited for
        ok = b.wait_y(y, status);
        if (!ok) break;
        load_pairs(shared_addr(b.extra->lse[y.at] + part * 32), of);
        ok = warp_wait(bar_scores, unsigned(i) & 1, status);
        if (!ok) break;
        fence_after_sync();
        tmem_load32(at_s, s);
        tmem_wait<32>(s);
        weights<E>(s, p, f, float(at - (key0 + row)), cut, [&](int c) { return of[c / 2]; });
        tmem_store16(at_s, p);
        tmem_stored();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) bar_arrive(bar_weights);

        ok = b.wait_x(x, status);
        if (!ok) break;
        load_pairs(shared_addr(b.extra->delta[x.at] + part * 32), of);
        ok = warp_wait(bar_dots, unsigned(i) & 1, status);
        if (!ok) break;
        fence_after_sync();
        float d[32];
        tmem_load32(at_dots, d);
        tmem_wait<32>(d);
        const auto delta = [&](int c) { return of[c / 2]; };
        slopes_of<T>(s, d, p, factor, cut, delta);
        tmem_store16(at_dots, p);
        tmem_stored();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) bar_arrive(shared_addr(&bars->slopes[i & 1]));
      }
    }
    // eight warps write grad_v (through v's place in shared memory), eight
    // grad_k, half of the elements to four warps
    if (ok) ok = warp_wait(shared_addr(n > 0 ? &bars->done : &bars->own_full), 0, status);
    fence_after_sync();
    const bool keys = part >= 2;
    const float scale = keys ? g.scale * b.inverse_factor(row) : power_of_two(-kLiftBits<T>);
    const uint32_t from = lanes + (keys ? kColumnsB : kColumnsA);
    const uint32_t tile_at = keys ? b.own0 : b.own1;
    const uint32_t place = tile_at + (quarter * 32 + lane) * 128;
    float* sums = nullptr;
    if (g.splits > 1)
      sums = g.parts + (((int64_t(split) * 2 + keys) * g.tokens + key0 + row) * kv_heads + kv) * g.width;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int c = (part % 2 * C + k) * 32;
      if (c >= g.width) continue;
      float o[32];
      if (n > 0) {
        tmem_load32(from + c, o);
        tmem_wait<32>(o);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = n > 0 ? o[i] * scale : 0.0f;
      if (sums) {
        if (key0 + row < g.tokens)
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            if (c + i < g.width) {
              reinterpret_cast<float4*>(sums + c + i)[0] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
              reinterpret_cast<float4*>(sums + c + i)[1] = make_float4(o[i + 4], o[i + 5], o[i + 6], o[i + 7]);
            }
      } else {
        store_units<E>(place, c, o);
      }
    }
    if (!sums) {
      fence_shared();
      group_sync(1 + keys, 256);
      if (threadIdx.x % 256 == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c * kChunk < g.width)
            store_head_box(keys ? &maps.grad_k : &maps.grad_v, c * kChunk, kv, key0, tile_at + c * kBoxBytes);
        wait_stores();
      }
    }
  }
  __syncwarp();
  chain_next();
  fence_before_sync();
  __syncthreads();
  if (warp == kMultiply) tmem_free(tmem, 512);
}

// ---- grad_q: 128 queries, a walk over keys ------------------------------------------------

template <class T, int C>
__device__ __forceinline__ void queries_cta(unsigned char* smem, const BackwardMaps& maps, const AttentionArgs& g,
                                            unsigned item) {
  using E = typename T::type;
  Backward<T, C> b;
  if (!b.begin(smem, g, 2)) return;
  const int warp = uniform(int(threadIdx.x / 32)), lane = threadIdx.x % 32;
  BackwardBarriers* bars = b.bars;
  int* status = g.status;
  chain_wait();

  const int head = int(item % unsigned(g.heads));
  const int query0 = (g.tiles - 1 - int(item / unsigned(g.heads))) * kRows;
  const int row = threadIdx.x % kRows;
  Spans span{};
  if (warp < kScoreWarps && query0 + row < g.tokens) span = spans_of(g, query0 + row);
  float bound = 0.0f;
  if (warp < kScoreWarps) bound = query_bound<T>(g, head, query0 + row);
  const bool alone = span.key_hi - span.key_lo == 1;
  b.load_own(&maps.q, &maps.grad_out, head, query0);
  const Reach reach = b.meet(span.key_lo, span.key_hi, query0 + row < g.tokens);
  const uint32_t tmem = uniform(bars->tmem);
  const int first = reach.first(), n = reach.last() - first;

  if (warp >= kScoreWarps) keep_registers<kOtherRegisters>();
  if (warp == kIdle) {
  } else if (warp == kLoad) {
    if (lane == 0) {
      const int kv = head / g.group;
      int x_key = first * kRows, y_key = x_key;
      const auto keys = [&](uint32_t dst, int, uint32_t bar) {
        load_head<C>(dst, &maps.k, kv, x_key, bar);
        x_key += kRows;
      };
      const auto values = [&](uint32_t dst, int, uint32_t bar) {
        load_head<C>(dst, &maps.v, kv, y_key, bar);
        y_key += kRows;
      };
      b.load_loop(n, 0, 0, status, keys, values);
    }
  } else if (warp == kMultiply2) {
    // scores
    if (n > 0) {
      const int steps = (g.width + 15) / 16;
      const uint32_t bar_read = shared_addr(&bars->scores_read);
      Place<kRingX> x;
      bool ok = warp_wait(shared_addr(&bars->own_full), 0, status);
      for (int i = 0; ok && i < n; ++i, x.next()) {
        ok = b.wait_x(x, status) && (i == 0 || warp_wait(bar_read, unsigned(i - 1) & 1, status));
        if (!ok) break;
        fence_after_sync();
        if (elect_one()) {
          mma_scores<T, C>(tmem + kColumnsS, b.own0, b.x_at(x.at), steps);
          commit(shared_addr(&bars->scores));
          commit(shared_addr(&bars->x_empty[x.at]));
        }
      }
      if (ok && elect_one()) commit(shared_addr(&bars->done));
    }
  } else if (warp == kMultiply) {
    // grad_out . v of a turn, then grad_q of the one before
    if (n > 0) {
      const int steps = (g.width + 15) / 16, width = steps * 16;
      const uint32_t bar_read = shared_addr(&bars->dots_read);
      Place<kRingX> x;
      Place<kRingY> y;
      const auto dots = [&] {
        mma_scores<T, C>(tmem + kColumnsDots, b.own1, b.y_at(y.at), steps);
        commit(shared_addr(&bars->dots));
        commit(shared_addr(&bars->y_empty[y.at]));
      };
      bool ok = warp_wait(shared_addr(&bars->own_full), 0, status) && b.wait_y(y, status);
      fence_after_sync();
      if (ok && elect_one()) dots();
      for (int i = 0; ok && i < n; ++i, x.next()) {
        if (i + 1 < n) {
          y.next();
          ok = b.wait_y(y, status) && warp_wait(bar_read, unsigned(i) & 1, status);
          if (!ok) break;
          fence_after_sync();
          if (elect_one()) dots();
        }
        ok = b.wait_x(x, status) && warp_wait(shared_addr(&bars->slopes[i & 1]), unsigned(i / 2) & 1, status);
        if (!ok) break;
        if (g.documents) clean_rows<C>(b.x_at(x.at), (first + i) * kRows, g);
        fence_after_sync();
        if (elect_one()) {
          mma_rows<T, 128>(tmem + kColumnsB, tmem + kColumnsA + (i & 1) * 64, 0, b.x_at(x.at), width, i > 0);
          commit(shared_addr(&bars->x_empty[x.at]));
        }
      }
      if (ok && elect_one()) commit(shared_addr(&bars->done));
    }
  } else if (warp < kScoreWarps) {
    take_registers<kScoreRegisters>();
    const int part = warp / 4, quarter = warp % 4;  // part: of the columns
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t at_s = lanes + kColumnsS + part * 32, at_dots = lanes + kColumnsDots + part * 32;
    const uint32_t bar_scores = shared_addr(&bars->scores), bar_dots = shared_addr(&bars->dots);
    const uint32_t bar_scores_read = shared_addr(&bars->scores_read);
    const uint32_t bar_dots_read = shared_addr(&bars->dots_read);
    const float factor = b.keep_factor(row, bound, alone);
    const int64_t pitch = int64_t(g.tiles) * kRows;
    const Pair lse = both(g.stats[head * pitch + query0 + row]);
    const Pair delta = both(g.stats[(g.heads + head) * pitch + query0 + row]);
    const Scores f(g, head);
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int tile_at = (first + i) * kRows, at = tile_at + part * 32;  // the first column's key
      const Cut cut(reach, tile_at, at, span.key_lo, span.key_hi);
      float s[32];
      uint32_t p[16];
      ok = warp_wait(bar_scores, unsigned(i) & 1, status);
      if (!ok) break;
      fence_after_sync();
      tmem_load32(at_s, s);
      tmem_wait<32>(s);
      fence_before_sync();
      __syncwarp();
      if (lane == 0) bar_arrive(bar_scores_read);
      weights<E>(s, p, f, float(at - (query0 + row)), cut, [&](int) { return lse; });

      ok = warp_wait(bar_dots, unsigned(i) & 1, status);
      if (!ok) break;
      fence_after_sync();
      float d[32];
      tmem_load32(at_dots, d);
      tmem_wait<32>(d);
      fence_before_sync();
      __syncwarp();
      if (lane == 0) bar_arrive(bar_dots_read);
      const auto less = [&](int) { return delta; };
      slopes_of<T>(s, d, p, factor, cut, less);
      // (grad_out . v of i comes behind the product with ds of i - 2: its place is free)
      tmem_store16(lanes + kColumnsA + (i & 1) * 64 + part * 16, p);
      tmem_stored();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) bar_arrive(shared_addr(&bars->slopes[i & 1]));
    }
    if (ok) ok = warp_wait(shared_addr(n > 0 ? &bars->done : &bars->own_full), 0, status);
    fence_after_sync();
    const float scale = g.scale * b.inverse_factor(row);
    const uint32_t place = b.own0 + (quarter * 32 + lane) * 128;
    // a quarter of the elements to four warps, C * 16 each
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int c = (part * C + k) * 16;
      if (c >= g.width) continue;
      float o[16];
      if (n > 0) {
        tmem_load16(lanes + kColumnsB + c, o);
        tmem_wait<16>(o);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = n > 0 ? o[i] * scale : 0.0f;
      store_units<E>(place, c, o);
    }
    fence_shared();
    group_sync(1, kScoreWarps * 32);
    if (threadIdx.x == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * kChunk < g.width)
          store_head_box(&maps.grad_q, c * kChunk, head, query0, b.own0 + c * kBoxBytes);
      wait_stores();
    }
  }
  __syncwarp();
  chain_next();
  fence_before_sync();
  __syncthreads();
  if (warp == kMultiply) tmem_free(tmem, 512);
}

// ---- both, in one launch -------------------------------------------------------------------

// The first CTAs take keys, the others queries, which get the SMs that the last
// of those leave.  (Two launches, of which the second one's CTAs started under
// the first one's end without a wait of their own, read what the launches
// before both had written, and nothing but their own wait makes that visible.)
template <class T, int C>
__global__ void __launch_bounds__(kAttentionThreads, 1)
    attention_backward_kernel(const __grid_constant__ BackwardMaps maps, const __grid_constant__ AttentionArgs g) {
  extern __shared__ __align__(1024) unsigned char smem[];
  if (blockIdx.x < g.key_items) keys_cta<T, C>(smem, maps, g, blockIdx.x);
  else queries_cta<T, C>(smem, maps, g, blockIdx.x - g.key_items);
}

template <class T, int C>
fadam_status launch_backward(const BackwardMaps& maps, AttentionArgs g, cudaStream_t stream) {
  auto* kernel = attention_backward_kernel<T, C>;
  if (const fadam_status st = launched_with<attention_backward_kernel<T, C>>("attention's backward pass")) return st;
  constexpr int kShared = int(kBackwardSmem<C>);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  // (tiles times heads are at most 2^30, and the key heads' splits no more than the heads: unsigned holds both)
  g.key_items = unsigned(int64_t(g.tiles) * (g.heads / g.group) * g.splits);
  return launch_chained("attention backward launch", kernel, g.key_items + int64_t(g.tiles) * g.heads,
                        kAttentionThreads, kShared, stream, maps, g);
}
template <class T>
fadam_status backward_of(const BackwardMaps& maps, const AttentionArgs& g, cudaStream_t stream) {
  return g.width <= kChunk ? launch_backward<T, 1>(maps, g, stream) : launch_backward<T, 2>(maps, g, stream);
}

}  // namespace fadam_ops
