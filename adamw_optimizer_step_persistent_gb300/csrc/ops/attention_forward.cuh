// Attention, forward.
//
// A CTA takes two tiles of 128 queries and walks over the keys that any of them
// sees, 128 at a time, once.  The tiles are the same rows of two query heads
// that share their keys, where an even number of heads does (they see the same
// keys, so that no turn is one tile's alone: 4096 packed tokens of 32 heads over
// 8 took 79 us with 256 rows of one head, 72 so), else 256 consecutive rows of
// one head.
//
// A turn: S = Q K^T on the tensor cores; two lanes to a query (of two warps, 64
// columns each: eight warps to a tile) take the row's maximum, exponentials and
// sum in registers and hand the exponentials, in 16 bits, back to tensor memory;
// O += P V.  Tensor memory: scores and O of both tiles (4 x 128 columns); P lies
// over the scores it came from.
//
// The two tiles take turns: while one's scores are worked on, the tensor cores
// work for the other, each fed by a warp of its own.  (One warp for both left
// them idle during its waits: 4000 cycles a turn of both tiles.)  The two pass a
// token: left alone, both tiles' products ran at the same time, and then both
// tiles' scores were worked on at the same time (4040; 3230 with the token).
//
// Bound by the chain of a tile's turn, some 1300 cycles for the scores and 1500
// for its two products: from shared memory both operands of Q K^T come at 687
// cycles for 128 x 128 x 128 where P V's one takes 569 and the tensor cores
// alone would take 512.  8192 causal tokens, 32 heads of 128, bf16: 382 us in a
// graph, 1.44 PFLOP/s of what is not masked, 410 back to back; tensor cores 59% active.
//
// The running maximum of a row need not be its true maximum: any reference
// gives the same quotient.  So O (in tensor memory) and the sum are only
// rescaled when the maximum has grown by more than 2^8, which after the first
// keys of a row hardly ever happens; exponentials stay below 2^8, in fp16 below
// 2^15, of which 2^7 keep small ones from its subnormals.
#pragma once

#include "attention.cuh"

namespace fadam_ops {

constexpr int kRing = 2;              // pairs of a tile of keys and one of values in flight
constexpr float kGrowth = 8.0f;

struct ForwardBarriers {
  uint64_t q_full[2], scores[2], weights[2], done[2];
  uint64_t go[2];             // the tensor cores are this tile's
  uint64_t k_full[kRing], k_empty[kRing], v_full[kRing], v_empty[kRing];
  Reach reach[8];
  float shared[2][2][kRows];  // what the two lanes of a row tell each other: tile, half, row
  uint32_t tmem;
};
template <int C>
constexpr size_t kForwardSmem = 1024 + (2 + 2 * kRing) * C * size_t(kBoxBytes) + sizeof(ForwardBarriers);

// (Capped scores have an instance of their own: with what they take in its loop the
// others' 8192 tokens took 405 us in a graph in place of 390.)
template <class T, int C, bool kCap>
__global__ void __launch_bounds__(kAttentionThreads, 1)
    attention_forward_kernel(const __grid_constant__ ForwardMaps maps, const __grid_constant__ AttentionArgs g) {
  using E = typename T::type;
  constexpr int kTile = C * kBoxBytes;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t q_tiles = (shared_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t ring = q_tiles + 2 * kTile;
  ForwardBarriers* bars =
      reinterpret_cast<ForwardBarriers*>(smem_raw + (ring + 2 * kRing * kTile - shared_addr(smem_raw)));
  const int warp = uniform(int(threadIdx.x / 32)), lane = threadIdx.x % 32;

  if (warp == kMultiply) tmem_alloc(shared_addr(&bars->tmem), 512);
  const unsigned columns = unsigned(g.pair_heads ? g.heads / 2 : g.heads);
  const int items = g.pair_heads ? g.tiles : (g.tiles + 1) / 2;
  if (warp == kLoad && lane == 0) {
    for (int t = 0; t < 2; ++t) {
      bar_init(shared_addr(&bars->q_full[t]), 1);
      bar_init(shared_addr(&bars->scores[t]), 1);
      bar_init(shared_addr(&bars->weights[t]), 8);
      bar_init(shared_addr(&bars->done[t]), 1);
      bar_init(shared_addr(&bars->go[t]), 1);
    }
    for (int i = 0; i < kRing; ++i) {
      bar_init(shared_addr(&bars->k_full[i]), 1);
      bar_init(shared_addr(&bars->v_full[i]), 1);
      bar_init(shared_addr(&bars->k_empty[i]), 2);  // both multiplying warps
      bar_init(shared_addr(&bars->v_empty[i]), 2);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  chain_wait();
  const int place = int(blockIdx.x / columns), item = g.order ? g.order[place] : items - 1 - place;
  const int head0 = int(blockIdx.x % columns) << g.pair_heads, row0 = item * kRows << (g.pair_heads ^ 1);
  const auto head_of = [&](int t) { return head0 + (t & g.pair_heads); };
  const auto row_of = [&](int t) { return row0 + (g.pair_heads ? 0 : t * kRows); };
  if (warp == kLoad && lane == 0) {
    // the queries, while the others find out which keys they see
    for (int t = 0; t < 2; ++t) {
      const uint32_t bar = shared_addr(&bars->q_full[t]);
      bar_expect(bar, kTile);
      load_head<C>(q_tiles + t * kTile, &maps.q, head_of(t), row_of(t), bar);
    }
  }
  // warps of scores: four and four to a tile, each four with half the columns
  const int tile = warp / 8 & 1, half = warp / 4 & 1, quarter = warp % 4;
  const int row = row_of(tile) + quarter * 32 + lane;
  Spans span{};
  if (warp < kScoreWarps) {
    if (row < g.tokens) span = spans_of(g, row);
    const Reach r = reach_of(span.key_lo, span.key_hi, row < g.tokens);
    if (lane == 0 && half == 0) bars->reach[tile * 4 + quarter] = r;
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = uniform(bars->tmem);
  Reach reach[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
    reach[t] = uniform(join(join(bars->reach[4 * t], bars->reach[4 * t + 1]),
                            join(bars->reach[4 * t + 2], bars->reach[4 * t + 3])));
  const int first = min(reach[0].first(), reach[1].first());
  const int last = max(reach[0].hi > reach[0].lo ? reach[0].last() : 0,
                       reach[1].hi > reach[1].lo ? reach[1].last() : 0);

  if (warp >= kScoreWarps) keep_registers<kOtherRegisters>();
  if (warp == kIdle) {
  } else if (warp == kLoad) {
    // ---- loads: keys and values in turn
    if (lane == 0) {
      const int kv = head0 / g.group;
      bool ok = true;
      Place<kRing> pair;  // an empty place passes for the parity before the first phase's
      for (int j = first; j < last; ++j, pair.next()) {
        ok = bar_wait(shared_addr(&bars->k_empty[pair.at]), pair.parity ^ 1, g.status);
        if (!ok) break;
        const uint32_t k_bar = shared_addr(&bars->k_full[pair.at]), v_bar = shared_addr(&bars->v_full[pair.at]);
        bar_expect(k_bar, kTile);
        load_head<C>(ring + 2 * pair.at * kTile, &maps.k, kv, j * kRows, k_bar);
        ok = bar_wait(shared_addr(&bars->v_empty[pair.at]), pair.parity ^ 1, g.status);
        if (!ok) break;
        bar_expect(v_bar, kTile);
        load_head<C>(ring + (2 * pair.at + 1) * kTile, &maps.v, kv, j * kRows, v_bar);
      }
      // every copy has landed and been used when the CTA ends
      for (int i = 0; i < kRing; ++i, pair.next()) {
        bar_wait(shared_addr(&bars->k_empty[pair.at]), pair.parity ^ 1, g.status);
        bar_wait(shared_addr(&bars->v_empty[pair.at]), pair.parity ^ 1, g.status);
      }
      for (int t = 0; t < 2; ++t) bar_wait(shared_addr(&bars->q_full[t]), 0, g.status);
    }
  } else if (warp == kMultiply || warp == kMultiply2) {
    // ---- tensor cores: a warp to a tile of queries
    const int t = warp == kMultiply ? 0 : 1;
    const Reach mine = t ? reach[1] : reach[0];
    if (first < last) {
      const int steps = (g.width + 15) / 16, n = steps * 16;
      const uint32_t queries = q_tiles + t * kTile, at_s = tmem + t * kRows, at_o = tmem + (2 + t) * kRows;
      const uint32_t bar_scores = shared_addr(&bars->scores[t]), bar_weights = shared_addr(&bars->weights[t]);
      const int begin = mine.first(), end = mine.last();
      const uint32_t my_go = shared_addr(&bars->go[t]), other_go = shared_addr(&bars->go[t ^ 1]);
      // the scores of j, and this warp's part in giving the keys' place back; the
      // other tile's products may follow from half way through
      const auto scores = [&](int j, int at) {
        if (j >= begin && j < end) {
          mma_scores<T, C>(at_s, queries, ring + 2 * at * kTile, steps, [&] { bar_arrive(other_go); });
          commit(bar_scores);
        } else {
          bar_arrive(other_go);
        }
        commit(shared_addr(&bars->k_empty[at]));
      };
      Place<kRing> keys, values;
      bool ok = warp_wait(shared_addr(&bars->k_full[0]), 0, g.status);
      if (ok && begin < end) ok = warp_wait(shared_addr(&bars->q_full[t]), 0, g.status);
      if (ok && t == 1) ok = warp_wait(my_go, 0, g.status);
      fence_after_sync();
      if (ok && elect_one()) scores(first, 0);
      keys.next();
      unsigned turn = 0, go = t;  // tile 0 of j comes behind tile 1's scores of j, tile 1 behind tile 0's of j + 1
      for (int j = first; ok && j < last; ++j) {
        const bool here = j >= begin && j < end, more = j + 1 < last;
        const uint32_t v_at = ring + (2 * values.at + 1) * kTile;
        ok = warp_wait(shared_addr(&bars->v_full[values.at]), values.parity, g.status);
        if (ok && more) ok = warp_wait(shared_addr(&bars->k_full[keys.at]), keys.parity, g.status);
        if (ok && here) {
          if (g.documents) clean_rows<C>(v_at, j * kRows, g);
          ok = warp_wait(bar_weights, turn, g.status);
          turn ^= 1;
        }
        ok = ok && warp_wait(my_go, go, g.status);
        go ^= 1;
        if (!ok) break;
        fence_after_sync();
        if (elect_one()) {
          if (here) {
            mma_rows<T, 64>(at_o, at_s, 64, v_at, n, j > begin);
            if (j + 1 == end) commit(shared_addr(&bars->done[t]));
          }
          commit(shared_addr(&bars->v_empty[values.at]));
          if (more) {
            scores(j + 1, keys.at);
          } else {
            bar_arrive(other_go);
          }
        }
        keys.next();
        values.next();
      }
    }
  } else {
    // ---- softmax: two lanes to a query, 64 columns each
    take_registers<kScoreRegisters>();
    const int t = tile, head = head_of(t), pair = 1 + warp / 8 * 4 + quarter;  // pair: their warps' barrier
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t at_s = lanes + t * kRows + half * 64;
    const uint32_t at_o = lanes + (2 + t) * kRows + half * C * 32;  // half of O's columns
    const int o_width = g.width - half * C * 32;
    const uint32_t bar_scores = shared_addr(&bars->scores[t]), bar_weights = shared_addr(&bars->weights[t]);
    float* told = &bars->shared[t][half][quarter * 32 + lane];
    const float* other = &bars->shared[t][half ^ 1][quarter * 32 + lane];
    const Scores f(g, head);
    constexpr float kLift = T::code == FADAM_DT_F16 ? 7.0f : 0.0f;
    float top = -INFINITY, sum = 0.0f;   // top: the reference that exponents are relative to
    bool ok = true;
    const Reach mine = t ? reach[1] : reach[0];
    const int begin = mine.first(), end = mine.last();
    for (int j = begin; j < end; ++j) {
      // (after a wait that gave up the turns go on without waiting: the two warps
      // of a pair must meet as often)
      ok = ok && warp_wait(bar_scores, unsigned(j - begin) & 1, g.status);
      fence_after_sync();
      float s[64];
      tmem_load32(at_s, s);
      tmem_load32(at_s + 32, s + 32);
      tmem_wait<64>(s);
      const int at = j * kRows + half * 64;  // the first column's key
      const float mul = f.finish<kCap>(s, float(at - row));
      // (most tiles that need a mask are cut on one side)
      if (mine.all_hi < (j + 1) * kRows) {
        const int hi = span.key_hi - at;
#pragma unroll
        for (int c = 0; c < 64; ++c) s[c] = c < hi ? s[c] : -INFINITY;
      }
      if (mine.all_lo > j * kRows) {
        const int lo = span.key_lo - at;
#pragma unroll
        for (int c = 0; c < 64; ++c) s[c] = c >= lo ? s[c] : -INFINITY;
      }
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 64; c += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = fmaxf(fmaxf(m[k], s[c + k]), s[c + 4 + k]);
      float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * mul;
      if (group_any(pair, 64, most > top + kGrowth)) {
        // (scores of j come behind the product with the values of j - 1: O is at rest)
        *told = most;
        group_sync(pair, 64);
        most = fmaxf(most, *other);
        // (a row that has not grown itself keeps its reference, and with it its bits)
        const float now = most > top + kGrowth ? most : top;
        const float factor = now == -INFINITY ? 1.0f : exp2_fast(top - now);
        top = now;
        sum *= factor;
        if (j > begin) {
#pragma unroll
          for (int c = 0; c < C * 32; c += 16)
            if (c < o_width) {
              float o[16];
              tmem_load16(at_o + c, o);
              tmem_wait<16>(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= factor;
              tmem_store16(at_o + c, reinterpret_cast<uint32_t*>(o));
            }
        }
      }
      const float from = top == -INFINITY ? 0.0f : top - kLift;
      const Pair mul_pair = both(mul), less = both(-from);
      Pair part[2] = {};
#pragma unroll
      for (int h = 0; h < 64; h += 32) {
        uint32_t p[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 z = split(fma2(make_pair(s[h + c], s[h + c + 1]), mul_pair, less));
          const float a = exp2_fast(z.x), b = exp2_fast(z.y);
          part[c / 2 % 2] = add2(part[c / 2 % 2], make_pair(a, b));
          p[c / 2] = pack2<E>(a, b);
        }
        tmem_store16(at_s + h / 2, p);
      }
      sum += sum2(add2(part[0], part[1]));
      tmem_stored();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) bar_arrive(bar_weights);
    }
    if (row_of(t) < g.tokens) {
      // O / sum, through the queries' place in shared memory
      group_sync(pair, 64);  // what was told has been read
      *told = sum;
      group_sync(pair, 64);
      sum = half ? *other + sum : sum + *other;
      // (a row that sees keys whose scores are all -infinity is NaN, 0 times infinity,
      // as an infinity elsewhere makes it)
      const bool none = span.key_lo >= span.key_hi;
      const float inverse = 1.0f / sum;
      if (ok) ok = warp_wait(shared_addr(begin < end ? &bars->done[t] : &bars->q_full[t]), 0, g.status);
      fence_after_sync();
      const uint32_t place = q_tiles + t * kTile + (quarter * 32 + lane) * 128;
#pragma unroll
      for (int k = 0; k < C * 32; k += 32)
        if (k < o_width) {
          const int c = half * C * 32 + k;
          float o[32];
          if (begin < end) {
            tmem_load32(at_o + k, o);
            tmem_wait<32>(o);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = none ? 0.0f : o[i] * inverse;
          store_units<E>(place, c, o);
        }
      if (row < g.tokens && half == 0)
        g.lse[int64_t(row) * g.heads + head] =
            none ? -INFINITY : (top - kLift + log2f(sum)) * kLn2;
      fence_shared();
      group_sync(9 + t, 256);
      if (threadIdx.x % 256 == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c * kChunk < g.width)
            store_head_box(&maps.out, c * kChunk, head, row_of(t), q_tiles + t * kTile + c * kBoxBytes);
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

template <class T, int C, bool kCap>
fadam_status launch_forward(const ForwardMaps& maps, const AttentionArgs& g, cudaStream_t stream) {
  auto* kernel = attention_forward_kernel<T, C, kCap>;
  if (const fadam_status st = launched_with<attention_forward_kernel<T, C, kCap>>("attention")) return st;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kForwardSmem<C>));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  const int64_t items = g.pair_heads ? int64_t(g.tiles) * (g.heads / 2) : int64_t((g.tiles + 1) / 2) * g.heads;
  return launch_chained("attention launch", kernel, items, kAttentionThreads, kForwardSmem<C>, stream, maps, g);
}
template <class T>
fadam_status forward_of(const ForwardMaps& maps, const AttentionArgs& g, cudaStream_t stream) {
  if (g.softcap > 0.0f)
    return g.width <= kChunk ? launch_forward<T, 1, true>(maps, g, stream) : launch_forward<T, 2, true>(maps, g, stream);
  return g.width <= kChunk ? launch_forward<T, 1, false>(maps, g, stream) : launch_forward<T, 2, false>(maps, g, stream);
}

}  // namespace fadam_ops
