// Attention: what its host code and its kernels' translation units share.
#pragma once

#include "fadam_seq.h"
#include "ops_internal.h"

namespace fadam_ops {

constexpr int kRows = 128;     // rows of a tile: a tensor-core instruction's lanes
constexpr int kChunk = 64;     // elements of a head in one block of shared memory (128 bytes a row)

// Which keys a token sees, and by which queries it is seen: [lo, hi) each.
struct Spans {
  int key_lo, key_hi, query_lo, query_hi;
};

struct AttentionArgs {
  int tokens, sequence, heads, group, width;   // group: query heads to a key head
  int tiles;                                   // of 128 tokens
  int causal;
  int pair_heads;                              // forward: a CTA's two tiles are the same rows of two heads
  float scale, softcap;
  float2 series[4];          // capped scores in units of log 2 near zero, for products x that are y caps: of x, x y^2,
                             // x y^4, x y^6, twice each
  const float* slopes;
  const Spans* spans;        // [tokens] where there are documents
  const int* order;          // forward: of what a CTA takes, or NULL: last ones first
  const int32_t* prefix;     // of the sequences, where there are none
  const int32_t* documents;  // the first and the last offset say what is padding
  int64_t n_documents;
  float* lse;                // [tokens, heads]
  int* status;

  // backward
  float* stats;              // [2][heads][tiles * 128]: -lse in units of log 2, then -delta; f16: a third,
                             // a grad_out row's largest magnitude
  unsigned* peaks;           // f16: [3][kv_heads][entries], bits of a key head's largest in a document:
                             // grad_out's magnitudes, delta's, sums of a v row's magnitudes
  int entries;               // one for each sequence, or one for each token, of which a document's first counts
  float* parts;              // fp32 sums of grad_k and grad_v by splits of the query heads
  int splits;
  unsigned key_items;        // CTAs of the first kind, which take keys
};

// One matrix [tokens, heads, width] of 16-bit elements for boxes of 128 tokens
// of one head, 64 elements each.
fadam_status head_map(CUtensorMap* map, const void* base, int64_t tokens, int heads, int width,
                      int64_t stride, int64_t head_stride);

struct ForwardMaps {
  CUtensorMap q, k, v, out;
};
struct BackwardMaps {
  CUtensorMap q, k, v, grad_out, grad_q, grad_k, grad_v;
};

// Instances: attention_{forward,backward}_{bf16,f16}.cu.
fadam_status attention_forward_bf16(const ForwardMaps&, const AttentionArgs&, cudaStream_t);
fadam_status attention_forward_f16(const ForwardMaps&, const AttentionArgs&, cudaStream_t);
fadam_status attention_backward_bf16(const BackwardMaps&, const AttentionArgs&, cudaStream_t);
fadam_status attention_backward_f16(const BackwardMaps&, const AttentionArgs&, cudaStream_t);

}  // namespace fadam_ops
