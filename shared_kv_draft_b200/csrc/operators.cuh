// Draft trees and rotary positions: what the plan's calls use of operators.cu.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

#include "orthrus.h"

namespace orthrus {

struct TreeAttnArgs {
  const void *q, *k_cache, *v_cache, *k_blk, *v_blk;
  const int *len, *n_nodes;
  const unsigned long long* mask;
  int B, Hkv, G, N, d, cap, blk_stride, words, bf16, out_type;
  float scale_log2;
  void* out;
  size_t out_lo;  // ORTHRUS_BF16_PLANES: elements from the hi to the lo plane
  int* status;
  // scratch, laid out by launch_tree_attention
  float4* part_o;   // [2 per CTA][d / 4][256 rows]
  float2* part_ml;  // [2 per CTA][256 rows]: (reference, sum of weights)
  int4* note;       // [CTAs]: (sequence, KV head, row group, last range) of a cut unit, or x < 0
};

// Embedding of a tree block: row m = b * nodes + i at position len[b] + depth[i]; node 0 is
// the pending token, padding nodes embed token 0. RoPE table as in the chain's embedding.
struct TreeEmbedArgs {
  int nodes, D, d, V;
  double theta;
  const int *pending, *tokens, *n_nodes, *depth, *len;
  const void* embed;  // bf16 [V][D]
  float* h;
  float2* rope;
  int* status;
};

bool tree_sizes_ok(int batch, int nodes);
// Scratch of one tree attention call over caches of `cap` rows (bytes); grows with each argument.
size_t tree_attn_scratch(int B, int Hkv, int G, int nodes, int d, int cap);
orthrus_status launch_tree_attention(const TreeAttnArgs& a, void* workspace, size_t bytes, cudaStream_t st);
orthrus_status launch_tree_layout(const int* parents, const int* n_nodes, int batch, int nodes, int* depth,
                                  unsigned long long* mask, int* status, cudaStream_t st);
orthrus_status launch_tree_embed(const TreeEmbedArgs& a, int rows, cudaStream_t st);

}  // namespace orthrus
