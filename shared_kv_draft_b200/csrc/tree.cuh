// Draft trees: the layout a tree's parents give (depths, visibility words), the block
// embedding of a tree at positions len + depth, and the greedy walk down the tree with the
// commit of the accepted path's K/V rows to the cache.
#pragma once
#include "operators.cuh"
#include "ptx.cuh"

namespace orthrus {

constexpr int kTreeMaxNodes = ORTHRUS_TREE_MAX_NODES;
constexpr int kTreeMaxWords = kTreeMaxNodes / 64;

__device__ __forceinline__ int tree_count(const int* n_nodes, int b, int nodes) {
  return n_nodes ? min(max(n_nodes[b], 0), nodes) : nodes;
}

// One CTA per sequence, one thread per node. The set of a node and its ancestors grows by
// pointer jumping: after round r a node holds its nearest 2^r ancestors and a pointer to the
// next one, so a chain of N nodes takes log2(N) rounds instead of N dependent loads. The
// depth is the size of the finished set less one. Bound by launch and shared-memory latency.
__global__ void __launch_bounds__(kTreeMaxNodes)
    tree_layout_kernel(const int* parents, const int* n_nodes, int nodes, int words, int* depth,
                       unsigned long long* mask, int* status) {
  __shared__ unsigned long long set[kTreeMaxWords][kTreeMaxNodes];
  __shared__ int next[kTreeMaxNodes];
  griddep_wait();
  griddep_launch();
  const int b = blockIdx.x, i = threadIdx.x;
  const int n = tree_count(n_nodes, b, nodes);
  if (i == 0 && n_nodes && n_nodes[b] != n) set_status(status, ORTHRUS_ERR_ARG);
  int up = -1;
  unsigned long long m[kTreeMaxWords] = {};
  if (i < n) {
    up = parents[(size_t)b * nodes + i];
    if (up < -1 || up >= i) {
      set_status(status, ORTHRUS_ERR_ARG);
      up = -1;
    }
#pragma unroll
    for (int w = 0; w < kTreeMaxWords; ++w) m[w] = (i >> 6) == w ? 1ull << (i & 63) : 0ull;
  }
  while (__syncthreads_or(up >= 0)) {
#pragma unroll
    for (int w = 0; w < kTreeMaxWords; ++w)
      if (w < words) set[w][i] = m[w];
    next[i] = up;
    __syncthreads();
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kTreeMaxWords; ++w)
        if (w < words) m[w] |= set[w][up];
      up = next[up];
    }
  }
  if (i >= nodes) return;
  int d = -1;
#pragma unroll
  for (int w = 0; w < kTreeMaxWords; ++w)
    if (w < words) {
      d += __popcll(m[w]);
      mask[((size_t)b * nodes + i) * words + w] = m[w];
    }
  depth[(size_t)b * nodes + i] = max(d, 0);
}

__global__ void tree_embed_kernel(const TreeEmbedArgs a) {
  griddep_wait();
  griddep_launch();
  const int m = blockIdx.x;
  const int b = m / a.nodes, i = m - b * a.nodes;
  int id = 0;
  if (i < tree_count(a.n_nodes, b, a.nodes)) id = i == 0 ? a.pending[b] : a.tokens[m];
  if (id < 0 || id >= a.V) {
    if (threadIdx.x == 0) set_status(a.status, ORTHRUS_ERR_ARG);
    id = 0;
  }
  const __nv_bfloat16* src = (const __nv_bfloat16*)a.embed + (size_t)id * a.D;
  float* dst = a.h + (size_t)m * a.D;
  for (int c = threadIdx.x * 2; c < a.D; c += blockDim.x * 2)
    *reinterpret_cast<float2*>(dst + c) = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(src + c));
  const int half = a.d / 2;
  const double pos = (double)a.len[b] + (double)a.depth[m];
  for (int j = threadIdx.x; j < half; j += blockDim.x) {
    const double ang = pos * pow(a.theta, -2.0 * (double)j / (double)a.d);
    a.rope[(size_t)m * half + j] = make_float2((float)cos(ang), (float)sin(ang));
  }
}

// Greedy walk, one warp per sequence: from node 0 to the lowest-indexed child whose token is
// the argmax at the current node, until there is none. A child has a higher index than its
// parent, so the walk ends whatever the parents hold. One CTA serves every sequence, so that
// all of them see the status word as it was before the call.
struct TreeWalkArgs {
  const int *parents, *tokens, *argmax, *n_nodes;
  int batch, nodes, capacity;
  const int* len;
  int *new_len, *pending, *accept_len, *path, *committed, *status;
};

constexpr int kWalkThreads = 1024;

__global__ void __launch_bounds__(kWalkThreads) tree_walk_kernel(const TreeWalkArgs a) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const bool failed = a.status && *(volatile const int*)a.status != 0;
  __syncthreads();
  for (int b = threadIdx.x >> 5; b < a.batch; b += blockDim.x >> 5) {
    const size_t base = (size_t)b * a.nodes;
    const int old = a.len[b];
    int n = a.n_nodes ? a.n_nodes[b] : a.nodes;
    bool ok = !failed && n > 0;
    if (n < 0 || n > a.nodes) {
      if (lane == 0) set_status(a.status, ORTHRUS_ERR_ARG);
      ok = false;
    }
    if (!ok) n = 0;
    int par[kTreeMaxNodes / 32], tok[kTreeMaxNodes / 32];
#pragma unroll
    for (int k = 0; k < kTreeMaxNodes / 32; ++k) {
      const int i = k * 32 + lane;
      par[k] = (i > 0 && i < n) ? a.parents[base + i] : -1;
      tok[k] = (i > 0 && i < n) ? a.tokens[base + i] : 0;
    }
    // path and tokens go out as they are found; the tails are filled afterwards
    int cur = 0, steps = 0, want = ok ? a.argmax[base] : 0;
    if (ok && lane == 0) a.path[base] = 0;
    while (ok) {
      unsigned int best = 0xffffffffu;
#pragma unroll
      for (int k = kTreeMaxNodes / 32 - 1; k >= 0; --k) {
        const int i = k * 32 + lane;
        if (par[k] == cur && tok[k] == want && i > cur) best = (unsigned int)i;
      }
      best = __reduce_min_sync(0xffffffffu, best);
      if (best == 0xffffffffu) break;
      ++steps;
      if (lane == 0) {
        a.path[base + steps] = (int)best;
        a.committed[base + steps - 1] = want;
      }
      cur = (int)best;
      want = a.argmax[base + cur];
    }
    if (ok && (old < 0 || old > a.capacity - (steps + 1))) {  // no room: nothing of this sequence is committed
      if (lane == 0) set_status(a.status, old < 0 ? ORTHRUS_ERR_ARG : ORTHRUS_ERR_CAPACITY);
      ok = false;
    }
    const int first = ok ? steps + 1 : 0;  // path entries kept
    __syncwarp();
    for (int i = lane; i < a.nodes; i += 32) {
      if (i >= first) a.path[base + i] = -1;
      if (i >= first) a.committed[base + i] = -1;
    }
    if (lane == 0) {
      if (ok) {
        a.committed[base + steps] = want;
        a.pending[b] = want;
      }
      a.accept_len[b] = ok ? steps : -1;
      a.new_len[b] = ok ? old + steps + 1 : old;
    }
    __syncwarp();
  }
}

// The path's K/V rows of one (layer, sequence, KV head), scratch row path[j] -> cache row
// old + j, old = new_len - (a + 1). 16-byte pieces; source and destination are different buffers.
struct TreeMoveArgs {
  const uint4 *k_blk, *v_blk;
  uint4 *k_cache, *v_cache;
  const int *accept_len, *new_len, *path;
  int batch, kv_heads, nodes, blk_stride, capacity, pieces;  // pieces: 16-byte pieces of a row
};

constexpr int kMoveThreads = 128;

__global__ void __launch_bounds__(kMoveThreads) tree_move_kernel(const TreeMoveArgs a) {
  griddep_wait();
  griddep_launch();
  const int z = blockIdx.x;  // (layer * batch + b) * kv_heads + head
  const int b = (z / a.kv_heads) % a.batch;
  const int acc = a.accept_len[b];
  if (acc < 0) return;
  const int old = a.new_len[b] - (acc + 1);
  const int total = (acc + 1) * a.pieces;
  for (int i = threadIdx.x; i < total; i += kMoveThreads) {
    const int j = i / a.pieces, c = i - j * a.pieces;
    const int node = a.path[(size_t)b * a.nodes + j];
    const size_t from = ((size_t)z * a.blk_stride + node) * a.pieces + c;
    const size_t to = ((size_t)z * a.capacity + old + j) * a.pieces + c;
    const uint4 k = a.k_blk[from], v = a.v_blk[from];
    a.k_cache[to] = k;
    a.v_cache[to] = v;
  }
}

}  // namespace orthrus
