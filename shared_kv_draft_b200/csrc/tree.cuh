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
// depth is the size of the finished set less one. Bound by launch and shared-memory latency: 1.6 us for one tree,
// 2.9 us for 64 of 256 nodes.
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
// parent, so the walk ends whatever the parents hold. The tree lies in registers, 32 nodes a
// register, loaded at once; a step is a comparison, a minimum over the warp and a shuffle. One CTA
// serves every sequence, so that all of them see the status word as it was before the call. Bound
// by latency: one round of loads, then about 50 cycles a step. Walk and move together: 4.3 us for one sequence, 14.9 us
// for 16 (36 layers, 8 KV heads, d = 128).
struct TreeWalkArgs {
  const int *parents, *tokens, *argmax, *n_nodes;
  int batch, nodes, capacity;
  const int* len;
  int *new_len, *pending, *accept_len, *path, *committed, *status;
};

constexpr int kWalkThreads = 1024;

// R: registers a lane holds of each array, at least nodes / 32
template <int R>
__global__ void __launch_bounds__(kWalkThreads) tree_walk_kernel(const TreeWalkArgs a) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  bool failed = false;
  const int laps = (a.batch + (blockDim.x >> 5) - 1) / (blockDim.x >> 5);
  for (int lap = 0; lap < laps; ++lap) {
    const int b = lap * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const bool mine = b < a.batch;
    const size_t base = (size_t)b * a.nodes;
    int par[R], tok[R], arg[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int i = k * 32 + lane;
      const bool in = mine && i < a.nodes;
      par[k] = in ? a.parents[base + i] : -1;
      tok[k] = in ? a.tokens[base + i] : 0;
      arg[k] = in ? a.argmax[base + i] : 0;
    }
    const int old = mine ? a.len[b] : 0;
    int n = mine ? (a.n_nodes ? a.n_nodes[b] : a.nodes) : 0;
    // the status word once, before any sequence of the call can change it
    if (lap == 0) failed = __syncthreads_or(a.status && *(volatile const int*)a.status != 0);
    if (!mine) continue;
    bool ok = !failed && n > 0;
    if (n < 0 || n > a.nodes) {
      if (lane == 0) set_status(a.status, ORTHRUS_ERR_ARG);
      ok = false;
    }
    if (!ok) n = 0;
    // lane l keeps entries l, l + 32, .. of the path and of the committed tokens
    int path[R], com[R], cur = 0, steps = 0, want = __shfl_sync(0xffffffffu, arg[0], 0);
#pragma unroll
    for (int k = 0; k < R; ++k) path[k] = com[k] = -1;
    if (lane == 0) path[0] = 0;
    while (ok) {
      unsigned int best = 0xffffffffu;
#pragma unroll
      for (int k = R - 1; k >= 0; --k) {
        const int i = k * 32 + lane;
        if (par[k] == cur && tok[k] == want && i > cur && i < n) best = (unsigned int)i;
      }
      best = __reduce_min_sync(0xffffffffu, best);
      if (best == 0xffffffffu) break;
      int next = arg[0];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (steps == k * 32 + lane) com[k] = want;
        if (steps + 1 == k * 32 + lane) path[k] = (int)best;
        if ((int)best >> 5 == k) next = arg[k];
      }
      ++steps;
      cur = (int)best;
      want = __shfl_sync(0xffffffffu, next, cur & 31);
    }
    if (ok && (old < 0 || old > a.capacity - (steps + 1))) {  // no room: nothing of this sequence is committed
      if (lane == 0) set_status(a.status, old < 0 ? ORTHRUS_ERR_ARG : ORTHRUS_ERR_CAPACITY);
      ok = false;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int i = k * 32 + lane;
      if (i < a.nodes) {
        a.path[base + i] = ok ? path[k] : -1;
        a.committed[base + i] = !ok ? -1 : (i == steps ? want : com[k]);
      }
    }
    if (lane == 0) {
      if (ok) a.pending[b] = want;
      a.accept_len[b] = ok ? steps : -1;
      a.new_len[b] = ok ? old + steps + 1 : old;
    }
  }
}

// The path's K/V rows, scratch row path[j] -> cache row old + j, old = new_len - (a + 1). A CTA moves the rows of
// `zs` (layer, KV head) pairs of one sequence in 16-byte pieces, two pairs of loads in flight a thread; source
// and destination are different buffers. Bound by memory for a batch (16 sequences: 3.4 TB/s with the walk), by launch
// and three dependent loads for one sequence.
struct TreeMoveArgs {
  const uint4 *k_blk, *v_blk;
  uint4 *k_cache, *v_cache;
  const int *accept_len, *new_len, *path;
  int layers, batch, kv_heads, nodes, blk_stride, capacity, pieces, zs;  // pieces: 16-byte pieces of a row
};

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) tree_move_kernel(const TreeMoveArgs a) {
  __shared__ int path[kTreeMaxNodes];
  griddep_wait();
  griddep_launch();
  const int b = blockIdx.y, acc = a.accept_len[b], old = a.new_len[b] - (acc + 1);
  for (int i = threadIdx.x; i < a.nodes; i += kMoveThreads) path[i] = a.path[(size_t)b * a.nodes + i];
  __syncthreads();
  if (acc < 0) return;
  const int z0 = blockIdx.x * a.zs, zn = min(a.zs, a.layers * a.kv_heads - z0);
  const int per = (acc + 1) * a.pieces, total = zn * per;
#pragma unroll 2
  for (int i = threadIdx.x; i < total; i += kMoveThreads) {
    const int zi = i / per, r = i - zi * per, j = r / a.pieces, c = r - j * a.pieces;
    const int layer = (z0 + zi) / a.kv_heads;
    const size_t z = ((size_t)layer * a.batch + b) * a.kv_heads + (z0 + zi - layer * a.kv_heads);
    const size_t from = (z * a.blk_stride + path[j]) * a.pieces + c, to = (z * a.capacity + old + j) * a.pieces + c;
    const uint4 k = __ldcs(a.k_blk + from), v = __ldcs(a.v_blk + from);
    a.k_cache[to] = k;
    a.v_cache[to] = v;
  }
}

}  // namespace orthrus
