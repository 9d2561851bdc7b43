// Attention of a draft tree over the KV cache and the tree's own K/V.
//
// Row (i, g) of KV head h (query head h G + g at tree node i) sees the cache rows
// [0, len[b]) and the tree rows j whose bit is set in the node's visibility words:
//     out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - m)
// with the running maximum m and sum in fp32; a row that sees nothing gives zeros.
#pragma once
#include "operators.cuh"
#include "ptx.cuh"

namespace orthrus {

__device__ __forceinline__ void tree_store(const TreeAttnArgs& a, size_t at, float x) {
  if (a.out_type == ORTHRUS_FP16) {
    ((__half*)a.out)[at] = __float2half_rn(x);
  } else {
    const __nv_bfloat16 hi = __float2bfloat16_rn(x);
    ((__nv_bfloat16*)a.out)[at] = hi;
    if (a.out_type == ORTHRUS_BF16_PLANES)
      ((__nv_bfloat16*)a.out)[a.out_lo + at] = __float2bfloat16_rn(x - __bfloat162float(hi));
  }
}

// One warp per row, one key at a time: the lanes hold d / 32 dims each.
template <int D>
__global__ void __launch_bounds__(128) tree_attention_kernel(const TreeAttnArgs a) {
  griddep_wait();
  griddep_launch();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const long long rows = (long long)a.B * a.Hkv * a.N * a.G;
  if (row >= rows) return;
  const int g = (int)(row % a.G), i = (int)(row / a.G % a.N), z = (int)(row / ((long long)a.G * a.N));
  const int b = z / a.Hkv, kvh = z - b * a.Hkv;
  int n = a.len[b];
  if (n < 0 || n > a.cap) {
    if (lane == 0) set_status(a.status, n < 0 ? ORTHRUS_ERR_ARG : ORTHRUS_ERR_CAPACITY);
    n = min(max(n, 0), a.cap);
  }
  const int live = a.n_nodes ? min(max(a.n_nodes[b], 0), a.N) : a.N;
  if (i >= live) return;
  auto value = [&](const void* p, size_t at) {
    return a.bf16 ? __bfloat162float(((const __nv_bfloat16*)p)[at]) : __half2float(((const __half*)p)[at]);
  };
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = value(a.q, (size_t)row * D + lane + 32 * e);
  auto step = [&](const void* kp, const void* vp, size_t at) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * value(kp, at + lane + 32 * e);
    s = warp_sum(s) * a.scale_log2;
    const float mn = fmaxf(m, s);
    const float f = mn == -INFINITY ? 1.f : exp2f(m - mn), p = mn == -INFINITY ? 0.f : exp2f(s - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * value(vp, at + lane + 32 * e);
    m = mn;
  };
  for (int j = 0; j < n; ++j) step(a.k_cache, a.v_cache, ((size_t)z * a.cap + j) * D);
  const unsigned long long* words = a.mask + ((size_t)b * a.N + i) * a.words;
  for (int j = 0; j < live; ++j)
    if ((words[j >> 6] >> (j & 63)) & 1ull) step(a.k_blk, a.v_blk, ((size_t)z * a.blk_stride + j) * D);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const size_t at = (((size_t)b * a.N + i) * a.Hkv * a.G + (size_t)kvh * a.G + g) * D;
#pragma unroll
  for (int e = 0; e < E; ++e) tree_store(a, at + lane + 32 * e, o[e] * inv);
}

}  // namespace orthrus
