// Rotary positions as an operator of its own: heads turned at explicit positions on their
// way from a projection's output to the attention's q layout and the KV cache, or, by the inverse, gradients
// of the turned heads on the way to gradients of the projection. A source has one stride for all of its heads:
// gradients that lie in the grouped q layout, or in cache rows, are brought to [batch][tokens][heads][d] first.
//
// Pair p of the first rot dims of a head, (x1, x2), at position t becomes
//     gain * (x1 cos a - x2 sin a,  x2 cos a + x1 sin a),   a = t f_p;
// the inverse uses -a, which with the same gain is the transposed map: the gradient. Dims
// past rot are copied. f_p comes from the host as turns per position (f_p / 2 pi, fp64).
// The angle needs more than fp32: at position 10^6 an fp32 product is off by 0.06 rad. The
// position times the turns is formed in fp64 (one product), its whole turns are dropped, and
// the rest, in [-1/2, 1/2] turns, goes through CUDA's sincospif in fp32: the angle is then
// off by about 2^-25 turns, like one fp32 rounding.
#pragma once
#include <limits.h>

#include "ptx.cuh"

namespace orthrus {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryMaxPairs = 128;
constexpr int kRotaryTokens = 8;  // tokens of one CTA at most
constexpr int kAnyType = -1;      // types of the parts at run time

struct RotaryArgs {
  double turns[kRotaryMaxPairs];
  orthrus_rotary_part part[ORTHRUS_ROTARY_MAX_PARTS];
  uint32_t per_group[ORTHRUS_ROTARY_MAX_PARTS];  // ceil(2^32 / group): h / group = its high product with h < 2^16
  int n_parts, head_dim, rot_dim, interleaved, inverse;
  float gain;
  int batch, tokens, tok_per_cta;
  int heads;               // of all parts
  uint32_t per_heads;      // ceil(2^32 / heads); one head has none (2^32)
  int units, slots;        // units of a head, heads that a CTA has in hand at a time
  const int* len;
  const int* offsets;
  int* status;
};

// N values from / to memory of type T, or `type` where T is kAnyType; N is 1, or 8 at 16-byte aligned addresses
template <int N, int T>
__device__ __forceinline__ void rot_load(const void* p, long long at, int type, float* x) {
  if (T != kAnyType) type = T;
  if constexpr (N == 8) {
    if (type == ORTHRUS_FP32) {
      const float4* q = reinterpret_cast<const float4*>((const float*)p + at);
      const float4 a = q[0], b = q[1];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
      const uint4 r = *reinterpret_cast<const uint4*>((const uint16_t*)p + at);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f;
        if (type == ORTHRUS_BF16) f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        else f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  } else {
    if (type == ORTHRUS_FP32) x[0] = ((const float*)p)[at];
    else if (type == ORTHRUS_BF16) x[0] = __bfloat162float(((const __nv_bfloat16*)p)[at]);
    else x[0] = __half2float(((const __half*)p)[at]);
  }
}

template <int N, int T>
__device__ __forceinline__ void rot_store(void* p, long long at, int type, bool bf16_values, float* x) {
  if (T != kAnyType) type = T;
  if (bf16_values) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = kv_value(x[i]);
  }
  if constexpr (N == 8) {
    if (type == ORTHRUS_FP32) {
      float4* q = reinterpret_cast<float4*>((float*)p + at);
      q[0] = make_float4(x[0], x[1], x[2], x[3]);
      q[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (type == ORTHRUS_BF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint4*>((uint16_t*)p + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    if (type == ORTHRUS_FP32) ((float*)p)[at] = x[0];
    else if (type == ORTHRUS_BF16) ((__nv_bfloat16*)p)[at] = __float2bfloat16_rn(x[0]);
    else ((__half*)p)[at] = __float2half_rn(x[0]);
  }
}

// A unit is N pairs of a head (2 N values), or 2 N values of its copied tail; N = 8, or 1 where the sizes, strides
// or addresses do not allow 16-byte accesses. A thread keeps its unit and goes through the heads of the CTA's
// tokens. Bound by memory: every value is read and written once (32768 tokens of 40 heads, bf16: 115 us, 5.8 TB/s, 89%
// of the copy rate; a tree's block 3 us, a launch). The angles of a token are computed once for all
// of its heads, and lie in shared memory so that the threads of a warp read consecutive 16 bytes.
template <int N, int SRC, int DST>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ float2 cs[kRotaryTokens * kRotaryMaxPairs];
  __shared__ long long from[kRotaryTokens][ORTHRUS_ROTARY_MAX_PARTS], to[kRotaryTokens][ORTHRUS_ROTARY_MAX_PARTS];
  griddep_wait();
  griddep_launch();
  const int pairs = a.rot_dim >> 1, rot_units = pairs / N;
  const int t0 = blockIdx.x * a.tok_per_cta, nt = min(a.tok_per_cta, a.batch * a.tokens - t0);
  // pair p = unit u's i-th: N = 8 keeps two neighbouring pairs (16 bytes) of all units together
  auto place = [&](int p) { return N == 1 ? p : ((p & 7) >> 1) * (2 * rot_units) + (p >> 3) * 2 + (p & 1); };
#pragma unroll 1
  for (int i = threadIdx.x; i < nt * pairs; i += kRotaryThreads) {
    const int k = i / pairs, p = i - k * pairs;
    const int m = t0 + k, b = m / a.tokens, t = m - b * a.tokens;
    const double pos = (double)(a.len ? a.len[b] : 0) + (double)(a.offsets ? a.offsets[m] : t);
    const double turns = pos * a.turns[p];
    const float r = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.f * r, &s, &c);
    cs[k * pairs + place(p)] = make_float2(c * a.gain, (a.inverse ? -s : s) * a.gain);
  }
  if (threadIdx.x < nt * a.n_parts) {
    const int k = threadIdx.x / a.n_parts, j = threadIdx.x - k * a.n_parts;
    const orthrus_rotary_part& p = a.part[j];
    const int m = t0 + k, b = m / a.tokens, t = m - b * a.tokens;
    long long row = t;
    bool ok = true;
    if (p.flags & ORTHRUS_ROTARY_APPEND) {
      row += a.len ? a.len[b] : 0;
      ok = row >= 0 && row < p.rows;
      if (!ok) set_status(a.status, ORTHRUS_ERR_CAPACITY);
    }
    from[k][j] = ok ? b * p.src_batch + t * p.src_token : LLONG_MIN;  // no such row: nothing is written
    to[k][j] = b * p.dst_batch + row * p.dst_token;
  }
  __syncthreads();
  const int slot = threadIdx.x / a.units, unit = threadIdx.x - slot * a.units;
  if (slot >= a.slots) return;
#pragma unroll 2
  for (int i = blockIdx.y * a.slots + slot; i < nt * a.heads; i += gridDim.y * a.slots) {
    const int k = a.heads == 1 ? i : (int)__umulhi((uint32_t)i, a.per_heads);
    int h = i - k * a.heads, j = 0;
    while (h >= a.part[j].heads) h -= a.part[j++].heads;
    const orthrus_rotary_part& p = a.part[j];
    if (from[k][j] == LLONG_MIN) continue;
    const int kv = p.group == 1 ? h : (int)__umulhi((uint32_t)h, a.per_group[j]);
    const long long src = from[k][j] + h * p.src_head;
    const long long dst = to[k][j] + kv * p.dst_kv + (h - kv * p.group) * p.dst_head;
    const bool bfv = (p.flags & ORTHRUS_ROTARY_BF16_VALUES) != 0;
    const bool turn = !(p.flags & ORTHRUS_ROTARY_COPY) && unit < rot_units;
    const int e1 = turn && !a.interleaved ? unit * N : 2 * unit * N, e2 = e1 + (turn && !a.interleaved ? pairs : N);
    float x[2 * N];
    rot_load<N, SRC>(p.src, src + e1, p.src_type, x);
    rot_load<N, SRC>(p.src, src + e2, p.src_type, x + N);
    if (turn) {
      const float2* c = cs + k * pairs;
      if (a.interleaved) {
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const float2 f = N == 1 ? c[unit] : c[(q >> 1) * (2 * rot_units) + unit * 2 + (q & 1)];
          const float u = x[2 * q], v = x[2 * q + 1];
          x[2 * q] = u * f.x - v * f.y;
          x[2 * q + 1] = v * f.x + u * f.y;
        }
      } else {
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const float2 f = N == 1 ? c[unit] : c[(q >> 1) * (2 * rot_units) + unit * 2 + (q & 1)];
          const float u = x[q], v = x[N + q];
          x[q] = u * f.x - v * f.y;
          x[N + q] = v * f.x + u * f.y;
        }
      }
    }
    rot_store<N, DST>(p.dst, dst + e1, p.dst_type, bfv, x);
    rot_store<N, DST>(p.dst, dst + e2, p.dst_type, bfv, x + N);
  }
}

}  // namespace orthrus
