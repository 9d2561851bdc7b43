// Rotary positions as an operator of its own: heads turned at explicit positions on their
// way from a projection's output to the attention's q layout and the KV cache (or from
// gradients of the turned heads back to gradients of the projection).
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
#include "ptx.cuh"

namespace orthrus {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryMaxPairs = 128;
constexpr int kRotaryTokens = 4;  // tokens of one CTA at most

struct RotaryArgs {
  double turns[kRotaryMaxPairs];
  orthrus_rotary_part part[ORTHRUS_ROTARY_MAX_PARTS];
  int n_parts, head_dim, rot_dim, interleaved, inverse;
  float gain;
  int batch, tokens, tok_per_cta, vec;
  int items[ORTHRUS_ROTARY_MAX_PARTS];  // units of work of one token: heads x units of a head
  int total_items;
  const int* len;
  const int* offsets;
  int* status;
};

// n values from / to memory of a run-time type; n is 1, or 8 at 16-byte aligned addresses
template <int N>
__device__ __forceinline__ void rot_load(const void* p, size_t at, int type, float* x) {
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

template <int N>
__device__ __forceinline__ void rot_store(void* p, size_t at, int type, bool bf16_values, float* x) {
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

// One unit of a head: N pairs (2 N values), or 2 N values of the copied tail.
template <int N>
__device__ __forceinline__ void rotary_unit(const RotaryArgs& a, const orthrus_rotary_part& p, const float2* cs,
                                            size_t src, size_t dst, int unit) {
  const int pairs = a.rot_dim >> 1;
  const bool bfv = (p.flags & ORTHRUS_ROTARY_BF16_VALUES) != 0;
  const bool turn = !(p.flags & ORTHRUS_ROTARY_COPY) && unit * N < pairs;
  int e1, e2;
  if (turn && !a.interleaved) {
    e1 = unit * N;
    e2 = e1 + pairs;
  } else {
    e1 = 2 * unit * N;
    e2 = e1 + N;
  }
  float x[N], y[N];
  rot_load<N>(p.src, src + e1, p.src_type, x);
  rot_load<N>(p.src, src + e2, p.src_type, y);
  if (turn) {
    if (a.interleaved) {
      // the 2 N values are N neighbouring pairs
      float z[2 * N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        z[i] = x[i];
        z[N + i] = y[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 c = cs[unit * N + i];
        const float u = z[2 * i], v = z[2 * i + 1];
        z[2 * i] = u * c.x - v * c.y;
        z[2 * i + 1] = v * c.x + u * c.y;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = z[i];
        y[i] = z[N + i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 c = cs[unit * N + i];
        const float u = x[i], v = y[i];
        x[i] = u * c.x - v * c.y;
        y[i] = v * c.x + u * c.y;
      }
    }
  }
  rot_store<N>(p.dst, dst + e1, p.dst_type, bfv, x);
  rot_store<N>(p.dst, dst + e2, p.dst_type, bfv, y);
}

__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ float2 cs[kRotaryTokens * kRotaryMaxPairs];
  griddep_wait();
  griddep_launch();
  const int pairs = a.rot_dim >> 1;
  const long long all = (long long)a.batch * a.tokens;
  const long long t0 = (long long)blockIdx.x * a.tok_per_cta;
  const int nt = (int)min((long long)a.tok_per_cta, all - t0);
  for (int i = threadIdx.x; i < nt * pairs; i += kRotaryThreads) {
    const int k = i / pairs, p = i - k * pairs;
    const long long m = t0 + k;
    const int b = (int)(m / a.tokens), t = (int)(m - (long long)b * a.tokens);
    const double pos = (double)(a.len ? a.len[b] : 0) + (double)(a.offsets ? a.offsets[m] : t);
    const double turns = pos * a.turns[p];
    const float r = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.f * r, &s, &c);
    cs[i] = make_float2(c * a.gain, (a.inverse ? -s : s) * a.gain);
  }
  __syncthreads();
  const int per_head = a.vec ? a.head_dim / 16 : a.head_dim / 2;
  for (int i = blockIdx.y * kRotaryThreads + threadIdx.x; i < nt * a.total_items; i += gridDim.y * kRotaryThreads) {
    const int k = i / a.total_items;
    int item = i - k * a.total_items, j = 0;
    while (j + 1 < a.n_parts && item >= a.items[j]) item -= a.items[j++];
    const orthrus_rotary_part& p = a.part[j];
    const long long m = t0 + k;
    const int b = (int)(m / a.tokens), t = (int)(m - (long long)b * a.tokens);
    const int h = item / per_head, unit = item - h * per_head;
    long long row = t;
    if (p.flags & ORTHRUS_ROTARY_APPEND) {
      row += a.len ? a.len[b] : 0;
      if (row < 0 || row >= p.rows) {
        if (unit == 0) set_status(a.status, ORTHRUS_ERR_CAPACITY);
        continue;
      }
    }
    const size_t src = (size_t)(b * p.src_batch + t * p.src_token + h * p.src_head);
    const int kv = h / p.group;
    const size_t dst = (size_t)(b * p.dst_batch + row * p.dst_token + kv * p.dst_kv + (h - kv * p.group) * p.dst_head);
    if (a.vec) rotary_unit<8>(a, p, cs + k * pairs, src, dst, unit);
    else rotary_unit<1>(a, p, cs + k * pairs, src, dst, unit);
  }
}

}  // namespace orthrus
