// Draft trees and rotary positions: launch geometry and the C-ABI entry points that need
// no plan (declared in include/orthrus.h).
#include "host.cuh"
#include "operators.cuh"
#include "orthrus.h"
#include "rotary.cuh"
#include "tree.cuh"
#include "tree_attention.cuh"

using namespace orthrus;

bool orthrus::tree_sizes_ok(int batch, int nodes) {
  return batch >= 1 && batch <= ORTHRUS_TREE_MAX_BATCH && nodes >= 1 && nodes <= ORTHRUS_TREE_MAX_NODES;
}

namespace {

// Two parts for each CTA: of the unit in which its range starts, and of the one in which it ends.
size_t tree_part_bytes(int ctas, int d) {
  return (size_t)2 * ctas * kTreeRows * ((size_t)d * 4 + 8) + (size_t)ctas * sizeof(int4);
}

long long tree_units(int B, int Hkv, int G, int nodes) {
  return (long long)B * Hkv * (((long long)nodes * G + kTreeRows - 1) / kTreeRows);
}

long long tree_tiles(int nodes, int cap) {  // of a unit, at most
  return ((long long)cap + kTreeKeys - 1) / kTreeKeys + (nodes + kTreeKeys - 1) / kTreeKeys;
}

// A CTA an SM, but where the capacity shows that the even division has fewer parts, not many more than those (a
// quarter, since the parts are rounded down): the SMs left free can start the join early (1 sequence of 1024 keys in a
// cache of that length: 11.3 us, with a CTA on every SM, as in a cache of 8192, 12.3)
int tree_ctas(int B, int Hkv, int G, int nodes, int cap) {
  const long long parts = (tree_tiles(nodes, cap) + kTreeMinTiles - 1) / kTreeMinTiles;
  return (int)std::min<long long>(num_sms(), tree_units(B, Hkv, G, nodes) * parts * 5 / 4);
}

}  // namespace

size_t orthrus::tree_attn_scratch(int B, int Hkv, int G, int nodes, int d, int cap) {
  return tree_part_bytes(tree_ctas(B, Hkv, G, nodes, cap), d);
}

namespace {

template <int D, bool BF16>
orthrus_status launch_tree_attention_as(const TreeAttnArgs& a, const CUtensorMap* m, int sms, cudaStream_t st) {
  if (!ensure_smem_attr(tree_attention_kernel<D, BF16>, TreeSmem<D>::kBytes)) return ORTHRUS_ERR_CUDA;
  const int units = (int)tree_units(a.B, a.Hkv, a.G, a.N);
  const long long tiles = tree_tiles(a.N, a.cap);
  if (launch(tree_attention_kernel<D, BF16>, dim3(sms), dim3(kTreeThreads), TreeSmem<D>::kBytes, st, m[0], m[1], m[2],
             m[3], m[4], a) != cudaSuccess)
    return ORTHRUS_ERR_CUDA;
  // no unit is cut where units and keys are few enough for the even division with one part a unit
  if (units <= sms && tiles <= kTreeMinTiles && kTreeUnit + tiles * kTreeCost2 <= kTreeSwitch + kTreeUnit + kTreeCost1)
    return ORTHRUS_OK;
  const dim3 grid(std::min(sms - 1, units), (std::min(kTreeRows, a.N * a.G) + 31) / 32);
  // few CTAs: the columns of a row over several
  const bool spread = (int)(grid.x * grid.y) < sms;
  const cudaError_t e = spread ? launch(tree_combine_kernel<1>, dim3(grid.x, grid.y, D / 32), dim3(kJoinThreads), 0, st, a, sms)
                               : launch(tree_combine_kernel<D / 32>, grid, dim3(kJoinThreads), 0, st, a, sms);
  return e == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ERR_CUDA;
}

}  // namespace

orthrus_status orthrus::launch_tree_attention(const TreeAttnArgs& args, void* workspace, size_t bytes, cudaStream_t st) {
  if (!encode_fn()) return ORTHRUS_ERR_CUDA;
  TreeAttnArgs a = args;
  // the costs of all tiles are counted in 31 bits
  if (tree_units(a.B, a.Hkv, a.G, a.N) * (kTreeUnit + tree_tiles(a.N, a.cap) * kTreeCost2) > INT32_MAX)
    return ORTHRUS_ERR_UNSUPPORTED;
  const int sms = tree_ctas(a.B, a.Hkv, a.G, a.N, a.cap);
  if (bytes < tree_part_bytes(sms, a.d)) return ORTHRUS_ERR_WORKSPACE;
  a.part_o = (float4*)workspace;
  a.part_ml = (float2*)(a.part_o + (size_t)2 * sms * kTreeRows * (a.d / 4));
  a.note = (int4*)(a.part_ml + (size_t)2 * sms * kTreeRows);
  const CUtensorMapDataType dt = a.bf16 ? kBF16 : kF16;
  const uint64_t z = (uint64_t)a.B * a.Hkv;
  CUtensorMap m[5];
  const bool ok = map2d(&m[0], a.q, a.d, z * a.N * a.G, 64, 32, dt) &&
                  map3d(&m[1], a.k_cache, a.d, a.cap, z, kTreeKeys, 1, dt) &&
                  map3d(&m[2], a.v_cache, a.d, a.cap, z, kTreeKeys, 1, dt) &&
                  map3d(&m[3], a.k_blk, a.d, a.blk_stride, z, kTreeKeys, 1, dt) &&
                  map3d(&m[4], a.v_blk, a.d, a.blk_stride, z, kTreeKeys, 1, dt);
  if (!ok) return ORTHRUS_ERR_ARG;
  if (a.d == 128)
    return a.bf16 ? launch_tree_attention_as<128, true>(a, m, sms, st)
                  : launch_tree_attention_as<128, false>(a, m, sms, st);
  return a.bf16 ? launch_tree_attention_as<64, true>(a, m, sms, st)
                : launch_tree_attention_as<64, false>(a, m, sms, st);
}

orthrus_status orthrus::launch_tree_layout(const int* parents, const int* n_nodes, int batch, int nodes, int* depth,
                                  unsigned long long* mask, int* status, cudaStream_t st) {
  const cudaError_t e = launch(tree_layout_kernel, dim3(batch), dim3(round_up(nodes, 32)), 0, st, parents, n_nodes,
                               nodes, (nodes + 63) / 64, depth, mask, status);
  return e == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ERR_CUDA;
}

orthrus_status orthrus::launch_tree_embed(const TreeEmbedArgs& a, int rows, cudaStream_t st) {
  return launch(tree_embed_kernel, dim3(rows), dim3(256), 0, st, a) == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ERR_CUDA;
}

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

orthrus_status launch_tree_commit(const TreeWalkArgs& w, TreeMoveArgs m, int n_layers, int head_dim, cudaStream_t st) {
  m.accept_len = w.accept_len;
  m.new_len = w.new_len;
  m.path = w.path;
  m.batch = w.batch;
  m.nodes = w.nodes;
  m.capacity = w.capacity;
  m.layers = n_layers;
  m.pieces = head_dim / 8;
  const int warps = std::min(kWalkThreads / 32, w.batch);
  void (*walk)(TreeWalkArgs) = w.nodes <= 64 ? tree_walk_kernel<2> : tree_walk_kernel<kTreeMaxNodes / 32>;
  if (launch(walk, dim3(1), dim3(32 * warps), 0, st, w) != cudaSuccess) return ORTHRUS_ERR_CUDA;
  // (layer, head) pairs to a CTA: one while the SMs are not full, then more, for longer streams of loads
  const long long pairs = (long long)n_layers * m.kv_heads;
  m.zs = (int)std::min<long long>(8, std::max(1ll, pairs * m.batch / (8 * num_sms())));
  if (launch(tree_move_kernel, dim3((unsigned)((pairs + m.zs - 1) / m.zs), m.batch), dim3(kMoveThreads), 0, st, m) !=
      cudaSuccess)
    return ORTHRUS_ERR_CUDA;
  return ORTHRUS_OK;
}

}  // namespace

extern "C" {

orthrus_status orthrus_tree_layout(const int32_t* parents, const int32_t* n_nodes, int32_t batch, int32_t nodes,
                                   int32_t* depth, uint64_t* mask, int32_t* status, orthrus_stream stream) {
  if (!parents || !depth || !mask || !tree_sizes_ok(batch, nodes) || !aligned(mask, 8)) return ORTHRUS_ERR_ARG;
  return launch_tree_layout(parents, n_nodes, batch, nodes, depth, (unsigned long long*)mask, status,
                            (cudaStream_t)stream);
}

size_t orthrus_tree_attention_workspace_bytes(int32_t batch, int32_t n_kv_heads, int32_t group, int32_t nodes,
                                              int32_t head_dim) {
  if (!tree_sizes_ok(batch, nodes) || n_kv_heads < 1 || group < 1 || group > 32 || (head_dim != 64 && head_dim != 128))
    return 0;
  return tree_part_bytes(num_sms(), head_dim);  // for any capacity
}

orthrus_status orthrus_tree_attention(const void* q, const void* k_cache, const void* v_cache, const void* k_blk,
                                      const void* v_blk, const int32_t* len, const int32_t* n_nodes,
                                      const uint64_t* mask, int32_t batch, int32_t n_kv_heads, int32_t group,
                                      int32_t nodes, int32_t head_dim, int32_t capacity, int32_t blk_stride,
                                      int32_t type, int32_t out_type, float scale, void* out, void* workspace,
                                      size_t workspace_bytes, int32_t* status, orthrus_stream stream) {
  if (!q || !k_cache || !v_cache || !k_blk || !v_blk || !len || !mask || !out || !workspace) return ORTHRUS_ERR_ARG;
  if (!tree_sizes_ok(batch, nodes) || n_kv_heads < 1 || group < 1 || capacity < 1 || blk_stride < nodes)
    return ORTHRUS_ERR_ARG;
  if (!(scale >= 0.f) || scale == INFINITY) return ORTHRUS_ERR_ARG;
  if (type != ORTHRUS_FP16 && type != ORTHRUS_BF16) return ORTHRUS_ERR_ARG;
  if (out_type != ORTHRUS_FP16 && out_type != ORTHRUS_BF16 && out_type != ORTHRUS_BF16_PLANES) return ORTHRUS_ERR_ARG;
  if (group > 32 || (head_dim != 64 && head_dim != 128)) return ORTHRUS_ERR_UNSUPPORTED;
  if ((long long)batch * n_kv_heads > (1 << 20)) return ORTHRUS_ERR_UNSUPPORTED;
  for (const void* p : {q, k_cache, v_cache, k_blk, v_blk, (const void*)out})
    if (!aligned(p, 16)) return ORTHRUS_ERR_ARG;
  if (!aligned(mask, 8) || !aligned(workspace, 256)) return ORTHRUS_ERR_ARG;
  if (workspace_bytes < tree_part_bytes(num_sms(), head_dim)) return ORTHRUS_ERR_WORKSPACE;
  TreeAttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_blk = k_blk;
  a.v_blk = v_blk;
  a.len = len;
  a.n_nodes = n_nodes;
  a.mask = (const unsigned long long*)mask;
  a.B = batch;
  a.Hkv = n_kv_heads;
  a.G = group;
  a.N = nodes;
  a.d = head_dim;
  a.cap = capacity;
  a.blk_stride = blk_stride;
  a.words = (nodes + 63) / 64;
  a.bf16 = type == ORTHRUS_BF16;
  a.out_type = out_type;
  a.scale_log2 = (float)(1.4426950408889634 * (scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)head_dim)));
  a.out = out;
  a.out_lo = (size_t)batch * nodes * n_kv_heads * group * head_dim;
  a.status = status;
  return launch_tree_attention(a, workspace, workspace_bytes, (cudaStream_t)stream);
}

orthrus_status orthrus_tree_commit(const int32_t* parents, const int32_t* tokens, const int32_t* argmax,
                                   const int32_t* n_nodes, const void* k_blk, const void* v_blk, int32_t blk_stride,
                                   void* k_cache, void* v_cache, int32_t n_layers, int32_t batch, int32_t n_kv_heads,
                                   int32_t capacity, int32_t head_dim, int32_t nodes, const int32_t* len,
                                   int32_t* new_len, int32_t* pending, int32_t* accept_len, int32_t* path,
                                   int32_t* committed, int32_t* status, orthrus_stream stream) {
  if (!parents || !tokens || !argmax || !k_blk || !v_blk || !k_cache || !v_cache || !len || !new_len || !pending ||
      !accept_len || !path || !committed)
    return ORTHRUS_ERR_ARG;
  if (!tree_sizes_ok(batch, nodes) || blk_stride < nodes || n_layers < 1 || n_kv_heads < 1 || capacity < 1 ||
      head_dim < 1)
    return ORTHRUS_ERR_ARG;
  if (head_dim % 8 || head_dim > 1024 || (long long)n_layers * batch * n_kv_heads > INT32_MAX)
    return ORTHRUS_ERR_UNSUPPORTED;
  for (const void* p : {k_blk, v_blk, (const void*)k_cache, (const void*)v_cache})
    if (!aligned(p, 16)) return ORTHRUS_ERR_ARG;
  TreeWalkArgs w;
  w.parents = parents;
  w.tokens = tokens;
  w.argmax = argmax;
  w.n_nodes = n_nodes;
  w.batch = batch;
  w.nodes = nodes;
  w.capacity = capacity;
  w.len = len;
  w.new_len = new_len;
  w.pending = pending;
  w.accept_len = accept_len;
  w.path = path;
  w.committed = committed;
  w.status = status;
  TreeMoveArgs m;
  m.k_blk = (const uint4*)k_blk;
  m.v_blk = (const uint4*)v_blk;
  m.k_cache = (uint4*)k_cache;
  m.v_cache = (uint4*)v_cache;
  m.kv_heads = n_kv_heads;
  m.blk_stride = blk_stride;
  return launch_tree_commit(w, m, n_layers, head_dim, (cudaStream_t)stream);
}

orthrus_status orthrus_rope_init(orthrus_rope* rope, int32_t head_dim, int32_t rot_dim, int32_t interleaved,
                                 float theta, int32_t scaling, float factor, int32_t original, float slow, float fast,
                                 float gain) {
  const orthrus_rope_numbers x = {theta, factor, slow, fast};
  return orthrus_rope_init_from(rope, head_dim, rot_dim, interleaved, &x, scaling, original, gain);
}

orthrus_status orthrus_rope_init_from(orthrus_rope* rope, int32_t head_dim, int32_t rot_dim, int32_t interleaved,
                                      const orthrus_rope_numbers* numbers, int32_t scaling, int32_t original,
                                      float gain) {
  if (!rope || !numbers || head_dim < 2 || head_dim > 2 * kRotaryMaxPairs || head_dim % 2 || rot_dim < 2 || rot_dim > head_dim ||
      rot_dim % 2)
    return ORTHRUS_ERR_ARG;
  const double theta = numbers->theta, factor = numbers->factor, slow = numbers->slow, fast = numbers->fast;
  if (!(theta > 1.0 && theta < INFINITY) || !(gain >= 0.f && gain < INFINITY) || scaling < ORTHRUS_ROPE_NONE ||
      scaling > ORTHRUS_ROPE_BY_INDEX)
    return ORTHRUS_ERR_ARG;
  if (scaling != ORTHRUS_ROPE_NONE && !(factor >= 1.0 && factor < INFINITY)) return ORTHRUS_ERR_ARG;
  const bool ramp = scaling == ORTHRUS_ROPE_BY_PARTS || scaling == ORTHRUS_ROPE_BY_INDEX;
  if (ramp && (original < 1 || !(slow > 0.0) || !(fast > slow) || !(fast < INFINITY))) return ORTHRUS_ERR_ARG;
  const double two_pi = 6.283185307179586476925;
  memset(rope, 0, sizeof(*rope));
  rope->head_dim = head_dim;
  rope->rot_dim = rot_dim;
  rope->interleaved = interleaved != 0;
  rope->gain = gain > 0.f ? gain : (ramp ? (float)(0.1 * std::log(factor) + 1.0) : 1.f);
  double lo = 0, hi = 0;
  if (scaling == ORTHRUS_ROPE_BY_INDEX) {
    auto index = [&](double rotations) {
      return rot_dim * std::log(original / (two_pi * rotations)) / (2.0 * std::log(theta));
    };
    lo = std::max(std::floor(index(fast)), 0.0);
    hi = std::min(std::ceil(index(slow)), (double)(rot_dim - 1));
    hi = std::max(hi, lo + 1e-3);
  }
  for (int p = 0; p < rot_dim / 2; ++p) {
    double f = std::pow(theta, -2.0 * p / rot_dim);
    if (scaling == ORTHRUS_ROPE_LINEAR) {
      f /= factor;
    } else if (ramp) {
      double keep;
      if (scaling == ORTHRUS_ROPE_BY_PARTS)
        keep = (original * f / two_pi - slow) / (fast - slow);
      else
        keep = 1.0 - (p - lo) / (hi - lo);
      keep = std::min(std::max(keep, 0.0), 1.0);
      f *= keep + (1.0 - keep) / factor;
    }
    rope->turns[p] = f / two_pi;
  }
  return ORTHRUS_OK;
}

orthrus_status orthrus_rotary(const orthrus_rope* rope, const orthrus_rotary_part* parts, int32_t n_parts,
                              int32_t batch, int32_t tokens, const int32_t* len, const int32_t* offsets,
                              int32_t inverse, int32_t* status, orthrus_stream stream) {
  if (!rope || !parts || n_parts < 1 || n_parts > ORTHRUS_ROTARY_MAX_PARTS || batch < 0 || tokens < 0)
    return ORTHRUS_ERR_ARG;
  if (rope->head_dim < 2 || rope->head_dim > 2 * kRotaryMaxPairs || rope->head_dim % 2 || rope->rot_dim < 2 ||
      rope->rot_dim > rope->head_dim || rope->rot_dim % 2)
    return ORTHRUS_ERR_ARG;
  RotaryArgs a;
  memcpy(a.turns, rope->turns, sizeof(a.turns));
  // 16-byte accesses: units of 8 pairs, every address of a unit a multiple of 8 elements (of
  // 4 for fp32, whose 8 values are two accesses; asked alike)
  bool vec = rope->head_dim % 16 == 0 && rope->rot_dim % 16 == 0;
  for (int i = 0; i < n_parts; ++i) {
    const orthrus_rotary_part& p = parts[i];
    if ((!p.src || !p.dst) && batch > 0 && tokens > 0) return ORTHRUS_ERR_ARG;  // an empty tensor may have no memory
    if (p.heads < 1 || p.group < 1 || p.heads % p.group || p.heads > 65536) return ORTHRUS_ERR_ARG;
    for (const int t : {p.src_type, p.dst_type})
      if (t != ORTHRUS_FP32 && t != ORTHRUS_BF16 && t != ORTHRUS_FP16) return ORTHRUS_ERR_ARG;
    if (p.flags & ~(ORTHRUS_ROTARY_COPY | ORTHRUS_ROTARY_APPEND | ORTHRUS_ROTARY_BF16_VALUES)) return ORTHRUS_ERR_ARG;
    if ((p.flags & ORTHRUS_ROTARY_APPEND) && p.rows < 1) return ORTHRUS_ERR_ARG;
    if (!aligned(p.src, p.src_type == ORTHRUS_FP32 ? 4 : 2) || !aligned(p.dst, p.dst_type == ORTHRUS_FP32 ? 4 : 2))
      return ORTHRUS_ERR_ARG;
    // values that would be written to one place (a broadcast destination)
    if ((!p.dst_batch && batch > 1) || (!p.dst_token && tokens > 1) || (!p.dst_kv && p.heads > p.group) ||
        (!p.dst_head && p.group > 1))
      return ORTHRUS_ERR_ARG;
    vec = vec && aligned(p.src, 16) && aligned(p.dst, 16);
    for (const int64_t s : {p.src_batch, p.src_token, p.src_head, p.dst_batch, p.dst_token, p.dst_kv, p.dst_head})
      vec = vec && s % 8 == 0;
    a.part[i] = p;
  }
  if (batch == 0 || tokens == 0) return ORTHRUS_OK;
  if ((long long)batch * tokens > INT32_MAX) return ORTHRUS_ERR_ARG;
  a.n_parts = n_parts;
  a.head_dim = rope->head_dim;
  a.rot_dim = rope->rot_dim;
  a.interleaved = rope->interleaved;
  a.inverse = inverse;
  a.gain = rope->gain;
  a.batch = batch;
  a.tokens = tokens;
  a.heads = 0;
  for (int i = 0; i < n_parts; ++i) {
    a.heads += parts[i].heads;
    a.per_group[i] = (uint32_t)(((1ull << 32) + parts[i].group - 1) / parts[i].group);
  }
  if (a.heads > 16384) return ORTHRUS_ERR_UNSUPPORTED;  // the reciprocals' products stay exact
  a.per_heads = (uint32_t)(((1ull << 32) + a.heads - 1) / a.heads);
  a.units = rope->head_dim / (vec ? 16 : 2);
  a.slots = kRotaryThreads / a.units;
  a.len = len;
  a.offsets = offsets;
  a.status = status;
  // many tokens: several to a CTA, whose angles are then a small part of its work; few: a CTA each, and
  // their heads over up to eight
  const long long all = (long long)batch * tokens;
  a.tok_per_cta = (int)std::min<long long>(kRotaryTokens, std::max(1ll, all / (8 * num_sms())));
  const long long gx = (all + a.tok_per_cta - 1) / a.tok_per_cta;
  int gy = 1;
  while (gy < 8 && gx * gy < num_sms() && gy * a.slots < a.heads) gy *= 2;
  // one pair of types for all parts in the usual cases
  bool same = vec;
  for (int i = 1; i < n_parts; ++i)
    same = same && parts[i].src_type == parts[0].src_type && parts[i].dst_type == parts[0].dst_type;
  const int from = parts[0].src_type, to = parts[0].dst_type;
  void (*kernel)(RotaryArgs) = vec ? rotary_kernel<8, kAnyType, kAnyType> : rotary_kernel<1, kAnyType, kAnyType>;
  if (same && from == ORTHRUS_FP32 && to == ORTHRUS_FP16) kernel = rotary_kernel<8, ORTHRUS_FP32, ORTHRUS_FP16>;
  if (same && from == ORTHRUS_FP32 && to == ORTHRUS_FP32) kernel = rotary_kernel<8, ORTHRUS_FP32, ORTHRUS_FP32>;
  if (same && from == ORTHRUS_BF16 && to == ORTHRUS_BF16) kernel = rotary_kernel<8, ORTHRUS_BF16, ORTHRUS_BF16>;
  if (same && from == ORTHRUS_FP16 && to == ORTHRUS_FP16) kernel = rotary_kernel<8, ORTHRUS_FP16, ORTHRUS_FP16>;
  return launch(kernel, dim3((unsigned)gx, gy), dim3(kRotaryThreads), 0, (cudaStream_t)stream, a) == cudaSuccess
             ? ORTHRUS_OK
             : ORTHRUS_ERR_CUDA;
}

}  // extern "C"
