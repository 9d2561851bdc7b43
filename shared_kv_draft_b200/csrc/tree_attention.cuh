// Attention of a draft tree over the KV cache and the tree's own K/V, on tcgen05.
//
// Row (i, g) of KV head h (query head h G + g at tree node i) sees the cache rows
// [0, len[b]) and the tree rows j whose bit is set in the node's visibility words:
//     out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(s_j - m),   s_j = log2(e) scale q.k_j
// in one pass over the keys with a running reference m per row; a row that sees nothing
// gives zeros.
//
// Bound: every key is read once for up to 256 rows (nodes x group) of a KV head. A key costs an SM, in cycles at
// 1965 MHz, 4 d / 22.5 for its bytes, 4 rows d / 5650 for the two products (the rates of a copy and of a large product
// over 148 SMs) and rows / 16 for the exponentials: at d = 128 and 256 rows 23, 23 and 16, with 128 rows 23, 12 and 8:
// HBM, with the products as long at 256 rows. At d = 64 and 256 rows 11, 12 and 16: the exponentials.
// Measured at d = 128: 128 rows or fewer 5.8 TB/s over a long cache (8 sequences of 16384 keys, 16 nodes x 4: 92 us, 89%
// of the copy rate; 112 us in a run of a second, at the card's power limit); 256 rows 3.7 TB/s and 0.94 PFLOP/s
// (4 of 32768 keys, 64 x 4: 143-150 us, and 169-174 us in a run of a second, at 1.5 GHz). There the loads alone take
// 100 us, the products with the loads 124, the softmax with the loads 120: q and K come to the first product from shared
// memory, 6 KB for 32 cycles of arithmetic (48 at 128 bytes a cycle), and the loads write there meanwhile. Measured at
// d = 64, 4 sequences of 32768 keys: 256 rows 120 us (the exponentials alone 58), 128 rows 80 us (the bytes alone 41): a
// tile is half as large there and takes nearly as long; which part of its chain sets the pace has not been taken apart.
// Short caches are bound by latency: launch, first loads, two or three tiles, and the second kernel (1 sequence of 1024
// keys: 11.3 us, in a cache for 8192 12.3).
//   Kept at 8 softmax warps of 64 keys a thread: 16 warps of 32 keys, which have to agree on the reference, took
// 174 us there; S in one buffer and P in two beside it, so that the next scores come sooner, 152.
//
// Split. A unit is (sequence, KV head, group of up to 256 rows); its keys come in tiles of 64, cache
// tiles first, then the tree's. The grid is a CTA an SM at most, and the lengths are on the device only,
// so the CTAs divide the units by themselves (TreeShare below), by the tiles' costs: a ragged
// batch loads every SM alike. A unit that one CTA has is finished there; of a unit that is cut,
// each CTA stores its part (unnormalised sums, the reference and the weights' sum per row, fp32),
// and tree_combine_kernel joins the parts in key order. The cuts follow from the lengths and sizes
// of the call, so results repeat bit for bit.
//
// One CTA: warp 8 loads (TMA, a ring of 160 KB in K and V tiles), warps 9 and 10 issue the MMAs, warps
// 0-3 and 4-7 are two softmax streams, one thread per row. TMEM holds two S buffers of 64 columns and
// the O of each stream; P (16 bit) overwrites its S and is read by the second product from there, so
// that shared memory is left to the ring. While the softmax works on one buffer, the next scores
// are written to the other.
//   More than 128 rows: stream s owns rows [128 s, 128 s + 128) of the group and sees every
//   tile, so a K/V tile is loaded once for both.
//   At most 128 rows: both streams own the same rows and take the tiles in turn; their sums
//   are joined when the segment ends.
//
// The accumulators stay in TMEM. The reference m of a row moves only when a tile's maximum
// exceeds it by more than 8 (a factor of 256), and only then is O rescaled. Weights carry a
// factor 2^7 that cancels in the quotient: between 2^15 (below fp16's 65504) and fp16's
// smallest step 2^-24 they keep 39 binades below the largest possible one. Scores, sums and
// the quotient are fp32; P is rounded to the operands' type for its product with V, because
// the tensor cores take 16-bit operands of one type: half a step, 2^-11 (fp16) or 2^-8 (bf16)
// of each weight.
//
// Rows of K and V that no row may see (past len, past the tree) can hold anything: their
// scores are replaced and their V rows are zeroed in shared memory before the product. A V
// value that is not finite in a live tree row is zeroed as well and added afterwards to the
// rows that see that node, so that 0 x NaN reaches nobody else.
#pragma once
#include "operators.cuh"
#include "ptx.cuh"
#include "tree_ring.cuh"

namespace orthrus {

constexpr int kTreeThreads = 384;  // 8 softmax warps, a load warp, two MMA warps, a note warp
constexpr int kTreeKeys = 64;      // keys of a tile: one visibility word
constexpr int kTreeRows = 256;     // rows of a unit
constexpr float kTreeSlack = 8.f;  // how far scores may exceed the reference (log2)
constexpr float kTreeShift = 7.f;  // factor on the weights (log2)
constexpr int kTreeLoadWarp = 8, kTreeMmaWarp = 9, kTreeNoteWarp = 11;  // MMA warps 9 and 10

template <int D>
struct TreeSmem {
  static constexpr int kTile = kTreeKeys * D * 2;  // bytes of a K or V tile
  static constexpr int kQTile = 128 * D * 2;       // of 128 rows of q
  static constexpr int kStages = D == 128 ? 10 : 20;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kQTile;
  static constexpr int kMisc = kRing + kStages * kTile;
  static constexpr int kBytes = 1024 + kMisc + 2048;  // 1024: alignment of the dynamic part
};

struct TreeMisc {
  uint64_t full[20], empty[20], q_full, q_empty;
  uint64_t s_full[4], p_full[4];  // [2 stream + buffer]
  uint64_t o_done[2], o_last[2], done[2], seg_done;
  uint32_t tmem;
  int bad_any;
  unsigned int bad[8];  // tree rows with values that are not finite (this segment)
  float2 ml[128];       // one stream's (reference, sum) for the other
};
static_assert(sizeof(TreeMisc) <= 2048, "misc area");

// ---- who works on what ------------------------------------------------------------------

// Relative times, in steps of about 0.4 us. A tile took 0.78 us with up to 128 rows (bound by its reads) and
// 1.06 us with 256 (d = 64, 4 x 32768 keys: 0.72 and 1.08); 3 : 4 instead of 2 : 3 cost 10% at 16 ragged sequences. What
// a unit costs beside its tiles (pipeline filled and drained, sums stored) is about 3 us; 6 or 10 instead of 8 cost
// nothing there.
constexpr int kTreeCost1 = 2, kTreeCost2 = 3;  // a tile with up to 128 rows, with more
constexpr int kTreeUnit = 8;                   // a unit
constexpr int kTreeSwitch = 10;                // how much longer than a range the even division's parts may be
// Tiles of a part at least, in the even division: more parts are quicker to compute and slower to join. One
// sequence of 1024 keys: 12.6 us with 2 or 3, 12.9 with 4 (with a CTA on every SM); a tree step of 100 keys 9.5, 7.9, 7.8.
constexpr int kTreeMinTiles = 3;

struct TreeSeq {
  int n, live, tiles, groups, big;  // clamped length, nodes, tiles of a unit, row groups, groups of more than 128 rows
  __device__ TreeSeq() {}
  __device__ TreeSeq(const TreeAttnArgs& a, int b)
      : TreeSeq(a.G, min(max(a.len[b], 0), a.cap), a.n_nodes ? min(max(a.n_nodes[b], 0), a.N) : a.N) {}
  __device__ TreeSeq(int G, int n_, int live_) {
    n = n_;
    live = live_;
    const int rows = live * G;
    groups = (rows + kTreeRows - 1) / kTreeRows;
    big = (rows + kTreeRows - 129) / kTreeRows;
    tiles = (n + kTreeKeys - 1) / kTreeKeys + (live + kTreeKeys - 1) / kTreeKeys;
  }
  __device__ int cost(int rg) const { return rg < big ? kTreeCost2 : kTreeCost1; }  // of a tile
  __device__ int unit(int rg) const { return kTreeUnit + tiles * cost(rg); }
  __device__ int head() const {  // of a KV head
    return groups * kTreeUnit + tiles * (big * kTreeCost2 + (groups - big) * kTreeCost1);
  }
};

// The division of the work. Even: every unit is cut into parts of its own, about as many as its share of
// the CTAs, and a CTA has one part. Line: the costs of all units form one line, cut into ranges of equal
// length, and a CTA has the tiles that start in its range, of one or several units (a unit's own cost lies
// with its first tile). The even division is taken where its largest part does not exceed a range by more than
// kTreeSwitch: with few units a CTA then never changes from one to another.
// (All costs fit 31 bits, which the host checks with the capacity.)
struct TreeShare {
  int total, ctas, each, more;  // line
  float per_cost;               // CTAs for a unit of cost: even
  bool even;
  __device__ int at(int c) const { return min(total, c * each + min(c, more)); }
  __device__ int parts(const TreeSeq& s, int rg) const {
    const int n = (int)(s.unit(rg) * per_cost), most = (s.tiles + kTreeMinTiles - 1) / kTreeMinTiles;
    return max(1, min(n, most));
  }
  __device__ int head_parts(const TreeSeq& s) const {
    return (s.big ? s.big * parts(s, 0) : 0) + (s.groups > s.big ? parts(s, s.groups - 1) : 0);
  }
  __device__ int largest(const TreeSeq& s) const {  // cost of a sequence's largest part
    int x = 0;
    for (int rg = 0; rg < s.groups; rg += max(1, s.groups - 1)) {
      const int n = parts(s, rg);
      x = max(x, kTreeUnit + (s.tiles + n - 1) / n * s.cost(rg));
    }
    return x;
  }
};

// The sequence of this lane among 32 from `base` on; empty past the last.
__device__ __forceinline__ TreeSeq tree_lane_seq(const TreeAttnArgs& a, int base) {
  TreeSeq s;
  s.n = s.live = s.tiles = s.groups = s.big = 0;
  const int b = base + (threadIdx.x & 31);
  return b < a.B ? TreeSeq(a, b) : s;
}

// The part of a unit that one CTA works on: tiles [t0, t1) of `tiles`.
struct TreeSeg {
  int b, kvh, rg, n, live, tiles, t0, t1, slot;
  bool two;  // more than 128 rows
  __device__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// A CTA's segments in order; every role walks them by itself.
struct TreeWalk {
  TreeSeq s;
  int b, kvh, rg, t, t1, c, left;  // left: the range's cost from the unit's start on (line)
  int part, parts;                 // of the unit (even)
  bool first;
  __device__ void none() { left = part = parts = 0; }
  // from the part or the cost `off` of sequence b on
  __device__ void begin(const TreeShare& d, const TreeSeq& it, int c_, int b_, int off) {
    s = it;
    c = c_;
    b = b_;
    first = true;
    const int head = d.even ? d.head_parts(s) : s.head();
    kvh = off / head;
    int r = off - kvh * head;
    const int n = d.even ? d.parts(s, 0) : s.unit(0);  // of a unit, all but the last
    rg = min(r / n, s.groups - 1);
    r -= rg * n;
    part = parts = 0;
    if (d.even) {
      part = r;
      parts = d.parts(s, rg);
      t = s.tiles * part / parts;
      t1 = s.tiles * (part + 1) / parts;
      left = 1;
    } else {
      const int w = s.cost(rg);
      left = d.at(c + 1) - d.at(c) + r;
      t = r == 0 ? 0 : max(1, (r - kTreeUnit + w - 1) / w);  // tile t > 0 starts at kTreeUnit + t w
      if (t >= s.tiles) {
        left -= s.unit(rg);
        t = 0;
        ++rg;
      }
    }
  }
  __device__ bool next(const TreeAttnArgs& a, TreeSeg& g) {
    if (left <= 0) return false;
    if (parts == 0) {
      if (rg >= s.groups) {
        rg = 0;
        ++kvh;
      }
      while (s.groups == 0 || kvh >= a.Hkv) {
        s = TreeSeq(a, ++b);
        kvh = 0;
      }
      const int w = s.cost(rg);
      t1 = min(s.tiles, max(1, (left - kTreeUnit + w - 1) / w));
    }
    g.b = b;
    g.kvh = kvh;
    g.rg = rg;
    g.n = s.n;
    g.live = s.live;
    g.tiles = s.tiles;
    g.t0 = t;
    g.t1 = t1;
    g.two = rg < s.big;
    g.slot = 2 * c + (first && t > 0 ? 0 : 1);
    first = false;
    if (parts == 0 && t1 == s.tiles) {
      left -= s.unit(rg);
      t = 0;
      ++rg;
    } else {
      left = 0;
    }
    return true;
  }
};

// Finds the division, and the start of CTA c's work in it. Every warp finds them by itself, a lane
// for a sequence, so that the start of the kernel has no barrier to wait at.
__device__ __forceinline__ TreeShare tree_start(const TreeAttnArgs& a, int c, int sms, TreeWalk& walk) {
  const int lane = threadIdx.x & 31;
  const TreeSeq first = tree_lane_seq(a, 0);
  TreeShare d;
  d.total = 0;
#pragma unroll 1
  for (int base = 0; base < a.B; base += 32) {
    const TreeSeq s = base ? tree_lane_seq(a, base) : first;
    d.total += __reduce_add_sync(0xffffffffu, s.head() * a.Hkv);
  }
  d.ctas = max(1, min(sms, d.total / (kTreeUnit + kTreeCost2)));  // every range holds a tile's start
  d.each = d.total / d.ctas;
  d.more = d.total - d.each * d.ctas;
  d.per_cost = (float)sms / (float)max(1, d.total);
  d.even = true;
  int all = 0;
#pragma unroll 1
  for (int base = 0; d.even && base < a.B; base += 32) {
    const TreeSeq s = base ? tree_lane_seq(a, base) : first;
    all += __reduce_add_sync(0xffffffffu, d.head_parts(s) * a.Hkv);
    d.even = __all_sync(0xffffffffu, d.largest(s) <= d.each + kTreeSwitch) && all <= sms;
  }
  if (d.even) d.ctas = all;
  const int mine = d.even ? c : d.at(c);
  int at = 0;
  walk.none();
  if (c >= d.ctas) return d;
#pragma unroll 1
  for (int base = 0; base < a.B; base += 32) {
    const TreeSeq s = base ? tree_lane_seq(a, base) : first;
    const int own = (d.even ? d.head_parts(s) : s.head()) * a.Hkv;
    int inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const int r = mine - at - (inc - own);
    const unsigned int hit = __ballot_sync(0xffffffffu, r >= 0 && r < own);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const TreeSeq it(a.G, __shfl_sync(0xffffffffu, s.n, src), __shfl_sync(0xffffffffu, s.live, src));
      walk.begin(d, it, c, base + src, __shfl_sync(0xffffffffu, r, src));
      break;
    }
    at += __shfl_sync(0xffffffffu, inc, 31);
  }
  return d;
}

// ---- TMEM helpers of this kernel -----------------------------------------------------------

// 64 consecutive columns of 32 lanes into registers (thread t of the warp reads lane base + t): two loads
// in flight, one wait.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float* v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]),
        "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]),
        "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 registers into 32 consecutive columns, without waiting (tmem_wait_st follows).
__device__ __forceinline__ void tmem_put32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// One thread of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Two fp32 values in one register pair: one instruction for both (1% off the short caches, half of one elsewhere).
__device__ __forceinline__ uint64_t pair2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair2(uint64_t r, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

__device__ __forceinline__ float max3(float x, float y, float z) { return fmaxf(fmaxf(x, y), z); }

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// MMAs whose shared-memory descriptors are given by their low word (address >> 4 in bits 0-13, leading
// byte offset lbo above): the high word (stride 1024 bytes, version 1, 128-byte swizzle) is the same for all.
constexpr uint32_t kTreeDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t lbo, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo | (lbo >> 4) << 16), "r"(b_lo | (lbo >> 4) << 16), "r"(idesc), "r"(accumulate), "r"(kTreeDescHi)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: A holds two 16-bit values along k in each 32-bit column.
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t lbo, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo | (lbo >> 4) << 16), "r"(idesc), "r"(accumulate), "r"(kTreeDescHi)
      : "memory");
}

// A warp's common value, told to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

template <bool BF16>
__device__ __forceinline__ uint32_t tree_pack(float x, float y) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool BF16>
__device__ __forceinline__ bool tree_finite(uint16_t bits) {
  constexpr uint32_t e = BF16 ? 0x7F80u : 0x7C00u;
  return (bits & e) != e;
}

// All eight: x 0 summed is zero, or NaN where a value is not finite.
template <bool BF16>
__device__ __forceinline__ bool tree_all_finite(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (BF16) {
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 s = zero;
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), zero, s);
    return __hbeq2(s, zero);
  } else {
    const __half2 zero = __floats2half2_rn(0.f, 0.f);
    __half2 s = zero;
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __hfma2(*reinterpret_cast<const __half2*>(&w[i]), zero, s);
    return __hbeq2(s, zero);
  }
}

// values out[at .. at + 8) of one row
__device__ __forceinline__ void tree_store8(const TreeAttnArgs& a, size_t at, const float* x) {
  if (a.out_type == ORTHRUS_BF16_PLANES) {
    __nv_bfloat16* o = (__nv_bfloat16*)a.out + at;
    st_split_x8(o, o + a.out_lo, x);
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = a.out_type == ORTHRUS_BF16 ? tree_pack<true>(x[2 * i], x[2 * i + 1]) : tree_pack<false>(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>((uint16_t*)a.out + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- the kernel -------------------------------------------------------------------------------

// Waits as in ptx.cuh; what a wait that is not over at once takes is one function for all of them, because
// this kernel is a few short loops whose time goes to instruction fetches when its code is large.
__device__ __noinline__ bool tree_wait_on(uint64_t* bar, uint32_t parity, int* status) {
  return mbar_wait(bar, parity, status);
}
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, int* status) {
  return mbar_try_wait(bar, parity) || tree_wait_on(bar, parity, status);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKb,
                          const __grid_constant__ CUtensorMap tmVb, const TreeAttnArgs a) {
  using S = TreeSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem + S::kQ;
  uint8_t* ring = smem + S::kRing;
  TreeMisc& ms = *reinterpret_cast<TreeMisc*>(smem + S::kMisc);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int kHalves = D / 64;
  constexpr int kHalf = kTreeKeys * 128, kQHalf = 128 * 128;  // bytes of 64 columns of a K/V tile, of a q tile
  constexpr uint32_t idS = BF16 ? idesc_bf16(128, kTreeKeys, false) : idesc_f16(128, kTreeKeys, false);
  constexpr uint32_t idO = BF16 ? idesc_bf16(128, D, true) : idesc_f16(128, D, true);

  if (warp == kTreeLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmKb);
    tma_prefetch_desc(&tmVb);
  }
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&ms.full[s], 1);
      mbar_init(&ms.empty[s], 2);
    }
    mbar_init(&ms.q_full, 1);
    mbar_init(&ms.q_empty, 2);
#pragma unroll 1
    for (int s = 0; s < 4; ++s) {
      mbar_init(&ms.s_full[s], 1);
      mbar_init(&ms.p_full[s], 4);
    }
    mbar_init(&ms.o_done[0], 1);
    mbar_init(&ms.o_done[1], 1);
    mbar_init(&ms.o_last[0], 1);
    mbar_init(&ms.o_last[1], 1);
    mbar_init(&ms.seg_done, 2);
    mbar_init(&ms.done[0], 1);
    mbar_init(&ms.done[1], 1);
    ms.bad_any = 0;
    for (int i = 0; i < 8; ++i) ms.bad[i] = 0u;
    fence_barrier_init();
  }
  // rows of q's tiles past the largest unit's last piece: zero, so that their scores, and the weights that nobody
  // writes over them, are zero too: products of zeros take less power, which is what a long run has too little of
  {
    const int rows = min(kTreeRows, a.N * a.G), r0 = (rows + 31) / 32 * 32, r1 = rows > 128 ? kTreeRows : 128;
    for (int i = threadIdx.x; i < (r1 - r0) * (D / 8); i += kTreeThreads) {
      const int q = i / (D / 8), c = i - q * (D / 8), row = r0 + q;
      *reinterpret_cast<uint4*>(sQ + (row >> 7) * S::kQTile + (c >> 3) * kQHalf + (row & 127) * 128 + (c & 7) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  if (warp == kTreeMmaWarp) {
    tmem_alloc(&ms.tmem, 512);
    tmem_relinquish();
  }
  griddep_wait();  // lengths, masks, q and K/V come from earlier kernels
  griddep_launch();
  TreeWalk walk;
  const TreeShare share = tree_start(a, blockIdx.x, gridDim.x, walk);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;

  // of every role: segments, ring position of the segment (tiles go through the ring in the order of
  // their use: `ahead` tiles of K, then V and K in turn), and whether no wait has run out. After that both
  // stand still; the load warp's are then the counts of the q and the tiles whose copies it has issued
  uint32_t seg = 0, base = 0;
  bool ok = true;
  // MMA warps: jobs of each stream so far, and the last segment's kind
  const bool issue = elect_one();
  const uint32_t mine = warp - kTreeMmaWarp;
  uint32_t c0 = 0, c1 = 0;
  bool was_two = false;
  // softmax: stream, row of the 128, jobs so far
  const int st = warp >> 2, r = (warp & 3) * 32 + lane;
  uint32_t cnt = 0, ends = 0;  // and segments in which the stream had a job
  // note warp: the unit's cost before the range (line)
  const int skipped = walk.left - (share.at(blockIdx.x + 1) - share.at(blockIdx.x));
  int4 note = make_int4(-1, 0, 0, 0);

  TreeSeg g;
#pragma unroll 1
  while (walk.next(a, g)) {
    const int nt = uniform(g.t1 - g.t0), ct = (g.n + kTreeKeys - 1) / kTreeKeys;
    const bool two = uniform(g.two);
    const int ahead = two ? 2 : 4;

    if (warp < 8) {
      // ---- softmax: thread = row ----
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + lanes + st * 128, tO = tmem + lanes + 256;
      const float sl = a.scale_log2;
      const int unit_rows = g.live * a.G - g.rg * kTreeRows;  // rows from this group on
      const int lrow = (two ? st * 128 : 0) + r;              // row within the group
      const bool row_ok = lrow < unit_rows;
      const bool warp_ok = lrow - lane < unit_rows;           // the warp has a row
      const int row = g.rg * kTreeRows + lrow, node = row_ok ? row / a.G : 0;
      const unsigned long long* words = a.mask + ((size_t)g.b * a.N + node) * a.words;
      // the word of the segment's first tree tile of this stream, ahead of its use
      const int every = two ? 1 : 2, k0 = two ? 0 : st;
      int kb = max(k0, ct - g.t0);
      kb += (kb - k0) & (every - 1);
      unsigned long long word = kb < nt ? words[kb + g.t0 - ct] : 0ull;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int k = k0; k < nt; k += every) {
        const int t = g.t0 + k, bt = t - ct;
        const bool blk = t >= ct;
        const int lim = blk ? g.live - bt * kTreeKeys : g.n - t * kTreeKeys;  // keys of the tile, if below 64
        const uint32_t buf = cnt & 1;
        if (ok) ok = tree_wait(&ms.s_full[2 * st + buf], (cnt >> 1) & 1, a.status);
        ok = __all_sync(0xffffffffu, ok);
        const bool part = blk || lim < kTreeKeys;
        if (part) {
          // thread r looks after half of key r & 63: V rows that nobody may see become zero, and values that are
          // not finite are marked and leave the product. With two streams on the tile both do it: each one's
          // products follow its own pass, and the later one finds values already marked. A key's row is 128
          // bytes of each half of the columns: the threads start at different 16 bytes of theirs, on different
          // banks. (The wait is after that for the scores: then the stage's earlier laps are over, and its parity
          // is this lap's.)
          const uint32_t pos = base + tree_pos_v(k, ahead, nt), s = pos % S::kStages;
          if (ok) ok = tree_wait(&ms.full[s], (pos / S::kStages) & 1, a.status);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            const int key = r & 63, q0 = (r >> 6) * 4 * kHalves;
            uint4* vr = reinterpret_cast<uint4*>(ring + s * S::kTile + key * 128);
            auto piece = [&](int q) -> uint4& { return vr[((q0 + q) >> 3) * (kHalf / 16) + ((q0 + q + key) & 7)]; };
            if (key >= lim) {
#pragma unroll
              for (int q = 0; q < 4 * kHalves; ++q) piece(q) = make_uint4(0u, 0u, 0u, 0u);
            } else if (blk) {
              bool fine = true;
#pragma unroll
              for (int q = 0; q < 4 * kHalves; ++q) fine = fine && tree_all_finite<BF16>(piece(q));
              if (!fine) {
                const int j = bt * kTreeKeys + key;
                atomicOr(&ms.bad[j >> 5], 1u << (j & 31));
                ms.bad_any = 1;
                __threadfence_block();
#pragma unroll 1
                for (int q = 0; q < 32 * kHalves; ++q) {
                  uint16_t* x = reinterpret_cast<uint16_t*>(&piece(q >> 3)) + (q & 7);
                  if (!tree_finite<BF16>(*x)) *x = 0;
                }
              }
            }
            fence_proxy_async_smem();
          }
        }
        if (ok && warp_ok) {
          tc_fence_after();
          float v[64];
          tmem_ld64(tS + buf * 64, v);
          if (part) {
            uint32_t s0 = ~0u, s1 = ~0u;
            if (lim < kTreeKeys) {
              s0 = lim >= 32 ? ~0u : (1u << lim) - 1u;
              s1 = lim > 32 ? (1u << (lim - 32)) - 1u : 0u;
            }
            if (blk) {
              s0 &= (uint32_t)word;
              s1 &= (uint32_t)(word >> 32);
              if (k + every < nt) word = words[bt + every];
            }
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (!((i < 32 ? s0 >> i : s1 >> (i - 32)) & 1u)) v[i] = -INFINITY;
          }
          float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int i = 4; i < 60; i += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], v[i + 2 * q], v[i + 2 * q + 1]);
          const float mt = max3(max3(mx[0], mx[1], v[60]), max3(mx[2], mx[3], v[61]), fmaxf(v[62], v[63])) * sl;
          if (k == k0) {
            m = mt;
          } else {
            const bool move = row_ok && mt > m + kTreeSlack;
            if (__any_sync(0xffffffffu, move)) {
              // the stream's last product is complete before its sums are scaled (the one before it is: these scores
              // were issued after it)
              ok = __all_sync(0xffffffffu, tree_wait(&ms.o_done[st], (cnt - 1) & 1, a.status));
              if (ok) {
                tc_fence_after();
                const float f = move ? fast_exp2(m - mt) : 1.f;
                l *= f;
                if (move) m = mt;
#pragma unroll 1
                for (int e = 0; e < D; e += 32) {
                  float o[32];
                  tmem_ld32(tO + st * 128 + e, o);
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] *= f;
                  tmem_st32(tO + st * 128 + e, o);
                }
              }
            }
          }
          const float shift = !row_ok ? INFINITY : m == -INFINITY ? 0.f : m - kTreeShift;  // no row: weights of zero
          const uint64_t scale2 = pair2(sl, sl), shift2 = pair2(-shift, -shift);
          uint64_t sum[2] = {0ull, 0ull};
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float p0, p1;
            unpair2(fma2(pair2(v[2 * i], v[2 * i + 1]), scale2, shift2), p0, p1);
            p0 = fast_exp2(p0);
            p1 = fast_exp2(p1);
            sum[i & 1] = add2(sum[i & 1], pair2(p0, p1));
            pk[i] = tree_pack<BF16>(p0, p1);
          }
          tmem_put32(tS + buf * 64, pk);
          float s0, s1;
          unpair2(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&ms.p_full[2 * st + buf]);
        ++cnt;
      }

      // ---- the segment's sums ----
      // a barrier of their own: of o_done's phases the last two may both be under way, or both over when a warp
      // comes here late, and a parity does not tell these apart
      if (two || nt > st) {
        if (ok) ok = tree_wait(&ms.o_last[st], ends & 1, a.status);
        ++ends;
      }
      ok = __all_sync(0xffffffffu, ok);
      float w0 = 1.f, w1 = 0.f;
      int e0 = 0, e1 = D;
      if (!two) {
        // both streams hold sums of the same rows: each joins one half of the columns
        if (st) ms.ml[r] = make_float2(m, l);
        named_bar_sync(1, 256);
        const float2 ml1 = ms.ml[r];
        named_bar_sync(2, 256);
        if (!st) ms.ml[r] = make_float2(m, l);
        named_bar_sync(1, 256);
        const float2 ml0 = ms.ml[r];
        m = fmaxf(ml0.x, ml1.x);
        const float ref = m == -INFINITY ? 0.f : m;
        w0 = fast_exp2(ml0.x - ref);
        w1 = fast_exp2(ml1.x - ref);
        l = ml0.y * w0 + ml1.y * w1;
        e0 = st ? D / 2 : 0;
        e1 = st ? D : D / 2;
      }
      bool bad = *(volatile int*)&ms.bad_any != 0;
      if (ok && warp_ok) {
        tc_fence_after();
        const bool whole = g.whole();
        if (whole) {  // the quotient's factor into the weights
          const float inv = l == 0.f ? 0.f : 1.f / l;
          w0 *= inv;
          w1 *= inv;
        }
        const size_t at = (((size_t)g.b * a.N + node) * a.Hkv * a.G + (size_t)g.kvh * a.G + (row - node * a.G)) * D;
        float4* po = a.part_o + (size_t)g.slot * (D / 4) * kTreeRows + lrow;
#pragma unroll 1
        for (int e = e0; e < e1; e += 16) {
          float o[16], x[16];
          tmem_ld16(tO + (two ? st * 128 : 0) + e, o);
          if (!two && nt > 1) {
            tmem_ld16(tO + 128 + e, x);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = o[i] * w0 + x[i] * w1;
          if (bad && row_ok) {
#pragma unroll 1
            for (int j = 0; j < g.live; ++j)
              if ((ms.bad[j >> 5] >> (j & 31) & 1u) && (words[j >> 6] >> (j & 63) & 1ull)) {
                const size_t vat = ((size_t)(g.b * a.Hkv + g.kvh) * a.blk_stride + j) * D + e;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float y = BF16 ? __bfloat162float(((const __nv_bfloat16*)a.v_blk)[vat + i])
                                       : __half2float(((const __half*)a.v_blk)[vat + i]);
                  if (!isfinite(y)) o[i] += y;
                }
              }
          }
          if (!row_ok) continue;
          if (whole) {
            tree_store8(a, at + e, o);
            tree_store8(a, at + e + 8, o + 8);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              po[(size_t)(e / 4 + i) * kTreeRows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (!whole && row_ok && (two || !st)) a.part_ml[(size_t)g.slot * kTreeRows + lrow] = make_float2(m, l);
      }
      tc_fence_before();
      bad = named_bar_or(2, 256, bad);  // O and the marks are read before the next segment writes them
      if (bad) {
        if (threadIdx.x < 8) ms.bad[threadIdx.x] = 0u;
        if (threadIdx.x == 0) ms.bad_any = 0;
        named_bar_sync(1, 256);
      }
    } else if (warp == kTreeLoadWarp) {
      // ---- loads: K and V in the order of their use, and q when the first K tiles are on their way (they
      // fill free stages while the last segment's scores still read its q) ----
      if (lane == 0 && ok) {
        // one row group: K and V are read once, and the parts of cut units stay in L2; several: the other
        // groups' CTAs read the same tiles
        const uint64_t once = a.N * a.G > kTreeRows ? policy_evict_normal() : policy_evict_first();
        const int z = g.b * a.Hkv + g.kvh, lead = min(ahead, nt);
#pragma unroll 1
        for (int p = 0; p < 2 * nt; ++p) {
          if (p == lead) {
            const int pieces = (min(kTreeRows, g.live * a.G - g.rg * kTreeRows) + 31) / 32;  // of q, 32 rows each
            if (seg > 0 && !(ok = tree_wait(&ms.q_empty, (seg - 1) & 1, a.status))) {
              base += p;
              break;
            }
            // rows of the 128-row tiles past the last piece keep what they hold: no sum of another row sees them
            mbar_arrive_expect_tx(&ms.q_full, pieces * (S::kQTile / 4));
            const int qrow = z * a.N * a.G + g.rg * kTreeRows;
#pragma unroll 1
            for (int h = 0; h < pieces; ++h)
              for (int e = 0; e < kHalves; ++e)
                tma_load_2d(sQ + (h >> 2) * S::kQTile + e * kQHalf + (h & 3) * (kQHalf / 4), &tmQ, &ms.q_full, e * 64,
                            qrow + h * 32);
          }
          // position p: K first, then V and K in turn, V last
          const bool val = p >= lead && (p >= 2 * nt - lead || ((p - lead) & 1) == 0);
          const int k = p < lead ? p : (p >= 2 * nt - lead ? p - nt : (p - lead) / 2 + (val ? 0 : lead));
          const uint32_t pos = base + p, s = pos % S::kStages, lap = pos / S::kStages;
          if (!(ok = tree_wait(&ms.empty[s], (lap & 1) ^ 1u, a.status))) {
            base += p;
            seg += p >= lead ? 1 : 0;
            break;
          }
          mbar_arrive_expect_tx(&ms.full[s], S::kTile);
          const int t = g.t0 + k;
          const bool blk = t >= ct;
          const CUtensorMap* map = val ? (blk ? &tmVb : &tmV) : (blk ? &tmKb : &tmK);
          const int y = (blk ? t - ct : t) * kTreeKeys;
          uint8_t* dst = ring + s * S::kTile;
#pragma unroll
          for (int e = 0; e < kHalves; ++e) tma_load_3d_hint(dst + e * kHalf, map, &ms.full[s], e * 64, y, z, once);
        }
      }
    } else if (warp <= kTreeMmaWarp + 1) {
      // ---- products: S = Q K^T, two jobs of a stream ahead of O += P V. With more than 128 rows the streams
      // have a warp each (the instruction latency of this loop, not the products, would otherwise set the
      // pace) and a stage is free after a commit of each; else the first warp serves both streams, sees every
      // stage in order, and commits twice. The whole warp runs the loop on warp-uniform values, one elected
      // thread issues.
      // seg_done: both warps have issued a segment's products and they are complete. Each warp sees every
      // phase: before its scores where the streams change hands (the S buffers' last readers were issued by
      // the other warp), else before its sums ----
      const bool early = two != was_two;
      was_two = two;
      if (ok && early && seg > 0) ok = tree_wait(&ms.seg_done, (seg - 1) & 1, a.status);
      if (two || mine == 0) {
        const uint32_t r_desc = uniform(smem_u32(ring) >> 4), tm = uniform(tmem);
        const uint32_t qd = uniform(smem_u32(sQ) >> 4) + (two ? mine * (S::kQTile >> 4) : 0);
        // job of tile k: its stream, and the stream's job number
        auto stream = [&](int k) { return two ? mine : (uint32_t)k & 1u; };
        auto job = [&](int k) { return two ? (mine ? c1 : c0) + k : ((k & 1) ? c1 : c0) + (k >> 1); };
        if (ok) ok = tree_wait(&ms.q_full, seg & 1, a.status);
#pragma unroll 1
        for (int k = -ahead; ok && k < nt; ++k) {
          if (k == 0 && !early && seg > 0 && !(ok = tree_wait(&ms.seg_done, (seg - 1) & 1, a.status))) break;
          if (k >= 0) {
            const uint32_t pos = base + tree_pos_v(k, ahead, nt), s = pos % S::kStages;
            const uint32_t sk = stream(k), n = job(k), buf = 2 * sk + (n & 1u);
            ok = tree_wait(&ms.p_full[buf], (n >> 1) & 1u, a.status) &&
                 tree_wait(&ms.full[s], (pos / S::kStages) & 1, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t to = tm + 256 + sk * 128, from = tm + buf * 64, vd = r_desc + s * (S::kTile >> 4);
            const uint32_t add = k >= (two ? 1 : 2) ? 1u : 0u;  // the stream's first job of the segment starts its sums
            if (issue) {
#pragma unroll
              for (int i = 0; i < kTreeKeys / 16; ++i)
                mma_ts_lo(to, from + i * 8, vd + i * (2048 >> 4), kHalf, idO, i > 0 ? 1u : add);
              mma_commit(&ms.o_done[sk]);
              if (k + (two ? 1 : 2) >= nt) mma_commit(&ms.o_last[sk]);
              mma_commit(&ms.empty[s]);
              if (!two) mma_commit(&ms.empty[s]);
            }
          }
          const int kn = k + ahead;
          if (kn < nt) {
            const uint32_t pos = base + tree_pos_k(kn, ahead), s = pos % S::kStages;
            const uint32_t buf = 2 * stream(kn) + (job(kn) & 1u);
            ok = tree_wait(&ms.full[s], (pos / S::kStages) & 1, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t to = tm + buf * 64, kd = r_desc + s * (S::kTile >> 4);
            if (issue) {
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
                mma_ss_lo(to, qd + (((i >> 2) * kQHalf + (i & 3) * 32) >> 4), kd + (((i >> 2) * kHalf + (i & 3) * 32) >> 4),
                          16, idS, i > 0 ? 1u : 0u);
              mma_commit(&ms.s_full[buf]);
              mma_commit(&ms.empty[s]);
              if (!two) mma_commit(&ms.empty[s]);
              if (kn == nt - 1) {
                mma_commit(&ms.q_empty);
                if (!two) mma_commit(&ms.q_empty);
              }
            }
          }
        }
        if (ok && issue) mma_commit(&ms.seg_done);
      } else {
        if (ok && !early && seg > 0) ok = tree_wait(&ms.seg_done, (seg - 1) & 1, a.status);
        if (ok && issue) mbar_arrive(&ms.seg_done);
      }
      c0 += two ? nt : (nt + 1) >> 1;
      c1 += two ? nt : nt >> 1;
    } else if (seg == 0 && g.t0 > 0) {
      // ---- for the joining kernel: whether this CTA has the second part of a unit that is cut ----
      const int c = blockIdx.x;
      int last = c;
      if (share.even) {
        last = walk.part == 1 ? c + walk.parts - 2 : -1;
      } else {
        const int u0 = share.at(c) - skipped, tail = u0 + kTreeUnit + (g.tiles - 1) * (two ? kTreeCost2 : kTreeCost1);
        if (share.at(c - 1) > u0) last = -1;
        else
          while (last + 1 < share.ctas && share.at(last + 1) <= tail) ++last;
      }
      if (last >= 0) note = make_int4(g.b, g.kvh, g.rg << 16 | min(kTreeRows, g.live * a.G - g.rg * kTreeRows), last);
    }
    if (ok) {
      base += 2 * nt;
      ++seg;
    }
  }

  if (warp == kTreeLoadWarp) {
    // copies in flight land before the CTA ends: the last q and the last use of each stage, of what was issued
    if (lane == 0) {
      bool landed = seg == 0 || tree_wait(&ms.q_full, (seg - 1) & 1, a.status);
#pragma unroll 1
      for (uint32_t k = tree_pos_last(base, S::kStages); landed && k < base; ++k)
        landed = tree_wait(&ms.full[k % S::kStages], (k / S::kStages) & 1, a.status);
    }
  } else if (warp >= kTreeMmaWarp && warp <= kTreeMmaWarp + 1) {
    if (issue) mma_commit(&ms.done[mine]);
    tree_wait(&ms.done[mine], 0, a.status);
  } else if (warp == kTreeNoteWarp && lane == 0) {
    a.note[blockIdx.x] = note;
  }
  if (blockIdx.x == 0 && warp < 8)
    for (int b = threadIdx.x; b < a.B; b += 256)
      if (a.len[b] < 0 || a.len[b] > a.cap) set_status(a.status, a.len[b] < 0 ? ORTHRUS_ERR_ARG : ORTHRUS_ERR_CAPACITY);

  tc_fence_before();
  __syncthreads();
  if (warp == kTreeMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- joining the parts of a cut unit ---------------------------------------------------------

// CTA x takes the x-th of the notes that name a cut unit, and joins 32 rows of its parts, thread = (row,
// 4 columns of each of E column groups), in key order:
//     out = sum_c w_c O_c / sum_c w_c l_c,   w_c = 2^(m_c - max m),
// P parts at a time with a running maximum, all their loads in flight together. Bound by the latency of
// two dependent loads from L2 (notes, parts), the wait for the first kernel, and fetching its own code: with
// E = 1, P = 16 instead of 8 takes 2 us longer at 18 parts.
constexpr int kJoinThreads = 256;

template <int E>
__global__ void __launch_bounds__(kJoinThreads) tree_combine_kernel(const TreeAttnArgs a, int sms) {
  constexpr int P = E == 1 ? 8 : 16 / E;
  __shared__ int before[kJoinThreads / 32];
  __shared__ int4 found;
  __shared__ int found_at;
  const int r = threadIdx.x & 31, part = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch();
  if (threadIdx.x == 0) found_at = -1;
  int left = blockIdx.x;
  for (int c = 1; c < sms; c += kJoinThreads) {
    const int4 note = c + (int)threadIdx.x < sms ? __ldcg(&a.note[c + threadIdx.x]) : make_int4(-1, 0, 0, 0);
    const unsigned int bal = __ballot_sync(0xffffffffu, note.x >= 0);
    __syncthreads();
    if (r == 0) before[part] = __popc(bal);
    __syncthreads();
    int at = __popc(bal & ((1u << r) - 1u)), all = 0;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      if (w < part) at += before[w];
      all += before[w];
    }
    if (note.x >= 0 && at == left) {
      found = note;
      found_at = c + threadIdx.x;
    }
    left -= all;
  }
  __syncthreads();
  if (found_at < 0) return;
  const int4 note = found;
  const int rg = note.z >> 16, rows = note.z & 0xffff, c0 = found_at - 1, n = note.w - c0 + 1;
  const int lrow = blockIdx.y * 32 + r;
  if ((int)blockIdx.y * 32 >= rows) return;
  const int e4 = blockIdx.z * 8 * E + part;  // and every 8th from there
  const float2* ml = a.part_ml + lrow;
  const float4* po = a.part_o + (size_t)e4 * kTreeRows + lrow;
  float top = -INFINITY, l = 0.f;
  float4 o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += P) {
    float2 m[P];
    float4 x[P][E];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      m[i] = make_float2(-INFINITY, 0.f);
      if (i0 + i < n) {
        // slot of part i: all but the first start inside the unit and use their CTA's first slot
        const size_t slot = (size_t)(2 * (c0 + i0 + i) + (i0 + i == 0 ? 1 : 0));
        m[i] = __ldcg(ml + slot * kTreeRows);
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] = __ldcg(po + (slot * (a.d / 4) + 8 * e) * kTreeRows);
      }
    }
    float next = top;
#pragma unroll
    for (int i = 0; i < P; ++i) next = fmaxf(next, m[i].x);
    const float ref = next == -INFINITY ? 0.f : next, f = fast_exp2(top - ref);
    top = next;
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = make_float4(o[e].x * f, o[e].y * f, o[e].z * f, o[e].w * f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (i0 + i < n) {
        const float w = fast_exp2(m[i].x - ref);
        l += m[i].y * w;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          o[e].x += x[i][e].x * w;
          o[e].y += x[i][e].y * w;
          o[e].z += x[i][e].z * w;
          o[e].w += x[i][e].w * w;
        }
      }
    }
  }
  if (lrow >= rows) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int row = rg * kTreeRows + lrow, node = row / a.G;
  const size_t to = (((size_t)note.x * a.N + node) * a.Hkv * a.G + (size_t)note.y * a.G + (row - node * a.G)) * a.d + e4 * 4;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float y[4] = {o[e].x * inv, o[e].y * inv, o[e].z * inv, o[e].w * inv};
    uint2* dst = reinterpret_cast<uint2*>((uint16_t*)a.out + to + 32 * e);
    if (a.out_type == ORTHRUS_FP16) {
      *dst = make_uint2(tree_pack<false>(y[0], y[1]), tree_pack<false>(y[2], y[3]));
    } else if (a.out_type == ORTHRUS_BF16) {
      *dst = make_uint2(tree_pack<true>(y[0], y[1]), tree_pack<true>(y[2], y[3]));
    } else {
      uint32_t h0, h1, l0, l1;
      split_bf16x2(y[0], y[1], h0, l0);
      split_bf16x2(y[2], y[3], h1, l1);
      *dst = make_uint2(h0, h1);
      *reinterpret_cast<uint2*>((uint16_t*)a.out + a.out_lo + to + 32 * e) = make_uint2(l0, l1);
    }
  }
}

}  // namespace orthrus
