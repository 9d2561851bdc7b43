// Order and bookkeeping of the loads of tree_attention.cuh: plain integer arithmetic, also for the host.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define ORTHRUS_HD __host__ __device__ __forceinline__
#else
#define ORTHRUS_HD inline
#endif

namespace orthrus {

// Ring positions of a segment's nt tiles: `ahead` tiles of K, then V and K in turn.
ORTHRUS_HD uint32_t tree_pos_k(int k, int ahead) { return k + (k >= ahead ? k - ahead + 1 : 0); }
ORTHRUS_HD uint32_t tree_pos_v(int k, int ahead, int nt) { return k + (k + ahead < nt ? k + ahead : nt); }

// First of the last uses of the stages, when positions 0 .. pos - 1 have been issued. (An earlier use of a stage had
// landed before the stage was filled again.)
ORTHRUS_HD uint32_t tree_pos_last(uint32_t pos, uint32_t stages) { return pos > stages ? pos - stages : 0; }

}  // namespace orthrus
