// Host helpers shared by the library's translation units: tensor-map encoding, launch
// attributes, the shared-memory opt-in.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <utility>
#include <vector>

namespace {

// ---------------------------------------------------------------------------
// driver entry point for tensor-map encoding (no link against libcuda)
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)p;
  }
  return fn;
}

constexpr CUtensorMapDataType kBF16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapDataType kF16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;

// 2D map of 16-bit elements over a row-major [rows][cols] matrix; box = box_cols x box_rows,
// 128-byte swizzle.
bool map2d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols, uint32_t box_rows,
           CUtensorMapDataType dt = kBF16) {
  EncodeTiledFn f = encode_fn();
  if (!f || !base) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  return f(m, dt, 2, const_cast<void*>(base), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3D map of 16-bit elements over [z][rows][cols]; box = 64 cols x box_rows rows x box_z.
bool map3d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t z, uint32_t box_rows = 128,
           uint32_t box_z = 1, CUtensorMapDataType dt = kBF16) {
  EncodeTiledFn f = encode_fn();
  if (!f || !base) return false;
  cuuint64_t dims[3] = {cols, rows, z};
  cuuint64_t strides[2] = {cols * 2, cols * rows * 2};
  cuuint32_t box[3] = {64, box_rows, box_z};
  cuuint32_t es[3] = {1, 1, 1};
  return f(m, dt, 3, const_cast<void*>(base), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 map of rank 3 or 4 with explicit strides (bytes, dims 1..rank-1) and box.
bool map_nd(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
            const uint32_t* box) {
  EncodeTiledFn f = encode_fn();
  if (!f || !base || rank < 3 || rank > 4) return false;
  cuuint64_t d[4], st[3];
  cuuint32_t b[4], es[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
  }
  for (int i = 0; i < rank - 1; ++i) st[i] = strides[i];
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, st, b, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D view of a row-major [rows][cols] bf16 matrix as (64 columns, rows, cols/64 chunks) with
// strides (row, 128 B): a box of (64, box_rows, 2) is two consecutive 64-wide k chunks.
bool map_kpair(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
  const uint64_t dims[3] = {64, rows, cols / 64};
  const uint64_t strides[2] = {cols * 2, 128};
  const uint32_t box[3] = {64, box_rows, 2};
  return map_nd(m, base, 3, dims, strides, box);
}

// An activation in two planes [2][rows][cols] (hi, then lo), as (64 columns, rows, plane): a box
// of (64, box_rows, 2) is one 64-wide k chunk of both planes.
bool map_planes(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
  const uint64_t dims[3] = {cols, rows, 2};
  const uint64_t strides[2] = {cols * 2, cols * rows * 2};
  const uint32_t box[3] = {64, box_rows, 2};
  return map_nd(m, base, 3, dims, strides, box);
}

// The same as (64 columns, rows, plane, cols/64 chunks): a box of (64, box_rows, 2, 2) is two
// consecutive 64-wide k chunks of both planes, laid out [chunk][plane][row][64], so that per
// chunk the hi rows and then the lo rows form one MMA operand of 2 box_rows rows.
bool map_kpair_planes(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
  const uint64_t dims[4] = {64, rows, 2, cols / 64};
  const uint64_t strides[3] = {cols * 2, cols * rows * 2, 128};
  const uint32_t box[4] = {64, box_rows, 2, 2};
  return map_nd(m, base, 4, dims, strides, box);
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int round_up(int x, int a) { return (x + a - 1) / a * a; }
int next_pow2(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

int num_sms() {
  static int n = 0;
  if (!n) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  }
  return n;
}

constexpr size_t kSmemLimit = 232448;  // opt-in shared memory per CTA on sm_100

// Programmatic dependent launch for every kernel: a kernel may begin its prologue and
// weight loads while its predecessor drains; its griddepcontrol.wait orders everything else.

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename F>
bool set_smem_attr(F* kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

// The dynamic shared-memory opt-in is a property of (kernel, device): it is set once per
// pair, under a lock, so that host threads and calls on a second GPU each get it.
template <typename F>
bool ensure_smem_attr(F* kernel, size_t bytes) {
  static std::mutex mu;
  static std::vector<std::pair<int, const void*>> done;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const std::pair<int, const void*> key(dev, (const void*)kernel);
  try {  // no exception leaves a C entry point
    std::lock_guard<std::mutex> lock(mu);
    if (std::find(done.begin(), done.end(), key) != done.end()) return true;
    if (!set_smem_attr(kernel, bytes)) return false;
    done.push_back(key);
  } catch (...) {
    return false;
  }
  return true;
}

}  // namespace
