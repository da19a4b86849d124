// Host-side helpers shared by the C-ABI layers: TMA descriptor encoding, device
// checks, workspace carving, GEMM geometry and NVTX ranges.
#pragma once
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include "../../include/flce.h"
#include "gemm_engine.cuh"

namespace flce {

constexpr size_t kAlign = 256;
inline PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
inline std::once_flag g_encode_once;

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  std::call_once(g_encode_once, [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}

// 2-D 16-bit tensor [outer, inner] (bf16, or fp16 when fp16) with row pitch
// `pitch_bytes`, 128-B swizzled boxes of box_inner x box_outer elements;
// out-of-range elements read as 0.
inline bool encode_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
               uint64_t pitch_bytes, uint32_t box_inner, uint32_t box_outer, bool fp16) {
  auto fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {pitch_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// TMA store map of a row-major [outer, inner] output for the epilogues'
// 32 x 32 blocks: fp32 with the 128-byte swizzle (128-byte box rows) or a
// 16-bit type with the 64-byte swizzle (64-byte box rows), the staging layouts
// of epilogues.cuh. Stores are clipped to [inner, outer].
inline bool encode_store_2d(CUtensorMap* m, void* base, uint64_t inner, uint64_t outer,
                     uint64_t pitch_bytes, bool fp32) {
  auto fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {pitch_bytes};
  cuuint32_t box[2] = {32, 32};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base,
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            fp32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int cdiv(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SM count and architecture of the current device (asked once per device).
inline flce_status_t device_info(int* sms) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> known[kMaxDev];  // SM count of a supported device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FLCE_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDev) {
    *sms = known[dev].load(std::memory_order_relaxed);
    if (*sms > 0) return FLCE_OK;
  }
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FLCE_ERR_CUDA;
  if (major != 10 || minor != 3) return FLCE_ERR_UNSUPPORTED;
  if (dev >= 0 && dev < kMaxDev) known[dev].store(*sms, std::memory_order_relaxed);
  return FLCE_OK;
}

struct Carver {
  uintptr_t base, cur, end;
  explicit Carver(void* b, size_t n)
      : base(reinterpret_cast<uintptr_t>(b)),
        cur((reinterpret_cast<uintptr_t>(b) + kAlign - 1) & ~(kAlign - 1)),
        end(reinterpret_cast<uintptr_t>(b) + n) {}
  template <class T>
  T* take(size_t count) {
    T* r = reinterpret_cast<T*>(cur);
    cur = (cur + count * sizeof(T) + kAlign - 1) & ~(kAlign - 1);
    return r;
  }
  size_t used() const { return cur - base; }
};

inline GemmGeom geom(int M, int N, int K, bool fp16) {
  GemmGeom g;
  std::memset(&g, 0, sizeof(g));
  g.ab_fp16 = fp16 ? 1 : 0;
  g.M = M;
  g.N = N;
  g.K = K;
  g.tiles_m = cdiv(M, kBM);
  g.tiles_n = cdiv(N, kBN);
  g.k_blocks = cdiv(K, kBK);
  g.raster_m_inner = 1;
  return g;
}

inline int grid_for(const GemmGeom& g, int sms) {
  const int tiles = g.tiles_m * g.tiles_n;
  return tiles < sms ? tiles : sms;
}


// NVTX range over a scope (host timeline; free unless a profiler is attached),
// so Nsight Systems shows each call and each backward vocabulary block.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace flce
