// Internal interface between the C-ABI layer of the layer operators
// (block_api.cu) and their kernel translation units.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "flce_internal.h"

namespace flce {

// Every kernel of the layer operators may start while its predecessor on the stream
// still runs (programmatic dependent launch): it sets up its barriers and TMEM and
// then waits, in all threads and before its first access to global memory, until
// the predecessor has completed and its writes are visible. It lets its own
// successor start in the same way once all its blocks are running.
#ifdef __CUDACC__
__device__ __forceinline__ void griddep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void griddep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class... P, class... A>
static cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                                    int cluster, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

struct PairArgs;
struct LinearArgs;
struct GatedArgs;
struct GradXArgs;
struct GradWArgs;

// GEMMs of the layer operators (block_gemm.cu). `two`: the gated operator's
// two-operand plan.
cudaError_t launch_linear(const PairArgs& g, const LinearArgs& ea, int sms, cudaStream_t st);
cudaError_t launch_gated(const PairArgs& g, const GatedArgs& ea, int sms, cudaStream_t st);
cudaError_t launch_grad_x(bool two, const PairArgs& g, const GradXArgs& ea, int sms,
                          cudaStream_t st);
cudaError_t launch_grad_w(bool two, const PairArgs& g, const GradWArgs& ea, int sms,
                          cudaStream_t st);

// Few-token products (block_small.cu): y [M, N] = epilogue of x Wt^T, with the
// weights on the MMA's rows. w: boxes of 128 features x 64 sum elements (64 x 64
// with the features contiguous, or for the gated projection); x: 64 sum elements x small_tokens(M) tokens.
struct SmallArgs {
  CUtensorMap w, w2, x, x2;  // x, x2: above 32 tokens only
  const uint16_t *xp, *xp2;  // x and the second segment's, [M, ld_x]
  const uint16_t* wp;        // weights [N, k_len] of the activation's argument, with keep
  int64_t ld_x;
  int k_len;                 // sum elements of a segment
  const uint16_t* bias;
  const uint16_t* res;
  uint16_t* keep;  // for the backward (block_epilogues.cuh): [M, N], or [2, M, N] (gated); or null
  uint16_t* y;
  int64_t ld_res, ld_y;
  int res_vec, y_vec;  // rows start on 16-byte boundaries
  int act, fp16;
  int relative;    // keep in the relative form
  int M, N;
  int k_blocks, k_split;  // blocks of 64 of the whole sum; those of the first segment
  int slices;             // K slices = cluster size: 1, 2, 4 or 8
  int* dev_err;
};
int small_tokens(int64_t M);  // tokens of a tile
int64_t small_tiles(int64_t M, int64_t N, bool two);
int64_t small_clusters(int64_t M, int slices);
int small_slices(int64_t M, int64_t N, int k_blocks, bool two);
cudaError_t launch_small(bool two, bool w_mn, const SmallArgs& a, cudaStream_t st);

// Element-wise parts of the backward passes (block_rowwise.cu).
struct DzArgs {
  const uint16_t* dy;  // [M, ld_dy]
  int64_t ld_dy;
  const uint16_t* slope;  // [M, N] kept slopes, or null (activation "none")
  uint16_t* dz;        // [M, ld_dz], or null: column sums only
  int64_t ld_dz;
  float* part;         // [dz_parts(M, N), N] column sums of dz, or null
  int M, N, fp16;
  float tail;          // of decode_slope (block_epilogues.cuh)
  int vec;             // dy, slope and dz rows start on 16-byte boundaries
};
int dz_parts(int64_t M, int64_t N);
cudaError_t launch_dz(const DzArgs& a, cudaStream_t st);
cudaError_t launch_db_sum(const float* part, int parts, int N, void* db, bool fp32, bool fp16,
                          cudaStream_t st);

struct GatedGradArgs {
  const uint16_t* dh;  // [M, ld_dh]
  int64_t ld_dh;
  const uint16_t* val;    // [M, F] kept a(g)
  const uint16_t* cross;  // [M, F] kept u a'(g)
  uint16_t* dg;           // [M, ld]
  uint16_t* du;           // [M, ld]
  int64_t ld;
  int M, F, fp16;
  int relative;           // val and cross in the relative form
};
// A copy of 16-bit rows to another pitch; both on 16-byte boundaries, cols a multiple of 8.
cudaError_t launch_repack(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst,
                          int rows, int cols, cudaStream_t st);
cudaError_t launch_gated_grad(const GatedGradArgs& a, cudaStream_t st);

}  // namespace flce
