// Internal interface between the C-ABI layer of the layer operators
// (block_api.cu) and their kernel translation units.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "flce_internal.h"

namespace flce {

struct LinearArgs;
struct GatedArgs;
struct GradXArgs;
struct GradWArgs;

// GEMMs of the layer operators (block_gemm.cu). `two`: the gated operator's
// two-operand plan.
cudaError_t launch_linear(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b,
                          const GemmGeom& g, const LinearArgs& ea, int* dev_err, int sms,
                          cudaStream_t st);
cudaError_t launch_gated(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b,
                         const GemmGeom& g, const GatedArgs& ea, int* dev_err, int sms,
                         cudaStream_t st);
cudaError_t launch_grad_x(GemmKind kind, bool two, const CUtensorMap& a, const CUtensorMap& b,
                          const GemmGeom& g, const GradXArgs& ea, int* dev_err, int sms,
                          cudaStream_t st);
cudaError_t launch_grad_w(GemmKind kind, bool two, const CUtensorMap& a, const CUtensorMap& b,
                          const GemmGeom& g, const GradWArgs& ea, int* dev_err, int sms,
                          cudaStream_t st);

// Element-wise parts of the backward passes (block_rowwise.cu).
struct DzArgs {
  const uint16_t* dy;  // [M, ld_dy]
  int64_t ld_dy;
  const uint16_t* z;   // [M, N] pre-activations, or null (activation "none")
  uint16_t* dz;        // [M, ld_dz], or null: column sums only
  int64_t ld_dz;
  float* part;         // [dz_parts(M, N), N] column sums of dz, or null
  int M, N, act, fp16;
  int vec;             // dy, z and dz rows start on 16-byte boundaries
};
int dz_parts(int64_t M, int64_t N);
cudaError_t launch_dz(const DzArgs& a, cudaStream_t st);

struct GatedGradArgs {
  const uint16_t* dh;  // [M, ld_dh]
  int64_t ld_dh;
  const uint16_t* g;   // [M, F]
  const uint16_t* u;   // [M, F]
  uint16_t* dg;        // [M, F]
  uint16_t* du;        // [M, F]
  int M, F, act, fp16;
};
cudaError_t launch_gated_grad(const GatedGradArgs& a, cudaStream_t st);

}  // namespace flce
