// The backward of the root-mean-square norm of fp32 rows.
#include "rms_norm_grad.cuh"

cudaError_t flce::norm_grad_fp32(const NormGradArgs& a, bool, bool wide, const GradShape& s, cudaStream_t st) {
  return launch_grad<kFp32, kFp32>(a, wide, s, st);
}
