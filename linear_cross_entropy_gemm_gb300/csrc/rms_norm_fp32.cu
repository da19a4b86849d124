// The root-mean-square norm of fp32 rows.
#include "rms_norm.cuh"

cudaError_t flce::norm_fp32(const NormArgs& a, bool, bool wide, cudaStream_t st) {
  return launch_norm<kFp32, kFp32>(a, wide, st);
}
