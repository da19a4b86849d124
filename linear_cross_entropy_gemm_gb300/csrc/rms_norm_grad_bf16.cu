// The backward of the root-mean-square norm of bf16 rows.
#include "rms_norm_grad.cuh"

cudaError_t flce::norm_grad_bf16(const NormGradArgs& a, bool stream_fp32, bool wide, const GradShape& s, cudaStream_t st) {
  return stream_fp32 ? launch_grad<kBf16, kFp32>(a, wide, s, st)
                     : launch_grad<kBf16, kBf16>(a, wide, s, st);
}
