// The root-mean-square norm of bf16 rows.
#include "rms_norm.cuh"

cudaError_t flce::norm_bf16(const NormArgs& a, bool stream_fp32, bool wide, cudaStream_t st) {
  return stream_fp32 ? launch_norm<kBf16, kFp32>(a, wide, st) : launch_norm<kBf16, kBf16>(a, wide, st);
}
