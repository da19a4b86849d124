// The root-mean-square norm of fp16 rows.
#include "rms_norm.cuh"

cudaError_t flce::norm_fp16(const NormArgs& a, bool stream_fp32, bool wide, cudaStream_t st) {
  return stream_fp32 ? launch_norm<kFp16, kFp32>(a, wide, st) : launch_norm<kFp16, kFp16>(a, wide, st);
}
