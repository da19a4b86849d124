// Internal interface of the root-mean-square norm: arguments of its kernels, which are compiled
// for each type of the operands apart.
#pragma once
#include <cuda_runtime.h>

#include "stream_ops.cuh"

namespace flce {

constexpr int kRowThreads = 512;  // of a row, at most
constexpr int kBlockRows = 4;     // rows of a block whose warps hold one each

struct NormArgs {
  const void *x, *w, *r;
  void *y, *h;
  float *rstd, *scales;
  int64_t ld_x, ld_r, ld_h, ld_y;
  int M, H;
  int w_fp32, blocks;  // blocks: scales of 128 columns, not of a row
  float eps;
  Dropout drop;
};

struct NormGradArgs {
  const void *dy, *h, *w, *dh;
  const float* rstd;
  void *dx, *dr;
  float* part;  // [rows of blocks, H] shares of dw, or null
  int64_t ld_dy, ld_h, ld_dh;
  int M, H;
  int w_fp32;
  Dropout drop;
};
// The backward's launch for M rows of H. It needs no device, as it sets the workspace's size.
struct GradShape {
  int nv, threads, rows, blocks;
};
// Whether rows to come are on their way into shared memory, and how many. An fp32 stream's would leave
// room for too few blocks: 8192 x 4096 92 us with them, 65 without; 16 bits 43 and 56.
__host__ __device__ constexpr bool grad_has_ring(int nv, int stream_size) {
  return nv <= 4 && stream_size == 2;
}
__host__ __device__ constexpr int grad_stages(int nv) { return nv <= 2 ? 3 : 2; }
inline size_t grad_ring(const GradShape& s, int x_size, int stream_size) {
  if (!grad_has_ring(s.nv, stream_size)) return 0;
  return static_cast<size_t>(grad_stages(s.nv)) * s.nv * (x_size + 2 * stream_size) * 8 * s.threads * s.rows;
}

// stream_fp32: the residual and h are fp32, not of the operands' type. wide: rows on 16-byte boundaries.
cudaError_t norm_bf16(const NormArgs& a, bool stream_fp32, bool wide, cudaStream_t st);
cudaError_t norm_fp16(const NormArgs& a, bool stream_fp32, bool wide, cudaStream_t st);
cudaError_t norm_fp32(const NormArgs& a, bool stream_fp32, bool wide, cudaStream_t st);
cudaError_t norm_grad_bf16(const NormGradArgs& a, bool stream_fp32, bool wide, const GradShape& s, cudaStream_t st);
cudaError_t norm_grad_fp16(const NormGradArgs& a, bool stream_fp32, bool wide, const GradShape& s, cudaStream_t st);
cudaError_t norm_grad_fp32(const NormGradArgs& a, bool stream_fp32, bool wide, const GradShape& s, cudaStream_t st);

}  // namespace flce
