// C ABI of the root-mean-square norm with the residual's addition, dropout on the branch that joins
// it, and an output in the operands' type or in 8 bits with scales (declared in include/flce.h).
//
//   h = r + D(x),   rstd = (mean_c h^2 + eps)^(-1/2),   y = w h rstd
//   8 bits: s = max |y| / 448 over the row or over 128 columns,  y8 = e4m3(y / s)
//   backward, g = dy w, xhat = h rstd:  e = dh + rstd (g - xhat mean_c(g xhat))
//   dr = e,   dx = D(e),   dw = sum_m dy xhat
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "block_internal.h"
#include "flce_host.h"
#include "rms_norm.h"
#include "stream_host.h"

namespace flce {

namespace {

// dw = the ordered sum of the blocks' shares: a cluster of up to 8 blocks takes 32 columns, each of its
// warps every so many'th share; the warps of a block and then the blocks add up in their order. 608 shares
// of 2048 columns: the backward 11.5 us with 4 blocks, 12.6 with one; 304 of 4096 alike.
constexpr int kSumThreads = 512, kSumBlocks = 8;
__global__ void __launch_bounds__(kSumThreads)
    share_sum_kernel(const float* part, int parts, int n, void* out, int type, int blocks) {
  __shared__ float s_sum[kSumThreads / 32][32], s_all[kSumBlocks][32];
  if (blocks > 1) cluster_arrive();
  griddep_wait();
  const int rank = blockIdx.x % blocks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = static_cast<int>(blockIdx.x / blocks) * 32 + lane, apart = blocks * (kSumThreads / 32);
  float sum = 0.f;
  for (int i = rank * (kSumThreads / 32) + warp; i < parts; i += 8 * apart) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = col < n && i + k * apart < parts ? part[static_cast<int64_t>(i + k * apart) * n + col] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += v[k];
  }
  griddep_launch();
  s_sum[warp][lane] = sum;
  __syncthreads();
  if (blocks > 1) cluster_wait();  // the first block runs: its memory may be written
  if (warp == 0) {
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kSumThreads / 32; ++w) sum += s_sum[w][lane];
    if (blocks > 1)
      cooperative_groups::this_cluster().map_shared_rank(s_all[rank], 0)[lane] = sum;
  }
  if (blocks > 1) {
    cooperative_groups::this_cluster().sync();
    sum = 0.f;
    for (int r = 0; r < blocks; ++r) sum += s_all[r][lane];
  }
  if (rank != 0 || warp != 0 || col >= n) return;
  if (type == kFp32)
    static_cast<float*>(out)[col] = sum;
  else
    static_cast<uint16_t*>(out)[col] = static_cast<uint16_t>(pack_16x2(sum, 0.f, type == kFp16) & 0xFFFFu);
}

cudaError_t launch_share_sum(const float* part, int parts, int n, void* out, int type, cudaStream_t st) {
  int blocks = 1;
  while (blocks < kSumBlocks && parts > blocks * 160) blocks *= 2;
  return launch_dependent(share_sum_kernel, dim3((n + 31) / 32 * blocks), kSumThreads, 0, blocks, st, part, parts, n,
                          out, type, blocks);
}

}  // namespace

flce_status_t check_norm(const flce_rms_norm_params_t* p) {
  if (!p || p->M < 0 || p->H <= 0) return FLCE_ERR_INVALID_ARG;
  if (p->M > (1LL << 30) || p->H > FLCE_RMS_NORM_MAX_H) return FLCE_ERR_UNSUPPORTED;
  if (!float_type_ok(p->dtype) || !wider_ok(p->stream_dtype, p->dtype) ||
      !wider_ok(p->weight_dtype, p->dtype) || p->scales < FLCE_SCALES_NONE ||
      p->scales > FLCE_SCALES_BLOCK || (p->dW_fp32 != 0 && p->dW_fp32 != 1))
    return FLCE_ERR_INVALID_ARG;
  for (const int64_t ld : {p->ld_x, p->ld_res, p->ld_h, p->ld_y})
    if (!pitch_ok(ld, p->H)) return FLCE_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || !(p->eps < INFINITY) || !(p->dropout >= 0.0) || !(p->dropout <= 1.0))
    return FLCE_ERR_INVALID_ARG;
  return FLCE_OK;
}

namespace {

// The registers of a row's threads, its ring and the time of its one sum decide. 8192 x 4096: 2 groups
// of 256 threads with 128 registers and two blocks on an SM 42.9 us, 3 blocks with 80 registers 52,
// 4 groups 69, 1 group of 512 threads 56.
GradShape grad_shape(int64_t M, int64_t H, int x_size, int stream_size, bool wide) {
  constexpr size_t kMemory = 220 * 1024;
  const int groups = static_cast<int>((H + 7) / 8);
  const auto with = [&](int nv) {
    GradShape s;
    s.nv = nv;
    s.threads = ((groups + nv - 1) / nv + 31) / 32 * 32;
    s.rows = nv == 1 && s.threads == 32 ? kBlockRows : 1;
    const int by_threads = (nv == 1 ? 1024 : 512) / (s.threads * s.rows);
    const int by_ring = static_cast<int>(kMemory / (grad_ring(s, x_size, stream_size) + 1024));
    s.blocks = by_threads < by_ring ? by_threads : by_ring;  // of an SM
    return s;
  };
  GradShape s = with(8);
  if (!wide) {
    // Value by value, many threads carry the accesses.
    s = with(groups <= 1024 ? 1 : groups <= 2048 ? 2 : 4);
    s.blocks = 1024 / (s.threads * s.rows);
  } else if (groups <= 256) {
    s = with(1);
  } else {
    const GradShape two = with(2), four = with(4);
    if (two.threads <= kRowThreads && two.blocks > 0)
      s = two;
    else if (four.threads <= kRowThreads && four.blocks > 0)
      s = four;
  }
  const int64_t all = 152 * static_cast<int64_t>(s.blocks > 0 ? s.blocks : 1), need = (M + s.rows - 1) / s.rows;
  s.blocks = static_cast<int>(need < all ? need : all);
  return s;
}
GradShape grad_shape(const flce_rms_norm_params_t* p, bool wide) {
  return grad_shape(p->M, p->H, type_size(p->dtype), type_size(p->stream_dtype), wide);
}

size_t grad_workspace(const flce_rms_norm_params_t* p) {
  // Whichever of the two the tensors' alignment asks for.
  const int wide = grad_shape(p, true).blocks, narrow = grad_shape(p, false).blocks;
  return static_cast<size_t>(wide > narrow ? wide : narrow) * p->H * sizeof(float) + kAlign;
}

}  // namespace
}  // namespace flce

extern "C" flce_status_t flce_rms_norm_forward(const flce_rms_norm_params_t* p, const void* x,
                                               const void* weight, const void* residual,
                                               const int64_t* seed, void* y, void* h, float* rstd,
                                               float* scales, void* stream) {
  using namespace flce;
  NvtxRange nvtx_range("flce_rms_norm_forward");
  const flce_status_t bad = check_norm(p);
  if (bad != FLCE_OK) return bad;
  const bool quantized = p->scales != FLCE_SCALES_NONE;
  if (p->M == 0) return FLCE_OK;
  if (!x || !y || quantized != (scales != nullptr)) return FLCE_ERR_INVALID_ARG;
  const int xb = type_size(p->dtype), sb = type_size(p->stream_dtype);
  if (!aligned_to(x, xb) || !aligned_to(weight, type_size(p->weight_dtype)) || !aligned_to(residual, sb) ||
      !aligned_to(h, sb) || (!quantized && !aligned_to(y, xb)) || !aligned_to(rstd, 4) ||
      !aligned_to(scales, 4) || !aligned_to(seed, 8))
    return FLCE_ERR_ALIGNMENT;
  int sms = 0;
  const flce_status_t ds = device_info(&sms);
  if (ds != FLCE_OK) return ds;
  NormArgs a;
  a.x = x;
  a.w = weight;
  a.r = residual;
  a.y = y;
  a.h = h;
  a.rstd = rstd;
  a.scales = scales;
  a.ld_x = pitch_of(p->ld_x, p->H);
  a.ld_r = pitch_of(p->ld_res, p->H);
  a.ld_h = pitch_of(p->ld_h, p->H);
  a.ld_y = pitch_of(p->ld_y, p->H);
  a.M = static_cast<int>(p->M);
  a.H = static_cast<int>(p->H);
  a.w_fp32 = p->weight_dtype == FLCE_DTYPE_FP32 ? 1 : 0;
  a.blocks = p->scales == FLCE_SCALES_BLOCK ? 1 : 0;
  a.eps = p->eps;
  if (!make_dropout(p->dropout, p->seed, p->offset, seed, &a.drop)) return FLCE_ERR_INVALID_ARG;
  const bool y16 = quantized ? aligned_to(y, 8) && (p->M <= 1 || a.ld_y % 8 == 0)
                             : rows16(y, a.ld_y, p->M, p->dtype);
  const bool wide = p->H % 8 == 0 && y16 && rows16(x, a.ld_x, p->M, p->dtype) &&
                   rows16(residual, a.ld_r, p->M, p->stream_dtype) &&
                   rows16(h, a.ld_h, p->M, p->stream_dtype) && aligned_to(weight, 16);
  const bool stream_fp32 = p->stream_dtype == FLCE_DTYPE_FP32;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->dtype == FLCE_DTYPE_BF16   ? norm_bf16(a, stream_fp32, wide, st)
                        : p->dtype == FLCE_DTYPE_FP16 ? norm_fp16(a, stream_fp32, wide, st)
                                                      : norm_fp32(a, stream_fp32, wide, st);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

extern "C" {

size_t flce_rms_norm_workspace_size(const flce_rms_norm_params_t* p) {
  if (flce::check_norm(p) != FLCE_OK || p->M == 0) return 0;
  return flce::grad_workspace(p);
}

flce_status_t flce_rms_norm_backward(const flce_rms_norm_params_t* p, const void* dy, const void* h,
                                     const void* weight, const float* rstd, const void* dh,
                                     const int64_t* seed, void* dx, void* dresidual, void* dW,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  using namespace flce;
  NvtxRange nvtx_range("flce_rms_norm_backward");
  const flce_status_t bad = check_norm(p);
  if (bad != FLCE_OK) return bad;
  if (p->scales != FLCE_SCALES_NONE) return FLCE_ERR_INVALID_ARG;
  const int xb = type_size(p->dtype), sb = type_size(p->stream_dtype), wb = p->dW_fp32 ? 4 : xb;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!aligned_to(dW, wb)) return FLCE_ERR_ALIGNMENT;
  if (p->M == 0) {
    if (dW && cudaMemsetAsync(dW, 0, static_cast<size_t>(p->H) * wb, st) != cudaSuccess)
      return FLCE_ERR_CUDA;
    return FLCE_OK;
  }
  if (!dx && !dresidual && !dW) return FLCE_OK;
  if (!dy || !h || !rstd) return FLCE_ERR_INVALID_ARG;
  // One buffer for both gradients: where they are equal.
  if (dx && dx == dresidual) {
    if (p->dropout != 0.0 || p->dtype != p->stream_dtype) return FLCE_ERR_INVALID_ARG;
    dresidual = nullptr;
  }
  if (!aligned_to(dy, xb) || !aligned_to(h, sb) || !aligned_to(weight, type_size(p->weight_dtype)) ||
      !aligned_to(dh, sb) || !aligned_to(rstd, 4) || !aligned_to(dx, xb) || !aligned_to(dresidual, sb) ||
      !aligned_to(seed, 8))
    return FLCE_ERR_ALIGNMENT;
  if (dW && !workspace) return FLCE_ERR_INVALID_ARG;
  if (dW && workspace_bytes < grad_workspace(p)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  const flce_status_t ds = device_info(&sms);
  if (ds != FLCE_OK) return ds;
  Carver cv(workspace, workspace_bytes);
  NormGradArgs a;
  a.dy = dy;
  a.h = h;
  a.w = weight;
  a.dh = dh;
  a.rstd = rstd;
  a.dx = dx;
  a.dr = dresidual;
  a.part = dW ? cv.take<float>(0) : nullptr;
  a.ld_dy = pitch_of(p->ld_y, p->H);
  a.ld_h = pitch_of(p->ld_h, p->H);
  a.ld_dh = pitch_of(p->ld_res, p->H);
  a.M = static_cast<int>(p->M);
  a.H = static_cast<int>(p->H);
  a.w_fp32 = p->weight_dtype == FLCE_DTYPE_FP32 ? 1 : 0;
  if (!make_dropout(p->dropout, p->seed, p->offset, seed, &a.drop)) return FLCE_ERR_INVALID_ARG;
  const bool wide = p->H % 8 == 0 && rows16(dy, a.ld_dy, p->M, p->dtype) &&
                   rows16(h, a.ld_h, p->M, p->stream_dtype) &&
                   rows16(dh, a.ld_dh, p->M, p->stream_dtype) && aligned_to(weight, 16) &&
                   aligned_to(dx, 16) && aligned_to(dresidual, 16);
  const GradShape s = grad_shape(p, wide);
  const bool stream_fp32 = p->stream_dtype == FLCE_DTYPE_FP32;
  cudaError_t e = p->dtype == FLCE_DTYPE_BF16   ? norm_grad_bf16(a, stream_fp32, wide, s, st)
                  : p->dtype == FLCE_DTYPE_FP16 ? norm_grad_fp16(a, stream_fp32, wide, s, st)
                                                : norm_grad_fp32(a, stream_fp32, wide, s, st);
  if (e == cudaSuccess && dW)
    e = launch_share_sum(a.part, s.blocks, a.H, dW, p->dW_fp32 ? FLCE_DTYPE_FP32 : p->dtype, st);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // extern "C"
