// Backward of the root-mean-square norm with the residual's addition.
//
//   g = dy w, xhat = h rstd:  e = dh + rstd (g - xhat mean_c(g xhat))
//   dr = e,   dx = D(e),   dw = sum_m dy xhat
//
// dh is the gradient that reaches h along the residual stream. A row stays in registers
// between its one sum and its stores; a block takes every gridDim-th row and keeps its
// columns' share of dw in registers too, so dy and h are read once for both results. The
// blocks' shares are added in a fixed order by a second kernel.
#include <algorithm>

#include <cuda_runtime.h>

#include "block_internal.h"
#include "flce_host.h"
#include "stream_host.h"
#include "stream_ops.cuh"

namespace flce {
namespace {

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

// Threads and groups as in the forward.
template <int XT, int ST, int NV, bool VEC>
__global__ void __launch_bounds__(1024) norm_grad_kernel(const __grid_constant__ NormGradArgs a) {
  __shared__ float s_sum[2][32];
  griddep_launch();
  griddep_wait();
  const int T = blockDim.x, t = threadIdx.x, n = a.H;
  const int lane_row = blockIdx.x * blockDim.y + threadIdx.y, step = gridDim.x * blockDim.y;
  const Key key = dropout_key(a.drop);
  float acc[NV * 8] = {};
  int turn = 0;
  for (int row = lane_row; row < a.M; row += step, turn ^= 1) {
    const uint8_t* dy = static_cast<const uint8_t*>(a.dy) + row * a.ld_dy * type_size(XT);
    const uint8_t* h = static_cast<const uint8_t*>(a.h) + row * a.ld_h * type_size(ST);
    const uint8_t* dh = static_cast<const uint8_t*>(a.dh) + row * a.ld_dh * type_size(ST);
    Raw8<XT> rd[NV];
    Raw8<ST> rh[NV], re[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * T + t) * 8;
      rd[j] = {};
      rh[j] = {};
      re[j] = {};
      if (col < n) {
        rd[j] = load8<XT, VEC>(dy, col, n);
        rh[j] = load8<ST, VEC>(h, col, n);
        if (a.dh) re[j] = load8<ST, VEC>(dh, col, n);
      }
    }
    const float rstd = a.rstd[row];
    float g[NV * 8];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * T + t) * 8;
      float d[8], v[8], w[8];
      unpack8<XT>(rd[j], d);
      unpack8<ST>(rh[j], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.f;
      if (a.w != nullptr && col < n) {
        if (a.w_fp32)
          unpack8<kFp32>(load8<kFp32, VEC>(a.w, col, n), w);
        else
          unpack8<XT>(load8<XT, VEC>(a.w, col, n), w);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xhat = v[e] * rstd;
        acc[8 * j + e] = fmaf(d[e], xhat, acc[8 * j + e]);
        g[8 * j + e] = d[e] * w[e];
        sum = fmaf(g[8 * j + e], xhat, sum);
      }
    }
    if (!a.dx && !a.dr) continue;
    const float c = row_reduce<false>(sum, s_sum[turn]) / static_cast<float>(n);
    uint8_t* dx = static_cast<uint8_t*>(a.dx) + static_cast<int64_t>(row) * n * type_size(XT);
    uint8_t* dr = static_cast<uint8_t*>(a.dr) + static_cast<int64_t>(row) * n * type_size(ST);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * T + t) * 8;
      if (col >= n) continue;
      float v[8], e8[8];
      unpack8<ST>(rh[j], v);
      unpack8<ST>(re[j], e8);
#pragma unroll
      for (int e = 0; e < 8; ++e) e8[e] = fmaf(rstd, g[8 * j + e] - v[e] * rstd * c, e8[e]);
      if (a.dr) store8<ST, VEC>(dr, col, n, e8);
      if (a.dx) {
        if (a.drop.threshold != 0) drop8(a.drop, key, row, j * T + t, e8);
        store8<XT, VEC>(dx, col, n, e8);
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(lane_row) * n;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * T + t) * 8;
    if (col < n) store8<kFp32, VEC>(part, col, n, acc + 8 * j);
  }
}

struct Shape {
  int nv, threads, rows, blocks;
};
// The launch for M rows of H; it needs no device, as it sets the size of the workspace.
Shape shape_of(int64_t M, int64_t H) {
  Shape s;
  const int groups = static_cast<int>((H + 7) / 8);
  s.nv = groups <= 1024 ? 1 : groups <= 2048 ? 2 : 4;
  s.threads = ((groups + s.nv - 1) / s.nv + 31) / 32 * 32;
  s.rows = s.threads == 32 ? 4 : 1;
  const int per_sm = std::max(1, 1024 / (s.threads * s.rows));
  s.blocks = static_cast<int>(std::min<int64_t>((M + s.rows - 1) / s.rows, 152 * per_sm));
  return s;
}

template <int XT, int ST, int NV>
cudaError_t launch_vec(const NormGradArgs& a, bool vec, const Shape& s, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(s.blocks));
  const dim3 block(static_cast<unsigned>(s.threads), static_cast<unsigned>(s.rows));
  return vec ? launch_dependent(norm_grad_kernel<XT, ST, NV, true>, grid, block, 0, 1, st, a)
             : launch_dependent(norm_grad_kernel<XT, ST, NV, false>, grid, block, 0, 1, st, a);
}
template <int XT, int ST>
cudaError_t launch_grad(const NormGradArgs& a, bool vec, const Shape& s, cudaStream_t st) {
  return s.nv == 1   ? launch_vec<XT, ST, 1>(a, vec, s, st)
         : s.nv == 2 ? launch_vec<XT, ST, 2>(a, vec, s, st)
                     : launch_vec<XT, ST, 4>(a, vec, s, st);
}
cudaError_t dispatch(const NormGradArgs& a, int xt, int st_type, bool vec, const Shape& s, cudaStream_t st) {
  if (xt == kFp32) return launch_grad<kFp32, kFp32>(a, vec, s, st);
  if (xt == kBf16)
    return st_type == kFp32 ? launch_grad<kBf16, kFp32>(a, vec, s, st)
                            : launch_grad<kBf16, kBf16>(a, vec, s, st);
  return st_type == kFp32 ? launch_grad<kFp16, kFp32>(a, vec, s, st)
                          : launch_grad<kFp16, kFp16>(a, vec, s, st);
}

size_t workspace_of(int64_t M, int64_t H) {
  const Shape s = shape_of(M, H);
  return static_cast<size_t>(s.blocks) * s.rows * H * sizeof(float) + kAlign;
}

}  // namespace
}  // namespace flce

extern "C" {

size_t flce_rms_norm_workspace_size(const flce_rms_norm_params_t* p) {
  if (flce::check_norm(p) != FLCE_OK || p->M == 0) return 0;
  return flce::workspace_of(p->M, p->H);
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
  if (dW && workspace_bytes < workspace_of(p->M, p->H)) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  const flce_status_t ds = device_info(&sms);
  if (ds != FLCE_OK) return ds;
  const Shape s = shape_of(p->M, p->H);
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
  const bool vec = p->H % 8 == 0 && rows16(dy, a.ld_dy, p->M, p->dtype) &&
                   rows16(h, a.ld_h, p->M, p->stream_dtype) &&
                   rows16(dh, a.ld_dh, p->M, p->stream_dtype) && aligned_to(weight, 16) &&
                   aligned_to(dx, 16) && aligned_to(dresidual, 16);
  cudaError_t e = dispatch(a, p->dtype, p->stream_dtype, vec, s, st);
  if (e == cudaSuccess && dW)
    e = launch_db_sum(a.part, s.blocks * s.rows, a.H, dW, p->dW_fp32 != 0 || p->dtype == FLCE_DTYPE_FP32,
                      p->dtype == FLCE_DTYPE_FP16, st);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // extern "C"
