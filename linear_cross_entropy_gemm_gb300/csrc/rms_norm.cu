// The root-mean-square norm with the residual's addition, dropout on the branch that joins
// it, and an output in the operands' type or in 8 bits with scales.
//
//   h = r + D(x),   rstd = (mean_c h^2 + eps)^(-1/2),   y = w h rstd
//   8 bits: s = max |y| / 448 over the row or over 128 columns,  y8 = e4m3(y / s)
//
// One pass: a row stays in its threads' registers from the loads to the stores, so x and r
// are read once and h and y written once. The norm is of the unrounded h: rounding it to
// 16 bits first would put 2^-9 of error into each y for nothing.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "block_internal.h"
#include "flce_host.h"
#include "stream_host.h"
#include "stream_ops.cuh"

namespace flce {
namespace {

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

__device__ __forceinline__ uint2 to_e4m3(const float* y, float inv) {
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    q[e] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * e] * inv, y[2 * e + 1] * inv), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// Scales below the smallest normal number are 0, and the values under them too: their
// inverses need not be finite.
__device__ __forceinline__ float scale_of(float largest, float* inv) {
  float s = __fdiv_rn(largest, 448.f);
  if (s < 1.17549435e-38f) s = 0.f;
  *inv = s == 0.f ? 0.f : __frcp_rn(s);
  return s;
}

// blockDim.x threads for a row, blockDim.y rows (one, unless a warp holds a row); a thread
// holds NV groups of 8 columns, blockDim.x groups apart.
template <int XT, int ST, int NV, bool VEC, bool Q>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float s_sum[32], s_max[32];
  griddep_launch();
  griddep_wait();
  const int row = blockIdx.x * blockDim.y + threadIdx.y, T = blockDim.x, t = threadIdx.x;
  if (row >= a.M) return;
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + row * a.ld_x * type_size(XT);
  const uint8_t* r = static_cast<const uint8_t*>(a.r) + row * a.ld_r * type_size(ST);
  const int n = a.H;
  float h[NV * 8];
  Raw8<ST> rr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * T + t) * 8;
    Raw8<XT> xr = {};
    rr[j] = {};
    if (col < n) {
      xr = load8<XT, VEC>(x, col, n);
      if (a.r) rr[j] = load8<ST, VEC>(r, col, n);
    }
    unpack8<XT>(xr, h + 8 * j);
  }
  if (a.drop.threshold != 0) {
    const Key key = dropout_key(a.drop);
#pragma unroll
    for (int j = 0; j < NV; ++j) drop8(a.drop, key, row, j * T + t, h + 8 * j);
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v[8];
    unpack8<ST>(rr[j], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[8 * j + e] += v[e];
      sum = fmaf(h[8 * j + e], h[8 * j + e], sum);
    }
  }
  sum = row_reduce<false>(sum, s_sum);
  const float rstd = rsqrtf(sum / static_cast<float>(n) + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
  uint8_t* ho = static_cast<uint8_t*>(a.h) + row * a.ld_h * type_size(ST);
  uint8_t* yo = static_cast<uint8_t*>(a.y) + row * a.ld_y * (Q ? 1 : type_size(XT));
  float most = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int col = (j * T + t) * 8;
    if (col < n) {
      if (a.h) store8<ST, VEC>(ho, col, n, h + 8 * j);
      float w[8];
      if (a.w == nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
      } else if (a.w_fp32) {
        unpack8<kFp32>(load8<kFp32, VEC>(a.w, col, n), w);
      } else {
        unpack8<XT>(load8<XT, VEC>(a.w, col, n), w);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) h[8 * j + e] *= rstd * w[e];
    }
    if constexpr (!Q) {
      if (col < n) store8<XT, VEC>(yo, col, n, h + 8 * j);
    } else {
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(h[8 * j + e]));
      if (a.blocks) {
        // 16 neighbouring threads hold 128 columns.
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        float inv;
        const float s = scale_of(m, &inv);
        if (col < n) {
          if ((t & 15) == 0) a.scales[static_cast<int64_t>(row) * ((n + 127) / 128) + col / 128] = s;
          const uint2 q = to_e4m3(h + 8 * j, inv);
          if constexpr (VEC) {
            *reinterpret_cast<uint2*>(yo + col) = q;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (col + e < n)
                yo[col + e] = static_cast<uint8_t>((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
          }
        }
      }
      most = max_nan(most, m);
    }
  }
  if constexpr (Q) {
    if (a.blocks) return;
    most = row_reduce<true>(most, s_max);
    float inv;
    const float s = scale_of(most, &inv);
    if (t == 0) a.scales[row] = s;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * T + t) * 8;
      if (col >= n) continue;
      const uint2 q = to_e4m3(h + 8 * j, inv);
      if constexpr (VEC) {
        *reinterpret_cast<uint2*>(yo + col) = q;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < n) yo[col + e] = static_cast<uint8_t>((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
      }
    }
  }
}

template <int XT, int ST, int NV, bool VEC>
cudaError_t launch_q(const NormArgs& a, dim3 grid, dim3 block, cudaStream_t st) {
  return a.scales ? launch_dependent(norm_kernel<XT, ST, NV, VEC, true>, grid, block, 0, 1, st, a)
                  : launch_dependent(norm_kernel<XT, ST, NV, VEC, false>, grid, block, 0, 1, st, a);
}
template <int XT, int ST, int NV>
cudaError_t launch_vec(const NormArgs& a, bool vec, dim3 grid, dim3 block, cudaStream_t st) {
  return vec ? launch_q<XT, ST, NV, true>(a, grid, block, st)
             : launch_q<XT, ST, NV, false>(a, grid, block, st);
}
template <int XT, int ST>
cudaError_t launch_norm(const NormArgs& a, bool vec, cudaStream_t st) {
  const int groups = (a.H + 7) / 8;
  const int nv = groups <= 1024 ? 1 : groups <= 2048 ? 2 : 4;
  const int threads = ((groups + nv - 1) / nv + 31) / 32 * 32;
  const int rows = threads == 32 ? 4 : 1;
  const dim3 block(static_cast<unsigned>(threads), static_cast<unsigned>(rows));
  const dim3 grid(static_cast<unsigned>((a.M + rows - 1) / rows));
  return nv == 1   ? launch_vec<XT, ST, 1>(a, vec, grid, block, st)
         : nv == 2 ? launch_vec<XT, ST, 2>(a, vec, grid, block, st)
                   : launch_vec<XT, ST, 4>(a, vec, grid, block, st);
}

cudaError_t dispatch(const NormArgs& a, int xt, int st_type, bool vec, cudaStream_t st) {
  if (xt == kFp32) return launch_norm<kFp32, kFp32>(a, vec, st);
  if (xt == kBf16)
    return st_type == kFp32 ? launch_norm<kBf16, kFp32>(a, vec, st) : launch_norm<kBf16, kBf16>(a, vec, st);
  return st_type == kFp32 ? launch_norm<kFp16, kFp32>(a, vec, st) : launch_norm<kFp16, kFp16>(a, vec, st);
}

}  // namespace

flce_status_t check_norm(const flce_rms_norm_params_t* p) {
  if (!p || p->M < 0 || p->H <= 0) return FLCE_ERR_INVALID_ARG;
  if (p->M > (1LL << 31) - 8 || p->H > FLCE_RMS_NORM_MAX_H) return FLCE_ERR_UNSUPPORTED;
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
  const bool vec = p->H % 8 == 0 && y16 && rows16(x, a.ld_x, p->M, p->dtype) &&
                   rows16(residual, a.ld_r, p->M, p->stream_dtype) &&
                   rows16(h, a.ld_h, p->M, p->stream_dtype) && aligned_to(weight, 16);
  const cudaError_t e = dispatch(a, p->dtype, p->stream_dtype, vec, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
