// Dropout from a counter-based generator, with the residual's addition:  y = r + D(x).
//
// The mask is a function of (seed, offset, row, column), so it is never stored: the backward,
// dx = D(dy), is the same call on dy.
#include <cuda_runtime.h>

#include "block_internal.h"
#include "flce_host.h"
#include "stream_host.h"
#include "stream_ops.cuh"

namespace flce {
namespace {

struct DropArgs {
  const void *x, *r;
  void* y;
  int64_t ld_x, ld_r, ld_y;
  int64_t M, H;
  Dropout drop;
};

// A thread takes 8 columns of a row: one counter's words.
template <int XT, int YT, bool VEC, class Index>
__global__ void __launch_bounds__(256) dropout_kernel(const __grid_constant__ DropArgs a) {
  griddep_launch();
  griddep_wait();
  const Index groups = static_cast<Index>((a.H + 7) / 8);
  const Index i = static_cast<Index>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= groups * static_cast<Index>(a.M)) return;
  const int64_t row = static_cast<int64_t>(i / groups);
  const uint32_t group = static_cast<uint32_t>(i - static_cast<Index>(row) * groups);
  const int64_t col = static_cast<int64_t>(group) * 8;
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + row * a.ld_x * type_size(XT);
  const uint8_t* r = static_cast<const uint8_t*>(a.r) + row * a.ld_r * type_size(YT);
  uint8_t* y = static_cast<uint8_t*>(a.y) + row * a.ld_y * type_size(YT);
  const Raw8<XT> xr = load8<XT, VEC>(x, col, a.H);
  Raw8<YT> rr = {};
  if (a.r) rr = load8<YT, VEC>(r, col, a.H);
  float v[8], u[8];
  unpack8<XT>(xr, v);
  unpack8<YT>(rr, u);
  if (a.drop.threshold != 0) drop8(a.drop, dropout_key(a.drop), static_cast<uint32_t>(row), group, v);
  if (a.r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += u[e];
  }
  store8<YT, VEC>(y, col, a.H, v);
}

template <int XT, int YT>
cudaError_t launch_drop(const DropArgs& a, bool vec, cudaStream_t st) {
  const uint64_t n = static_cast<uint64_t>(a.M) * static_cast<uint64_t>((a.H + 7) / 8);
  const uint64_t blocks = (n + 255) / 256;
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  const bool small = n < (1ull << 32) - 256;
  auto kernel = vec ? small ? dropout_kernel<XT, YT, true, uint32_t> : dropout_kernel<XT, YT, true, uint64_t>
                    : small ? dropout_kernel<XT, YT, false, uint32_t> : dropout_kernel<XT, YT, false, uint64_t>;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(blocks)), 256, 0, 1, st, a);
}

cudaError_t dispatch(const DropArgs& a, int xt, int yt, bool vec, cudaStream_t st) {
  if (xt == kFp32)
    return yt == kFp32   ? launch_drop<kFp32, kFp32>(a, vec, st)
           : yt == kBf16 ? launch_drop<kFp32, kBf16>(a, vec, st)
                         : launch_drop<kFp32, kFp16>(a, vec, st);
  if (xt == kBf16)
    return yt == kFp32 ? launch_drop<kBf16, kFp32>(a, vec, st) : launch_drop<kBf16, kBf16>(a, vec, st);
  return yt == kFp32 ? launch_drop<kFp16, kFp32>(a, vec, st) : launch_drop<kFp16, kFp16>(a, vec, st);
}

}  // namespace
}  // namespace flce

extern "C" flce_status_t flce_dropout(const flce_dropout_params_t* p, const void* x, const void* residual,
                                      const int64_t* seed, void* y, void* stream) {
  using namespace flce;
  NvtxRange nvtx_range("flce_dropout");
  if (!p || p->M < 0 || p->H < 0 || !float_type_ok(p->dtype) || !float_type_ok(p->out_dtype) ||
      (p->out_dtype != p->dtype && p->out_dtype != FLCE_DTYPE_FP32 && p->dtype != FLCE_DTYPE_FP32))
    return FLCE_ERR_INVALID_ARG;
  for (const int64_t ld : {p->ld_x, p->ld_res, p->ld_y})
    if (!pitch_ok(ld, p->H)) return FLCE_ERR_INVALID_ARG;
  DropArgs a;
  if (!make_dropout(p->dropout, p->seed, p->offset, seed, &a.drop)) return FLCE_ERR_INVALID_ARG;
  // A counter holds the row and the group of columns in 32 bits each, and the grid its blocks in 31.
  if (p->M > (1LL << 31) || p->H > (1LL << 34) ||
      (p->H > 0 && p->M > 0 && (p->H + 7) / 8 > ((1LL << 31) - 1) * 256 / p->M))
    return FLCE_ERR_UNSUPPORTED;
  if (p->M == 0 || p->H == 0) return FLCE_OK;
  if (!x || !y) return FLCE_ERR_INVALID_ARG;
  const int xb = type_size(p->dtype), yb = type_size(p->out_dtype);
  if (!aligned_to(x, xb) || !aligned_to(residual, yb) || !aligned_to(y, yb) || !aligned_to(seed, 8))
    return FLCE_ERR_ALIGNMENT;
  int sms = 0;
  const flce_status_t ds = device_info(&sms);
  if (ds != FLCE_OK) return ds;
  a.x = x;
  a.r = residual;
  a.y = y;
  a.ld_x = pitch_of(p->ld_x, p->H);
  a.ld_r = pitch_of(p->ld_res, p->H);
  a.ld_y = pitch_of(p->ld_y, p->H);
  a.M = p->M;
  a.H = p->H;
  const bool vec = p->H % 8 == 0 && rows16(x, a.ld_x, p->M, p->dtype) &&
                   rows16(residual, a.ld_r, p->M, p->out_dtype) && rows16(y, a.ld_y, p->M, p->out_dtype);
  const cudaError_t e = dispatch(a, p->dtype, p->out_dtype, vec, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
