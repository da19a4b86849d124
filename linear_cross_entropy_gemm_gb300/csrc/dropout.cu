// Dropout from a counter-based generator, with the residual's addition:  y = r + D(x).
//
// The mask is a function of (seed, offset, row, column), so it is never stored: the backward,
// dx = D(dy), is the same call on dy. Bound by HBM, and by the generator's instructions (10 rounds for 8
// columns) close behind: 8192 x 14336 bf16 85 us (5.5 TB/s; a copy of it 72).
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

// A thread takes the same group of 8 columns, one counter's words, of kRows rows, blockDim.y apart: their
// loads are in flight together, and the generator's keys are made once for all of them.
constexpr int kRows = 4, kThreads = 256;

template <int XT, int YT>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropArgs a, uint32_t across) {
  griddep_launch();
  griddep_wait();
  const uint32_t down = blockIdx.x / across;
  const int64_t group = static_cast<int64_t>(blockIdx.x - down * across) * blockDim.x + threadIdx.x;
  const int64_t col = group * 8, first = static_cast<int64_t>(down) * (blockDim.y * kRows) + threadIdx.y;
  if (col >= a.H) return;
  const auto row_of = [](const void* p, int64_t row, int64_t ld, int size) {
    return static_cast<const uint8_t*>(p) + row * ld * size;
  };
  Raw8<XT> xr[kRows];
  Raw8<YT> rr[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = first + i * blockDim.y;
    rr[i] = {};
    if (row >= a.M) break;
    xr[i] = load8<XT, true>(row_of(a.x, row, a.ld_x, type_size(XT)), col, a.H);
    if (a.r) rr[i] = load8<YT, true>(row_of(a.r, row, a.ld_r, type_size(YT)), col, a.H);
  }
  Keys keys;
  if (a.drop.threshold != 0) keys = dropout_keys(a.drop);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = first + i * blockDim.y;
    if (row >= a.M) break;
    float v[8];
    unpack8<XT>(xr[i], v);
    if (a.drop.threshold != 0)
      drop8(a.drop, keys, static_cast<uint32_t>(row), static_cast<uint32_t>(group), v);
    if (a.r) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        f32x2_split(fadd2(f32x2(v[2 * e], v[2 * e + 1]), pair_of(rr[i], e)), v[2 * e], v[2 * e + 1]);
    }
    store8<YT, true>(static_cast<uint8_t*>(a.y) + row * a.ld_y * type_size(YT), col, a.H, v);
  }
}

// Rows off the 16-byte boundaries go value by value: a warp takes 256 columns of kRows rows, its
// accesses next to each other; a lane makes the random bits of a group, and takes those of the columns
// that it moves. 8192 x 4095 bf16 37 us; 89 with a thread for 8 neighbouring columns.
template <int XT, int YT>
__global__ void __launch_bounds__(kThreads)
    dropout_strided_kernel(const __grid_constant__ DropArgs a, uint32_t segments, int64_t warps) {
  __shared__ uint4 s_bits[kThreads / 32][32];
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp;
  if (id >= warps) return;
  const int64_t down = id / segments, segment = id - down * segments, col = segment * 256 + lane;
  const int left = static_cast<int>(a.H - segment * 256 < 256 ? a.H - segment * 256 : 256) - lane;
  const uint32_t group = static_cast<uint32_t>(segment) * 32 + lane;
  const uint16_t* bits = reinterpret_cast<const uint16_t*>(s_bits[warp]) + lane;
  Keys keys;
  if (a.drop.threshold != 0) keys = dropout_keys(a.drop);
#pragma unroll 2
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = down * kRows + i;
    if (row >= a.M) return;
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + (row * a.ld_x + col) * type_size(XT);
    const uint8_t* r = static_cast<const uint8_t*>(a.r) + (row * a.ld_r + col) * type_size(YT);
    uint8_t* y = static_cast<uint8_t*>(a.y) + (row * a.ld_y + col) * type_size(YT);
    float v[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = 32 * e < left ? load_value<XT>(x, 32 * e) : 0.f;
      u[e] = 0.f;
    }
    if (a.r) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = 32 * e < left ? load_value<YT>(r, 32 * e) : 0.f;
    }
    if (a.drop.threshold != 0) {
      s_bits[warp][lane] = drop_bits(a.drop, keys, static_cast<uint32_t>(row), group);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = bits[32 * e] >= a.drop.threshold ? v[e] * a.drop.scale : 0.f;
      __syncwarp();
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (32 * e < left) store_value<YT>(y, 32 * e, a.r ? v[e] + u[e] : v[e]);
  }
}

template <int XT, int YT>
cudaError_t launch_drop(const DropArgs& a, bool wide, cudaStream_t st) {
  const int64_t groups = (a.H + 7) / 8;
  if (!wide) {
    const int64_t segments = (groups + 31) / 32, warps = segments * ((a.M + kRows - 1) / kRows);
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_dependent(dropout_strided_kernel<XT, YT>, dim3(static_cast<unsigned>(blocks)), kThreads, 0, 1, st,
                            a, static_cast<uint32_t>(segments), warps);
  }
  // Blocks across a row, all of nearly the same width.
  const int64_t across = (groups + kThreads - 1) / kThreads;
  const int64_t even = (groups + across - 1) / across;
  const unsigned x = even <= 16 ? static_cast<unsigned>(even) : static_cast<unsigned>((even + 31) / 32 * 32);
  const unsigned y = kThreads / x;
  const int64_t down = (a.M + y * kRows - 1) / (y * kRows);
  if (across > 0x7FFFFFFF / down) return cudaErrorInvalidValue;
  return launch_dependent(dropout_kernel<XT, YT>, dim3(static_cast<unsigned>(across * down)), dim3(x, y), 0, 1, st, a,
                          static_cast<uint32_t>(across));
}

cudaError_t dispatch(const DropArgs& a, int xt, int yt, bool wide, cudaStream_t st) {
  if (xt == kFp32)
    return yt == kFp32   ? launch_drop<kFp32, kFp32>(a, wide, st)
           : yt == kBf16 ? launch_drop<kFp32, kBf16>(a, wide, st)
                         : launch_drop<kFp32, kFp16>(a, wide, st);
  if (xt == kBf16)
    return yt == kFp32 ? launch_drop<kBf16, kFp32>(a, wide, st) : launch_drop<kBf16, kBf16>(a, wide, st);
  return yt == kFp32 ? launch_drop<kFp16, kFp32>(a, wide, st) : launch_drop<kFp16, kFp16>(a, wide, st);
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
  // A counter holds the row and the group of columns in 32 bits each; the grid has fewer than 2^31
  // blocks of 4 rows or more and half of 256 groups or more, or of 64 rows and more.
  if (p->M > (1LL << 31) || p->H > (1LL << 34) ||
      (p->H > 0 && p->M > 0 && (p->H + 7) / 8 > (1LL << 31) * 256 / p->M))
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
  const bool wide = p->H % 8 == 0 && rows16(x, a.ld_x, p->M, p->dtype) &&
                   rows16(residual, a.ld_r, p->M, p->out_dtype) && rows16(y, a.ld_y, p->M, p->out_dtype);
  const cudaError_t e = dispatch(a, p->dtype, p->out_dtype, wide, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
