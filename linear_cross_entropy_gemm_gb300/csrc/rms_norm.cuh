// Kernels of the root-mean-square norm's forward, for one type of the operands (rms_norm.cu says
// what they compute).
//
// One pass: a row stays in its threads' registers from the loads to the stores, so x and r
// are read once and h and y written once. The norm is of the unrounded h: rounding it to
// 16 bits first would put up to 2^-8 of error into each y (bf16) for nothing. Bound by HBM: 8192 x 4096 bf16
// with a residual 40.9 us (6.6 TB/s; a copy runs at 6.8), with dropout 42.5, to 8 bits 37.4 (a
// scale for a row) and 39.6 (for 128 columns), fp32 80.7. Rows off the 16-byte boundaries go value by
// value and are bound by their accesses: 8192 x 4095 68 us, 8192 x 4100 77 (one block of 544
// threads on an SM, where 512 leave room for two).
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "block_internal.h"
#include "rms_norm.h"
#include "stream_ops.cuh"

namespace flce {
namespace {

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

template <Layout L>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int j, int T, int t, int n, const float* y, float inv) {
  const uint2 q = to_e4m3(y, inv);
  if constexpr (L == kWide) {
    const int col = column<L>(j, 0, T, t);
    if (col < n) *reinterpret_cast<uint2*>(row + col) = q;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = column<L>(j, e, T, t);
      if (col < n) row[col] = static_cast<uint8_t>((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
    }
  }
}

// blockDim.x threads for a row, blockDim.y rows (one, unless a warp holds a row); a thread
// holds NV groups of 8 columns.
template <int XT, int ST, int NV, Layout L, bool Q>
__global__ void __launch_bounds__(L == kStrided ? 1024 : kRowThreads) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float s_sum[32], s_max[32];
  extern __shared__ __align__(16) uint8_t smem[];  // kStrided: the dropout's random bits
  griddep_launch();
  griddep_wait();
  const int row = blockIdx.x * blockDim.y + threadIdx.y, T = blockDim.x, t = threadIdx.x;
  if (row >= a.M) return;
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + row * a.ld_x * type_size(XT);
  const uint8_t* r = static_cast<const uint8_t*>(a.r) + row * a.ld_r * type_size(ST);
  const int n = a.H;
  float h[NV * 8];
  Raw8<XT> xr[NV];
  Raw8<ST> rr[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    xr[j] = load_group<XT, L>(x, j, T, t, n);
    rr[j] = {};
    if (a.r) rr[j] = load_group<ST, L>(r, j, T, t, n);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) unpack8<XT>(xr[j], h + 8 * j);
  if (a.drop.threshold != 0) {
    const Keys keys = dropout_keys(a.drop);
    if constexpr (L != kStrided) {
#pragma unroll
      for (int j = 0; j < NV; ++j) drop8(a.drop, keys, row, j * T + t, h + 8 * j);
    } else {
      // Eight columns share a counter: a thread makes neighbours' bits, and takes its own.
      uint4* bits = reinterpret_cast<uint4*>(smem) + threadIdx.y * (NV * T);
#pragma unroll
      for (int j = 0; j < NV; ++j) bits[j * T + t] = drop_bits(a.drop, keys, row, j * T + t);
      if (T == 32)
        __syncwarp();
      else
        __syncthreads();
      const uint16_t* own = reinterpret_cast<const uint16_t*>(bits);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          h[8 * j + e] = own[column<L>(j, e, T, t)] >= a.drop.threshold ? h[8 * j + e] * a.drop.scale : 0.f;
    }
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
    if (a.h) store_group<ST, L>(ho, j, T, t, n, h + 8 * j);
    float w[8];
    if (a.w == nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.f;
    } else if (a.w_fp32) {
      unpack8<kFp32>(load_group<kFp32, L>(a.w, j, T, t, n), w);
    } else {
      unpack8<XT>(load_group<XT, L>(a.w, j, T, t, n), w);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) h[8 * j + e] *= rstd * w[e];
    if constexpr (!Q) {
      store_group<XT, L>(yo, j, T, t, n, h + 8 * j);
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
        const int col = column<L>(j, 0, T, t);
        if ((t & 15) == 0 && col < n) a.scales[static_cast<int64_t>(row) * ((n + 127) / 128) + col / 128] = s;
        store_e4m3<L>(yo, j, T, t, n, h + 8 * j, inv);
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
    for (int j = 0; j < NV; ++j) store_e4m3<L>(yo, j, T, t, n, h + 8 * j, inv);
  }
}

template <int XT, int ST, int NV, Layout L>
cudaError_t launch_q(const NormArgs& a, dim3 grid, dim3 block, size_t smem, cudaStream_t st) {
  return a.scales ? launch_dependent(norm_kernel<XT, ST, NV, L, true>, grid, block, smem, 1, st, a)
                  : launch_dependent(norm_kernel<XT, ST, NV, L, false>, grid, block, smem, 1, st, a);
}
template <int XT, int ST, Layout L>
cudaError_t launch_nv(const NormArgs& a, int nv, dim3 grid, dim3 block, size_t smem, cudaStream_t st) {
  if constexpr (L == kWide)
    if (nv == 8) return launch_q<XT, ST, 8, L>(a, grid, block, smem, st);
  return nv == 1   ? launch_q<XT, ST, 1, L>(a, grid, block, smem, st)
         : nv == 2 ? launch_q<XT, ST, 2, L>(a, grid, block, smem, st)
                   : launch_q<XT, ST, 4, L>(a, grid, block, smem, st);
}
template <int XT, int ST>
cudaError_t launch_norm(const NormArgs& a, bool wide, cudaStream_t st) {
  const int groups = (a.H + 7) / 8;
  const bool bits = a.drop.threshold != 0;
  const Layout layout = wide ? kWide : (a.scales && a.blocks) || (bits && groups > 2048) ? kNarrow : kStrided;
  // Blocks of 64 to 256 threads, several of them on an SM, overlap one's reduction with another's loads:
  // 8192 x 4096 with dropout 42.6 us with 4 groups for a thread, 44.3 with 2, 53.6 with 1, 47.1 with
  // 8; 65536 x 256 20.5 us with 1, 24.4 with 2. Value by value the accesses are many and small,
  // and more threads carry them; so do a few rows (1 x 4096 1.9 us with 1 group, 2.7 with 4; 256 x 8192
  // 4.3 with 2, 4.5 with 4).
  int nv = groups <= 64 ? 1 : groups <= 256 ? 2 : groups <= (XT == kFp32 ? 2048 : 1024) ? 4 : 8;
  if (layout == kWide && a.M <= 256)
    nv = groups <= 512 ? 1 : groups <= 1024 ? 2 : groups <= (XT == kFp32 ? 2048 : 1024) ? 4 : 8;
  if (layout == kStrided) nv = groups <= 1024 ? 1 : groups <= 2048 ? 2 : 4;
  if (layout == kNarrow) nv = 8;
  const int threads = ((groups + nv - 1) / nv + 31) / 32 * 32;
  const int rows = threads == 32 ? kBlockRows : 1;
  const dim3 block(static_cast<unsigned>(threads), static_cast<unsigned>(rows));
  const dim3 grid(static_cast<unsigned>((a.M + rows - 1) / rows));
  if (layout == kNarrow) return launch_q<XT, ST, 8, kNarrow>(a, grid, block, 0, st);
  if (layout == kWide) return launch_nv<XT, ST, kWide>(a, nv, grid, block, 0, st);
  const size_t smem = bits ? static_cast<size_t>(threads) * nv * rows * 16 : 0;
  return launch_nv<XT, ST, kStrided>(a, nv, grid, block, smem, st);
}

}  // namespace
}  // namespace flce
