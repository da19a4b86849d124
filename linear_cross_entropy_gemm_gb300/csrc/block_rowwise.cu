// Element-wise (HBM-bound) parts of the layer operators' backward passes:
//   dz     : dz = dy a'(z) in the operands' type, with its fp32 column sums
//            (the bias gradient's partials)
//   gated  : dg = dh u a'(g), du = dh a(g)
// a'(z), a(g) and u a'(g) are what the forward kept (block_epilogues.cuh): reading them
// takes a few operations a value where recomputing an activation took thirty.
#include <cuda_runtime.h>

#include "block_epilogues.cuh"
#include "block_internal.h"

namespace flce {

__device__ __forceinline__ void unpack8(const uint4& u, bool f16, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = unpack_16(w[e] & 0xFFFFu, f16);
    v[2 * e + 1] = unpack_16(w[e] >> 16, f16);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8], bool f16) {
  uint4 u;
  u.x = pack_16x2(v[0], v[1], f16);
  u.y = pack_16x2(v[2], v[3], f16);
  u.z = pack_16x2(v[4], v[5], f16);
  u.w = pack_16x2(v[6], v[7], f16);
  return u;
}

// A block takes 256 columns (32 threads x 8) of one part's rows, 8 rows at a
// time; a thread keeps the fp32 sums of its columns, and the eight row groups
// are added in a fixed order at the end. With rows off the 16-byte boundaries
// a thread's columns are 32 apart instead of adjacent, so that a warp's
// accesses stay contiguous.
constexpr int kDzCols = 256, kDzRowGroups = 8;

static int dz_rows_per_part(int64_t M, int64_t N) {
  // About two waves of 8 blocks on each of 152 SMs.
  const int64_t ct = (N + kDzCols - 1) / kDzCols;
  int64_t parts = (2 * 8 * 152 + ct - 1) / ct;
  int64_t rows = (M + parts - 1) / parts;
  rows = (rows + kDzRowGroups - 1) / kDzRowGroups * kDzRowGroups;
  return static_cast<int>(rows);
}

int dz_parts(int64_t M, int64_t N) {
  const int64_t rows = dz_rows_per_part(M, N);
  return static_cast<int>((M + rows - 1) / rows);
}

__global__ void __launch_bounds__(32 * kDzRowGroups) dz_kernel(const DzArgs a, int rows_per_part) {
  __shared__ float s_sum[kDzRowGroups][kDzCols];
  griddep_launch();
  griddep_wait();
  const int cg = threadIdx.x & 31, rg = threadIdx.x >> 5;
  const bool f16 = a.fp16 != 0, vec = a.vec != 0;
  const int col0 = blockIdx.x * kDzCols;
  const int r_lo = blockIdx.y * rows_per_part;
  const int r_hi = min(a.M, r_lo + rows_per_part);
  float sum[8] = {};
  const int vcol = col0 + cg * 8;
  if (vec && vcol + 8 <= a.N) {
    // Four rows at a time: their loads are in flight together.
    const bool scaled = a.slope != nullptr;
    for (int r = r_lo + rg; r < r_hi; r += 4 * kDzRowGroups) {
      uint4 d[4], q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r + i * kDzRowGroups;
        if (row >= r_hi) break;
        d[i] = *reinterpret_cast<const uint4*>(a.dy + static_cast<size_t>(row) * a.ld_dy + vcol);
        if (scaled)
          q[i] =
              *reinterpret_cast<const uint4*>(a.slope + static_cast<size_t>(row) * a.N + vcol);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r + i * kDzRowGroups;
        if (row >= r_hi) break;
        float v[8];
        unpack8(d[i], f16, v);
        if (scaled) {
          const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[2 * j] *= decode_slope(w[j] & 0xFFFFu, a.tail);
            v[2 * j + 1] *= decode_slope(w[j] >> 16, a.tail);
          }
        }
        if (a.dz)
          *reinterpret_cast<uint4*>(a.dz + static_cast<size_t>(row) * a.ld_dz + vcol) =
              pack8(v, f16);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[j];
      }
    }
  } else {
    const int first = vec ? vcol : col0 + cg, step = vec ? 1 : 32;
    for (int r = r_lo + rg; r < r_hi; r += kDzRowGroups) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = first + j * step;
        if (c >= a.N) continue;
        float v = unpack_16(a.dy[static_cast<size_t>(r) * a.ld_dy + c], f16);
        if (a.slope) v *= decode_slope(a.slope[static_cast<size_t>(r) * a.N + c], a.tail);
        if (a.dz) a.dz[static_cast<size_t>(r) * a.ld_dz + c] = to16(v, f16);
        sum[j] += v;
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) s_sum[rg][vec ? cg * 8 + j : j * 32 + cg] = sum[j];
  __syncthreads();
  const int c = threadIdx.x;
  if (col0 + c < a.N) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kDzRowGroups; ++k) t += s_sum[k][c];
    a.part[static_cast<size_t>(blockIdx.y) * a.N + col0 + c] = t;
  }
}

cudaError_t launch_dz(const DzArgs& a, cudaStream_t st) {
  const dim3 grid((a.N + kDzCols - 1) / kDzCols, dz_parts(a.M, a.N));
  return launch_dependent(dz_kernel, grid, 32 * kDzRowGroups, 0, 1, st, a,
                          dz_rows_per_part(a.M, a.N));
}

// db = the ordered sum of the parts: a block takes 32 columns, its 32 warps every 32nd
// part each, and the warps' sums are added in warp order.
constexpr int kDbSumWarps = 32;
__global__ void __launch_bounds__(32 * kDbSumWarps)
    db_sum_kernel(const float* part, int parts, int N, void* db, int fp32, int fp16) {
  __shared__ float s_sum[kDbSumWarps][33];
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (col < N) {
#pragma unroll 8
    for (int i = w; i < parts; i += kDbSumWarps) t += part[static_cast<size_t>(i) * N + col];
  }
  s_sum[w][lane] = t;
  __syncthreads();
  if (w != 0 || col >= N) return;
#pragma unroll
  for (int k = 1; k < kDbSumWarps; ++k) t += s_sum[k][lane];
  if (fp32)
    static_cast<float*>(db)[col] = t;
  else
    static_cast<uint16_t*>(db)[col] = to16(t, fp16 != 0);
}

cudaError_t launch_db_sum(const float* part, int parts, int N, void* db, bool fp32, bool fp16,
                          cudaStream_t st) {
  return launch_dependent(db_sum_kernel, dim3(static_cast<unsigned>((N + 31) / 32)),
                          32 * kDbSumWarps, 0, 1, st, part, parts, N, db, fp32 ? 1 : 0,
                          fp16 ? 1 : 0);
}

// A block copies 1024 groups of 8 columns, a thread four of them 256 apart. Index: the 32-
// or 64-bit type that holds rows * cols / 8.
template <class Index>
__global__ void __launch_bounds__(256) repack_kernel(const uint16_t* src, int64_t ld_src,
                                                     uint16_t* dst, int64_t ld_dst, int rows,
                                                     int cols) {
  griddep_launch();
  griddep_wait();
  const Index c8 = static_cast<Index>(cols / 8), n = c8 * static_cast<Index>(rows);
  const Index first = static_cast<Index>(blockIdx.x) * 1024 + threadIdx.x;
  uint4 v[4];
  size_t to[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const Index i = first + 256 * k;
    if (i >= n) break;
    const Index row = i / c8;
    const size_t col = static_cast<size_t>(i - row * c8) * 8;
    v[k] = __ldcs(
        reinterpret_cast<const uint4*>(src + static_cast<size_t>(row) * ld_src + col));
    to[k] = static_cast<size_t>(row) * ld_dst + col;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (first + 256 * k < n) *reinterpret_cast<uint4*>(dst + to[k]) = v[k];
}

cudaError_t launch_repack(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst,
                          int rows, int cols, cudaStream_t st) {
  const uint64_t n = static_cast<uint64_t>(rows) * (cols / 8), blocks = (n + 1023) / 1024;
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  return n < (1ull << 32) - 1024
             ? launch_dependent(repack_kernel<uint32_t>, grid, 256, 0, 1, st, src, ld_src, dst,
                                ld_dst, rows, cols)
             : launch_dependent(repack_kernel<uint64_t>, grid, 256, 0, 1, st, src, ld_src, dst,
                                ld_dst, rows, cols);
}

// One thread takes 8 columns of one row: three 16-byte loads, two 16-byte
// stores. Index: the 32- or 64-bit type that holds M F / 8. Made for each form of the kept
// values: 32 registers, so that an SM is full (8192 x 14336 in 160 us; 168 with both forms
// in one kernel of 40; __ldcs loads 162).
template <class Index, bool RELATIVE>
__global__ void __launch_bounds__(256) gated_grad_kernel(const GatedGradArgs a) {
  griddep_launch();
  griddep_wait();
  const Index f8 = static_cast<Index>(a.F / 8);
  const Index i = static_cast<Index>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= f8 * static_cast<Index>(a.M)) return;
  const Index row = i / f8;
  const size_t col = static_cast<size_t>(i - row * f8) * 8;
  const size_t at = static_cast<size_t>(i) * 8;
  const bool f16 = a.fp16 != 0;
  float d[8], g[8], u[8];
  // Ordinary loads: the kernel is resident while the one before it still writes these.
  const uint4 dv = *reinterpret_cast<const uint4*>(a.dh + static_cast<size_t>(row) * a.ld_dh + col);
  const uint4 gv = *reinterpret_cast<const uint4*>(a.cross + at);
  const uint4 uv = *reinterpret_cast<const uint4*>(a.val + at);
  unpack8(dv, f16, d);
  if constexpr (RELATIVE) {
    decode_group_relative(gv, g);
    decode_group_relative(uv, u);
  } else {
    decode_group(gv, g);
    decode_group(uv, u);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    g[j] *= d[j];
    u[j] *= d[j];
  }
  const size_t to = static_cast<size_t>(row) * a.ld + col;
  *reinterpret_cast<uint4*>(a.dg + to) = pack8(g, f16);
  *reinterpret_cast<uint4*>(a.du + to) = pack8(u, f16);
}

cudaError_t launch_gated_grad(const GatedGradArgs& a, cudaStream_t st) {
  const uint64_t n = static_cast<uint64_t>(a.M) * (a.F / 8);
  const uint64_t blocks = (n + 255) / 256;
  if (blocks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  const bool small = n < (1ull << 32) - 256;
  auto kernel = a.relative != 0
                    ? small ? gated_grad_kernel<uint32_t, true> : gated_grad_kernel<uint64_t, true>
                    : small ? gated_grad_kernel<uint32_t, false> : gated_grad_kernel<uint64_t, false>;
  return launch_dependent(kernel, grid, 256, 0, 1, st, a);
}

}  // namespace flce
