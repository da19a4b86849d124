// Kernels of the root-mean-square norm's backward, for one type of the operands (rms_norm.cu says
// what they compute).
//
// One pass: a block takes every gridDim-th row and keeps its columns' share of dw in
// registers, so dy, h and dh are read once for both results. On 16-byte rows the next two are on
// their way into shared memory, each thread its own part and for itself alone, while one is
// worked on. The blocks' shares are added in a fixed order by a second kernel. Bound by HBM, and
// by instructions close behind: the arithmetic is on packed pairs, and products of 16-bit values
// take them as they are. 8192 x 4096 bf16 with dh 45 to 47 us (6.0 TB/s, dw's sum 5 of it), with dropout
// 57 (the generator's ten rounds for 8 columns), fp32 84. Rows off the 16-byte boundaries go value
// by value, by up to 1024 threads: 8192 x 4095 86 us (512 threads with twice the columns 118).
//
// dw takes h as it is stored: in 16 bits its rounding adds as much error to dw as dw's own to 16 bits.
// The sum before rounding is not in memory, and keeping it would cost more bytes than the pass has.
#pragma once
#include <cuda_runtime.h>

#include "block_internal.h"
#include "rms_norm.h"
#include "stream_ops.cuh"

namespace flce {
namespace {

// Copies of 16 bytes from global to shared memory, in the background; done once the group that
// holds them is waited for.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// blockDim.x threads for a row, blockDim.y rows at a time (one, unless a warp holds a row); a thread
// holds NV groups of 8 columns.
template <int XT, int ST, int NV, Layout L, bool DROP>
__global__ void __launch_bounds__(L == kStrided ? 1024 : NV == 1 ? 256 : kRowThreads, L == kWide && NV == 1 ? 4 : 1)
    norm_grad_kernel(const __grid_constant__ NormGradArgs a) {
  constexpr bool kRing = L == kWide && grad_has_ring(NV, type_size(ST));
  constexpr int kStages = grad_stages(NV);
  constexpr int XV = type_size(XT) / 2, SV = type_size(ST) / 2;  // 16-byte words of a group
  constexpr int kWords = NV * (XV + 2 * SV);
  __shared__ float s_sum[2][32];
  extern __shared__ __align__(16) uint8_t smem[];
  griddep_wait();
  const int T = blockDim.x, t = threadIdx.x, n = a.H;
  const int first = blockIdx.x * blockDim.y + threadIdx.y, step = gridDim.x * blockDim.y;
  // The generator's keys: value by value, in shared memory, as the registers are few.
  __shared__ Keys s_keys;
  Keys keys;
  if constexpr (DROP && L == kWide) keys = dropout_keys(a.drop);
  if constexpr (DROP && L != kWide) {
    if (threadIdx.y * T + t == 0) s_keys = dropout_keys(a.drop);
    __syncthreads();
  }
  Raw8<XT> wr[NV];
  uint64_t acc[NV * 4];  // pairs of columns
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    constexpr float ones[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    wr[j] = pack8<XT>(ones);
    if (a.w && (XT == kFp32 || !a.w_fp32)) wr[j] = load_group<XT, L>(a.w, j, T, t, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[4 * j + i] = f32x2(0.f, 0.f);
  }
  // An fp32 weight beside 16-bit operands is loaded for each row.
  const bool wider = XT != kFp32 && a.w && a.w_fp32;
  const auto weights = [&](int j, uint64_t* w) {
    if (wider) {
      const Raw8<kFp32> r = load_group<kFp32, L>(a.w, j, T, t, n);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pair_of(r, i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pair_of(wr[j], i);
    }
  };
  const int threads = T * blockDim.y, me = threadIdx.y * T + t;
  uint4* ring = reinterpret_cast<uint4*>(smem) + me;
  const auto word = [&](int stage, int i) { return ring + (stage * kWords + i) * threads; };
  const auto row_of = [](const void* p, int row, int64_t ld, int size) {
    return static_cast<const uint8_t*>(p) + row * ld * size;
  };
  const auto fetch = [&](int row, int stage) {
    if (row < a.M) {
      const uint8_t* dy = row_of(a.dy, row, a.ld_dy, type_size(XT)) + t * XV * 16;
      const uint8_t* h = row_of(a.h, row, a.ld_h, type_size(ST)) + t * SV * 16;
      const uint8_t* dh = row_of(a.dh, row, a.ld_dh, type_size(ST)) + t * SV * 16;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if ((j * T + t) * 8 >= n) break;
#pragma unroll
        for (int i = 0; i < XV; ++i) copy16(word(stage, j * XV + i), dy + (j * T * XV + i) * 16);
#pragma unroll
        for (int i = 0; i < SV; ++i) {
          copy16(word(stage, NV * XV + j * SV + i), h + (j * T * SV + i) * 16);
          if (a.dh) copy16(word(stage, NV * (XV + SV) + j * SV + i), dh + (j * T * SV + i) * 16);
        }
      }
    }
    copies_end();
  };
  Raw8<XT> rd[NV];
  Raw8<ST> rh[NV], re[NV];
  int turn = 0, stage = 0;
  float next_rstd = first < a.M ? a.rstd[first] : 0.f;
  if constexpr (kRing) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(first + i * step, i);
  }
  for (int row = first; row < a.M; row += step, turn ^= 1) {
    const float rstd = next_rstd;
    if (row + step < a.M) next_rstd = a.rstd[row + step];
    if constexpr (kRing) {
      copies_wait<kStages - 2>();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        rd[j] = {};
        rh[j] = {};
        re[j] = {};
        if (column<L>(j, 0, T, t) >= n) break;
#pragma unroll
        for (int i = 0; i < XV; ++i) rd[j].w[i] = *word(stage, j * XV + i);
#pragma unroll
        for (int i = 0; i < SV; ++i) {
          rh[j].w[i] = *word(stage, NV * XV + j * SV + i);
          if (a.dh) re[j].w[i] = *word(stage, NV * (XV + SV) + j * SV + i);
        }
      }
      // Into the words of the row before: this thread has read them.
      fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        rd[j] = load_group<XT, L>(row_of(a.dy, row, a.ld_dy, type_size(XT)), j, T, t, n);
        rh[j] = load_group<ST, L>(row_of(a.h, row, a.ld_h, type_size(ST)), j, T, t, n);
        re[j] = {};
        if (a.dh) re[j] = load_group<ST, L>(row_of(a.dh, row, a.ld_dh, type_size(ST)), j, T, t, n);
      }
    }
    uint64_t sums = f32x2(0.f, 0.f);
    const uint64_t rstd2 = f32x2(rstd, rstd);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t w[4];
      weights(j, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint64_t dv;
        if constexpr (XT == ST)
          dv = pair_product(rd[j], rh[j], i);
        else
          dv = fmul2(pair_of(rd[j], i), pair_of(rh[j], i));
        acc[4 * j + i] = ffma2(dv, rstd2, acc[4 * j + i]);
        sums = ffma2(dv, w[i], sums);
      }
    }
    if (!a.dx && !a.dr) continue;
    float sum, other;
    f32x2_split(sums, sum, other);
    const float c = row_reduce<false>(sum + other, s_sum[turn]) * rstd / static_cast<float>(n);
    const float along = -(rstd * rstd) * c;
    const uint64_t along2 = f32x2(along, along);
    uint8_t* dx = static_cast<uint8_t*>(a.dx) + static_cast<int64_t>(row) * n * type_size(XT);
    uint8_t* dr = static_cast<uint8_t*>(a.dr) + static_cast<int64_t>(row) * n * type_size(ST);
    const uint16_t* bits = nullptr;
    if constexpr (DROP && L != kWide) {
      // Eight columns share a counter: a thread makes neighbours' bits, and takes its own.
      uint4* made = reinterpret_cast<uint4*>(smem) + threadIdx.y * (NV * T);
      T == 32 ? __syncwarp() : __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j) made[j * T + t] = drop_bits(a.drop, s_keys, row, j * T + t);
      T == 32 ? __syncwarp() : __syncthreads();
      bits = reinterpret_cast<const uint16_t*>(made);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t w[4];
      float g[8];
      weights(j, w);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f32x2_split(ffma2(pair_of(rh[j], i), along2,
                          ffma2(fmul2(pair_of(rd[j], i), w[i]), rstd2, pair_of(re[j], i))),
                    g[2 * i], g[2 * i + 1]);
      if (a.dr) store_group<ST, L>(dr, j, T, t, n, g);
      if (a.dx) {
        if constexpr (DROP && L == kWide) drop8(a.drop, keys, row, j * T + t, g);
        if constexpr (DROP && L != kWide) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            g[e] = bits[column<L>(j, e, T, t)] >= a.drop.threshold ? g[e] * a.drop.scale : 0.f;
        }
        store_group<XT, L>(dx, j, T, t, n, g);
      }
    }
  }
  if constexpr (kRing) copies_wait<0>();
  // Not before: blocks of the next kernel that wait on an SM keep this one's from it (20000 x 2048
  // 67 us so, 54 with the call here).
  griddep_launch();
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * n;
  if (blockDim.y > 1) {
    // The warps' shares, in their order.
    __shared__ uint64_t shares[kBlockRows - 1][NV == 1 ? 4 : 1][32];
    if constexpr (NV == 1) {
      if (threadIdx.y > 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) shares[threadIdx.y - 1][i][t] = acc[i];
      __syncthreads();
      if (threadIdx.y > 0) return;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        for (int r = 0; r < static_cast<int>(blockDim.y) - 1; ++r) acc[i] = fadd2(acc[i], shares[r][i][t]);
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f32x2_split(acc[4 * j + i], v[2 * i], v[2 * i + 1]);
    store_group<kFp32, L>(part, j, T, t, n, v);
  }
}

template <int XT, int ST, int NV, bool DROP>
cudaError_t launch_nv(const NormGradArgs& a, bool wide, const GradShape& s, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(s.blocks));
  const dim3 block(static_cast<unsigned>(s.threads), static_cast<unsigned>(s.rows));
  auto kernel = norm_grad_kernel<XT, ST, NV, kWide, DROP>;
  if constexpr (NV <= 4)
    if (!wide) kernel = norm_grad_kernel<XT, ST, NV, kStrided, DROP>;
  const size_t smem = wide ? grad_ring(s, type_size(XT), type_size(ST))
                      : DROP ? static_cast<size_t>(NV) * s.threads * s.rows * 16 : 0;
  // Beyond 48 KiB, of which the kernel's own arrays take under 4, it is asked for: always the most that this
  // kernel can need, so that no call lowers what another is about to launch with.
  if (smem > 44 * 1024) {
    const size_t most = wide ? grad_ring({NV, NV == 1 ? 256 : kRowThreads, 1, 1}, type_size(XT), type_size(ST))
                             : static_cast<size_t>(NV) * 1024 * 16;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kernel, grid, block, smem, 1, st, a);
}
template <int XT, int ST, int NV>
cudaError_t launch_drop(const NormGradArgs& a, bool wide, const GradShape& s, cudaStream_t st) {
  return a.drop.threshold != 0 ? launch_nv<XT, ST, NV, true>(a, wide, s, st)
                               : launch_nv<XT, ST, NV, false>(a, wide, s, st);
}
template <int XT, int ST>
cudaError_t launch_grad(const NormGradArgs& a, bool wide, const GradShape& s, cudaStream_t st) {
  return s.nv == 1   ? launch_drop<XT, ST, 1>(a, wide, s, st)
         : s.nv == 2 ? launch_drop<XT, ST, 2>(a, wide, s, st)
         : s.nv == 4 ? launch_drop<XT, ST, 4>(a, wide, s, st)
                     : launch_drop<XT, ST, 8>(a, wide, s, st);
}

}  // namespace
}  // namespace flce
