// Few-token products: the layer operators' GEMMs with the operands swapped.
//
// With M tokens far below a 256-row tile the product is bound by streaming the
// weights from HBM, so the weights take the MMA's 128 rows (TMEM lanes) and the
// tokens its columns:
//
//   D[f, m] = sum_k Wt[f, k] x[m, k],   128 features x NT tokens, NT = 16 .. 128
//
// and a tile wastes at most 15 of the columns it computes. One CTA per tile and K
// slice: the slices of a tile form a cluster (1, 2, 4 or 8 CTAs), so that even a
// narrow layer keeps every SM streaming. The cluster joins its slices through
// distributed shared memory, each CTA adding the fp32 partial sums of its share
// of the features in rank order (the result does not depend on timing) and
// applying the epilogue: no scratch memory, no second launch.
//
// Warp 0 streams (W, x) slices by TMA through a ring, warp 1 issues the MMAs, and
// four warps move the accumulator to shared memory.
#include <cuda_runtime.h>

#include "block_epilogues.cuh"
#include "block_internal.h"

namespace flce {

constexpr int kSmThreads = 192;
constexpr int kWTileBytes = 128 * kBK * 2;  // one weight slice, 16 KiB

// Ring stages: two CTAs per SM up to 64 tokens (their loads overlap each other's
// epilogues), one above.
template <int NT, bool TWO>
struct SmallShape {
  static constexpr int kStage = (TWO ? 2 : 1) * kWTileBytes + NT * kBK * 2;
  static constexpr int kRing = NT <= 64 ? 108 * 1024 : 208 * 1024;
  static constexpr int kStages = kRing / kStage;
  // An MMA waits about 137 cycles for the one before it on the same accumulator, far
  // longer than its own products take here: the four K steps of a slice go to up to
  // four accumulators, as many as TMEM holds for the CTAs of an SM.
  static constexpr int kAcc = (TWO ? 2 : 1) * NT;
  static constexpr int kWays = kAcc * 4 <= (NT <= 64 ? 256 : 512) ? 4 : 2;
  static constexpr int kTmem = kWays * kAcc;  // columns: a power of two, at least 64
  static constexpr int kPartial = (TWO ? 2 : 1) * NT * 128 * 4;  // joins reuse the ring
  static constexpr int kBody = kStages * kStage > kPartial ? kStages * kStage : kPartial;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kBody) + kBarrierBytes;
  static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KiB a CTA may use");
  static_assert((2 * kStages + 1) * 8 + 8 <= kBarrierBytes, "barriers do not fit");
};

// 32 lanes x 16 consecutive fp32 columns.
__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 8 consecutive 16-bit values of a row: one 16-byte access where `vec`, else as many
// as there are.
__device__ __forceinline__ void load8(const uint16_t* p, int n, bool vec, bool f16, float (&v)[8]) {
  if (vec && n >= 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = unpack_16(w[e] & 0xFFFFu, f16);
      v[2 * e + 1] = unpack_16(w[e] >> 16, f16);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? unpack_16(p[j], f16) : 0.f;
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int n, bool vec, bool f16, const float (&v)[8]) {
  if (vec && n >= 8) {
    uint4 u;
    u.x = pack_16x2(v[0], v[1], f16);
    u.y = pack_16x2(v[2], v[3], f16);
    u.z = pack_16x2(v[4], v[5], f16);
    u.w = pack_16x2(v[6], v[7], f16);
    *reinterpret_cast<uint4*>(p) = u;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = to16(v[j], f16);
  }
}

// W_MN: the weights' features are contiguous and its rows are the sum (dx: W and
// dz), else its rows are the features. TWO: two weight tensors with one x (gated
// forward). The two-segment sum of the gated dx is `k_split` < `k_blocks`.
template <int NT, bool TWO, bool W_MN>
__global__ void __launch_bounds__(kSmThreads)
    small_gemm_kernel(const __grid_constant__ SmallArgs a) {
  using S = SmallShape<NT, TWO>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBody);
  uint64_t* empty = full + S::kStages;
  uint64_t* done = empty + S::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int slices = a.slices;
  const int rank = static_cast<int>(blockIdx.x) % slices;  // = the CTA's rank in its cluster
  const int f0 = static_cast<int>(blockIdx.x) / slices * 128;
  const int m0 = static_cast<int>(blockIdx.y) * NT;
  const int kb_lo = static_cast<int>(static_cast<int64_t>(a.k_blocks) * rank / slices);
  const int kb_hi = static_cast<int>(static_cast<int64_t>(a.k_blocks) * (rank + 1) / slices);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&a.w);
    tma_prefetch_desc(&a.x);
  }
  if (warp == 1) tmem_alloc(tmem_slot, S::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      int s = 0, issued = 0;
      uint32_t ph = 0;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!mbar_wait(&empty[s], ph ^ 1, abort_flag, a.dev_err)) break;
        mbar_arrive_expect_tx(&full[s], S::kStage);
        uint8_t* w = smem + s * S::kStage;
        const bool second = kb >= a.k_split;
        const int k0 = (second ? kb - a.k_split : kb) * kBK;
        const CUtensorMap* mw = second ? &a.w2 : &a.w;
        if constexpr (!W_MN) {
          tma_load_2d(w, mw, &full[s], k0, f0, pol);
          if constexpr (TWO) tma_load_2d(w + kWTileBytes, &a.w2, &full[s], k0, f0, pol);
        } else {
          tma_load_2d(w, mw, &full[s], f0, k0, pol);
          tma_load_2d(w + kMnBoxBytes, mw, &full[s], f0 + 64, k0, pol);
        }
        tma_load_2d(w + (TWO ? 2 : 1) * kWTileBytes, second ? &a.x2 : &a.x, &full[s], k0, m0, pol);
        ++issued;
        if (++s == S::kStages) {
          s = 0;
          ph ^= 1;
        }
      }
      // Drain: the last load issued into each stage must land before the ring is reused.
      for (int i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i)
        mbar_drain(&full[i % S::kStages], static_cast<uint32_t>((i / S::kStages) & 1));
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_f16kind_f32(128, NT, W_MN, false, a.fp16 != 0);
      int s = 0;
      uint32_t ph = 0;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!mbar_wait(&full[s], ph, abort_flag, a.dev_err)) break;
        tc_fence_after();
        const uint32_t w = smem_u32(smem + s * S::kStage);
        const uint32_t x = w + (TWO ? 2 : 1) * kWTileBytes;
#pragma unroll
        for (int kk = 0; kk < kBK / kUmmaK; ++kk) {
          const uint64_t xd = smem_desc_sw128(x + kk * (kUmmaK * 2), 16, 1024);
          const uint32_t acc = kb != kb_lo || kk >= S::kWays ? 1u : 0u;
          const uint32_t d = tmem_base + (kk % S::kWays) * S::kAcc;
#pragma unroll
          for (int h = 0; h < (TWO ? 2 : 1); ++h) {
            const uint32_t wh = w + h * kWTileBytes;
            const uint64_t wd = W_MN
                                    ? smem_desc_sw128(wh + kk * (kUmmaK * 128), kMnBoxBytes, 1024)
                                    : smem_desc_sw128(wh + kk * (kUmmaK * 2), 16, 1024);
            umma_bf16(d + h * NT, wd, xd, idesc, acc);
          }
        }
        umma_commit(&empty[s]);
        if (++s == S::kStages) {
          s = 0;
          ph ^= 1;
        }
      }
      umma_commit(done);
      mbar_drain(done, 0);
    }
  }
  // The producer and the issuer leave their branches only when every load has
  // landed and every MMA is done, so the ring may be overwritten.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const int tokens = min(NT, a.M - m0);
  float* part = reinterpret_cast<float*>(smem);  // [TWO ? 2 : 1][NT tokens][128 features]
  if (warp >= 2) {
    const int quad = warp & 3;
    const uint32_t base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll
    for (int h = 0; h < (TWO ? 2 : 1); ++h) {
#pragma unroll 1
      for (int c = 0; c < tokens; c += 16) {
        float v[16];
        tmem_ld_16cols(base + h * NT + c, v);
#pragma unroll
        for (int w = 1; w < S::kWays; ++w) {
          float q[16];
          tmem_ld_16cols(base + w * S::kAcc + h * NT + c, q);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] += q[j];
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(h * NT + c + j) * 128 + quad * 32 + lane] = v[j];
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, S::kTmem);
  if (slices > 1) cluster_sync();

  // This CTA's features: [f_lo, f_lo + 128 / slices) of the tile, 8 at a time.
  const int groups = 16 / slices;
  const int g_lo = rank * groups;
  const bool f16 = a.fp16 != 0;
  const uint32_t part_addr = smem_u32(part);
  for (int i = threadIdx.x; i < tokens * groups; i += kSmThreads) {
    const int t = i / groups, gi = g_lo + (i - t * groups);
    const int col = f0 + gi * 8, n = a.N - col;
    if (n <= 0) continue;
    float v[TWO ? 2 : 1][8];
#pragma unroll
    for (int h = 0; h < (TWO ? 2 : 1); ++h) {
      const uint32_t off = part_addr + static_cast<uint32_t>(((h * NT + t) * 128 + gi * 8) * 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[h][j] = 0.f;
      for (int r = 0; r < slices; ++r) {
        const uint32_t at = slices > 1 ? mapa_shared(off, r) : off;
        const float4 p = ld_cluster_f4(at), q = ld_cluster_f4(at + 16);
        v[h][0] += p.x;
        v[h][1] += p.y;
        v[h][2] += p.z;
        v[h][3] += p.w;
        v[h][4] += q.x;
        v[h][5] += q.y;
        v[h][6] += q.z;
        v[h][7] += q.w;
      }
    }
    const size_t row = static_cast<size_t>(m0 + t);
    if constexpr (TWO) {
      if (a.keep) {
        store8(a.keep + row * a.N + col, n, true, f16, v[0]);
        store8(a.keep + (static_cast<size_t>(a.M) + row) * a.N + col, n, true, f16, v[1]);
      }
      act_all(a.act, v[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[0][j] *= v[TWO ? 1 : 0][j];
    } else {
      if (a.bias) {
        float b[8];
        load8(a.bias + col, n, true, f16, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[0][j] += b[j];
      }
      if (a.keep) store8(a.keep + row * a.N + col, n, a.N % 8 == 0, f16, v[0]);
      act_all(a.act, v[0]);
      if (a.res) {
        float r[8];
        load8(a.res + row * a.ld_res + col, n, a.res_vec != 0, f16, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[0][j] += r[j];
      }
    }
    store8(a.y + row * a.ld_y + col, n, a.y_vec != 0, f16, v[0]);
  }
  // No CTA leaves while another may still read its partial sums.
  if (slices > 1) cluster_sync();
}

template <int NT, bool TWO, bool W_MN>
static cudaError_t launch_t(const SmallArgs& a, cudaStream_t st) {
  using S = SmallShape<NT, TWO>;
  auto kernel = small_gemm_kernel<NT, TWO, W_MN>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.slices);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + 127) / 128 * a.slices),
                     static_cast<unsigned>((a.M + NT - 1) / NT));
  cfg.blockDim = dim3(kSmThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

int small_tokens(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

int small_slices(int64_t M, int64_t N, int k_blocks) {
  const int64_t nt = small_tokens(M);
  const int64_t tiles = (N + 127) / 128 * ((M + nt - 1) / nt);
  int s = 1;
  const int64_t places = nt <= 64 ? 304 : 152;
  while (s < 8 && tiles * s * 2 <= places && 2 * s <= k_blocks) s *= 2;
  return s;
}

cudaError_t launch_small(bool two, bool w_mn, const SmallArgs& a, cudaStream_t st) {
#define FLCE_SMALL(NT)                                            \
  return two    ? launch_t<NT, true, false>(a, st)                \
         : w_mn ? launch_t<NT, false, true>(a, st)                \
                : launch_t<NT, false, false>(a, st)
  switch (small_tokens(a.M)) {
    case 16: FLCE_SMALL(16);
    case 32: FLCE_SMALL(32);
    case 64: FLCE_SMALL(64);
    default: FLCE_SMALL(128);
  }
#undef FLCE_SMALL
}

}  // namespace flce
