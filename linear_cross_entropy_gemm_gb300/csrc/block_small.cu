// Few-token products: the layer operators' GEMMs with the operands swapped.
//
// With M tokens far below a 256-row tile the product is bound by streaming the
// weights from HBM, so the weights take the MMA's 128 rows (TMEM lanes) and the
// tokens its columns:
//
//   D[f, m] = sum_k Wt[f, k] x[m, k],   128 features x NT tokens, NT = 16, 32, 64, 128
//
// and a tile computes up to half of its columns for nothing (33 tokens take 64, 129 two
// tiles of 128), which the stream of weights hides. A tile of the gated
// projection has 64 rows of each weight, so that its ring stage is no larger. One CTA per tile and K
// slice: the slices of a tile form a cluster (1, 2, 4 or 8 CTAs), so that even a
// narrow layer keeps every SM streaming. The slices join through distributed shared
// memory: each CTA sends the others the fp32 partial sums of their share of the
// features, adds what it got in rank order (the result does not depend on timing) and
// applies the epilogue: no scratch memory, no second launch.
//
// Warp 0 streams (W, x) slices by TMA through a ring, warp 1 issues the MMAs, and
// four warps move the accumulator to shared memory. Up to 32 tokens those four also
// bring x into the ring, by plain loads a ring's length ahead: so small a tensor is
// slow to load by TMA when every SM shares it (gated 1 token x 4096 x 14336 45 us, 38 us
// with plain loads).
#include <cuda_runtime.h>

#include "block_epilogues.cuh"
#include "block_internal.h"

namespace flce {

constexpr int kSmThreads = 192;
constexpr int kWTileBytes = 128 * kBK * 2;  // one weight slice, 16 KiB

// Ring stages: two CTAs per SM up to 64 tokens (their loads overlap each other's
// epilogues), one above.
template <int NT>
struct SmallShape {
  static constexpr int kStage = kWTileBytes + NT * kBK * 2;
  static constexpr int kRing = NT <= 64 ? 108 * 1024 : 208 * 1024;
  static constexpr int kStages = kRing / kStage;
  static constexpr int kTmem = NT < 32 ? 32 : NT;  // TMEM columns
  static constexpr bool kPlainX = NT <= 32;        // x by plain loads
  static constexpr int kXChunks = NT * 8 / 128;    // 16-byte words of a slice for each of 128 threads
  static constexpr int kPartial = NT * 128 * 4;    // joins reuse the ring
  static constexpr int kBody = kStages * kStage > kPartial ? kStages * kStage : kPartial;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kBody) + kBarrierBytes;
  static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KiB a CTA may use");
  static_assert((2 * kStages + 1) * 8 + 8 <= kBarrierBytes, "barriers do not fit");
};

// 32 lanes x 16 consecutive fp32 columns: the load is complete after tmem_wait_16.
__device__ __forceinline__ void tmem_issue_16(uint32_t taddr, uint32_t (&r)[16]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
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

// Thread t's 16-byte words of x in slice kb: eight threads to a token's 64 sum elements;
// zeros past the sum's end and past the last token.
template <int CHUNKS>
__device__ __forceinline__ void fetch_x(const SmallArgs& a, int kb, int m0, int t,
                                        uint4 (&v)[CHUNKS]) {
  const bool second = kb >= a.k_split;
  const int col = (second ? kb - a.k_split : kb) * kBK + (t & 7) * 8, n = a.k_len - col;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int m = m0 + (t >> 3) + c * 16;
    v[c] = make_uint4(0u, 0u, 0u, 0u);
    if (m >= a.M || n <= 0) continue;
    const uint16_t* p = (second ? a.xp2 : a.xp) + static_cast<size_t>(m) * a.ld_x + col;
    if (n >= 8) {
      v[c] = *reinterpret_cast<const uint4*>(p);
    } else {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < n) w[j >> 1] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
      v[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// W_MN: the weights' features are contiguous and its rows are the sum (dx: W and
// dz), else its rows are the features. TWO: two weight tensors with one x (gated
// forward); rows 0 .. 63 of a tile are the first's, 64 .. 127 the second's. The
// two-segment sum of the gated dx is `k_split` < `k_blocks`.
// The bound of one block is for ptxas, which otherwise stops at 64 registers and spills (32 x
// 14336 x 4096 23.45 us, 22.99 us); two blocks of 148 fit an SM.
template <int NT, bool TWO, bool W_MN>
__global__ void __launch_bounds__(kSmThreads, 1)
    small_gemm_kernel(const __grid_constant__ SmallArgs a) {
  using S = SmallShape<NT>;
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
  constexpr int kOut = TWO ? 64 : 128;  // output features of a tile
  const int f0 = static_cast<int>(blockIdx.x) / slices * kOut;
  const int m0 = static_cast<int>(blockIdx.y) * NT;
  const int kb_lo = static_cast<int>(static_cast<int64_t>(a.k_blocks) * rank / slices);
  const int kb_n = static_cast<int>(static_cast<int64_t>(a.k_blocks) * (rank + 1) / slices) - kb_lo;
  // Tiles start at different places of their slice and go round it, so that the CTAs of
  // an x do not all read the same few lines of it at the same time.
  const int turn = static_cast<int>(blockIdx.x) / slices * 5 % kb_n;
  const auto block = [&](int j) { return kb_lo + (j + turn < kb_n ? j + turn : j + turn - kb_n); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], S::kPlainX ? 5 : 1);  // the producer, and the warps that bring x
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&a.w);
    if constexpr (!S::kPlainX) tma_prefetch_desc(&a.x);
  }
  if (warp == 1) tmem_alloc(tmem_slot, S::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch();

  griddep_wait();

  if (warp == 0) {
    const uint64_t pol = l2_policy_evict_normal();
    int s = 0, issued = 0;
    uint32_t ph = 0;
    for (int j = 0; j < kb_n; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1, abort_flag, a.dev_err))) break;
      const int kb = block(j);
      uint8_t* w = smem + s * S::kStage;
      const bool second = kb >= a.k_split;
      const int k0 = (second ? kb - a.k_split : kb) * kBK;
      const CUtensorMap* mw = second ? &a.w2 : &a.w;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[s], S::kPlainX ? kWTileBytes : S::kStage);
        if constexpr (TWO) {
          tma_load_2d(w, &a.w, &full[s], k0, f0, pol);
          tma_load_2d(w + kWTileBytes / 2, &a.w2, &full[s], k0, f0, pol);
        } else if constexpr (!W_MN) {
          tma_load_2d(w, mw, &full[s], k0, f0, pol);
        } else {
          tma_load_2d(w, mw, &full[s], f0, k0, pol);
          tma_load_2d(w + kMnBoxBytes, mw, &full[s], f0 + 64, k0, pol);
        }
        if constexpr (!S::kPlainX)
          tma_load_2d(w + kWTileBytes, second ? &a.x2 : &a.x, &full[s], k0, m0, pol);
      }
      __syncwarp();
      ++issued;
      if (++s == S::kStages) {
        s = 0;
        ph ^= 1;
      }
    }
    // Drain: the last load issued into each stage must land before the ring is reused.
    for (int i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i)
      mbar_drain(&full[i % S::kStages], static_cast<uint32_t>((i / S::kStages) & 1));
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f16kind_f32(128, NT, W_MN, false, a.fp16 != 0);
    const uint32_t s0 = smem_u32(smem);
    const uint64_t w0 = smem_desc_sw128(s0, W_MN ? kMnBoxBytes : 16, 1024);
    const uint64_t x0 = smem_desc_sw128(s0 + kWTileBytes, 16, 1024);
    int s = 0;
    uint32_t ph = 0;
    for (int j = 0; j < kb_n; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], ph, abort_flag, a.dev_err))) break;
      tc_fence_after();
      const uint64_t off = static_cast<uint64_t>(s) * (S::kStage / 16);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kBK / kUmmaK; ++kk) {
          const uint64_t wd = w0 + off + kk * (W_MN ? 128 : 2), xd = x0 + off + kk * 2;
          const uint32_t acc = j != 0 || kk != 0 ? 1u : 0u;
          umma_bf16(tmem_base, wd, xd, idesc, acc);
        }
        umma_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == S::kStages) {
        s = 0;
        ph ^= 1;
      }
    }
    if (elect_one()) umma_commit(done);
    __syncwarp();
    mbar_drain(done, 0);
  } else if constexpr (S::kPlainX) {
    const int t = static_cast<int>(threadIdx.x) - 64;
    uint4 ahead[S::kStages][S::kXChunks];
#pragma unroll
    for (int i = 0; i < S::kStages; ++i)
      if (i < kb_n) fetch_x<S::kXChunks>(a, block(i), m0, t, ahead[i]);
    uint32_t ph = 0;
    bool ok = true;
    for (int j = 0; j < kb_n && ok; j += S::kStages) {
#pragma unroll
      for (int i = 0; i < S::kStages; ++i) {
        if (j + i >= kb_n || !ok) break;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[i], ph ^ 1, abort_flag, a.dev_err));
        if (!ok) break;
        uint8_t* x = smem + i * S::kStage + kWTileBytes;
#pragma unroll
        for (int c = 0; c < S::kXChunks; ++c) {
          const int row = (t >> 3) + c * 16, word = (t & 7) ^ (row & 7);  // the 128-byte swizzle
          *reinterpret_cast<uint4*>(x + row * 128 + word * 16) = ahead[i][c];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[i]);
        if (j + i + S::kStages < kb_n)
          fetch_x<S::kXChunks>(a, block(j + i + S::kStages), m0, t, ahead[i]);
      }
      ph ^= 1;
    }
  }
  // The producer and the issuer leave their branches only when every load has
  // landed and every MMA is done, so the ring may be overwritten: by this CTA, and
  // once the whole cluster is here, by the others.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (slices > 1) cluster_sync();
  tc_fence_after();

  const int tokens = min(NT, a.M - m0);
  // Received partial sums, fp32 [slices][products][NT tokens][own features].
  constexpr int kProducts = TWO ? 2 : 1;
  const int own = kOut / slices;  // output features that this CTA writes
  const float* part = reinterpret_cast<const float*>(smem);
  if (warp >= 2) {
    const int quad = warp & 3, lane_row = quad * 32 + lane;
    const int h = lane_row / kOut, f = lane_row - h * kOut;
    const uint32_t base = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const int to = f / own;  // rank that writes feature f
    const uint32_t mine =
        smem_u32(smem) +
        static_cast<uint32_t>(((rank * kProducts + h) * NT * own + f - to * own) * 4);
    const uint32_t dst = slices > 1 ? mapa_shared(mine, static_cast<uint32_t>(to)) : mine;
#pragma unroll 1
    for (int c = 0; c < tokens; c += 16) {
      uint32_t r[16];
      tmem_issue_16(base + c, r);
      tmem_wait_16(r);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (c + j >= tokens) break;
        st_cluster_f32(dst + static_cast<uint32_t>((c + j) * own * 4), __uint_as_float(r[j]));
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (slices > 1) cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, S::kTmem);

  // This CTA's features: [rank * own, rank * own + own) of the tile, 8 at a time.
  const int groups = own / 8;
  const bool f16 = a.fp16 != 0;
  // relu's signs (signs_again) are looked at by whole warps, in a loop of its own.
  const auto finish = [&](auto with_signs) {
    constexpr bool kSigns = decltype(with_signs)::value;
    for (int i0 = warp * 32; i0 < tokens * groups; i0 += kSmThreads) {
      const int i = i0 + lane, t = i / groups, gl = i - t * groups;
      const int col = f0 + rank * own + gl * 8, n = a.N - col;
      const bool mine = i < tokens * groups && n > 0;
      if (!mine && !kSigns) continue;
      float v[kProducts][8];
      const size_t row = static_cast<size_t>(m0 + t);
      uint32_t near = 0, above = 0;
      if (mine) {
#pragma unroll
        for (int h = 0; h < kProducts; ++h) {
          const float* p = part + (h * NT + t) * own + gl * 8;
          const int step = kProducts * NT * own;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[h][j] = p[j];
#pragma unroll
          for (int r = 1; r < 8; ++r) {
            if (r < slices) {
              const float4 q0 = *reinterpret_cast<const float4*>(p + r * step);
              const float4 q1 = *reinterpret_cast<const float4*>(p + r * step + 4);
              v[h][0] += q0.x;
              v[h][1] += q0.y;
              v[h][2] += q0.z;
              v[h][3] += q0.w;
              v[h][4] += q1.x;
              v[h][5] += q1.y;
              v[h][6] += q1.z;
              v[h][7] += q1.w;
            }
          }
        }
        float largest = 0.f;
        if constexpr (kSigns) largest = largest_of(v[0]);
        if (!TWO && a.bias) {
          float b[8];
          load8(a.bias + col, n, true, f16, b);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[0][j] += b[j];
        }
        if constexpr (kSigns) {
          near = near_zero(v[0], largest, a.k_len);
          if (n < 8) near &= (1u << n) - 1u;
        }
      }
      if constexpr (kSigns) {
        if (__any_sync(0xffffffffu, near != 0))
          above = signs_again(SignArgs{a.xp, a.wp, a.bias, a.ld_x, a.k_len}, f16,
                              static_cast<int>(row), col, near, lane);
        if (!mine) continue;
      }
      if constexpr (TWO) {
        float (&u)[8] = v[kProducts - 1];
        if (a.keep) {
          float x[8];
          act_cross(a.act, v[0], u, x);
          if constexpr (kSigns) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if ((near >> j) & 1u) x[j] = ((above >> j) & 1u) ? u[j] : 0.f;
          }
          uint16_t* k = a.keep + row * a.N + col;
          uint32_t w[4];
          encode_groups(a.relative != 0, v[0], w);
          *reinterpret_cast<uint4*>(k) = make_uint4(w[0], w[1], w[2], w[3]);
          encode_groups(a.relative != 0, x, w);
          *reinterpret_cast<uint4*>(k + static_cast<size_t>(a.M) * a.N) =
              make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          act_all(a.act, v[0]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[0][j] *= u[j];
      } else {
        if (a.keep) {
          uint32_t w[4];
          with_act(a.act, [&](auto act) {
            constexpr int kAct = decltype(act)::value;
            if (a.relative != 0)
              act_keep_slopes<kAct, true>(v[0], w);
            else
              act_keep_slopes<kAct, false>(v[0], w);
          });
          if constexpr (kSigns) put_signs(near, above, w);
          uint16_t* k = a.keep + row * a.N + col;
          if (a.N % 8 == 0) {
            *reinterpret_cast<uint4*>(k) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j < n) k[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
          }
        } else {
          act_all(a.act, v[0]);
        }
        if (a.res) {
          float r[8];
          load8(a.res + row * a.ld_res + col, n, a.res_vec != 0, f16, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[0][j] += r[j];
        }
      }
      store8(a.y + row * a.ld_y + col, n, a.y_vec != 0, f16, v[0]);
    }
  };
  if constexpr (!W_MN) {
    if (a.keep && a.act == kActRelu) {
      finish(std::true_type());
      return;
    }
  }
  finish(std::false_type());
}

template <int NT, bool TWO, bool W_MN>
static cudaError_t launch_t(const SmallArgs& a, cudaStream_t st) {
  using S = SmallShape<NT>;
  auto kernel = small_gemm_kernel<NT, TWO, W_MN>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  constexpr int kOut = TWO ? 64 : 128;
  const dim3 grid(static_cast<unsigned>((a.N + kOut - 1) / kOut * a.slices),
                  static_cast<unsigned>((a.M + NT - 1) / NT));
  return launch_dependent(kernel, grid, kSmThreads, S::kSmem, a.slices, st, a);
}

int small_tokens(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// Tiles of a product, and the clusters of 1, 2, 4 and 8 CTAs that run at once (as the
// runtime says) with one CTA to an SM (128 tokens) and with two.
int64_t small_tiles(int64_t M, int64_t N, bool two) {
  const int64_t nt = small_tokens(M), out = two ? 64 : 128;
  return (N + out - 1) / out * ((M + nt - 1) / nt);
}
int64_t small_clusters(int64_t M, int slices) {
  constexpr int kOne[] = {152, 76, 36, 15}, kTwo[] = {304, 152, 74, 36};
  const int i = slices == 8 ? 3 : slices / 2;
  return small_tokens(M) <= 64 ? kTwo[i] : kOne[i];
}
int small_slices(int64_t M, int64_t N, int k_blocks, bool two) {
  const int64_t tiles = small_tiles(M, N, two);
  int s = 1;
  while (s < 8 && tiles <= small_clusters(M, 2 * s) && 2 * s <= k_blocks) s *= 2;
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
