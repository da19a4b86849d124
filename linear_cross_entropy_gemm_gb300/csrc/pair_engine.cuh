// The layer operators' GEMM: D[M, N] = A[M, K] B[N, K]^T on CTA pairs, with a
// tile width that is chosen per problem.
//
// Like gemm_engine.cuh's pair kernels it is persistent and warp-specialised (warp 0
// TMA, warp 1 MMA, the others the epilogue) and computes tiles of 256 rows with
// cta_group::2. It differs in what bounds layers, whose sums are short and whose
// tiles are few:
//   - A tile is HALVES x bn columns wide, bn <= 256 a multiple of 32, so that the
//     tiles can be cut to fill the GPU's last wave. HALVES = 1 double-buffers the
//     accumulator: a tile's epilogue runs beside the next tile's MMAs. HALVES = 2
//     issues two MMAs per K step that share A and fill TMEM with one tile.
//   - Shared memory bounds the narrower tiles: for 64 sum elements a CTA writes and
//     reads 16 KiB of A and 64 bn bytes of B twice at 128 bytes a cycle, 256 + bn cycles,
//     beside 2 bn cycles of tensor work (measured: 338 cycles at bn = 64, 424 at
//     128, 444 at 192, 627 at 256, where the two meet; 1104 for two halves of 256,
//     whose B tiles share the A).
//   - The issuing warps stay converged and elect their thread, and a stage of the
//     HALVES = 1 ring holds 128 sum elements: with 64 and a diverged thread a stage took
//     550 cycles at any width.
//   - A long sum with few tiles is split: the 2 or 3 pairs of a cluster take a part of one
//     tile's sum each, send one another the fp32 partial sums of a share of its columns
//     through distributed shared memory and add them in rank order (SPLIT; the result
//     does not depend on timing).
//   - 8 epilogue warps (two per SM sub-partition): the drain of a tile has to fit
//     beside the next tile's short sum.
// An operand is K-major (rows of the sum) or MN-major, as there, and a product may
// have two operands of one kind (OperandPlan).
//
//   full[s]   (even CTA) : both CTAs' TMA bytes of stage s
//   empty[s]  (each CTA) : pair MMA commit, multicast to both CTAs
//   tfull[a]  (each CTA) : pair MMA commit after a tile's last K step
//   tempty[a] (even CTA) : one arrival per epilogue thread of both CTAs
#pragma once
#include <cstdint>
#include <cuda.h>

#include "block_internal.h"
#include "gemm_engine.cuh"

namespace flce {

// Where the operands come from. Most products have one A and one B; the gated
// feed-forward products have two of one kind (gate and up).
//   kTwoB : a tile's columns are the same rows of B and of B2, so both products of a
//           token and an output column land in one TMEM lane: bn / 2 rows of each, one
//           from each CTA. Such tiles have one half.
//   kTwoK : the sum runs over A B^T and then A2 B2^T, each zero-filled to whole stages.
//   kTwoA : the first m_split 256-row tiles take A, the others A2.
enum OperandPlan : int { kOneEach = 0, kTwoB = 1, kTwoK = 2, kTwoA = 3 };

struct PairArgs {
  CUtensorMap a, b, a2, b2;
  int tiles_m, tiles_n;  // tiles of 256 rows, tiles of the output columns below
  int k_stages;          // stages of the whole sum
  int k_split;           // kTwoK: stages of the first product
  int m_split;           // kTwoA: 256-row tiles of the first A
  int halves, bn;        // accumulator columns of a tile: halves x bn
  int slices;            // pairs that share a tile's sum: 1, 2 or 3
  int band_m;            // raster: bands of this many row tiles
  int fp16;
  int* dev_err;
};

__host__ __device__ constexpr int pair_lk(int halves) { return 128 / halves; }  // sum elements of a stage
// Output columns of a tile.
__host__ __device__ constexpr int pair_cols(OperandPlan plan, int halves, int bn) {
  return plan == kTwoB ? bn / 2 : halves * bn;
}

template <int HALVES>
struct PairShape {
  static constexpr int kLK = pair_lk(HALVES);
  static constexpr int kABytes = 128 * kLK * 2;
  static constexpr int kBBytes = 128 * kLK * 2;  // of one half, at most
  static constexpr int kStage = kABytes + HALVES * kBBytes;
  static constexpr int kStages = HALVES == 1 ? 3 : 4;
  static constexpr int kAccs = HALVES == 1 ? 2 : 1;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStage +
                                  8 * kStageBytes + kBarrierBytes;
  static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KiB a CTA may use");
};
constexpr int kLEpiWarps = 8;
constexpr int kLThreads = 64 + 32 * kLEpiWarps;

// Waits until at most the last committed bulk store of this thread still reads its source.
__device__ __forceinline__ void bulk_wait_group_read1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

// One lane of a converged warp, known to the compiler as such.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// D (+)= A B^T by the pair, keeping A in the tensor core's collector for the next
// MMA (`fill`), or taking it from there for the last time (`lastuse`).
__device__ __forceinline__ void umma_pair_a_fill(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16.collector::a::fill [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_pair_a_last(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16.collector::a::lastuse [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A warp's staging of 32 x 32 blocks on their way to TMA stores: two buffers of 2 KiB
// for 16-bit blocks, so that one is built while the one before it is still read, or
// one of 4 KiB for fp32 blocks. It lives for the whole kernel: `turn` goes on from
// tile to tile.
struct Staging {
  uint8_t* buf;
  int turn;
};

// What an epilogue warp drains: the 32-column chunks [c_lo, c_hi) of a tile. Chunk c
// lies in half c / per, `width` output columns wide; a half's last chunk ends with it: where
// the width is no multiple of 32, that chunk starts early and repeats 16 columns
// with the same values.
struct TileSlice {
  int c_lo, c_hi, per, width;
  int up_off;  // kTwoB: accumulator columns from B's product to B2's
  __device__ __forceinline__ void at(int c, int& acc_col, int& out_col) const {
    const int h = c / per, cc = min((c - h * per) * 32, width - 32);
    acc_col = h * kBN + cc;
    out_col = h * width + cc;
  }
};

// Where an epilogue reads 32 accumulator columns of its row: TMEM; or, of a split tile,
// TMEM plus what the other pairs sent, fp32 float4 [slices - 1][chunks][4 lane
// quarters][8][32 rows].
struct TmemAcc {
  uint32_t taddr;
  __device__ __forceinline__ void load(int col, float (&v)[32]) const {
    tmem_ld_32cols(taddr + static_cast<uint32_t>(col), v);
  }
};
struct SplitAcc {
  uint32_t taddr;     // of the pair's first own chunk
  int product_cols;   // TMEM columns from one product's own chunks to the other's
  const float4* row;  // of this lane, in its quarter
  int slices, own, chunks;  // own: chunks of one product; chunks: of all
  __device__ __forceinline__ void load(int col, float (&v)[32]) const {
    const int lc = col >> 5, h = lc / own;
    tmem_ld_32cols(taddr + static_cast<uint32_t>(h * product_cols + (lc - h * own) * 32), v);
    for (int r = 0; r < slices - 1; ++r) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 t = row[static_cast<size_t>(r * chunks + lc) * 1024 + q * 32];
        v[4 * q] += t.x;
        v[4 * q + 1] += t.y;
        v[4 * q + 2] += t.z;
        v[4 * q + 3] += t.w;
      }
    }
  }
};
// Copies `bytes` of this CTA's shared memory to another CTA of the cluster, completing
// them on a barrier there. Addresses 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_copy_to_cta(uint32_t dst_cluster, uint32_t src, uint32_t bytes,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst_cluster),
      "r"(src), "r"(bytes), "r"(bar_cluster)
      : "memory");
}

__device__ __forceinline__ void pair_coords(const PairArgs& g, int t, int& tm, int& tn) {
  const int per = g.band_m * g.tiles_n, b = t / per, r = t - b * per;
  const int height = min(g.band_m, g.tiles_m - b * g.band_m);
  tn = r / height;
  tm = b * g.band_m + (r - tn * height);
}

template <class Epi, int HALVES, bool SPLIT>
__global__ void __launch_bounds__(kLThreads, 1)
    pair_gemm_kernel(const __grid_constant__ PairArgs g,
                     const __grid_constant__ typename Epi::Args ea) {
  using S = PairShape<HALVES>;
  constexpr bool kAMN = Epi::kAMN, kBMN = Epi::kBMN;
  constexpr OperandPlan kPlan = Epi::kPlan;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* stage = smem + S::kStages * S::kStage;  // epilogue staging
  uint64_t* full = reinterpret_cast<uint64_t*>(stage + kLEpiWarps * kStageBytes);
  uint64_t* empty = full + S::kStages;
  uint64_t* tfull = empty + S::kStages;
  uint64_t* tempty = tfull + S::kAccs;
  uint64_t* done_bar = tempty + S::kAccs;
  uint64_t* xbar = done_bar + 1;  // SPLIT: the other pairs' partial sums have arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(xbar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  static_assert(HALVES == 1 || (!SPLIT && kPlan != kTwoB), "forms of one half");
  const int slices = SPLIT ? g.slices : 1;
  const uint32_t cta = cluster_ctarank(), rank = cta & 1;  // in the cluster, in the pair
  const uint32_t even = cta & ~1u;
  const uint16_t both = static_cast<uint16_t>(3u << even);  // the pair's CTAs
  const bool leader = rank == 0;
  const int num_tiles = g.tiles_m * g.tiles_n;
  // Tiles go round the clusters of the grid; a split launch has one cluster per tile.
  const int cluster = static_cast<int>(blockIdx.x) / (2 * slices);
  const int nclusters = SPLIT ? num_tiles : static_cast<int>(gridDim.x) / 2;
  const int slice = static_cast<int>(cta >> 1);
  const int kb_lo = SPLIT ? g.k_stages * slice / slices : 0;
  const int kb_hi = SPLIT ? g.k_stages * (slice + 1) / slices : g.k_stages;
  const int bn = g.bn;
  const int cols = pair_cols(kPlan, HALVES, bn);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < S::kAccs; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * 32 * kLEpiWarps);
    }
    mbar_init(done_bar, 1);
    if constexpr (SPLIT) mbar_init(xbar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    // Chunks of 16 KiB from each other pair: its share of the tile's bn / 32 chunks.
    if constexpr (SPLIT)
      mbar_arrive_expect_tx(xbar, static_cast<uint32_t>((slices - 1) * (bn / 32 / slices) * 16384));
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&g.a);
    tma_prefetch_desc(&g.b);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch();
  griddep_wait();

  if (warp == 0) {
    // -------------------------------------------------- TMA producer (both CTAs)
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t full0 = mapa_shared(smem_u32(&full[0]), even);
    const int b_boxes = (bn / 2 + 63) / 64;  // MN-major B: boxes of 64 columns
    const uint32_t b_bytes = kBMN ? static_cast<uint32_t>(b_boxes * 64 * S::kLK * 2)
                                  : static_cast<uint32_t>(bn / 2 * S::kLK * 2);
    int s = 0;
    uint32_t ph = 0;
    long long issued = 0;
    bool ok = true;
    for (int t = cluster; t < num_tiles && ok; t += nclusters) {
      int tm, tn;
      pair_coords(g, t, tm, tn);
      int m0 = tm * 256 + static_cast<int>(rank) * 128;
      const CUtensorMap *pa = &g.a, *pb = &g.b;
      int n0 = tn * cols + static_cast<int>(rank) * (bn / 2);
      if constexpr (kPlan == kTwoB) {
        n0 = tn * cols;
        if (!leader) pb = &g.b2;
      }
      if constexpr (kPlan == kTwoA) {
        if (tm >= g.m_split) {
          pa = &g.a2;
          m0 -= g.m_split * 256;
        }
      }
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1, abort_flag, g.dev_err));
        if (!ok) break;
        int k0 = kb * S::kLK;
        if constexpr (kPlan == kTwoK) {
          if (kb >= g.k_split) {
            pa = &g.a2;
            pb = &g.b2;
            k0 -= g.k_split * S::kLK;
          }
        }
        uint8_t* a = smem + s * S::kStage;
        const uint32_t fb = full0 + static_cast<uint32_t>(s) * 8u;
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * (S::kABytes + HALVES * b_bytes));
          if constexpr (!kAMN) {
#pragma unroll
            for (int j = 0; j < S::kLK / 64; ++j)
              tma_load_2d_pair(a + j * 128 * 128, pa, fb, k0 + j * 64, m0, pol);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tma_load_2d_pair(a + j * 128 * S::kLK, pa, fb, m0 + j * 64, k0, pol);
          }
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            uint8_t* b = a + S::kABytes + h * S::kBBytes;
            const int nh = n0 + h * bn;
            if constexpr (!kBMN) {
#pragma unroll
              for (int j = 0; j < S::kLK / 64; ++j)
                tma_load_2d_pair(b + j * 128 * 128, pb, fb, k0 + j * 64, nh, pol);
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (j < b_boxes)
                  tma_load_2d_pair(b + j * 128 * S::kLK, pb, fb, nh + j * 64, k0, pol);
            }
          }
        }
        __syncwarp();
        ++issued;
        if (++s == S::kStages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // Drain: a stage's loads have landed once the pair MMA that read it committed.
    for (long long i = (issued > S::kStages ? issued - S::kStages : 0); i < issued; ++i)
      mbar_drain(&empty[i % S::kStages], static_cast<uint32_t>((i / S::kStages) & 1));
  } else if (warp == 1) {
    if (leader) {
      // ----------------------------------------------- MMA issuer (even CTA)
      // The LBO of an MN-major operand is the distance of its two 64-column boxes.
      const uint32_t idesc = idesc_f16kind_f32(256, bn, kAMN, kBMN, g.fp16 != 0);
      const uint32_t s0 = smem_u32(smem);
      const uint64_t a0 = smem_desc_sw128(s0, kAMN ? 128 * S::kLK : 16, 1024);
      const uint64_t b0 = smem_desc_sw128(s0 + S::kABytes, kBMN ? 128 * S::kLK : 16, 1024);
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int t = cluster; t < num_tiles && ok; t += nclusters) {
        ok = __all_sync(0xffffffffu, mbar_wait(&tempty[acc], aph ^ 1, abort_flag, g.dev_err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kBN);
        for (int kb = kb_lo; kb < kb_hi; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ph, abort_flag, g.dev_err));
          if (!ok) break;
          tc_fence_after();
          const uint64_t as = a0 + static_cast<uint64_t>(s) * (S::kStage / 16);
          const uint64_t bs = b0 + static_cast<uint64_t>(s) * (S::kStage / 16);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < S::kLK / kUmmaK; ++kk) {
              // Offsets of the K step in 16-byte units.
              const uint32_t km = (kk >> 2) * (128 * 128 / 16) + (kk & 3) * 2, mn = kk * 128;
              const uint64_t ad = as + (kAMN ? mn : km), bd = bs + (kBMN ? mn : km);
              const uint32_t accumulate = kb != kb_lo || kk != 0 ? 1u : 0u;
              if constexpr (HALVES == 1) {
                umma_bf16_pair(d, ad, bd, idesc, accumulate);
              } else {
                umma_pair_a_fill(d, ad, bd, idesc, accumulate);
                umma_pair_a_last(d + kBN, ad, bd + S::kBBytes / 16, idesc, accumulate);
              }
            }
            umma_commit_pair(&empty[s], both);
          }
          __syncwarp();
          if (++s == S::kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if constexpr (!SPLIT) {
          if (elect_one()) umma_commit_pair(&tfull[acc], both);
          __syncwarp();
        }
        if (++acc == S::kAccs) {
          acc = 0;
          aph ^= 1;
        }
      }
      if (elect_one()) umma_commit_pair(done_bar, both);
      __syncwarp();
    }
    // Both CTAs: every pair MMA must finish before TMEM is released.
    mbar_drain(done_bar, 0);
  } else if constexpr (!SPLIT) {
    // -------------------------------------------------------- epilogue (both CTAs)
    const int quad = warp & 3;
    TileSlice sl;
    sl.width = kPlan == kTwoB ? cols : bn;
    sl.per = (sl.width + 31) / 32;
    sl.up_off = bn / 2;
    const int chunks = HALVES * sl.per, first = (chunks + 1) / 2;
    sl.c_lo = warp < 6 ? 0 : first;
    sl.c_hi = warp < 6 ? first : chunks;
    Staging st{stage + (warp - 2) * kStageBytes, 0};
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), even);
    int acc = 0;
    uint32_t aph = 0;
    for (int t = cluster; t < num_tiles; t += nclusters) {
      int tm, tn;
      pair_coords(g, t, tm, tn);
      if (!mbar_wait(&tfull[acc], aph, abort_flag, g.dev_err)) break;
      tc_fence_after();
      const TmemAcc from{tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                         static_cast<uint32_t>(acc * kBN)};
      Epi::tile(ea, g, tm, tm * 256 + static_cast<int>(rank) * 128 + quad * 32, tn * cols, lane,
                from, st, sl);
      tc_fence_before();
      tmem_release_arrive_cluster(tempty0 + static_cast<uint32_t>(acc) * 8u);
      if (++acc == S::kAccs) {
        acc = 0;
        aph ^= 1;
      }
    }
    if (lane == 0) bulk_wait_group0();  // this warp's epilogue stores have completed
  }
  if constexpr (SPLIT) {
    // The ring is free once every CTA of the cluster is here: its loads have landed and
    // its MMAs are done.
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    // Output chunk oc of the tile goes to the pair oc / own (with kTwoB both its products).
    const int products = kPlan == kTwoB ? 2 : 1;
    const int own = bn / 32 / products / slices;  // output chunks of a pair
    const int quad = warp & 3, e = warp - 2;
    if (warp >= 2) {
      // Sent chunks are built above the received ones, 4 KiB a warp and chunk.
      const uint32_t recv = smem_u32(smem);
      const uint32_t send = recv + static_cast<uint32_t>((slices - 1) * products * own * 16384);
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll 1
      for (int c = e >> 2; c < bn / 32; c += 2) {
        const int h = c / (own * slices), oc = c - h * own * slices, to = oc / own;
        if (to == slice) continue;
        const int lc = h * own + oc - to * own;
        const int slot = slice - (slice > to ? 1 : 0);  // the receiver has none of its own
        const uint32_t src = send + static_cast<uint32_t>(
                                        ((to - (to > slice ? 1 : 0)) * products * own + lc) * 16384 +
                                        quad * 4096);
        const uint32_t dst =
            recv + static_cast<uint32_t>((slot * products * own + lc) * 16384 + quad * 4096);
        float v[32];
        tmem_ld_32cols(taddr + static_cast<uint32_t>(c * 32), v);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                           src + static_cast<uint32_t>(q * 512 + lane * 16)),
                       "f"(v[4 * q]), "f"(v[4 * q + 1]), "f"(v[4 * q + 2]), "f"(v[4 * q + 3])
                       : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        const uint32_t there = static_cast<uint32_t>(2 * to) + rank;
        if (lane == 0)
          bulk_copy_to_cta(mapa_shared(dst, there), src, 4096, mapa_shared(smem_u32(xbar), there));
        __syncwarp();
      }
      int tm, tn;
      pair_coords(g, cluster, tm, tn);
      Staging st{stage + e * kStageBytes, 0};
      TileSlice sl;
      sl.width = own * 32;
      sl.per = own;
      sl.up_off = own * 32;
      const int first = (own + 1) / 2;
      sl.c_lo = e < 4 ? 0 : first;
      sl.c_hi = e < 4 ? first : own;
      const SplitAcc from{taddr + static_cast<uint32_t>(slice * own * 32), own * slices * 32,
                          reinterpret_cast<const float4*>(smem) + quad * 256 + lane, slices, own,
                          products * own};
      if (mbar_wait(xbar, 0, abort_flag, g.dev_err))
        Epi::tile(ea, g, tm, tm * 256 + static_cast<int>(rank) * 128 + quad * 32,
                tn * cols + slice * own * 32, lane, from, st, sl);
      tc_fence_before();
      if (lane == 0) bulk_wait_group0();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

}  // namespace flce
