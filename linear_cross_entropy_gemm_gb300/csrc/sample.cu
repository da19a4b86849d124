// Sampling from logits with temperature, top-k, top-p and min-p, from given random numbers.
//
//   w_i = exp((z_i - max z) / T);  order: by z falling, then by index
//   S_k: the first k.  S_p: those of S_k before which less than p sum(S_k) lies.
//   S = { i in S_p : w_i >= min_p }.  token = lowest i with  sum_{j <= i, j in S} w_j > u sum(S)
//
// A token is a comparison of two long sums, so a rounding anywhere in a row of 100000 terms
// could move it. The weights are therefore whole numbers of 2^-43 of the largest, each right to
// 2^-35 of itself: their sums are exact in any order, and the same for any split of a row
// over threads and blocks.
//
// A cluster of blocks takes a row, each warp a contiguous stretch of it. All three limits keep a
// prefix of the same order, so one cut, a (logit, index) pair, says what is kept. It is
// found from a histogram of the logits' distance from the largest, whose bins bracket it, and
// then by sorting the few elements of the bracket; a bracket that holds too many (equal
// logits, flat distributions) is halved until it does not.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "block_internal.h"
#include "flce_host.h"
#include "stream_host.h"
#include "stream_ops.cuh"

namespace cg = cooperative_groups;

namespace flce {
namespace {

constexpr int kThreadsS = 512, kWarpsS = kThreadsS / 32;
constexpr int kMaxCluster = 8;
constexpr int kFrac = 43;                  // fraction bits of a weight
constexpr uint64_t kOne = 1ull << kFrac;
constexpr int kTable = 1024;               // 2^(i / kTable)
constexpr int kPerOctave = 64;             // histogram bins to a factor of 2
constexpr int kBins = 46 * kPerOctave;     // weights below 2^-44 are 0
constexpr int kList = 2048;                // elements that are sorted
constexpr uint64_t kAll = ~0ull;

struct Table {
  uint64_t v[kTable];
};
constexpr Table make_table() {
  Table t{};
  for (int i = 0; i < kTable; ++i) {
    const double x = 0.693147180559945309417 * i / kTable;
    double term = 1.0, sum = 1.0;
    for (int k = 1; k < 24; ++k) {
      term *= x / k;
      sum += term;
    }
    t.v[i] = static_cast<uint64_t>(sum * static_cast<double>(kOne) + 0.5);
  }
  return t;
}
__device__ const Table kExp2 = make_table();

struct SampleArgs {
  const void* logits;
  const float *u, *temperatures, *top_ps, *min_ps;
  const int32_t* top_ks;
  int64_t* tokens;
  int64_t ld;
  int B, V, cluster, stretch;  // stretch: elements of a warp, a multiple of 8
  float temperature, top_p, min_p;
  int top_k;
};

struct Shared {
  uint64_t table[kTable];
  uint32_t hist[kBins];
  uint64_t list[kList];
  uint64_t red[kWarpsS][2];
  uint64_t peers[2][kMaxCluster][2];
  uint64_t warp_sum[kWarpsS];
  uint32_t scan[kWarpsS];
  float scan_mass[kWarpsS], within[2];
  uint32_t listed;
  uint64_t cut;
  int bins[2];
  float c_hi, c_lo;
  double p;
};

// A row's order as a number: larger for larger z, and for the lower index among equals.
// A NaN is above everything.
__device__ __forceinline__ uint32_t order_of(float z) {
  if (z != z) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(z + 0.f);  // -0 and 0 are equal
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);
}
__device__ __forceinline__ uint64_t place_of(float z, int index) {
  return static_cast<uint64_t>(order_of(z)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int mask) {
  return __shfl_xor_sync(0xffffffffu, v, mask);
}

template <int TYPE>
struct Row {
  const SampleArgs& a;
  Shared& s;
  const uint8_t* z;   // the row
  int shift;          // its first element's distance from a 16-byte boundary, in elements
  int rank, first, last;  // this warp's positions, index + shift
  int lane, warp, turn;
  float top, c_hi, c_lo, bin_scale;

  __device__ void sync() const {
    if (a.cluster == 1)
      __syncthreads();
    else
      cg::this_cluster().sync();
  }

  // f(index of the first, 8 values) over this warp's stretch; -inf where there is no element.
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int at = first + lane * 8; at < last; at += 256) {
      const int i = at - shift;
      float v[8];
      if (i >= 0 && i + 8 <= a.V) {
        unpack8<TYPE>(load8<TYPE, true>(z, i, a.V), v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = i + e >= 0 && i + e < a.V ? load_value<TYPE>(z, i + e) : -INFINITY;
      }
      f(i, v);
    }
  }

  // The sums (or the largest) of two numbers over the cluster, in every thread.
  template <bool MAX>
  __device__ __forceinline__ void reduce(uint64_t& x, uint64_t& y) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t p = shfl64(x, o), q = shfl64(y, o);
      x = MAX ? max(x, p) : x + p;
      y = MAX ? max(y, q) : y + q;
    }
    if (lane == 0) {
      s.red[warp][0] = x;
      s.red[warp][1] = y;
    }
    __syncthreads();
    if (warp == 0) {
      x = lane < kWarpsS ? s.red[lane][0] : 0;
      y = lane < kWarpsS ? s.red[lane][1] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t p = shfl64(x, o), q = shfl64(y, o);
        x = MAX ? max(x, p) : x + p;
        y = MAX ? max(y, q) : y + q;
      }
      if (lane < a.cluster) {
        uint64_t* to = a.cluster == 1 ? s.peers[turn][0]
                                      : cg::this_cluster().map_shared_rank(s.peers[turn][rank], lane);
        to[0] = x;
        to[1] = y;
      }
    }
    sync();
    x = y = 0;
    for (int i = 0; i < a.cluster; ++i) {
      x = MAX ? max(x, s.peers[turn][i][0]) : x + s.peers[turn][i][0];
      y = MAX ? max(y, s.peers[turn][i][1]) : y + s.peers[turn][i][1];
    }
    turn ^= 1;
  }

  // exp((z - top) / T) in units of 2^-43. (z - top) log2(e) / T as a pair of floats is right
  // to 2^-42; the table takes its first 10 fraction bits, a polynomial the rest.
  __device__ __forceinline__ uint64_t weight(float v) const {
    if (v == top) return kOne;
    const float d = v - top;
    const float hi = __fmul_rn(d, c_hi);
    if (!(hi > -45.f)) return 0;
    const float back = d - v;
    const float err = (v - (d - back)) + (-top - back);
    const float lo = __fmaf_rn(d, c_hi, -hi) + __fmaf_rn(d, c_lo, __fmul_rn(err, c_hi));
    const float magic = 12288.f;  // its last bit is 2^-10
    const float near = hi + magic;
    const int k = __float_as_int(near) - __float_as_int(magic);
    const float r = (hi - (near - magic)) + lo;
    const float q = r * fmaf(r, fmaf(r, 0.05550411f, 0.24022651f), 0.69314718f);
    const uint64_t base = s.table[k & (kTable - 1)];
    const float part = static_cast<float>(static_cast<uint32_t>(base >> 20)) * q * 131072.f;
    const int64_t w = static_cast<int64_t>(base) + (static_cast<int64_t>(__float2int_rn(part)) << 3);
    const int down = -(k >> 10);
    return (static_cast<uint64_t>(w) + ((1ull << down) >> 1)) >> down;
  }
  // The histogram bin, kBins where the weight is 0: falls with the logit.
  __device__ __forceinline__ int bin(float v) const {
    const float d = v == top ? 0.f : (top - v) * bin_scale;
    return d < static_cast<float>(kBins) ? static_cast<int>(d) : kBins;
  }

  __device__ void histogram() {
    for (int i = threadIdx.x; i < kBins; i += kThreadsS) s.hist[i] = 0;
    __syncthreads();
    each([&](int, const float* v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int b = bin(v[e]);
        if (b < kBins) atomicAdd(&s.hist[b], 1u);
      }
    });
    sync();
    if (a.cluster > 1) {
      // Block r adds its share of the bins over all blocks, into the first block's copy.
      auto cl = cg::this_cluster();
      for (int i = rank * kThreadsS + threadIdx.x; i < kBins; i += a.cluster * kThreadsS) {
        uint32_t n = 0;
        for (int r = 0; r < a.cluster; ++r) n += cl.map_shared_rank(s.hist, r)[i];
        cl.map_shared_rank(s.hist, 0)[i] = n;
      }
      sync();
    }
  }

  __device__ static float bin_weight(int i) {
    return exp2f(-(static_cast<float>(i) + 0.5f) / kPerOctave);
  }

  // In the first block: the bins [s.bins[0], s.bins[1]] in which the cut must lie: the one that
  // holds the k-th element, or, with p < 1, those where the weight before an element can
  // reach p of the sum over the first k. A bin's weight is known from its count to half a
  // bin's width, 0.55 %; two such sums are compared, and `slack` is more than both errors.
  __device__ void bracket(uint64_t k, float p) {
    constexpr float slack = 0.016f;
    if (rank == 0) {
      constexpr int kEach = (kBins + kThreadsS - 1) / kThreadsS;
      const int b = min(static_cast<int>(threadIdx.x) * kEach, kBins), b_end = min(b + kEach, kBins);
      uint32_t n = 0;
      float m = 0.f;
      for (int i = b; i < b_end; ++i) {
        n += s.hist[i];
        m += static_cast<float>(s.hist[i]) * bin_weight(i);
      }
      uint32_t n_scan = n;
      float m_scan = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, n_scan, o);
        const float y = __shfl_up_sync(0xffffffffu, m_scan, o);
        if (lane >= o) {
          n_scan += x;
          m_scan += y;
        }
      }
      if (lane == 31) {
        s.scan[warp] = n_scan;
        s.scan_mass[warp] = m_scan;
      }
      if (threadIdx.x == 0) s.bins[0] = s.bins[1] = kBins - 1;
      __syncthreads();
      uint32_t n_before = n_scan - n;
      float m_before = m_scan - m, total = 0.f;
      for (int w = 0; w < kWarpsS; ++w) {
        if (w < warp) {
          n_before += s.scan[w];
          m_before += s.scan_mass[w];
        }
        total += s.scan_mass[w];
      }
      // The sum over the first k: between what lies before the k-th element's bin and its end.
      if (threadIdx.x == 0) s.within[0] = s.within[1] = total;
      __syncthreads();
      if (n_before < k && k <= n_before + n) {
        uint32_t c = n_before;
        float x = m_before;
        int i = b;
        while (c + s.hist[i] < k) {
          x += static_cast<float>(s.hist[i]) * bin_weight(i);
          c += s.hist[i++];
        }
        if (p >= 1.f) s.bins[0] = s.bins[1] = i;
        s.within[0] = x;
        s.within[1] = x + static_cast<float>(s.hist[i]) * bin_weight(i);
      }
      __syncthreads();
      if (p < 1.f) {
        const float low = p * s.within[0] * (1.f - slack), high = p * s.within[1] * (1.f + slack);
        float x = m_before;
        for (int i = b; i < b_end; ++i) {
          x += static_cast<float>(s.hist[i]) * bin_weight(i);
          if (x >= low) atomicMin(&s.bins[0], i);
          if (x >= high) atomicMin(&s.bins[1], i);
        }
      }
    }
    if (a.cluster > 1 && rank == 0) {
      __syncthreads();
      if (threadIdx.x > 0 && threadIdx.x < a.cluster) {
        int* to = cg::this_cluster().map_shared_rank(s.bins, threadIdx.x);
        to[0] = s.bins[0];
        to[1] = s.bins[1];
      }
    }
    sync();
  }

  // The cut: the lowest place that is kept, where at most k elements and those before which
  // less than `mass` lies are. Elements below `floor` do not count. k, mass: kAll for none.
  __device__ uint64_t find_cut(uint64_t k, uint64_t mass, uint64_t floor, int b0, int b1) {
    // What lies above the bracket, and what is in it.
    const bool weigh = mass != kAll;
    uint64_t above_n = 0, above_m = 0, in_lo = kAll, in_hi = 0, in_n = 0, none = 0;
    each([&](int i, const float* v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int b = bin(v[e]);
        if (b > b1) continue;
        const uint64_t at = place_of(v[e], i + e);
        if (at < floor) continue;
        if (b < b0) {
          above_n += 1;
          if (weigh) above_m += weight(v[e]);
        } else {
          in_n += 1;
          in_lo = min(in_lo, at);
          in_hi = max(in_hi, at);
        }
      }
    });
    reduce<false>(above_n, above_m);
    reduce<false>(in_n, none);
    in_lo = ~in_lo;
    reduce<true>(in_lo, in_hi);
    in_lo = ~in_lo;
    if (in_n == 0) return floor;
    uint64_t lo = in_lo, hi = in_hi + 1;  // the bracket [lo, hi)
    while (in_n > kList) {
      const uint64_t mid = lo + (hi - lo) / 2;
      uint64_t n = 0, m = 0;
      each([&](int i, const float* v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint64_t at = place_of(v[e], i + e);
          if (at >= mid && at < hi) {
            n += 1;
            if (weigh) m += weight(v[e]);
          }
        }
      });
      reduce<false>(n, m);
      if (above_n + n < k && above_m + m < mass) {
        above_n += n;
        above_m += m;
        hi = mid;
        in_n -= n;
      } else {
        lo = mid;
        in_n = n;
      }
    }
    if (rank == 0 && threadIdx.x == 0) s.listed = 0;
    sync();
    {
      uint32_t* listed = a.cluster == 1 ? &s.listed : cg::this_cluster().map_shared_rank(&s.listed, 0);
      uint64_t* list = a.cluster == 1 ? s.list : cg::this_cluster().map_shared_rank(s.list, 0);
      each([&](int i, const float* v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint64_t at = place_of(v[e], i + e);
          if (at >= lo && at < hi) {
            const uint32_t n = atomicAdd(listed, 1u);
            if (n < kList) list[n] = at;
          }
        }
      });
    }
    sync();
    if (rank == 0) {
      const int n = min(static_cast<int>(s.listed), kList);
      sort_list(n);
      cut_list(n, k, mass, above_n, above_m, hi);
      if (threadIdx.x < a.cluster && a.cluster > 1)
        *cg::this_cluster().map_shared_rank(&s.cut, threadIdx.x) = s.cut;
    }
    sync();
    return s.cut;
  }

  // The list by falling place, in this block.
  __device__ void sort_list(int n) {
    int size = 1;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += kThreadsS) s.list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1) {
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int t = threadIdx.x; t < size / 2; t += kThreadsS) {
          const int x = 2 * t - (t & (j - 1)), y = x + j;
          const uint64_t p = s.list[x], q = s.list[y];
          if ((p < q) == ((x & k) == 0)) {
            s.list[x] = q;
            s.list[y] = p;
          }
        }
        __syncthreads();
      }
    }
  }

  // s.cut from the sorted list: the last place that is kept, or `hi` where none is.
  __device__ void cut_list(int n, uint64_t k, uint64_t mass, uint64_t above_n, uint64_t above_m,
                           uint64_t hi) {
    constexpr int kEach = kList / kThreadsS;
    uint64_t w[kEach], sum = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x * kEach + e;
      w[e] = i < n && mass != kAll ? weight(value_of(static_cast<uint32_t>(s.list[i] >> 32))) : 0;
      sum += w[e];
    }
    uint64_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += x;
    }
    if (lane == 31) s.warp_sum[warp] = scan;
    if (threadIdx.x == 0) s.cut = hi;
    __syncthreads();
    uint64_t before = above_m + scan - sum;
    for (int i = 0; i < warp; ++i) before += s.warp_sum[i];
    int kept = -1;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x * kEach + e;
      if (i < n && above_n + i < k && before < mass) kept = i;
      before += w[e];
    }
    // What is kept is a prefix: the last one's thread sees that the next is not.
    if (kept >= 0) {
      const uint64_t at = s.list[kept];
      atomicMin(reinterpret_cast<unsigned long long*>(&s.cut), static_cast<unsigned long long>(at));
    }
    __syncthreads();
  }

  // Draws from the elements at or above `cut` whose weight is at least `least`.
  __device__ void draw(uint64_t cut, uint64_t least, float u, int64_t* token) {
    uint64_t sum = 0;
    each([&](int i, const float* v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (v[e] == -INFINITY || place_of(v[e], i + e) < cut) continue;
        const uint64_t w = weight(v[e]);
        if (w >= least) sum += w;
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += shfl64(sum, o);
    if (lane == 0) s.warp_sum[warp] = sum;
    __syncthreads();
    uint64_t block = 0, before = 0;
    for (int i = 0; i < kWarpsS; ++i) {
      if (i < warp) before += s.warp_sum[i];
      block += s.warp_sum[i];
    }
    if (threadIdx.x < a.cluster) {
      uint64_t* to = a.cluster == 1
                         ? s.peers[turn][0]
                         : cg::this_cluster().map_shared_rank(s.peers[turn][rank], threadIdx.x);
      to[0] = block;
    }
    sync();
    uint64_t all = 0;
    for (int i = 0; i < a.cluster; ++i) {
      if (i < rank) before += s.peers[turn][i][0];
      all += s.peers[turn][i][0];
    }
    turn ^= 1;
    // The sums are whole: one is above u all where it is above the whole part of that.
    uint64_t target = 0;
    if (lane == 0 && u > 0.f) {
      const double t = static_cast<double>(u) * static_cast<double>(all);
      target = t < static_cast<double>(all) ? static_cast<uint64_t>(t) : all - 1;
      if (target >= all) target = all - 1;
    }
    target = __shfl_sync(0xffffffffu, target, 0);
    if (target < before || target >= before + sum) return;
    // This warp's stretch holds it.
    for (int at = first; at < last; at += 256) {
      const int i = at + lane * 8 - shift;
      uint64_t w[8], mine = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = i + e;
        w[e] = 0;
        if (j >= 0 && j < a.V && at + lane * 8 < last) {
          const float v = load_value<TYPE>(z, j);
          if (v != -INFINITY && place_of(v, j) >= cut) {
            const uint64_t x = weight(v);
            if (x >= least) w[e] = x;
          }
        }
        mine += w[e];
      }
      uint64_t scan = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += x;
      }
      uint64_t c = before + scan - mine;
      if (target >= c && target < c + mine) {
        int e = 0;
#pragma unroll
        for (int k = 0; k < 7; ++k) {
          if (e == k && target >= c + w[k]) {
            c += w[k];
            e = k + 1;
          }
        }
        *token = i + e;
      }
      before += __shfl_sync(0xffffffffu, scan, 31);
      if (target < before) return;
    }
  }

  __device__ void run(int row) {
    const float temperature = a.temperatures ? a.temperatures[row] : a.temperature;
    int64_t top_k = a.top_ks ? a.top_ks[row] : a.top_k;
    float p = a.top_ps ? a.top_ps[row] : a.top_p;
    const float min_p = a.min_ps ? a.min_ps[row] : a.min_p;
    if (threadIdx.x == 0) {
      const double c = 1.4426950408889634074 / fmax(static_cast<double>(temperature), 1e-30);
      s.c_hi = static_cast<float>(c);
      s.c_lo = static_cast<float>(c - static_cast<double>(s.c_hi));
    }
    for (int i = threadIdx.x; i < kTable; i += kThreadsS) s.table[i] = kExp2.v[i];
    uint64_t best = 0, none = 0;
    each([&](int i, const float* v) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (v[e] != -INFINITY) best = max(best, place_of(v[e], i + e));
    });
    reduce<true>(best, none);
    c_hi = s.c_hi;
    c_lo = s.c_lo;
    bin_scale = c_hi * kPerOctave;
    const uint32_t order = static_cast<uint32_t>(best >> 32);
    int64_t* token = a.tokens + row;
    if (best == 0 || order == 0xFFFFFFFFu) {  // nothing to choose from, or a NaN
      if (rank == 0 && threadIdx.x == 0) *token = -1;
      return;
    }
    top = value_of(order);
    if (top_k <= 0 || top_k > a.V) top_k = a.V;
    const bool greedy = !(temperature > 0.f) || top_k == 1 || !(p > 0.f);
    if (greedy) {
      if (rank == 0 && threadIdx.x == 0)
        *token = static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
      return;
    }
    const bool by_k = top_k < a.V, by_p = p < 1.f;
    uint64_t cut = 0;
    if (by_k || by_p) histogram();
    if (by_k) {
      bracket(top_k, 1.f);
      cut = find_cut(top_k, kAll, 0, s.bins[0], s.bins[1]);
    }
    if (by_p) {
      uint64_t all = 0, zero = 0;
      each([&](int i, const float* v) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (v[e] != -INFINITY && place_of(v[e], i + e) >= cut) all += weight(v[e]);
      });
      reduce<false>(all, zero);
      if (threadIdx.x == 0) s.p = ceil(static_cast<double>(p) * static_cast<double>(all));
      bracket(top_k, p);
      const uint64_t mass = static_cast<uint64_t>(s.p);
      cut = find_cut(kAll, mass < 1 ? 1 : mass, cut, s.bins[0], s.bins[1]);
    }
    // min_p above 1 keeps the largest.
    const float share = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;
    // share 2^43 is exact in 32 bits' mantissa; the least whole number at or above it.
    const uint64_t least = static_cast<uint64_t>(__float2ull_ru(share * static_cast<float>(kOne)));
    draw(cut, least, a.u[row], token);
  }
};

template <int TYPE>
__global__ void __launch_bounds__(kThreadsS) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  griddep_launch();
  griddep_wait();
  const int row = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
  const uint8_t* z = static_cast<const uint8_t*>(a.logits) + row * a.ld * type_size(TYPE);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(z) % 16) / type_size(TYPE);
  const int64_t begin = static_cast<int64_t>(rank * kWarpsS + warp) * a.stretch;
  const int64_t end = min(begin + a.stretch, static_cast<int64_t>(a.V) + shift);
  Row<TYPE> r{a, *reinterpret_cast<Shared*>(smem), z, shift, rank,
              static_cast<int>(min(begin, end)), static_cast<int>(end), lane, warp, 0};
  r.run(row);
  // No block leaves while another may still write into its memory.
  r.sync();
}

cudaError_t launch_sample(const SampleArgs& a, int type, cudaStream_t st) {
  auto kernel = type == kFp32 ? sample_kernel<kFp32> : type == kBf16 ? sample_kernel<kBf16> : sample_kernel<kFp16>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(sizeof(Shared)));
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(a.B) * a.cluster), kThreadsS, sizeof(Shared),
                          a.cluster, st, a);
}

}  // namespace
}  // namespace flce

extern "C" flce_status_t flce_sample(const flce_sample_params_t* p, const void* logits, const float* u,
                                     const float* temperatures, const int32_t* top_ks,
                                     const float* top_ps, const float* min_ps, int64_t* tokens,
                                     void* stream) {
  using namespace flce;
  NvtxRange nvtx_range("flce_sample");
  if (!p || p->B < 0 || p->V <= 0 || !float_type_ok(p->dtype) || !pitch_ok(p->ld, p->V))
    return FLCE_ERR_INVALID_ARG;
  if (p->V > FLCE_SAMPLE_MAX_V || p->B > (1LL << 28)) return FLCE_ERR_UNSUPPORTED;
  if ((!temperatures && !(p->temperature >= 0.f)) || (!top_ks && p->top_k < 0) ||
      (!top_ps && (!(p->top_p >= 0.f) || !(p->top_p <= 1.f))) ||
      (!min_ps && (!(p->min_p >= 0.f) || !(p->min_p <= 1.f))))
    return FLCE_ERR_INVALID_ARG;
  if (p->B == 0) return FLCE_OK;
  if (!logits || !u || !tokens) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(logits, type_size(p->dtype)) || !aligned_to(u, 4) || !aligned_to(temperatures, 4) ||
      !aligned_to(top_ks, 4) || !aligned_to(top_ps, 4) || !aligned_to(min_ps, 4) || !aligned_to(tokens, 8))
    return FLCE_ERR_ALIGNMENT;
  int sms = 0;
  const flce_status_t ds = device_info(&sms);
  if (ds != FLCE_OK) return ds;
  SampleArgs a;
  a.logits = logits;
  a.u = u;
  a.temperatures = temperatures;
  a.top_ks = top_ks;
  a.top_ps = top_ps;
  a.min_ps = min_ps;
  a.tokens = tokens;
  a.ld = pitch_of(p->ld, p->V);
  a.B = static_cast<int>(p->B);
  a.V = static_cast<int>(p->V);
  a.temperature = p->temperature;
  a.top_k = p->top_k;
  a.top_p = p->top_p;
  a.min_p = p->min_p;
  // Blocks for a row: as many as fill the GPU, each with 4096 elements at least.
  int cluster = 1;
  while (cluster < kMaxCluster && 2 * cluster * p->B <= 2 * sms && p->V >= 2 * cluster * 4096) cluster *= 2;
  a.cluster = cluster;
  const int64_t warps = static_cast<int64_t>(cluster) * kWarpsS;
  a.stretch = static_cast<int>(((p->V + 8 + warps - 1) / warps + 7) / 8 * 8);
  const cudaError_t e = launch_sample(a, p->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
