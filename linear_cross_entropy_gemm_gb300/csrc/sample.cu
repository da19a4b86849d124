// Sampling from logits with temperature, top-k, top-p and min-p, from given random numbers.
//
//   w_i = exp((z_i - max z) / T);  order: by z falling, then by index
//   S_k: the first k.  S_p: those of S_k before which less than p sum(S_k) lies.
//   S = { i in S_p : w_i >= min_p }.  token = lowest i with  sum_{j <= i, j in S} w_j > u sum(S)
//
// A token is a comparison of two long sums, so a rounding anywhere in a row of 100000 terms
// could move it. The weights are therefore whole numbers of 2^-43 of the power of two at or above the
// largest (of the largest itself where z / T is far from 0), each right to 2^-32 of itself: their
// sums are exact in any order, and the same for any split of a row over threads and blocks.
//
// A cluster of blocks takes a row, each warp a contiguous stretch of it. All three limits keep a
// prefix of the same order, so one cut, a (logit, index) pair, says what is kept.
//   One pass finds the largest, and from the threads' largest a logit that enough elements reach.
//   The list: a second pass lists those that reach it (and adds up the others' weight, by the hardware's
//   2^x, where p alone limits); cut and draw are among the listed. Where the error of that sum could
//   move the cut it is made again in whole numbers.
//   The row: where k is large or the kept ones are many, a histogram of the distances from the largest
//   brackets the cut, one pass of exact weights sums what lies above the bracket and lists what lies in
//   it, and a bracket with too many (equal logits) is halved until it has not. Sums of parts of the
//   warps' stretches say where the draw falls.
//
// The bytes are the logits once (512 x 128256 bf16: 131 MB, 19.4 us), but the second pass comes from L2
// at best, and an exact weight takes about 35 instructions. Measured at that size: the largest
// alone 48 us, top-k 50 59, the whole distribution 106, p = 0.95 83 where some tens of words
// matter and 237 where 106000 do. One row of 128256: 6, 13, 12, 18 and 39 us: the clusters'
// exchanges and the first block's work on the list, each a few us of waiting.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "block_internal.h"
#include "flce_host.h"
#include "stream_host.h"
#include "stream_ops.cuh"

namespace cg = cooperative_groups;

namespace flce {
namespace {

constexpr int kThreadsS = 256, kWarpsS = kThreadsS / 32;
constexpr int kPerSm = 4;                  // blocks of an SM: 64 registers for a thread
constexpr int kMaxCluster = 8;
constexpr int kFrac = 43;                  // fraction bits of a weight
constexpr uint64_t kOne = 1ull << kFrac;
constexpr int kTable = 1024;               // 2^(i / kTable)
constexpr int kTableFrac = 55;
constexpr int kAhead = 4;                  // loads of a thread in flight,
constexpr int kStep = kAhead * 256;        //   elements of a warp's
constexpr int kParts = 32;                 // sums of a warp's stretch, at most
constexpr int kList = 1536;                // elements that are listed
constexpr int kNotes = 2 * kList;          // groups that are looked at again
constexpr int kMostK = 1000;               // top-k up to this goes by the list
constexpr int kWanted = 512;               // the list's least length where only p says how much is needed
constexpr int kNear = 8, kNearBins = 512;  // bins to a factor of 2 and bins: of the loads' largest,
constexpr int kPerOctave = 64, kBins = 46 * kPerOctave;  //   of all elements; weights below 2^-44 are 0
constexpr float kSureSlack = 0.016f, kLikelySlack = 0.0004f;
constexpr int kItemBits = 9;               // bins of a list
constexpr int kFew = 64;                   // items that are compared with each other
constexpr int kPairs = kThreadsS / 2;      // lists up to this length are compared in pairs
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
    t.v[i] = static_cast<uint64_t>(sum * static_cast<double>(1ull << kTableFrac) + 0.5);
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
  int B, V, cluster, stretch, part;  // elements of a warp, a multiple of 8; of a part of them, of kStep
  float temperature, top_p, min_p;
  int top_k;
};

// Two arrays of a block share memory where one of them is done with when the other is made.
struct Shared {
  union {
    uint32_t hist[kBins];
    uint32_t near_hist[kNearBins];
    struct {
      uint64_t item_mass[1 << kItemBits];
      uint32_t item_hist[1 << kItemBits];
    };
    uint64_t bucket[kThreadsS];
  };
  uint64_t list[kList];      // places; in the first block those of all blocks, kList / cluster for each
  union {
    uint64_t table[kTable];  // without a list
    uint64_t item[kList];    // the list, one after another,
  };
  uint64_t heft[kList];      //   and its weights
  uint16_t few[kList];       // items of one bin or bucket
  uint64_t red[kWarpsS][2];
  uint64_t peers[2][kMaxCluster][2];
  uint64_t warp_sum[kWarpsS], warp_kept[kWarpsS];
  uint64_t kept[kWarpsS][kParts];  // weights that are kept, by parts of the warps' stretches
  uint64_t cut, cut_mass;    // the last place that is kept, the weight up to and including it
  uint64_t x_before, x_count;
  uint64_t rests[kMaxCluster];
  uint32_t owns[kMaxCluster];
  float thresholds[kMaxCluster][2];
  uint32_t scan[kWarpsS];
  float scan_mass[kWarpsS], within[2], mine[2];
  uint32_t owned, noted, few_n, above;
  int x_bin, verdict;
  int bins[2];
  float c_hi, c_lo;
};
enum Verdict { kDone = 0, kInexact = 1, kTooShort = 2 };

// A row's order as a number: larger for larger z, and for the lower index among equals.
__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);  // -0 and 0 are equal
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);
}
__device__ __forceinline__ uint64_t place_of(float z, int index) {
  return static_cast<uint64_t>(order_of(z)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}
__device__ __forceinline__ float place_value(uint64_t place) {
  return value_of(static_cast<uint32_t>(place >> 32));
}
__device__ __forceinline__ int place_index(uint64_t place) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(place));
}

// The last index that is at or above a place, among those of its logit.
__device__ __forceinline__ uint32_t place_last(uint64_t place) {
  return 0xFFFFFFFFu - static_cast<uint32_t>(place);
}

// To a sum of 64 bits in shared memory, in two halves: there is no such instruction for the whole.
__device__ __forceinline__ void add64(uint64_t* sum, uint64_t v) {
  uint32_t* half = reinterpret_cast<uint32_t*>(sum);
  const uint32_t low = static_cast<uint32_t>(v), old = atomicAdd(half, low);
  const uint32_t high = static_cast<uint32_t>(v >> 32) + (old + low < old ? 1 : 0);
  if (high != 0) atomicAdd(half + 1, high);
}

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int mask) {
  return __shfl_xor_sync(0xffffffffu, v, mask);
}

// x f, rounded down or up to a whole number, exactly: f in [0, 1).
template <bool UP>
__device__ __forceinline__ uint64_t times(uint64_t x, float f) {
  const uint32_t b = __float_as_uint(f);
  const int e = static_cast<int>(b >> 23);
  const uint64_t m = (b & 0x7FFFFFu) | (e > 0 ? 0x800000u : 0u);
  const int down = 150 - (e > 0 ? e : 1);  // f = m 2^-down, at least 24
  const uint64_t lo = x * m, hi = __umul64hi(x, m);
  uint64_t whole, rest;
  if (down < 64) {
    whole = hi << (64 - down) | lo >> down;
    rest = lo << (64 - down);
  } else if (down < 128) {
    whole = down == 64 ? hi : hi >> (down - 64);
    rest = lo | (down == 64 ? 0 : hi << (128 - down));
  } else {
    whole = 0;
    rest = lo | hi;
  }
  return whole + (UP && rest != 0 ? 1 : 0);
}

// The weight before which elements are kept: p `of`, and the first one always.
__device__ __forceinline__ uint64_t share_of(uint64_t of, float p) {
  const uint64_t m = times<true>(of, p);
  return m > 0 ? m : 1;
}

// The largest of eight; a NaN if there is one.
template <int TYPE>
__device__ __forceinline__ float largest(const Raw8<TYPE>& r) {
  if constexpr (TYPE == kFp32) {
    float v[8];
    unpack8<TYPE>(r, v);
    return max_nan(max_nan(max_nan(v[0], v[1]), max_nan(v[2], v[3])),
                   max_nan(max_nan(v[4], v[5]), max_nan(v[6], v[7])));
  } else {
    const uint4& w = r.w[0];
    uint32_t m;
    if constexpr (TYPE == kBf16)
      asm("{.reg .b32 a, b;\n max.NaN.bf16x2 a, %1, %2;\n max.NaN.bf16x2 b, %3, %4;\n"
          " max.NaN.bf16x2 %0, a, b;}" : "=r"(m) : "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w));
    else
      asm("{.reg .b32 a, b;\n max.NaN.f16x2 a, %1, %2;\n max.NaN.f16x2 b, %3, %4;\n"
          " max.NaN.f16x2 %0, a, b;}" : "=r"(m) : "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w));
    return max_nan(unpack_16(m & 0xFFFFu, TYPE == kFp16), unpack_16(m >> 16, TYPE == kFp16));
  }
}
template <int TYPE>
__device__ __forceinline__ Raw8<TYPE> nothing() {
  const uint32_t w = TYPE == kFp32 ? 0xFF800000u : TYPE == kBf16 ? 0xFF80FF80u : 0xFC00FC00u;
  Raw8<TYPE> r;
  for (auto& x : r.w) x = make_uint4(w, w, w, w);
  return r;
}

// exp((z - top) / T) in units of 2^-43, for z / T of any size: (z - top) log2(e) / T as a pair of
// floats is right to 2^-42, and then as in Row::weight_near.
__device__ __noinline__ uint64_t weight_far(float v, float top, float c_hi, float c_lo, const uint64_t* table) {
  if (v == top) return kOne;
  const float d = v - top;
  const float hi = __fmul_rn(d, c_hi);
  if (!(hi > -45.f)) return 0;
  const float back = d - v;
  const float err = (v - (d - back)) + (-top - back);
  const float lo = __fmaf_rn(d, c_hi, -hi) + __fmaf_rn(d, c_lo, __fmul_rn(err, c_hi));
  const float near = hi + 12288.f;
  const int k = __float_as_int(near) - 0x46400000;
  const float r = (hi - (near - 12288.f)) + lo;
  const uint64_t t = table[k & (kTable - 1)];
  const float part = __int_as_float(static_cast<int>(t >> 32) + 0x3F000000) *
                     (r * __fmaf_rn(r, 0.24022651f * 0x1p40f, 0.69314718f * 0x1p40f));
  const uint64_t w = t + static_cast<int64_t>(__float2int_rn(part)) * 32768;
  const int down = (kTableFrac - kFrac) - (k >> 10);
  return (w + (1ull << (down - 1))) >> down;
}

template <int TYPE>
struct Row {
  const SampleArgs& a;
  Shared& s;
  const uint8_t* z;   // the row
  int shift;          // its first element's distance from a 16-byte boundary, in elements
  int rank, first, last;  // this warp's positions, index + shift
  int lane, warp, turn;
  float top, c_hi, c_lo, lowest;
  int octave;         // weights are 2^(z log2(e) / T - octave)
  bool far;           // z log2(e) / T is too large for weight_near
  int index_bits;     // of the largest index,
  uint32_t place_mask;  //   all of them set

  __device__ void sync() const {
    if (a.cluster == 1)
      __syncthreads();
    else
      cg::this_cluster().sync();
  }
  template <class T>
  __device__ T* of_block(T* p, int r) const {
    return a.cluster == 1 ? p : cg::this_cluster().map_shared_rank(p, r);
  }

  // The 8 values at a position, -inf where there is no element; `group`: of this warp's stretch.
  __device__ __forceinline__ Raw8<TYPE> group(int at) const {
    return at >= last ? nothing<TYPE>() : any_group(at);
  }
  __device__ __forceinline__ Raw8<TYPE> any_group(int at) const {
    const int i = at - shift;
    if (i >= 0 && i + 8 <= a.V) return load8<TYPE, true>(z, i, a.V);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = i + e >= 0 && i + e < a.V ? load_value<TYPE>(z, i + e) : -INFINITY;
    return pack8<TYPE>(v);
  }
  // f(which of the loads, position, 8 values as they are) over this warp's stretch.
  template <class F>
  __device__ __forceinline__ void each_raw(F f) const {
    for (int base = first; base < last; base += kStep) {
      const int at = base + lane * 8;
      Raw8<TYPE> r[kAhead];
#pragma unroll
      for (int g = 0; g < kAhead; ++g) r[g] = group(at + g * 256);
#pragma unroll
      for (int g = 0; g < kAhead; ++g) f(g, at + g * 256, r[g]);
    }
  }
  // f(position, 8 values as they are), the next ones on their way: a body that is long is not
  // repeated for each of several loads, which the instruction cache would not hold.
  template <class F>
  __device__ __forceinline__ void each_group(F f) const {
    Raw8<TYPE> next = group(first + lane * 8);
#pragma unroll 1
    for (int base = first; base < last; base += 256) {
      const Raw8<TYPE> r = next;
      next = group(base + 256 + lane * 8);
      f(base + lane * 8, r);
    }
  }
  // f(index, value) for the groups that hold one of at least `least`.
  template <class F>
  __device__ __forceinline__ void each(float least, F f) const {
    each_group([&](int at, const Raw8<TYPE>& r) {
      if (!(largest<TYPE>(r) >= least)) return;
      float v[8];
      unpack8<TYPE>(r, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) f(at - shift + e, v[e]);
    });
  }
  // The same, f returning weights: they go to s.kept, by parts of this warp's stretch. after(position)
  // follows each group.
  template <class F, class G>
  __device__ __forceinline__ void each_kept(float least, F f, G after) const {
    uint64_t sum = 0;
    int part = 0, left = a.part;
    each_group([&](int at, const Raw8<TYPE>& r) {
      if (largest<TYPE>(r) >= least) {
        float v[8];
        unpack8<TYPE>(r, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += f(at - shift + e, v[e]);
        after(at);
      }
      left -= 256;
      if (left == 0 || at - lane * 8 + 256 >= last) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += shfl64(sum, o);
        if (lane == 0) s.kept[warp][part] = sum;
        sum = 0;
        ++part;
        left = a.part;
      }
    });
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
        uint64_t* to = of_block(s.peers[turn][rank], lane);
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

  // 2^(z log2(e) / T - octave) in units of 2^-43, octave being the largest's. Adding 12288 rounds
  // z log2(e) / T to 10 fraction bits, for which there is the table; what is left, at most
  // 2^-11, is right to 2^-35, and a polynomial of two terms gives the rest to 2^-37. Its roundings in
  // fp32 are of a number below 2^-11.5: four of them by 2^-24, and the table's entry cut to 24 bits
  // by 2^-23, or 2^-32.7 of the weight with everything (2^-35.9 in the mean square, 2^-33.2 the most
  // of 200000 weights at each of eight settings).
  __device__ __forceinline__ uint64_t weight_near(float v, const uint64_t* table) const {
    const float x = fmaxf(v, lowest);
    const float near = __fmaf_rn(x, c_hi, 12288.f);
    const float r = __fmaf_rn(x, c_lo, __fmaf_rn(x, c_hi, 12288.f - near));
    const int k = __float_as_int(near);
    const uint64_t t = table[k & (kTable - 1)];
    const float part = __int_as_float(static_cast<int>(t >> 32) + 0x3F000000) *  // 1 .. 2
                       (r * __fmaf_rn(r, 0.24022651f * 0x1p40f, 0.69314718f * 0x1p40f));
    const uint64_t w = t + static_cast<int64_t>(__float2int_rn(part)) * 32768;
    const int down = (kTableFrac - kFrac) + octave + (0x46400000 >> 10) - (k >> 10);
    return (w + (1ull << (down - 1))) >> down;
  }
  template <bool FAR>
  __device__ __forceinline__ uint64_t weight(float v, const uint64_t* table) const {
    return FAR ? weight_far(v, top, c_hi, c_lo, table) : weight_near(v, table);
  }
  __device__ uint64_t any_weight(float v, const uint64_t* table) const {
    return far ? weight<true>(v, table) : weight<false>(v, table);
  }

  // A bin of `per` to a factor of 2, `bins` where it is beyond the last: falls with the logit.
  __device__ __forceinline__ int bin(float v, float per, int bins) const {
    const float d = v == top ? 0.f : (top - v) * (c_hi * per);
    return d < static_cast<float>(bins) ? static_cast<int>(d) : bins;
  }
  __device__ __forceinline__ int bin(float v) const { return bin(v, kPerOctave, kBins); }
  // The least logit whose bin is below b, to the bit; a NaN, which none reaches, for b = 0. By a
  // whole warp: its lanes try 32 places between the ends.
  __device__ float above_bin(int b) const {
    if (b <= 0) return __int_as_float(0x7FC00000);
    uint32_t lo = order_of(-INFINITY), hi = order_of(top);
    while (lo < hi) {
      const uint32_t step = (hi - lo) / 32 + 1, probe = min(lo + lane * step, hi);
      const uint32_t below = __ballot_sync(0xffffffffu, bin(value_of(probe)) < b);
      if (below == 0) {
        lo = min(lo + 31 * step, hi - 1) + 1;
      } else {
        const int at = __ffs(below) - 1;
        hi = min(lo + at * step, hi);
        if (at > 0) lo = min(lo + (at - 1) * step + 1, hi);
      }
    }
    return value_of(hi);
  }

  // ---- the whole row: a histogram of all elements, merged in the first block

  __device__ void histogram() {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreadsS) s.hist[i] = 0;
    __syncthreads();
    each(-INFINITY, [&](int, float v) {
      const int b = bin(v);
      if (b < kBins) atomicAdd(&s.hist[b], 1u);
    });
    sync();
    if (a.cluster > 1) {
      // Block r adds its share of the bins over all blocks, into the first block's copy.
      for (int i = rank * kThreadsS + threadIdx.x; i < kBins; i += a.cluster * kThreadsS) {
        uint32_t n = 0;
        for (int r = 0; r < a.cluster; ++r) n += of_block(s.hist, r)[i];
        of_block(s.hist, 0)[i] = n;
      }
      sync();
    }
  }

  // The same by a call, where it is rarely needed: inlined once more it costs the callers registers.
  __device__ __noinline__ static void histogram_apart(Row r) { r.histogram(); }

  // The weight of a bin's elements, relative to the largest: of its middle, or, as 16-bit logits are
  // few in a bin or none, of the middle of those that it can hold. The bin's middle is not by way of a
  // logit: where z / T is far from 0, fp32's step is as wide as a bin, and rounding to it puts 2 % on a weight.
  __device__ float bin_weight(int i) const {
    float x = -(static_cast<float>(i) + 0.5f) / kPerOctave;
    if (TYPE != kFp32 && c_hi >= 1e-30f) {
      constexpr uint32_t kBelow = TYPE == kBf16 ? 0xFFFFu : 0x1FFFu;  // the bits that fp32 has below
      const float scale = c_hi * kPerOctave, upper = top - static_cast<float>(i) / scale;
      const uint32_t u = order_of(upper), l = order_of(upper - 1.f / scale);
      const uint32_t high = u & 0x80000000u ? u & ~kBelow : ((u + 1) & ~kBelow) - 1;
      const uint32_t low = l & 0x80000000u ? (l + kBelow) & ~kBelow : l | kBelow;
      if (low <= high) x = (0.5f * (value_of(low) + value_of(high)) - top) * c_hi;
    }
    return top < INFINITY ? exp2f(x) : 1.f;  // below +infinity no element is in a bin
  }

  // In the first block: the bins [s.bins[0], s.bins[1]] in which the cut must lie: the one that
  // holds the k-th element, or, with p < 1, those where the weight before an element can
  // reach p of the sum over the first k. A bin's weight is known from its count to half a
  // bin's width, 0.55 %; two such sums are compared, and kSureSlack is more than both errors.
  __device__ void bracket(uint64_t k, float p, float slack = kSureSlack) {
    if (rank == 0) {
      constexpr int kEach = (kBins + kThreadsS - 1) / kThreadsS;
      const int b = min(static_cast<int>(threadIdx.x) * kEach, kBins), b_end = min(b + kEach, kBins);
      uint32_t n = 0;
      float m = 0.f, in_bin[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const uint32_t c = b + j < b_end ? s.hist[b + j] : 0;
        in_bin[j] = c > 0 ? static_cast<float>(c) * bin_weight(b + j) : 0.f;
        n += c;
        m += in_bin[j];
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
      if (threadIdx.x == 0) {
        s.bins[0] = s.bins[1] = kBins - 1;
        s.above = 0;
      }
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
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const uint32_t h = b + j < b_end ? s.hist[b + j] : 0;
          if (c < k && k <= c + h) {
            if (p >= 1.f) s.bins[0] = s.bins[1] = b + j;
            s.above = c;
            s.within[0] = x;
            s.within[1] = x + in_bin[j];
          }
          c += h;
          x += in_bin[j];
        }
      }
      __syncthreads();
      if (p < 1.f) {
        const float low = p * s.within[0] * (1.f - slack), high = p * s.within[1] * (1.f + slack);
        float x = m_before;
        int at_low = kBins, at_high = kBins;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          x += in_bin[j];
          if (b + j >= b_end) continue;
          if (x >= low) at_low = min(at_low, b + j);
          if (x >= high) at_high = min(at_high, b + j);
        }
        if (at_low < kBins) atomicMin(&s.bins[0], at_low);
        if (at_high < kBins) atomicMin(&s.bins[1], at_high);
      }
    }
    share_bins();
  }

  // The same once the weight above s.bins[0] is known: `needed` more reaches the cut, in units of
  // `heaviest`, the largest's weight.
  __device__ void narrow(uint64_t needed, uint64_t heaviest) {
    if (rank == 0) {
      constexpr int kEach = (kBins + kThreadsS - 1) / kThreadsS;
      const int b0 = s.bins[0], b1 = s.bins[1];
      const int b = max(static_cast<int>(threadIdx.x) * kEach, b0);
      const int b_end = min(static_cast<int>(threadIdx.x + 1) * kEach, b1 + 1);
      float m = 0.f;
      for (int i = b; i < b_end; ++i) m += static_cast<float>(s.hist[i]) * bin_weight(i);
      float m_scan = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, m_scan, o);
        if (lane >= o) m_scan += y;
      }
      if (lane == 31) s.scan_mass[warp] = m_scan;
      __syncthreads();  // the bins have been read
      if (threadIdx.x == 0) s.bins[0] = s.bins[1] = b1;
      float x = m_scan - m;
      for (int w = 0; w < warp; ++w) x += s.scan_mass[w];
      __syncthreads();
      const float to = static_cast<float>(needed) / static_cast<float>(heaviest);
      for (int i = b; i < b_end; ++i) {
        x += static_cast<float>(s.hist[i]) * bin_weight(i);
        if (x >= to * 0.993f) atomicMin(&s.bins[0], i);
        if (x >= to * 1.007f) atomicMin(&s.bins[1], i);
      }
    }
    share_bins();
  }

  // s.bins and s.above of the first block to all.
  __device__ void share_bins() {
    if (a.cluster > 1 && rank == 0) {
      __syncthreads();
      if (threadIdx.x > 0 && threadIdx.x < a.cluster) {
        int* to = of_block(s.bins, threadIdx.x);
        to[0] = s.bins[0];
        to[1] = s.bins[1];
        *of_block(&s.above, threadIdx.x) = s.above;
      }
    }
    sync();
  }

  // Groups that are looked at again once a pass is over, by as many threads as there are: in the pass a
  // warp would go through the code for each value of a few of its lanes.
  __device__ void clear_notes() {
    if (threadIdx.x == 0) s.owned = s.noted = 0;
    __syncthreads();
  }
  __device__ __forceinline__ void note(uint32_t* notes, int at) {
    const uint32_t n = atomicAdd(&s.noted, 1u);
    if (n < kNotes) notes[n] = at;
  }
  // f(index, value) of the groups noted; s.owned is more than kList where they were too many.
  template <class F>
  __device__ __forceinline__ void look_again(const uint32_t* notes, F f) {
    __syncthreads();
    const uint32_t n = s.noted;
    if (n > kNotes && threadIdx.x == 0) s.owned = kList + 1;
    const uint32_t end = n <= kNotes ? n : 0;
    if (threadIdx.x >= end) return;
    int next_at = notes[threadIdx.x];
    Raw8<TYPE> next = any_group(next_at);
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < end; i += kThreadsS) {
      const int at = next_at;
      float v[8];
      unpack8<TYPE>(next, v);
      if (i + kThreadsS < end) {
        next_at = notes[i + kThreadsS];
        next = any_group(next_at);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) f(at - shift + e, v[e]);
    }
  }

  // Notes a place, in this block's s.heft.
  __device__ __forceinline__ void own(uint64_t place) {
    const uint32_t n = atomicAdd(&s.owned, 1u);
    if (n < kList) s.heft[n] = place;
  }
  // The blocks' places into the first one's list. Their number, the same in every thread; above
  // kList nothing is listed. sum: over the cluster.
  __device__ uint64_t gather(uint64_t& sum) {
    __syncthreads();
    const uint32_t mine = s.owned;
    uint64_t n = threadIdx.x == 0 ? mine : 0;
    const int at = turn;
    reduce<false>(sum, n);
    if (n > kList) return n;
    uint32_t before = 0;
    for (int r = 0; r < rank; ++r) before += static_cast<uint32_t>(s.peers[at][r][1]);
    uint64_t* list = of_block(s.list, 0);
    for (uint32_t i = threadIdx.x; i < mine; i += kThreadsS) list[before + i] = s.heft[i];
    sync();
    return n;
  }

  // The cut within places [lo, hi), which hold it: the last place before which less than k and less
  // than `mass` lie, above_n and above_m of them at or above hi. n: how many there are; listed: whether
  // they are in the list. moved: whether more elements than those above hi and of the list are kept.
  template <bool FAR>
  __device__ uint64_t cut_between(uint64_t lo, uint64_t hi, uint64_t n, bool listed, uint64_t k, uint64_t mass,
                                  uint64_t above_n, uint64_t above_m, bool& moved) {
    const bool weigh = mass != kAll;
    uint64_t none = 0;
    while (!listed) {
      while (n > kList && hi - lo > 1) {
        const uint64_t mid = lo + (hi - lo) / 2;
        uint64_t c = 0, m = 0;
        each(place_value(mid), [&](int i, float v) {
          const uint64_t at = place_of(v, i);
          if (at >= mid && at < hi) {
            c += 1;
            if (weigh) m += weight<FAR>(v, s.table);
          }
        });
        reduce<false>(c, m);
        if (above_n + c < k && above_m + m < mass) {
          above_n += c;
          above_m += m;
          moved |= c > 0;
          hi = mid;
          n -= c;
        } else {
          lo = mid;
          n = c;
        }
      }
      if (threadIdx.x == 0) s.owned = 0;
      __syncthreads();
      each(place_value(lo), [&](int i, float v) {
        const uint64_t at = place_of(v, i);
        if (at >= lo && at < hi) own(at);
      });
      n = gather(none);
      listed = n <= kList;
    }
    if (rank == 0) {
      const int listed_n = static_cast<int>(n);
      if (weigh) {
        for (int i = threadIdx.x; i < listed_n; i += kThreadsS)
          s.heft[i] = weight<FAR>(place_value(s.list[i]), s.table);
        __syncthreads();
      }
      cut_items(s.list, listed_n, lo, hi, k, mass, above_n, above_m);
      if (weigh) {
        // The kept ones' weights, to their parts of s.kept.
        for (int i = threadIdx.x; i < listed_n; i += kThreadsS) {
          if (s.list[i] < s.cut) continue;
          const int at = place_index(s.list[i]) + shift, w_at = at / a.stretch;
          uint64_t* to = &s.kept[w_at % kWarpsS][at % a.stretch / a.part];
          atomicAdd(reinterpret_cast<unsigned long long*>(of_block(to, w_at / kWarpsS)),
                    static_cast<unsigned long long>(s.heft[i]));
        }
      }
      if (threadIdx.x < a.cluster && a.cluster > 1) {
        *of_block(&s.cut, threadIdx.x) = s.cut;
        *of_block(&s.cut_mass, threadIdx.x) = s.cut_mass;
      }
    }
    sync();
    return s.cut;
  }

  // The place of the k-th element, from the histogram.
  __device__ uint64_t cut_by_count(uint64_t k) {
    bracket(k, 1.f);
    const float from = above_bin(s.bins[0] + 1), to = above_bin(s.bins[0]);
    const uint64_t lo = static_cast<uint64_t>(order_of(from)) << 32;
    const uint64_t hi = s.bins[0] == 0 ? kAll : static_cast<uint64_t>(order_of(to)) << 32;
    if (threadIdx.x == 0) s.owned = 0;
    __syncthreads();
    each(from, [&](int i, float v) {
      if (v >= from && !(v >= to)) own(place_of(v, i));
    });
    uint64_t none = 0;
    const uint64_t n = gather(none);
    bool moved = false;
    return cut_between<false>(lo, hi, n, n <= kList, k, kAll, s.above, 0, moved);
  }

  // The last place of those at or above `floor`, the k-th one's, before which less than p of their
  // weight lies. s.kept is what is at or above it, unless `moved`.
  template <bool FAR, bool FLOOR>
  __device__ uint64_t cut_by_mass(uint64_t k, float p, uint64_t floor, uint64_t heaviest, bool& moved) {
    const float least = FLOOR ? place_value(floor) : -INFINITY;
    const uint32_t least_index = place_last(floor);
    // The bins' middles are nearer to the truth than they have to be: first a bracket that is likely to
    // hold the cut, which the exact sums confirm or refute.
    for (float slack = kLikelySlack;; slack = kSureSlack) {
      bracket(k, p, slack);
      const float above = above_bin(s.bins[0]), lower = fmaxf(above_bin(s.bins[1] + 1), least);
      clear_kept();
      clear_notes();
      uint64_t all = 0, none = 0;
      uint32_t* notes = reinterpret_cast<uint32_t*>(s.list);
      bool hit = false;
      each_kept(
          least,
          [&](int i, float v) {
            uint64_t w = weight<FAR>(v, s.table);
            if (FLOOR) w = v > least || (v == least && static_cast<uint32_t>(i) <= least_index) ? w : 0;
            all += w;
            hit |= v >= lower && !(v >= above);
            return v >= above ? w : 0;
          },
          [&](int at) {
            if (hit && at < last) note(notes, at);
            hit = false;
          });
      look_again(notes, [&](int i, float v) {
        if (v >= lower && !(v >= above) && !(FLOOR && v == least && static_cast<uint32_t>(i) > least_index))
          own(place_of(v, i));
      });
      uint64_t sum = s.kept[warp][lane];
      reduce<false>(all, sum);
      const uint64_t mass = share_of(all, p), n = gather(none);
      const uint64_t lo = static_cast<uint64_t>(order_of(lower)) << 32;
      const uint64_t hi = s.bins[0] == 0 ? kAll : static_cast<uint64_t>(order_of(above)) << 32;
      const bool sure = slack == kSureSlack;
      if (sum < mass && n <= kList) {
        const uint64_t cut =
            cut_between<FAR>(floor > lo ? floor : lo, hi, n, true, kAll, mass, 0, sum, moved);
        if (sure || s.cut_mass >= mass) return cut;
        histogram_apart(*this);  // the items' sums have had its place
      } else if (sure) {
        return narrow_cut<FAR>(above, least, least_index, floor, mass, sum, heaviest, moved);
      }
    }
  }
  // The same where the bracket holds too many: once more, from the weight above it.
  template <bool FAR>
  __device__ uint64_t narrow_cut(float above, float least, uint32_t least_index, uint64_t floor, uint64_t mass,
                                 uint64_t sum, uint64_t heaviest, bool& moved) {
    narrow(mass - sum, heaviest);
    const float upper = above_bin(s.bins[0]), lower = fmaxf(above_bin(s.bins[1] + 1), least);
    const uint64_t lo = static_cast<uint64_t>(order_of(lower)) << 32;
    const uint64_t hi = s.bins[0] == 0 ? kAll : static_cast<uint64_t>(order_of(upper)) << 32;
    if (threadIdx.x == 0) s.owned = 0;
    __syncthreads();
    uint64_t more = 0;
    each(lower, [&](int i, float v) {
      if (v < lower || v >= above) return;
      if (v == least && static_cast<uint32_t>(i) > least_index) return;
      if (v >= upper)
        more += weight<FAR>(v, s.table);
      else
        own(place_of(v, i));
    });
    moved |= true;  // s.kept lacks these
    const uint64_t n = gather(more);
    return cut_between<FAR>(floor > lo ? floor : lo, hi, n, n <= kList, kAll, mass, 0, sum + more, moved);
  }

  // u all, rounded down: the sums are whole, and one is above u all where it is above this.
  __device__ static uint64_t target_of(uint64_t all, float u) {
    if (!(u > 0.f)) return 0;
    return u < 1.f ? times<false>(all, u) : all - 1;
  }

  // Exclusive sums of (n, m) over the block's threads, and the totals.
  __device__ void scan(uint32_t n, uint64_t m, uint32_t& n_before, uint64_t& m_before, uint32_t& n_all,
                       uint64_t& m_all) {
    uint32_t sn = n;
    uint64_t sm = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sn, o);
      const uint64_t y = __shfl_up_sync(0xffffffffu, sm, o);
      if (lane >= o) {
        sn += x;
        sm += y;
      }
    }
    __syncthreads();  // the last scan has been read
    if (lane == 31) {
      s.scan[warp] = sn;
      s.warp_sum[warp] = sm;
    }
    __syncthreads();
    n_before = sn - n;
    m_before = sm - m;
    n_all = 0;
    m_all = 0;
#pragma unroll
    for (int w = 0; w < kWarpsS; ++w) {
      const uint32_t x = s.scan[w];
      const uint64_t y = s.warp_sum[w];
      if (w < warp) {
        n_before += x;
        m_before += y;
      }
      n_all += x;
      m_all += y;
    }
  }

  // A place without the bits in which no two differ: those that a 16-bit logit lacks, and those above
  // the largest index. Rises with the places of elements.
  __device__ __forceinline__ uint64_t key_of(uint64_t place) const {
    constexpr int kLacks = TYPE == kBf16 ? 16 : TYPE == kFp16 ? 13 : 0;
    const uint32_t order = static_cast<uint32_t>(place >> 32) >> kLacks, index = place_last(place);
    return static_cast<uint64_t>(order) << index_bits | (place_mask - min(index, place_mask));
  }

  // Among n items, with their weights in s.heft (not read with mass kAll), those in [lo, hi): s.cut is
  // the last place before which less than k and less than `mass` lie, above_n and above_m of them at or
  // above hi; s.cut_mass the weight up to it. lo, and all the weight, where the items end before both
  // are reached. By bins of equal stretches of keys, then those of one bin.
  __device__ void cut_items(const uint64_t* items, int n, uint64_t lo, uint64_t hi, uint64_t k, uint64_t mass,
                            uint64_t above_n, uint64_t above_m) {
    const bool weigh = mass != kAll;
    // The ends need not be elements' places: outwards, to a logit's first and last key.
    uint64_t key_lo = key_of(lo) >> index_bits << index_bits, key_hi = key_of(hi - 1) | place_mask;
    ++key_hi;
    while (true) {
      const int top_bit = 63 - __clzll(static_cast<long long>(key_hi - key_lo - 1 | 1));
      const int down = max(0, top_bit + 1 - kItemBits);
      s.item_mass[threadIdx.x] = s.item_mass[threadIdx.x + kThreadsS] = 0;
      s.item_hist[threadIdx.x] = s.item_hist[threadIdx.x + kThreadsS] = 0;
      if (threadIdx.x == 0) {
        s.x_bin = -1;
        s.few_n = 0;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += kThreadsS) {
        const uint64_t at = items[i], key = key_of(at);
        if (at < lo || at >= hi || key < key_lo || key >= key_hi) continue;
        const int b = static_cast<int>((key_hi - 1 - key) >> down);
        atomicAdd(&s.item_hist[b], 1u);
        if (weigh) add64(&s.item_mass[b], s.heft[i]);
      }
      __syncthreads();
      const int b = 2 * threadIdx.x;
      uint32_t c0 = s.item_hist[b], c = c0 + s.item_hist[b + 1], c_before, c_all;
      uint64_t m0 = s.item_mass[b], m = m0 + s.item_mass[b + 1], m_before, m_all;
      scan(c, m, c_before, m_before, c_all, m_all);
      uint64_t x_n = above_n + c_before, x_m = above_m + m_before;
      if (threadIdx.x == 0) {
        s.cut = lo;
        s.cut_mass = above_m + m_all;
      }
      __syncthreads();
      if (x_n < k && x_m < mass && (x_n + c >= k || x_m + m >= mass)) {
        const bool second = x_n + c0 < k && x_m + m0 < mass;
        s.x_bin = b + (second ? 1 : 0);
        s.x_count = second ? x_n + c0 : x_n;
        s.x_before = second ? x_m + m0 : x_m;
      }
      __syncthreads();
      const int x = s.x_bin;
      if (x < 0) return;
      above_n = s.x_count;
      above_m = s.x_before;
      const uint32_t in_bin = s.item_hist[x];
      key_hi -= static_cast<uint64_t>(x) << down;
      if (key_hi - key_lo > 1ull << down) key_lo = key_hi - (1ull << down);
      if (in_bin <= kFew) break;
      __syncthreads();
    }
    for (int i = threadIdx.x; i < n; i += kThreadsS) {
      const uint64_t at = items[i], key = key_of(at);
      if (at >= lo && at < hi && key >= key_lo && key < key_hi) s.few[atomicAdd(&s.few_n, 1u)] = static_cast<uint16_t>(i);
    }
    __syncthreads();
    const uint32_t few = s.few_n;
    if (threadIdx.x < few) {
      const uint64_t at = items[s.few[threadIdx.x]], w = weigh ? s.heft[s.few[threadIdx.x]] : 0;
      uint64_t before = above_m, count = above_n;
      for (uint32_t j = 0; j < few; ++j) {
        const bool above = items[s.few[j]] > at;
        if (weigh) before += above ? s.heft[s.few[j]] : 0;
        count += above ? 1 : 0;
      }
      if (count < k && before < mass && (count + 1 >= k || before + w >= mass)) {
        s.cut = at;
        s.cut_mass = before + w;
      }
    }
    __syncthreads();
  }

  __device__ void clear_kept() {
    static_assert(kParts == 32, "one for each lane");
    s.kept[warp][lane] = 0;
    __syncwarp();
  }
  // The elements at or above `cut` that weigh at least `least` into s.kept; those below `low` are
  // known to weigh less.
  template <bool FAR>
  __device__ void weigh_kept(uint64_t cut, uint64_t least, float low) {
    const float edge = cut > 0 ? place_value(cut) : -INFINITY;
    const uint32_t edge_index = place_last(cut);
    clear_kept();
    const auto nothing_more = [](int) {};
    if (cut == 0 && least == 0) {
      each_kept(-INFINITY, [&](int, float v) { return weight<FAR>(v, s.table); }, nothing_more);
      return;
    }
    each_kept(
        fmaxf(low, edge),
        [&](int i, float v) {
          const uint64_t w = weight<FAR>(v, s.table);
          return (v > edge || (v == edge && static_cast<uint32_t>(i) <= edge_index)) && w >= least ? w : 0;
        },
        nothing_more);
  }
  // Draws from them.
  template <bool FAR>
  __device__ void draw(uint64_t cut, uint64_t least, float low, float u, int64_t* token) {
    const float edge = cut > 0 ? place_value(cut) : -INFINITY;
    const uint32_t edge_index = place_last(cut);
    __syncwarp();
    const uint64_t part = s.kept[warp][lane];
    uint64_t scan = part;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += x;
    }
    if (lane == 31) s.warp_kept[warp] = scan;
    __syncthreads();
    uint64_t block = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kWarpsS; ++i) {
      if (i < warp) before += s.warp_kept[i];
      block += s.warp_kept[i];
    }
    const uint64_t sum = s.warp_kept[warp];
    if (threadIdx.x < a.cluster) *of_block(s.peers[turn][rank], threadIdx.x) = block;
    sync();
    uint64_t all = 0;
    for (int i = 0; i < a.cluster; ++i) {
      if (i < rank) before += s.peers[turn][i][0];
      all += s.peers[turn][i][0];
    }
    turn ^= 1;
    const uint64_t target = target_of(all, u), part_before = before + scan - part;
    if (target >= part_before && target < part_before + part) {
      s.x_bin = warp * kParts + lane;
      s.x_before = part_before;
    }
    if (!__syncthreads_or(target >= before && target < before + sum)) return;
    // This block holds it, in this part of a warp's stretch.
    const int stretch_begin = (rank * kWarpsS + s.x_bin / kParts) * a.stretch;
    const int begin = stretch_begin + s.x_bin % kParts * a.part;
    const int end = min(min(begin + a.part, stretch_begin + a.stretch), a.V + shift);
    before = s.x_before;
    constexpr int kMine = 4;
    for (int at = begin; at < end; at += kThreadsS * kMine) {
      const int i = at + static_cast<int>(threadIdx.x) * kMine - shift;
      uint64_t w[kMine], mine = 0;
#pragma unroll
      for (int e = 0; e < kMine; ++e) {
        const bool on = i + e >= 0 && i + e + shift < end;
        const float v = on ? load_value<TYPE>(z, i + e) : -INFINITY;
        w[e] = weight<FAR>(v, s.table);
        const bool in =
            on && v >= low && (v > edge || (v == edge && static_cast<uint32_t>(i + e) <= edge_index)) && w[e] >= least;
        w[e] = in ? w[e] : 0;
        mine += w[e];
      }
      uint32_t none, none_all;
      uint64_t c, total;
      this->scan(0, mine, none, c, none_all, total);
      c += before;
#pragma unroll
      for (int e = 0; e < kMine; ++e) {
        if (target >= c && target < c + w[e]) *token = i + e;
        c += w[e];
      }
      before += total;
    }
  }

  __device__ void fill_table() {
    for (int i = threadIdx.x; i < kTable; i += kThreadsS) s.table[i] = kExp2.v[i];
  }
  // Everything from passes over the row. by_list: the list has had the table's place.
  template <bool FAR>
  __device__ void from_row(bool by_list, int64_t top_k, float p, uint64_t heaviest, uint64_t least, float low,
                           float u, int64_t* token) {
    if (by_list) {
      __syncthreads();
      fill_table();
      __syncthreads();
    }
    const bool by_k = top_k < a.V, by_p = p < 1.f;
    uint64_t cut = 0;
    if (by_k || by_p) histogram();
    if (by_k) cut = cut_by_count(top_k);
    bool moved = false;
    if (by_k && by_p) histogram();  // its place has been in use
    if (by_p)
      cut = by_k ? cut_by_mass<FAR, true>(top_k, p, cut, heaviest, moved)
                 : cut_by_mass<FAR, false>(top_k, p, 0, heaviest, moved);
    if (!by_p || least > 0 || moved) weigh_kept<FAR>(cut, least, low);
    draw<FAR>(cut, least, low, u, token);
  }

  // ---- the list of candidates: all elements that reach a logit

  // This block's largest logit of each thread's loads is m. Finds the row's largest (its order, or
  // 0xFFFFFFFF for a NaN), and where `wanted` is not 0 a logit that at least so many elements
  // reach, from the m's: each block offers the one that `wanted` of its own reach, and the one that
  // its share of them reach. The highest of the former will do, and the lowest of the latter.
  __device__ uint32_t find_top(const float (&m)[kAhead], uint32_t wanted, float& threshold) {
    float most = max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) s.scan_mass[warp] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarpsS; ++w) most = max_nan(most, s.scan_mass[w]);
    c_hi = s.c_hi;
    c_lo = s.c_lo;
    if (wanted > 0) {
      const float scale = c_hi * kNear;
      // What is beyond the last bin has no weight.
      if (threadIdx.x < 2) s.mine[threadIdx.x] = (most - kNearBins / scale) - fabsf(most) * 1e-6f;
#pragma unroll
      for (int g = 0; g < kAhead; ++g) {
        const float d = m[g] == most ? 0.f : (most - m[g]) * scale;
        if (d < static_cast<float>(kNearBins) && most > -INFINITY) atomicAdd(&s.near_hist[static_cast<int>(d)], 1u);
      }
      __syncthreads();
      static_assert(kNearBins == 2 * kThreadsS, "two bins for a thread");
      const uint32_t n0 = s.near_hist[2 * threadIdx.x], n = n0 + s.near_hist[2 * threadIdx.x + 1];
      uint32_t sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      if (lane == 31) s.scan[warp] = sum;
      __syncthreads();
      uint32_t before = sum - n;
      for (int w = 0; w < warp; ++w) before += s.scan[w];
      const uint32_t share = (wanted + a.cluster - 1) / a.cluster;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t k = i == 0 ? wanted : share;
        if (before < k && k <= before + n) {
          // The bins' edges are rounded: a little further.
          const float b = static_cast<float>(2 * threadIdx.x + (before + n0 < k ? 1 : 0)) + 1.01f;
          s.mine[i] = (most - b / scale) - fabsf(most) * 1e-6f;
        }
      }
      __syncthreads();
    }
    if (a.cluster > 1) cluster_wait();  // all blocks run: their memory may be written
    if (threadIdx.x < a.cluster) {
      of_block(s.peers[turn][rank], threadIdx.x)[0] = most != most ? 0xFFFFFFFFull : order_of(most);
      float* to = of_block(s.thresholds[rank], threadIdx.x);
      to[0] = wanted > 0 ? s.mine[0] : -INFINITY;
      to[1] = wanted > 0 ? s.mine[1] : -INFINITY;
    }
    sync();
    uint64_t best = 0;
    float one = -INFINITY, each_one = INFINITY;
    for (int r = 0; r < a.cluster; ++r) {
      best = max(best, s.peers[turn][r][0]);
      one = fmaxf(one, s.thresholds[r][0]);
      each_one = fminf(each_one, s.thresholds[r][1]);
    }
    turn ^= 1;
    threshold = fmaxf(one, each_one);
    return static_cast<uint32_t>(best);
  }

  // 2^((z - top) log2(e) / T), by the hardware's.
  __device__ __forceinline__ float about(float v) const {
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"((v - top) * c_hi));
    return w;
  }
  // Whether those that reach `threshold` seem to weigh less than p of all: from the loads' largest, and from
  // the middle of each warp's stretch. The list would be for nothing (512 rows of 128256, p = 0.95: 27 of
  // 166 us that a block of a flat row takes); asking takes 3.
  __device__ bool seems_flat(const float (&m)[kAhead], float threshold, float p) {
    float listed = 0.f, rest = 0.f, v[8];
#pragma unroll
    for (int g = 0; g < kAhead; ++g) listed += m[g] >= threshold ? about(m[g]) : 0.f;
    const int steps = (last - first) / 256;
    unpack8<TYPE>(group(first + steps / 2 * 256 + lane * 8), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) rest += v[e] >= threshold ? 0.f : about(v[e]);
    uint64_t x = static_cast<uint64_t>(listed * 0x1p20f);
    uint64_t y = static_cast<uint64_t>(rest * static_cast<float>(steps + 1) * 0x1p20f);
    reduce<false>(x, y);
    return 2.f * static_cast<float>(x) * (1.f - p) < static_cast<float>(y) * p;
  }

  // Lists the elements that reach `threshold`, in the first block. `weigh`: the weight of all
  // others, by the hardware's 2^x, in the weights' units. Their number, the same in every thread; above
  // kList they are not listed.
  __device__ int list_above(float threshold, bool weigh, uint64_t heaviest) {
    const uint32_t room = kList / a.cluster;
    uint64_t* list = of_block(s.list, 0);
    const float shift_by = top * c_hi;
    float sum = 0.f;
    clear_notes();
    uint32_t* notes = reinterpret_cast<uint32_t*>(s.item);
    each_raw([&](int, int at, const Raw8<TYPE>& raw) {
      if (weigh) {
        float v[8], w[8];
        unpack8<TYPE>(raw, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w[e]) : "f"(fmaf(v[e], c_hi, -shift_by)));
          w[e] = v[e] >= threshold ? 0.f : w[e];
        }
        sum += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
      }
      if (largest<TYPE>(raw) >= threshold && at < last) note(notes, at);
    });
    look_again(notes, [&](int i, float v) {
      if (v >= threshold && v != -INFINITY) {
        const uint32_t n = atomicAdd(&s.owned, 1u);
        if (n < room) list[rank * room + n] = place_of(v, i);
        if (n < kList) s.heft[n] = place_of(v, i);
      }
    });
    uint64_t rest = 0;
    if (weigh) {
      rest = __float2ull_rn(sum * static_cast<float>(heaviest));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) rest += shfl64(rest, o);
      if (lane == 0) s.red[warp][0] = rest;
    }
    __syncthreads();
    if (threadIdx.x < a.cluster) {
      rest = 0;
      if (weigh)
        for (int w = 0; w < kWarpsS; ++w) rest += s.red[w][0];
      *of_block(&s.rests[rank], threadIdx.x) = rest;
      *of_block(&s.owns[rank], threadIdx.x) = s.owned;
    }
    sync();
    uint32_t n = 0, before = 0, most = 0;
    for (int r = 0; r < a.cluster; ++r) {
      if (r < rank) before += min(s.owns[r], kList + 0u);
      n += min(s.owns[r], kList + 1u);
      most = max(most, s.owns[r]);
    }
    if (n <= kList && most > room) {
      // More than a block's room: once more, one block's after the other's.
      const uint32_t mine = s.owns[rank];
      for (uint32_t i = threadIdx.x; i < mine; i += kThreadsS) list[before + i] = s.heft[i];
      sync();
    }
    return static_cast<int>(n);
  }

  // In the first block: the items and their weights from the list.
  __device__ void take_list(uint64_t& rest) {
    uint32_t room = kList / a.cluster, most = 0;
    for (int r = 0; r < a.cluster; ++r) most = max(most, s.owns[r]);
    int n = 0;
    rest = 0;
    for (int r = 0; r < a.cluster; ++r) {
      const uint32_t m = s.owns[r], from = most > room ? n : r * room;
      rest += s.rests[r];
      for (uint32_t i = threadIdx.x; i < m; i += kThreadsS) s.item[n + i] = s.list[from + i];
      n += static_cast<int>(m);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreadsS) s.heft[i] = any_weight(place_value(s.item[i]), kExp2.v);
    __syncthreads();
  }

  // The token from a list of up to kPairs items: two threads compare an item with the others.
  __device__ int draw_pairs(int n, uint64_t k, float p, uint64_t rest, uint64_t error, uint64_t least, float u,
                            int64_t* token) {
    const int mine = threadIdx.x >> 1, half = threadIdx.x & 1;
    const bool on = mine < n;
    const uint64_t at = on ? s.item[mine] : 0, w = on ? s.heft[mine] : 0;
    uint32_t count = 0;
    uint64_t before = 0;
    for (int j = half; j < n; j += 2) {
      const bool above = s.item[j] > at;
      count += above ? 1 : 0;
      before += above ? s.heft[j] : 0;
    }
    count += __shfl_xor_sync(0xffffffffu, count, 1);
    before += shfl64(before, 1);
    bool kept = on && count < k;
    if (p < 1.f) {
      uint64_t sum = kept && half == 0 ? w : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += shfl64(sum, o);
      if (lane == 0) s.warp_sum[warp] = sum;
      __syncthreads();
      uint64_t listed = 0;
#pragma unroll
      for (int i = 0; i < kWarpsS; ++i) listed += s.warp_sum[i];
      const uint64_t of = listed + rest;
      const uint64_t mass = share_of(of - (of < error ? of : error), p), most = share_of(of + error, p);
      if (most > listed) return kTooShort;
      if (__syncthreads_or(kept && before >= mass && before < most)) return kInexact;
      kept = kept && before < mass;
    }
    kept = kept && w >= least;
    if (half == 0) s.list[mine] = kept ? w : 0;
    __syncthreads();
    uint64_t all = 0, c = 0;
    const uint32_t index = static_cast<uint32_t>(at);  // falls with the index
    for (int j = half; j < n; j += 2) {
      const uint64_t x = s.list[j];
      all += x;
      c += static_cast<uint32_t>(s.item[j]) > index ? x : 0;
    }
    all += shfl64(all, 1);
    c += shfl64(c, 1);
    const uint64_t target = target_of(all, u);
    if (kept && half == 0 && target >= c && target < c + w) *token = place_index(at);
    return kDone;
  }

  // The token, from the items at or above s.cut with weights of at least `least`: by buckets of
  // neighbouring indices.
  __device__ void draw_buckets(int n, uint64_t least, float u, int64_t* token) {
    int down = 0;
    while (((a.V - 1) >> down) >= kThreadsS) ++down;
    const uint64_t cut = s.cut;
    s.bucket[threadIdx.x] = 0;
    if (threadIdx.x == 0) s.few_n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreadsS) {
      const uint64_t at = s.item[i], w = s.heft[i];
      if (at >= cut && w >= least)
        add64(&s.bucket[place_index(at) >> down], w);
    }
    __syncthreads();
    uint32_t none, none_all;
    uint64_t before, all;
    const uint64_t mine = s.bucket[threadIdx.x];
    scan(0, mine, none, before, none_all, all);
    const uint64_t target = target_of(all, u);
    if (target >= before && target < before + mine) {
      s.x_bin = threadIdx.x;
      s.x_before = before;
    }
    __syncthreads();
    const int x = s.x_bin;
    for (int i = threadIdx.x; i < n; i += kThreadsS) {
      const uint64_t at = s.item[i];
      if (at >= cut && place_index(at) >> down == x && s.heft[i] >= least)
        s.few[atomicAdd(&s.few_n, 1u)] = static_cast<uint16_t>(i);
    }
    __syncthreads();
    const uint32_t few = s.few_n;
    for (uint32_t i = threadIdx.x; i < few; i += kThreadsS) {
      const int index = place_index(s.item[s.few[i]]);
      uint64_t c = s.x_before;
      for (uint32_t j = 0; j < few; ++j)
        c += place_index(s.item[s.few[j]]) < index ? s.heft[s.few[j]] : 0;
      if (target >= c && target < c + s.heft[s.few[i]]) *token = index;
    }
  }

  // The token from the list, where it holds all that is kept. Otherwise the cut hangs on what `rest` is
  // within `error` (kInexact), or on elements that are not listed (kTooShort).
  __device__ int from_items(int n, float threshold, uint64_t k, float p, uint64_t rest, uint64_t error,
                            uint64_t least, float u, int64_t* token) {
    if (n <= kPairs) return draw_pairs(n, k, p, rest, error, least, u, token);
    const uint64_t lo = static_cast<uint64_t>(order_of(threshold)) << 32;
    const uint64_t hi = static_cast<uint64_t>(order_of(top) + 1) << 32;
    uint64_t listed = 0, cut = lo;
    if (k == kAll) {
      uint32_t none, none_all;
      uint64_t m = 0, before;
      for (int i = threadIdx.x; i < n; i += kThreadsS) m += s.heft[i];
      scan(0, m, none, before, none_all, listed);
    } else {
      cut_items(s.item, n, lo, hi, k, p < 1.f ? kAll - 1 : kAll, 0, 0);
      listed = s.cut_mass;
      cut = s.cut;
    }
    if (p < 1.f) {
      const uint64_t of = listed + rest;
      const uint64_t mass = share_of(of - (of < error ? of : error), p), most = share_of(of + error, p);
      if (most > listed) return kTooShort;
      __syncthreads();
      cut_items(s.item, n, cut, hi, kAll, mass, 0, 0);
      if (s.cut_mass < most) return kInexact;
    }
    draw_buckets(n, least, u, token);
    return kDone;
  }
  // Whether the token was drawn from the elements that reach `threshold`.
  __device__ bool from_list(float threshold, int64_t top_k, float p, uint64_t heaviest, uint64_t least,
                            float u, int64_t* token) {
    const bool by_k = top_k < a.V;
    const uint64_t k = by_k ? top_k : kAll;
    const int n = list_above(threshold, !by_k, heaviest);
    if (n > kList) return false;
    int verdict = kTooShort;
    uint64_t rest = 0;
    if (rank == 0) {
      take_list(rest);
      // The hardware's 2^x and its argument, a thread's sums, and top c, whose rounding grows with
      // it; each weight is rounded by half a unit.
      const float off = 0x1p-18f + (fabsf(top * c_hi) + static_cast<float>(a.stretch / 256 + 8)) * 0x1p-24f;
      const uint64_t error = by_k ? 0 : static_cast<uint64_t>(static_cast<float>(rest) * off) + a.V;
      verdict = from_items(n, threshold, k, p, rest, error, least, u, token);
      if (threadIdx.x < a.cluster) *of_block(&s.verdict, threadIdx.x) = verdict;
    }
    sync();
    if (s.verdict == kInexact) {
      // The others' weight once more, as whole numbers.
      rest = 0;
      uint64_t none = 0;
      each(-INFINITY, [&](int, float v) {
        if (v < threshold) rest += any_weight(v, kExp2.v);
      });
      reduce<false>(rest, none);
      if (rank == 0) {
        verdict = from_items(n, threshold, k, p, rest, 0, least, u, token);
        if (threadIdx.x < a.cluster) *of_block(&s.verdict, threadIdx.x) = verdict;
      }
      sync();
    }
    return s.verdict == kDone;
  }

  __device__ void run(int row) {
    const float temperature = a.temperatures ? a.temperatures[row] : a.temperature;
    int64_t top_k = a.top_ks ? a.top_ks[row] : a.top_k;
    const float p = a.top_ps ? a.top_ps[row] : a.top_p;
    const float min_p = a.min_ps ? a.min_ps[row] : a.min_p;
    const float u = a.u[row];
    if (threadIdx.x == 0) {
      const double c = 1.4426950408889634074 / fmax(static_cast<double>(temperature), 1e-30);
      s.c_hi = static_cast<float>(c);
      s.c_lo = static_cast<float>(c - static_cast<double>(s.c_hi));
    }
    if (top_k <= 0 || top_k > a.V) top_k = a.V;
    const bool greedy = !(temperature > 0.f) || top_k == 1 || !(p > 0.f);
    const bool by_k = top_k < a.V, by_p = p < 1.f;
    const bool list = !greedy && (by_k ? top_k <= kMostK : by_p) && temperature < 1e30f;
    // The loads' largest tell where the list begins if there are enough of them.
    const int loads = min(a.cluster * kThreadsS * kAhead, a.V / 8);
    const int wanted = by_k ? static_cast<int>(min(top_k, static_cast<int64_t>(kMostK))) : min(loads / 2, kWanted);
    const bool near = list && wanted > 0 && loads >= 2 * wanted;
    if (!list && !greedy) fill_table();
    float m[kAhead];
#pragma unroll
    for (int g = 0; g < kAhead; ++g) m[g] = -INFINITY;
    each_raw([&](int g, int, const Raw8<TYPE>& raw) { m[g] = max_nan(m[g], largest<TYPE>(raw)); });
    float threshold;
    const uint32_t order = find_top(m, near ? wanted : 0, threshold);
    int64_t* token = a.tokens + row;
    top = value_of(order);
    if (order == 0xFFFFFFFFu || top == -INFINITY) {  // a NaN, or nothing to choose from
      if (rank == 0 && threadIdx.x == 0) *token = -1;
      return;
    }
    if (greedy) {
      uint64_t at = 0, none = 0;
      each(top, [&](int i, float v) {
        if (v == top) at = max(at, place_of(top, i));
      });
      reduce<true>(at, none);
      if (rank == 0 && threadIdx.x == 0) *token = place_index(at);
      return;
    }
    index_bits = 32 - __clz(a.V);
    place_mask = (1u << index_bits) - 1;
    const float high = top * c_hi;
    far = !(fabsf(high) < 3900.f) || c_hi < 1e-30f;
    octave = far ? 0 : static_cast<int>(ceilf(high));
    lowest = far ? -INFINITY : top - 47.f / c_hi;
    // min_p above 1 keeps the largest. Elements well below the limit need no weight; below +infinity no
    // logit says how far.
    const float share = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;
    const uint64_t heaviest = share > 0.f || by_p ? any_weight(top, kExp2.v) : 0;
    const uint64_t least = share < 1.f ? times<true>(heaviest, share) : heaviest;  // 0 where all weigh enough
    const float low = share > 0.f && c_hi > 1e-30f && top < INFINITY
                          ? top + (log2f(share) - 0.01f) / c_hi - fabsf(top) * 1e-6f : -INFINITY;
    // Where p alone limits, the others' weight is by the hardware's 2^x, whose argument must be right to
    // less than 1: from_list's bound on its error is linear in the argument's. Else from the row.
    if (list && (by_k || fabsf(high) < 0x1p24f)) {
      const bool in_vain = near && !by_k && seems_flat(m, threshold, p);
      if ((near && !in_vain) || a.V <= kList / a.cluster) {
        if (!near || in_vain) threshold = -INFINITY;
        if (from_list(threshold, top_k, p, heaviest, least, u, token)) return;
      }
      if (by_k) {
        histogram();
        bracket(wanted, 1.f);
        threshold = above_bin(s.bins[0] + 1);
        if (from_list(threshold, top_k, p, heaviest, least, u, token)) return;
      }
    }
    if (far)
      from_row<true>(list, top_k, p, heaviest, least, low, u, token);
    else
      from_row<false>(list, top_k, p, heaviest, least, low, u, token);
  }
};

static_assert(kPerSm * (sizeof(Shared) + 1024) <= 227 * 1024, "as many blocks as an SM is to hold");

template <int TYPE>
__global__ void __launch_bounds__(kThreadsS, kPerSm) sample_kernel(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  if (a.cluster > 1) cluster_arrive();
  for (int i = threadIdx.x; i < kNearBins; i += kThreadsS) s.near_hist[i] = 0;
  griddep_wait();
  const int row = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
  const uint8_t* z = static_cast<const uint8_t*>(a.logits) + row * a.ld * type_size(TYPE);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(z) % 16) / type_size(TYPE);
  const int64_t begin = static_cast<int64_t>(rank * kWarpsS + warp) * a.stretch;
  const int64_t end = min(begin + a.stretch, static_cast<int64_t>(a.V) + shift);
  Row<TYPE> r{a, s, z, shift, rank, static_cast<int>(min(begin, end)), static_cast<int>(end), lane, warp, 0};
  r.run(row);
  // Not before: blocks of the next kernel that wait on an SM keep this one's from it.
  griddep_launch();
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
  // Blocks for a row: as many as give two waves of them, each with 16 KiB at least. 512 x 128256, p = 0.95,
  // rows of mixed certainty: 1 block 241 us, 2 234, 4 258; 1 x 128256 with 8.
  int cluster = 1;
  while (cluster < kMaxCluster && 2 * cluster * p->B <= 2 * kPerSm * sms &&
         p->V * type_size(p->dtype) >= 2 * cluster * 16384)
    cluster *= 2;
  a.cluster = cluster;
  const int64_t warps = static_cast<int64_t>(cluster) * kWarpsS;
  a.stretch = static_cast<int>(((p->V + 8 + warps - 1) / warps + 7) / 8 * 8);
  const int steps = (a.stretch + kStep - 1) / kStep;
  a.part = (steps + kParts - 1) / kParts * kStep;
  const cudaError_t e = launch_sample(a, p->dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}
