// Device helpers of the operators on the residual stream: rows of bf16, fp16 or fp32 in
// groups of 8 columns, sums over the threads of a row, and the dropout mask.
#pragma once
#include <cstdint>

#include "../../include/flce.h"
#include "sm103_primitives.cuh"

namespace flce {

constexpr int kBf16 = FLCE_DTYPE_BF16, kFp16 = FLCE_DTYPE_FP16, kFp32 = FLCE_DTYPE_FP32;

__host__ __device__ constexpr int type_size(int type) { return type == kFp32 ? 4 : 2; }

// Eight values as they are in memory.
template <int TYPE>
struct Raw8 {
  uint4 w[TYPE == kFp32 ? 2 : 1];
};

template <int TYPE>
__device__ __forceinline__ float load_value(const void* row, int64_t col) {
  if constexpr (TYPE == kFp32) return static_cast<const float*>(row)[col];
  return unpack_16(static_cast<const uint16_t*>(row)[col], TYPE == kFp16);
}
template <int TYPE>
__device__ __forceinline__ void store_value(void* row, int64_t col, float v) {
  if constexpr (TYPE == kFp32)
    static_cast<float*>(row)[col] = v;
  else
    static_cast<uint16_t*>(row)[col] =
        static_cast<uint16_t>(pack_16x2(v, 0.f, TYPE == kFp16) & 0xFFFFu);
}

template <int TYPE>
__device__ __forceinline__ void unpack8(const Raw8<TYPE>& r, float* v) {
#pragma unroll
  for (int i = 0; i < (TYPE == kFp32 ? 2 : 1); ++i) {
    const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (TYPE == kFp32) {
        v[4 * i + e] = __uint_as_float(w[e]);
      } else {
        v[2 * e] = unpack_16(w[e] & 0xFFFFu, TYPE == kFp16);
        v[2 * e + 1] = unpack_16(w[e] >> 16, TYPE == kFp16);
      }
    }
  }
}
template <int TYPE>
__device__ __forceinline__ Raw8<TYPE> pack8(const float* v) {
  Raw8<TYPE> r;
#pragma unroll
  for (int i = 0; i < (TYPE == kFp32 ? 2 : 1); ++i) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (TYPE == kFp32)
        w[e] = __float_as_uint(v[4 * i + e]);
      else
        w[e] = pack_16x2(v[2 * e], v[2 * e + 1], TYPE == kFp16);
    }
    r.w[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

// Values 2 i and 2 i + 1 as a packed pair of floats, on which one instruction does two sums or
// products.
template <int TYPE>
__device__ __forceinline__ uint64_t pair_of(const Raw8<TYPE>& r, int i) {
  const uint4& u = r.w[TYPE == kFp32 ? i / 2 : 0];
  if constexpr (TYPE == kFp32) {
    return i % 2 ? f32x2(__uint_as_float(u.z), __uint_as_float(u.w))
                 : f32x2(__uint_as_float(u.x), __uint_as_float(u.y));
  } else {
    const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
    return f32x2(unpack_16(w & 0xFFFFu, TYPE == kFp16), unpack_16(w >> 16, TYPE == kFp16));
  }
}

// a b of values 2 i and 2 i + 1 of two groups, exact in fp32 for 16-bit types: the products
// take the halves of a word as they are.
template <int TYPE>
__device__ __forceinline__ uint64_t pair_product(const Raw8<TYPE>& a, const Raw8<TYPE>& b, int i) {
  if constexpr (TYPE == kFp32) {
    return fmul2(pair_of(a, i), pair_of(b, i));
  } else {
    const uint4 &u = a.w[0], &v = b.w[0];
    const uint32_t x = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
    const uint32_t y = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    float lo, hi;
    if constexpr (TYPE == kBf16)
      asm("{.reg .b16 a, b, c, d;\n mov.b32 {a, b}, %2;\n mov.b32 {c, d}, %3;\n"
          " fma.rn.f32.bf16 %0, a, c, 0f00000000;\n fma.rn.f32.bf16 %1, b, d, 0f00000000;}"
          : "=f"(lo), "=f"(hi) : "r"(x), "r"(y));
    else
      asm("{.reg .b16 a, b, c, d;\n mov.b32 {a, b}, %2;\n mov.b32 {c, d}, %3;\n"
          " fma.rn.f32.f16 %0, a, c, 0f00000000;\n fma.rn.f32.f16 %1, b, d, 0f00000000;}"
          : "=f"(lo), "=f"(hi) : "r"(x), "r"(y));
    return f32x2(lo, hi);
  }
}

// Columns col .. col + 7 of a row. VEC: the row starts on a 16-byte boundary and n is a
// multiple of 8; otherwise value by value, and values at or past n read as 0.
template <int TYPE, bool VEC>
__device__ __forceinline__ Raw8<TYPE> load8(const void* row, int64_t col, int64_t n) {
  Raw8<TYPE> r;
  if constexpr (VEC) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) +
                                                    col * type_size(TYPE));
    r.w[0] = p[0];
    if constexpr (TYPE == kFp32) r.w[1] = p[1];
  } else {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = col + e < n ? load_value<TYPE>(row, col + e) : 0.f;
    r = pack8<TYPE>(v);  // exact: the values are of this type
  }
  return r;
}
template <int TYPE, bool VEC>
__device__ __forceinline__ void store8(void* row, int64_t col, int64_t n, const float* v) {
  if constexpr (VEC) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(row) + col * type_size(TYPE));
    const Raw8<TYPE> r = pack8<TYPE>(v);
    p[0] = r.w[0];
    if constexpr (TYPE == kFp32) p[1] = r.w[1];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < n) store_value<TYPE>(row, col + e, v[e]);
  }
}

// How a thread's groups of 8 columns lie. kWide: 8 neighbours, moved 16 bytes at a time; rows off
// the 16-byte boundaries go value by value, either with a warp's accesses next to each other
// (kStrided), or, where a scale covers 128 columns, as in kWide (kNarrow).
enum Layout { kWide, kStrided, kNarrow };

template <Layout L>
__device__ __forceinline__ int column(int j, int e, int T, int t) {
  return L == kStrided ? (j * 8 + e) * T + t : (j * T + t) * 8 + e;
}
template <int TYPE, Layout L>
__device__ __forceinline__ Raw8<TYPE> load_group(const void* row, int j, int T, int t, int n) {
  if constexpr (L == kWide) {
    if (column<L>(j, 0, T, t) >= n) return {};
    return load8<TYPE, true>(row, column<L>(j, 0, T, t), n);
  } else {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = column<L>(j, e, T, t);
      v[e] = col < n ? load_value<TYPE>(row, col) : 0.f;
    }
    return pack8<TYPE>(v);
  }
}
template <int TYPE, Layout L>
__device__ __forceinline__ void store_group(void* row, int j, int T, int t, int n, const float* v) {
  if constexpr (L == kWide) {
    if (column<L>(j, 0, T, t) < n) store8<TYPE, true>(row, column<L>(j, 0, T, t), n, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = column<L>(j, e, T, t);
      if (col < n) store_value<TYPE>(row, col, v[e]);
    }
  }
}

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2,
// 3", 2011): four random words for a counter of four words and a key of two. The ten rounds'
// keys are the same for all counters of a call: a thread makes them once (in shared
// memory they cost more: 8192 x 4096 forward 48 us for 43).
struct Keys {
  uint32_t k0[10], k1[10];
};
__device__ __forceinline__ Keys philox_keys(uint64_t seed) {
  Keys k;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    k.k0[i] = static_cast<uint32_t>(seed) + i * 0x9E3779B9u;
    k.k1[i] = static_cast<uint32_t>(seed >> 32) + i * 0xBB67AE85u;
  }
  return k;
}
__device__ __forceinline__ uint4 philox(uint4 c, const Keys& k) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k.k0[i], static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k.k1[i], static_cast<uint32_t>(a));
  }
  return c;
}

// The dropout of a call: an element is dropped where its 16 random bits are below
// `threshold`, and scaled otherwise. Sixteen bits for an element, not 32: the generator's ten
// rounds take some 60 instructions for a counter's four words, which with 32 bits would be
// more time than the memory takes; p is kept to 2^-16, and the scale is the exact inverse of
// what is kept, so that the mean is right for the p that is drawn.
struct Dropout {
  uint32_t threshold;  // 0: no dropout, 65536: everything
  float scale;         // 65536 / (65536 - threshold), 0 where everything is dropped
  uint64_t seed, offset;
  const int64_t* seed_at;  // the seed in device memory instead, or null
};
__device__ __forceinline__ Keys dropout_keys(const Dropout& d) {
  return philox_keys(d.seed_at ? static_cast<uint64_t>(*d.seed_at) : d.seed);
}
// The random bits of columns 8 group .. 8 group + 7 of a row, two in a word, the lower first.
__device__ __forceinline__ uint4 drop_bits(const Dropout& d, const Keys& k, uint32_t row, uint32_t group) {
  return philox(make_uint4(group, row, static_cast<uint32_t>(d.offset), static_cast<uint32_t>(d.offset >> 32)),
                k);
}
// v[e] = D(v[e]) of those columns. A half is compared where it is, or in the upper place.
__device__ __forceinline__ void drop8(const Dropout& d, const Keys& k, uint32_t row, uint32_t group, float* v) {
  const uint4 r = drop_bits(d, k, row, group);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  // At least the threshold: above the last word whose upper half is below it.
  const uint32_t last = (d.threshold - 1) << 16 | 0xFFFFu;
  const uint64_t scale = f32x2(d.scale, d.scale);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float lo, hi;
    f32x2_split(fmul2(f32x2(v[2 * e], v[2 * e + 1]), scale), lo, hi);
    v[2 * e] = (w[e] << 16) > last ? lo : 0.f;
    v[2 * e + 1] = w[e] > last ? hi : 0.f;
  }
}

// The larger one; a NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum (or largest) over a row's threads, in every one of them and in a fixed order: a warp
// alone, or all of a block's blockDim.x / 32 warps through `s` (32 floats, not in use by an
// earlier call).
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, u) : v + u;
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? s[lane] : 0.f;  // 0 is neutral for the sums, and for largest magnitudes
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, u) : v + u;
  }
  return v;
}

}  // namespace flce
