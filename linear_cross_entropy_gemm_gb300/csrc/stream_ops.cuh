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

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2,
// 3", 2011): four random words for a counter of four words and a key of two.
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// The dropout of a call: an element is dropped where its 16 random bits are below
// `threshold`, and scaled otherwise. Sixteen bits for an element, not 32: the generator's ten
// rounds are two products and two three-way XORs each, which for a counter of four words
// would cost as much time as the memory does; p is kept to 2^-16, and the scale is the
// exact inverse of what is kept, so that the mean is right for the p that is drawn.
struct Dropout {
  uint32_t threshold;  // 0: no dropout, 65536: everything
  float scale;         // 65536 / (65536 - threshold), 0 where everything is dropped
  uint64_t seed, offset;
  const int64_t* seed_at;  // the seed in device memory instead, or null
};
struct Key {
  uint32_t k0, k1;
};
__device__ __forceinline__ Key dropout_key(const Dropout& d) {
  uint64_t s = d.seed;
  if (d.threshold != 0 && d.seed_at) s = static_cast<uint64_t>(*d.seed_at);
  return {static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32)};
}
// v[e] = D(v[e]) of columns 8 group .. 8 group + 7 of a row.
__device__ __forceinline__ void drop8(const Dropout& d, Key k, uint32_t row, uint32_t group, float* v) {
  const uint4 r = philox(make_uint4(group, row, static_cast<uint32_t>(d.offset),
                                    static_cast<uint32_t>(d.offset >> 32)), k.k0, k.k1);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = (w[e] & 0xFFFFu) >= d.threshold ? v[2 * e] * d.scale : 0.f;
    v[2 * e + 1] = (w[e] >> 16) >= d.threshold ? v[2 * e + 1] * d.scale : 0.f;
  }
}

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
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
