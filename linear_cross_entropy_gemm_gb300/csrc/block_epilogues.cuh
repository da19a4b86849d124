// Activations and GEMM epilogues of the layer operators: the linear layer
// (bias, activation, residual), the gated feed-forward projection, and the
// gradients of both.
//
//   linear   z = x W^T + b,  y = a(z) + r
//   gated    g = x Wg^T, u = x Wu^T,  h = a(g) u
//
// Everything between the fp32 accumulator and the one rounding of each output
// stays in fp32; the kept z, g and u are rounded copies for the backward pass,
// and the forward's own output is computed from the unrounded values.
#pragma once
#include <cstdint>
#include <type_traits>

#include "epilogues.cuh"
#include "pair_engine.cuh"

namespace flce {

// flce_activation_t (include/flce.h).
enum Activation : int {
  kActNone = 0,
  kActRelu = 1,
  kActGelu = 2,
  kActGeluTanh = 3,
  kActSilu = 4,
  kActSigmoid = 5
};

constexpr float kGeluC = 0.7978845608028654f;    // sqrt(2 / pi)
constexpr float kGeluC3 = 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// 1 / (1 + e^-z) from ex2 and the approximate division: relative error a few
// 2^-22, far below the 16-bit rounding of anything made from it. e^-z
// overflows to +inf for z < -88, and the quotient is then 0, its limit.
__device__ __forceinline__ float sigmoid_f(float z) {
  return __fdividef(1.f, 1.f + fast_exp2(-kLog2e * z));
}
// gelu_tanh: (1 + tanh w) / 2 = 1 / (1 + e^-2w), w = c (z + 0.044715 z^3).
__device__ __forceinline__ float gelu_tanh_gate(float z) {
  return sigmoid_f(2.f * kGeluC * z * fmaf(kGeluC3 * z, z, 1.f));
}
// gelu: Phi(z) = 1 - Q(z) with, for x = |z| / sqrt(2), Q = erfc(x) / 2 and
// erfc(x) = (a1 t + ... + a5 t^5) e^(-x^2) + e, t = 1 / (1 + p x), |e| <= 1.5e-7
// (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26, after
// Hastings). A third of erff's instructions, no branch, and e^(-z^2 / 2) is the
// density that the derivative needs. gauss: e^(-z^2 / 2).
__device__ __forceinline__ float gelu_cdf(float z, float& gauss) {
  const float t = __fdividef(1.f, fmaf(0.3275911f * kInvSqrt2, fabsf(z), 1.f));
  gauss = fast_exp2(-0.5f * kLog2e * z * z);
  float q = fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
  q = fmaf(t, q, 0.5f * 1.421413741f);
  q = fmaf(t, q, 0.5f * -0.284496736f);
  q = fmaf(t, q, 0.5f * 0.254829592f);
  q *= t * gauss;
  return z < 0.f ? q : 1.f - q;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;  // a NaN stays one
  if constexpr (ACT == kActGelu) {
    float gauss;
    return z * gelu_cdf(z, gauss);
  }
  if constexpr (ACT == kActGeluTanh) return z * gelu_tanh_gate(z);
  if constexpr (ACT == kActSilu) return z * sigmoid_f(z);
  if constexpr (ACT == kActSigmoid) return sigmoid_f(z);
  return z;
}

// a(z) and a'(z).
template <int ACT>
__device__ __forceinline__ void act_value_slope(float z, float& val, float& slope) {
  if constexpr (ACT == kActRelu) {
    val = z < 0.f ? 0.f : z;
    slope = z > 0.f ? 1.f : 0.f;
  } else if constexpr (ACT == kActGelu) {
    float gauss;
    const float c = gelu_cdf(z, gauss);
    val = z * c;
    slope = fmaf(z * kInvSqrt2Pi, gauss, c);
  } else if constexpr (ACT == kActGeluTanh) {
    const float p = gelu_tanh_gate(z);
    val = z * p;
    // Beyond |z| = 64 p is 0 or 1 and the second term is 0; its polynomial must not overflow.
    const float zc = fminf(fmaxf(z, -64.f), 64.f);
    slope = fmaf(zc * p * (1.f - p), 2.f * kGeluC * fmaf(3.f * kGeluC3 * zc, zc, 1.f), p);
  } else if constexpr (ACT == kActSilu) {
    const float p = sigmoid_f(z);
    val = z * p;
    slope = fmaf(val, 1.f - p, p);
  } else if constexpr (ACT == kActSigmoid) {
    val = sigmoid_f(z);
    slope = val * (1.f - val);
  } else {
    val = z;
    slope = 1.f;
  }
}

// Calls f with the activation as a compile-time constant: one branch around a
// loop over values, none inside it.
template <class Fn>
__device__ __forceinline__ void with_act(int act, Fn f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>()); return;
    case kActGelu: f(std::integral_constant<int, kActGelu>()); return;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); return;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); return;
    case kActSigmoid: f(std::integral_constant<int, kActSigmoid>()); return;
    default: f(std::integral_constant<int, kActNone>());
  }
}

template <int N>
__device__ __forceinline__ void act_all(int act, float (&v)[N]) {
  with_act(act, [&](auto a) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = act_value<decltype(a)::value>(v[j]);
  });
}

// A 16-bit [rows, cols] output: through a TMA store map of 32 x 32 boxes where
// its rows start on 16-byte boundaries, else by plain stores.
struct Out16 {
  CUtensorMap map;
  uint16_t* ptr;
  int64_t ld;
  int use_map;
};

// As tma_block_16 (epilogues.cuh: the box and its swizzle), through the two buffers
// of the warp's staging.
__device__ __forceinline__ void staged_block_16(const CUtensorMap* map, int x, int y,
                                                const float (&v)[32], bool fp16, Staging& st,
                                                int lane) {
  if (lane == 0) bulk_wait_group_read1();
  __syncwarp();
  uint4* stage = reinterpret_cast<uint4*>(st.buf + st.turn * 2048);
  st.turn ^= 1;
  uint32_t w[16];
  if (fp16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_f16x2(v[2 * j], v[2 * j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    stage[lane * 4 + (q ^ ((lane >> 1) & 3))] =
        make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, stage, x, y);
    bulk_commit_group();
  }
}

// One row (this lane's) of a warp's 32 x 32 block at (row0, col0). Warp-uniform
// but for the values; rows and columns outside the output are clipped.
__device__ __forceinline__ void put_block_16(const Out16& o, int rows, int cols, int row0, int col0,
                                             const float (&v)[32], bool fp16, Staging& st,
                                             int lane) {
  if (row0 >= rows || col0 >= cols) return;
  if (o.use_map) {
    staged_block_16(&o.map, col0, row0, v, fp16, st, lane);
  } else if (row0 + lane < rows) {
    uint16_t* p = o.ptr + static_cast<size_t>(row0 + lane) * o.ld + col0;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (col0 + j < cols) p[j] = to16(v[j], fp16);
  }
}

// Two 16-bit values of a word.
template <bool F16>
__device__ __forceinline__ void unpack_2(uint32_t w, float& lo, float& hi) {
  if constexpr (F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  } else {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
  }
}

// v[j] += src[j] for 32 values at a 16-byte boundary.
template <bool F16>
__device__ __forceinline__ void add_32(const uint16_t* src, float (&v)[32]) {
  uint4 u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) u[q] = reinterpret_cast<const uint4*>(src)[q];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t w[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = q * 8 + 2 * e;
      float lo, hi;
      unpack_2<F16>(w[e], lo, hi);
      f32x2_split(fadd2(f32x2(v[j], v[j + 1]), f32x2(lo, hi)), v[j], v[j + 1]);
    }
  }
}

// The same for the first ncol of a row's 32 columns (16-bit); vec: at a 16-byte boundary.
__device__ __forceinline__ void add_row_16(const uint16_t* src, int ncol, bool vec, bool fp16,
                                           float (&v)[32]) {
  if (vec && ncol >= 32) {
    if (fp16)
      add_32<true>(src, v);
    else
      add_32<false>(src, v);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < ncol) v[j] += unpack_16(src[j], fp16);
  }
}

// The epilogues drain one warp's 32 rows from row0 (lane = row - row0) of its chunks
// of a tile whose columns start at col_base. Chunks come in rising column order, so the
// first one past the output is the last one looked at.

// --------------------------------------------------------- linear: forward
struct LinearArgs {
  const uint16_t* bias;  // [N] or null
  const uint16_t* res;   // [M, ld_res] or null; may be the output itself
  int64_t ld_res;
  int res_vec;           // the residual's rows start on 16-byte boundaries
  int act, fp16, keep;   // keep: also write z
  int M, N;
  Out16 y, z;
};

struct LinearEpi {
  static constexpr bool kAMN = false, kBMN = false;
  static constexpr OperandPlan kPlan = kOneEach;
  using Args = LinearArgs;
  template <class Acc>
  __device__ static void tile(const Args& a, const PairArgs&, int, int row0, int col_base, int lane,
                              const Acc& acc, Staging& st, const TileSlice& sl) {
    const int row = row0 + lane;
    const bool f16 = a.fp16 != 0;
#pragma unroll 1
    for (int c = sl.c_lo; c < sl.c_hi; ++c) {
      int acc_col, col0;
      sl.at(c, acc_col, col0);
      col0 += col_base;
      if (col0 >= a.N || row0 >= a.M) break;  // uniform over the warp
      float v[32];
      acc.load(acc_col, v);
      if (a.bias) add_row_16(a.bias + col0, a.N - col0, true, f16, v);
      if (a.keep) put_block_16(a.z, a.M, a.N, row0, col0, v, f16, st, lane);
      act_all(a.act, v);
      if (a.res && row < a.M)
        add_row_16(a.res + static_cast<size_t>(row) * a.ld_res + col0, a.N - col0, a.res_vec != 0,
                   f16, v);
      put_block_16(a.y, a.M, a.N, row0, col0, v, f16, st, lane);
    }
  }
};

// ---------------------------------------------------------- gated: forward
struct GatedArgs {
  int act, fp16, keep;
  int M, F;
  Out16 h, g, u;
};

struct GatedEpi {
  static constexpr bool kAMN = false, kBMN = false;
  static constexpr OperandPlan kPlan = kTwoB;
  using Args = GatedArgs;
  template <class Acc>
  __device__ static void tile(const Args& a, const PairArgs&, int, int row0, int col_base, int lane,
                              const Acc& acc, Staging& st, const TileSlice& sl) {
    const bool f16 = a.fp16 != 0;
#pragma unroll 1
    for (int c = sl.c_lo; c < sl.c_hi; ++c) {
      int acc_col, col0;
      sl.at(c, acc_col, col0);
      col0 += col_base;
      if (col0 >= a.F || row0 >= a.M) break;  // uniform over the warp
      float g[32], u[32];
      acc.load(acc_col, g);
      acc.load(sl.up_off + acc_col, u);
      if (a.keep) {
        put_block_16(a.g, a.M, a.F, row0, col0, g, f16, st, lane);
        put_block_16(a.u, a.M, a.F, row0, col0, u, f16, st, lane);
      }
      act_all(a.act, g);
#pragma unroll
      for (int j = 0; j < 32; ++j) g[j] *= u[j];
      put_block_16(a.h, a.M, a.F, row0, col0, g, f16, st, lane);
    }
  }
};

// --------------------------------------------------- gradients of both
// dx [M, K] in the operands' type: dz W, or dg Wg + du Wu in one sum.
struct GradXArgs {
  int fp16, M, K;
  Out16 dx;
};

template <OperandPlan PLAN>
struct GradXEpi {
  static constexpr bool kAMN = false, kBMN = true;
  static constexpr OperandPlan kPlan = PLAN;
  using Args = GradXArgs;
  template <class Acc>
  __device__ static void tile(const Args& a, const PairArgs&, int, int row0, int col_base, int lane,
                              const Acc& acc, Staging& st, const TileSlice& sl) {
#pragma unroll 1
    for (int c = sl.c_lo; c < sl.c_hi; ++c) {
      int acc_col, col0;
      sl.at(c, acc_col, col0);
      col0 += col_base;
      if (col0 >= a.K || row0 >= a.M) break;  // uniform over the warp
      float v[32];
      acc.load(acc_col, v);
      put_block_16(a.dx, a.M, a.K, row0, col0, v, a.fp16 != 0, st, lane);
    }
  }
};

// dW [N, K] = dz^T x, in fp32 or the operands' type; with two dz (gated), the
// first m_split row tiles are dWg and the others dWu.
struct GradWArgs {
  CUtensorMap out, out2;
  int out16, fp16;
  int N, K;  // rows of one dW, columns
};

template <OperandPlan PLAN>
struct GradWEpi {
  static constexpr bool kAMN = true, kBMN = true;
  static constexpr OperandPlan kPlan = PLAN;
  using Args = GradWArgs;
  template <class Acc>
  __device__ static void tile(const Args& a, const PairArgs& g, int tm, int row0, int col_base,
                              int lane, const Acc& acc, Staging& st, const TileSlice& sl) {
    const CUtensorMap* out = &a.out;
    if constexpr (PLAN == kTwoA) {
      if (tm >= g.m_split) {
        out = &a.out2;
        row0 -= g.m_split * 256;
      }
    }
#pragma unroll 1
    for (int c = sl.c_lo; c < sl.c_hi; ++c) {
      int acc_col, col0;
      sl.at(c, acc_col, col0);
      col0 += col_base;
      if (col0 >= a.K || row0 >= a.N) break;  // uniform over the warp
      float v[32];
      acc.load(acc_col, v);
      if (a.out16)
        staged_block_16(out, col0, row0, v, a.fp16 != 0, st, lane);
      else
        tma_block_f32(out, col0, row0, v, st.buf, lane);
    }
  }
};

}  // namespace flce
