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

#include "epilogues.cuh"

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
__device__ __forceinline__ float gelu_cdf(float z) { return fmaf(0.5f, erff(z * kInvSqrt2), 0.5f); }

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;  // a NaN stays one
    case kActGelu: return z * gelu_cdf(z);
    case kActGeluTanh: return z * gelu_tanh_gate(z);
    case kActSilu: return z * sigmoid_f(z);
    case kActSigmoid: return sigmoid_f(z);
    default: return z;
  }
}

// a(z) and a'(z).
__device__ __forceinline__ void act_value_slope(int act, float z, float& val, float& slope) {
  switch (act) {
    case kActRelu:
      val = z < 0.f ? 0.f : z;
      slope = z > 0.f ? 1.f : 0.f;
      return;
    case kActGelu: {
      const float c = gelu_cdf(z);
      val = z * c;
      slope = fmaf(z * kInvSqrt2Pi, fast_exp2(-0.5f * kLog2e * z * z), c);
      return;
    }
    case kActGeluTanh: {
      const float p = gelu_tanh_gate(z);
      val = z * p;
      // Beyond |z| = 64 p is 0 or 1 and the second term is 0; its polynomial must not overflow.
      const float zc = fminf(fmaxf(z, -64.f), 64.f);
      slope = fmaf(zc * p * (1.f - p), 2.f * kGeluC * fmaf(3.f * kGeluC3 * zc, zc, 1.f), p);
      return;
    }
    case kActSilu: {
      const float p = sigmoid_f(z);
      val = z * p;
      slope = fmaf(val, 1.f - p, p);
      return;
    }
    case kActSigmoid: {
      val = sigmoid_f(z);
      slope = val * (1.f - val);
      return;
    }
    default:
      val = z;
      slope = 1.f;
  }
}

// The activation of 32 values: one branch for the chunk, not one per value.
__device__ __forceinline__ void act_32(int act, float (&v)[32]) {
  switch (act) {
    case kActNone: return;
    case kActRelu:
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = act_value(kActRelu, v[j]);
      return;
    case kActGelu:
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = act_value(kActGelu, v[j]);
      return;
    case kActGeluTanh:
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = act_value(kActGeluTanh, v[j]);
      return;
    case kActSilu:
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = act_value(kActSilu, v[j]);
      return;
    default:
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = act_value(kActSigmoid, v[j]);
  }
}

// A 16-bit [rows, cols] output: through a TMA store map of 32 x 32 boxes where
// its rows start on 16-byte boundaries, else by plain stores.
struct Out16 {
  CUtensorMap map;
  uint16_t* ptr;
  int64_t ld;
  int use_map;
};

// One row (this lane's) of a warp's 32 x 32 block at (row0, col0). Warp-uniform
// but for the values; rows and columns outside the output are clipped.
__device__ __forceinline__ void put_block_16(const Out16& o, int rows, int cols, int row0, int col0,
                                             const float (&v)[32], bool fp16, void* stage,
                                             int lane) {
  if (row0 >= rows || col0 >= cols) return;
  if (o.use_map) {
    tma_block_16(&o.map, col0, row0, v, fp16, stage, lane);
  } else if (row0 + lane < rows) {
    uint16_t* p = o.ptr + static_cast<size_t>(row0 + lane) * o.ld + col0;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (col0 + j < cols) p[j] = to16(v[j], fp16);
  }
}

// v[j] += src[j] of one row's 32 columns (16-bit); vec: 16-byte loads allowed.
__device__ __forceinline__ void add_row_16(const uint16_t* src, int ncol, bool vec, bool fp16,
                                           float (&v)[32]) {
  if (vec && ncol >= 32) {
    const uint4* p = reinterpret_cast<const uint4*>(src);
    uint4 u[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = p[q];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t w[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[q * 8 + 2 * e] += unpack_16(w[e] & 0xFFFFu, fp16);
        v[q * 8 + 2 * e + 1] += unpack_16(w[e] >> 16, fp16);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < ncol) v[j] += unpack_16(src[j], fp16);
  }
}

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
  static constexpr int kWideWarps = 8, kStageNeed = 32 * 32 * 2;
  using Args = LinearArgs;
  __device__ static void tile(const Args& a, const GemmGeom&, int tm, int tn, int row_in_tile,
                              int lane, int quad, uint32_t taddr, void* stage,
                              const EpiSlice& sl) {
    const int row = tm * kBM + row_in_tile, row0 = tm * kBM + quad * 32;
    const bool f16 = a.fp16 != 0;
#pragma unroll 1
    for (int c = sl.c_lo; c < sl.c_hi; ++c) {
      const int col0 = tn * kBN + c * 32;
      if (col0 >= a.N || row0 >= a.M) break;  // uniform over the warp
      float v[32];
      tmem_ld_32cols(taddr + c * 32, v);
      if (a.bias) {
        float bv[32];
        load_bias32<true>(a.bias, col0, a.N, bv, f16);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += bv[j];
      }
      if (a.keep) put_block_16(a.z, a.M, a.N, row0, col0, v, f16, stage, lane);
      act_32(a.act, v);
      if (a.res && row < a.M)
        add_row_16(a.res + static_cast<size_t>(row) * a.ld_res + col0, a.N - col0, a.res_vec != 0,
                   f16, v);
      put_block_16(a.y, a.M, a.N, row0, col0, v, f16, stage, lane);
    }
  }
};

// ---------------------------------------------------------- gated: forward
struct GatedArgs {
  SecondOperand second;  // b2: Wu
  int act, fp16, keep;
  int M, F;
  Out16 h, g, u;
};

struct GatedEpi {
  static constexpr bool kAMN = false, kBMN = false;
  static constexpr OperandPlan kPlan = kTwoB;
  static constexpr int kWideWarps = 8, kStageNeed = 32 * 32 * 2;
  using Args = GatedArgs;
  __device__ static void tile(const Args& a, const GemmGeom&, int tm, int tn, int, int lane,
                              int quad, uint32_t taddr, void* stage, const EpiSlice& sl) {
    const int row0 = tm * kBM + quad * 32;
    const bool f16 = a.fp16 != 0;
#pragma unroll 1
    for (int c = sl.c_lo; c < sl.c_hi; ++c) {
      const int col0 = tn * sl.up_off + c * 32;
      if (col0 >= a.F || row0 >= a.M) break;  // uniform over the warp
      float g[32], u[32];
      tmem_ld_32cols(taddr + c * 32, g);
      tmem_ld_32cols(taddr + sl.up_off + c * 32, u);
      if (a.keep) {
        put_block_16(a.g, a.M, a.F, row0, col0, g, f16, stage, lane);
        put_block_16(a.u, a.M, a.F, row0, col0, u, f16, stage, lane);
      }
      act_32(a.act, g);
#pragma unroll
      for (int j = 0; j < 32; ++j) g[j] *= u[j];
      put_block_16(a.h, a.M, a.F, row0, col0, g, f16, stage, lane);
    }
  }
};

// --------------------------------------------------- gradients of both
// dx [M, K] in the operands' type: dz W, or dg Wg + du Wu in one sum.
struct GradXArgs {
  SecondOperand second;
  int fp16, M, K;
  Out16 dx;
};

template <OperandPlan PLAN>
struct GradXEpi {
  static constexpr bool kAMN = false, kBMN = true;
  static constexpr OperandPlan kPlan = PLAN;
  static constexpr int kWideWarps = 8, kStageNeed = 32 * 32 * 2;
  using Args = GradXArgs;
  __device__ static void tile(const Args& a, const GemmGeom&, int tm, int tn, int, int lane,
                              int quad, uint32_t taddr, void* stage, const EpiSlice& sl) {
    const int row0 = tm * kBM + quad * 32;
#pragma unroll 1
    for (int c = sl.c_lo; c < sl.c_hi; ++c) {
      const int col0 = tn * kBN + c * 32;
      if (col0 >= a.K || row0 >= a.M) break;  // uniform over the warp
      float v[32];
      tmem_ld_32cols(taddr + c * 32, v);
      put_block_16(a.dx, a.M, a.K, row0, col0, v, a.fp16 != 0, stage, lane);
    }
  }
};

// dW [N, K] = dz^T x, in fp32 or the operands' type; with two dz (gated), the
// first m_split 256-row tiles are dWg and the others dWu.
struct GradWArgs {
  SecondOperand second;
  CUtensorMap out, out2;
  int out16, fp16;
  int N, K;  // rows of one dW, columns
};

template <OperandPlan PLAN>
struct GradWEpi {
  static constexpr bool kAMN = true, kBMN = true;
  static constexpr OperandPlan kPlan = PLAN;
  static constexpr int kWideWarps = 8, kStageNeed = 32 * 32 * 4;
  using Args = GradWArgs;
  __device__ static void tile(const Args& a, const GemmGeom&, int tm, int tn, int, int lane,
                              int quad, uint32_t taddr, void* stage, const EpiSlice& sl) {
    const CUtensorMap* out = &a.out;
    int row0 = tm * kBM + quad * 32;
    if constexpr (PLAN == kTwoA) {
      if (tm >= 2 * a.second.m_split) {
        out = &a.out2;
        row0 -= 2 * a.second.m_split * kBM;
      }
    }
#pragma unroll 1
    for (int c = sl.c_lo; c < sl.c_hi; ++c) {
      const int col0 = tn * kBN + c * 32;
      if (col0 >= a.K || row0 >= a.N) break;  // uniform over the warp
      float v[32];
      tmem_ld_32cols(taddr + c * 32, v);
      if (a.out16)
        tma_block_16(out, col0, row0, v, a.fp16 != 0, stage, lane);
      else
        tma_block_f32(out, col0, row0, v, stage, lane);
    }
  }
};

}  // namespace flce
