// Activations and GEMM epilogues of the layer operators: the linear layer
// (bias, activation, residual), the gated feed-forward projection, and the
// gradients of both.
//
//   linear   z = x W^T + b,  y = a(z) + r
//   gated    g = x Wg^T, u = x Wu^T,  h = a(g) u
//
// Everything between the fp32 accumulator and the one rounding of each output
// stays in fp32.
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

// Activations work on packed fp32 pairs: an epilogue beside a short sum is bound by its
// instructions, and a packed one does the work of two.
__device__ __forceinline__ uint64_t splat(float c) { return f32x2(c, c); }
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint64_t rcp2(uint64_t x) {
  float a, b;
  f32x2_split(x, a, b);
  return f32x2(rcp_approx(a), rcp_approx(b));
}
__device__ __forceinline__ uint64_t exp2_2(uint64_t x) {
  float a, b;
  f32x2_split(x, a, b);
  return f32x2(fast_exp2(a), fast_exp2(b));
}
// 1 / (1 + e^-z) from ex2 and the approximate reciprocal: relative error (|z| + 4) 2^-24 for
// negative z, whose exponent is rounded to fp32 (5e-6 at z = -87), and 2^-22 above, far
// below the 16-bit rounding of anything made from it. 0 under z = -87.3, where fp32's normal
// numbers end (e^-z overflows to +inf soon after, and its reciprocal is 0).
__device__ __forceinline__ uint64_t sigmoid2(uint64_t z) {
  return rcp2(fadd2(exp2_2(fmul2(z, splat(-kLog2e))), splat(1.f)));
}
// Phi(z) = Q(|z|) below 0 and 1 - Q(|z|) above, Q(x) = erfc(x / sqrt(2)) / 2 = P(t) e^(-x^2 / 2)
// with t = 1 / (1 + p x). P, of degree 6 without a constant term, is fitted to the least
// largest relative error of Q: 1.3e-6 up to x = 2.5, 1e-5 to 6, 8e-5 to 14, so that the negative
// tail of gelu keeps its relative precision. A third of erff's instructions, no branch, and
// e^(-z^2 / 2) is the density that the derivative needs. gauss: e^(-z^2 / 2).
__device__ __forceinline__ uint64_t gelu_cdf2(uint64_t z, uint64_t& gauss) {
  constexpr uint64_t kSign = 0x8000000080000000ull;
  const uint64_t t = rcp2(ffma2(z & ~kSign, splat(0.296984851f), splat(1.f)));
  gauss = exp2_2(fmul2(fmul2(z, z), splat(-0.5f * kLog2e)));
  uint64_t q = ffma2(t, splat(-0.0836496651f), splat(0.244700462f));
  q = ffma2(t, q, splat(-0.0478213876f));
  q = ffma2(t, q, splat(0.158557892f));
  q = ffma2(t, q, splat(0.109055996f));
  q = ffma2(t, q, splat(0.119156331f));
  q = fmul2(fmul2(q, t), gauss);
  float a, b, qa, qb, ra, rb;
  f32x2_split(z, a, b);
  f32x2_split(q, qa, qb);
  f32x2_split(ffma2(q, splat(-1.f), splat(1.f)), ra, rb);
  return f32x2(a < 0.f ? qa : ra, b < 0.f ? qb : rb);
}
// gelu_tanh: (1 + tanh w) / 2 = 1 / (1 + e^-2w), w = c (z + 0.044715 z^3).
__device__ __forceinline__ uint64_t gelu_tanh_gate2(uint64_t z) {
  return sigmoid2(
      fmul2(fmul2(z, splat(2.f * kGeluC)), ffma2(fmul2(z, z), splat(kGeluC3), splat(1.f))));
}

// a(z) and a'(z) of two values.
template <int ACT>
__device__ __forceinline__ void act2(uint64_t z, uint64_t& val, uint64_t& slope) {
  if constexpr (ACT == kActRelu) {
    float a, b;
    f32x2_split(z, a, b);
    val = f32x2(a < 0.f ? 0.f : a, b < 0.f ? 0.f : b);  // a NaN stays one
    slope = f32x2(a > 0.f ? 1.f : 0.f, b > 0.f ? 1.f : 0.f);
  } else if constexpr (ACT == kActGelu) {
    uint64_t gauss;
    const uint64_t c = gelu_cdf2(z, gauss);
    val = fmul2(z, c);
    slope = ffma2(fmul2(z, splat(kInvSqrt2Pi)), gauss, c);
  } else if constexpr (ACT == kActGeluTanh) {
    const uint64_t p = gelu_tanh_gate2(z);
    val = fmul2(z, p);
    // Beyond |z| = 64 p is 0 or 1 and the second term is 0; its polynomial must not overflow.
    float a, b;
    f32x2_split(z, a, b);
    const uint64_t zc = f32x2(fminf(fmaxf(a, -64.f), 64.f), fminf(fmaxf(b, -64.f), 64.f));
    const uint64_t poly =
        ffma2(fmul2(zc, zc), splat(6.f * kGeluC * kGeluC3), splat(2.f * kGeluC));
    slope = ffma2(fmul2(fmul2(zc, p), ffma2(p, splat(-1.f), splat(1.f))), poly, p);
  } else if constexpr (ACT == kActSilu) {
    const uint64_t p = sigmoid2(z);
    val = fmul2(z, p);
    slope = ffma2(val, ffma2(p, splat(-1.f), splat(1.f)), p);
  } else if constexpr (ACT == kActSigmoid) {
    // With e = e^-|z| and r = 1 / (1 + e): sigmoid is r above 0 and e r below, its slope e r^2 on
    // both sides. 1 - r would lose it where r rounds to 1.
    constexpr uint64_t kSign = 0x8000000080000000ull;
    const uint64_t e = exp2_2(fmul2(z | kSign, splat(kLog2e))), r = rcp2(fadd2(e, splat(1.f)));
    const uint64_t er = fmul2(e, r);
    float a, b, ra, rb, ea, eb;
    f32x2_split(z, a, b);
    f32x2_split(r, ra, rb);
    f32x2_split(er, ea, eb);
    val = f32x2(a < 0.f ? ea : ra, b < 0.f ? eb : rb);
    slope = fmul2(er, r);
  } else {
    val = z;
    slope = splat(1.f);
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

// v = a(v).
template <int N>
__device__ __forceinline__ void act_all(int act, float (&v)[N]) {
  if (act == kActNone) return;
  with_act(act, [&](auto a) {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      uint64_t val, slope;
      act2<decltype(a)::value>(f32x2(v[j], v[j + 1]), val, slope);
      f32x2_split(val, v[j], v[j + 1]);
    }
  });
}

// ------------------------------------------------------- kept for the backward
// The backward's error should be that of its own roundings. What the forward keeps in 16
// bits a value takes one of two forms (flce_keep_t).
//
// Linear: the slope a'(z), which lies in (-0.13, 1.13) for every activation, as a fixed
// point number of 2^-15 steps from -0.25 (0 and 1 are exact; 65535: NaN). Far from 0 that is
// finer than the operands' types; the slope of a saturated unit is lost in it.
// FLCE_KEEP_RELATIVE: below 2^-6 the slopes of a saturated unit (sigmoid: all; the others: z
// under -2) take the codes that the fixed form leaves unused, as floating point numbers of 9
// bits: 45312 + the bits above the 14th of |a'| 2^-82, which go on with the fixed form's step at
// 2^-6, are off by 2^-10 of the slope down to 2^-44 and by 2^-54 below. Around the zeros of
// a' at z = -1.3 .. -0.7 the steps stay fixed. Every other code is that of the fixed form.
//
// Gated: a(g) and u a'(g), whose range has no bound, in groups of 8 columns that share
// an exponent: value = q 2^(eb - 140) 16384 / 16383, q a 15-bit integer, eb the exponent
// field of the group's largest magnitude, at least 14. A value's word is 2 q + bit j of
// eb, j its place in the group, so that a 16-byte load holds all it needs. An infinity or NaN
// is q = -16384, reads as NaN and leaves its neighbours alone: eb is that of the largest finite
// one. Off by at most 2^-14 of the largest, whatever their own size.
// FLCE_KEEP_RELATIVE: the same groups, with value 2^(126 - eb), of magnitude 1 at most, as an fp16
// number, whose second highest bit is then 0 and makes room for bit j of eb. Off by 2^-11 of
// the value itself or, under 2^-13 of the group's largest, by 2^-24 of that: the rounding of
// fp16 operands, an eighth of bf16's. (14 bits of magnitude as steps of 2^-13 above 1/8 and 10-bit
// numbers below took 10 us more of 55 at 1834 x 512 x 11208 and were 0.2 % off beside a feature
// 1000 times as large.) An infinity or NaN has 14 low bits of ones.
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr float kRound = 12582912.f;  // 1.5 * 2^23: x + kRound holds round(x) in its low bits

// Codes of two slopes in one word.
__device__ __forceinline__ uint32_t encode_slopes(uint64_t s) {
  float a, b;
  f32x2_split(ffma2(s, splat(32768.f), splat(kRound + 8192.f)), a, b);
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410);
}

constexpr uint32_t kTailCode = 45312u;  // above the fixed code of any slope, (1.13 + 0.25) 2^15
template <int ACT>
__device__ __forceinline__ uint32_t encode_slopes_relative(uint64_t z, uint64_t s) {
  constexpr uint64_t kSign = 0x8000000080000000ull;
  constexpr uint32_t kAdd = 0x2000u + (kTailCode << 14);  // rounds, and moves to the codes
  float za, zb, sa, sb, ta, tb, fa, fb;
  f32x2_split(z, za, zb);
  f32x2_split(s, sa, sb);
  f32x2_split(fmul2(s & ~kSign, splat(0x1p-82f)), ta, tb);
  f32x2_split(ffma2(s, splat(32768.f), splat(kRound + 8192.f)), fa, fb);
  // Not of a NaN: no comparison holds.
  const bool low_a = ACT == kActSigmoid ? sa < 0x1p-6f : sa > -0x1p-6f && za < -2.f;
  const bool low_b = ACT == kActSigmoid ? sb < 0x1p-6f : sb > -0x1p-6f && zb < -2.f;
  return __byte_perm(low_a ? (__float_as_uint(ta) + kAdd) >> 14 : __float_as_uint(fa),
                     low_b ? (__float_as_uint(tb) + kAdd) >> 14 : __float_as_uint(fb), 0x5410);
}

// v = a(v), and the codes of the slopes.
template <int ACT, bool RELATIVE, int N>
__device__ __forceinline__ void act_keep_slopes(float (&v)[N], uint32_t (&w)[N / 2]) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    uint64_t val, slope;
    const uint64_t z = f32x2(v[j], v[j + 1]);
    act2<ACT>(z, val, slope);
    if constexpr (RELATIVE && ACT != kActNone && ACT != kActRelu)
      w[j / 2] = encode_slopes_relative<ACT>(z, slope);
    else
      w[j / 2] = encode_slopes(slope);
    f32x2_split(val, v[j], v[j + 1]);
  }
}
// v = a(v), and x = u a'(v).
template <int N>
__device__ __forceinline__ void act_cross(int act, float (&v)[N], const float (&u)[N], float (&x)[N]) {
  with_act(act, [&](auto a) {
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      uint64_t val, slope;
      act2<decltype(a)::value>(f32x2(v[j], v[j + 1]), val, slope);
      f32x2_split(val, v[j], v[j + 1]);
      f32x2_split(fmul2(f32x2(u[j], u[j + 1]), slope), x[j], x[j + 1]);
    }
  });
}
// A kept slope in either form. tail: 2^82, with the sign that the activation's slope has where
// the unit is saturated.
__device__ __forceinline__ float decode_slope(uint32_t code, float tail) {
  const float q = __uint_as_float(0x4B000000u + code) - 8388608.f;
  const float low = __uint_as_float((code - kTailCode) << 14) * tail;
  const float v = code >= kTailCode ? low : fmaf(q, 1.f / 32768.f, -0.25f);
  return code == 65535u ? __uint_as_float(0x7FFFFFFFu) : v;
}

__device__ __forceinline__ uint32_t largest_bits(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  return m;
}
// The words of 8 values whose largest finite magnitude has the bits m.
__device__ __forceinline__ uint4 group_words(const float* v, uint32_t m) {
  const uint32_t eb = max(m >> 23, 14u);
  const float scale = __uint_as_float((267u - eb) << 23) * (16383.f / 16384.f);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x, y;
    f32x2_split(ffma2(f32x2(v[2 * i], v[2 * i + 1]), splat(scale), splat(kRound)), x, y);
    const uint32_t t = eb >> (2 * i);
    w[i] = ((__byte_perm(__float_as_uint(x), __float_as_uint(y), 0x5410) << 1) & 0xFFFEFFFEu) |
           (t & 1u) | ((t & 2u) << 15);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 2^x of an exponent field f = x + 127, below 1 too (x = -127, -128).
__device__ __forceinline__ float exp2_of_field(int f) {
  return __uint_as_float(f > 0 ? static_cast<uint32_t>(f) << 23 : 0x00800000u >> (1 - f));
}
// The same in the relative form.
__device__ __forceinline__ uint4 group_words_relative(const float* v, uint32_t m) {
  const uint32_t eb = max(m >> 23, 1u);
  const uint64_t scale = splat(exp2_of_field(253 - static_cast<int>(eb)));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f32x2_split(fmul2(f32x2(v[2 * i], v[2 * i + 1]), scale), a, b);
    const uint32_t t = eb >> (2 * i);
    w[i] = (pack_f16x2(a, b) & 0xBFFFBFFFu) | ((t & 1u) << 14) | ((t & 2u) << 29);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// A group's words, its exponent that of the largest finite value.
template <bool RELATIVE>
__device__ __forceinline__ uint4 group_words_any(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    m = max(m, b < kInfBits ? b : 0u);
  }
  const uint4 u = RELATIVE ? group_words_relative(v, m) : group_words(v, m);
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if ((__float_as_uint(v[j]) & 0x7FFFFFFFu) < kInfBits) continue;
    const int at = 16 * (j & 1);
    w[j / 2] = RELATIVE ? w[j / 2] | (0x3FFFu << at)
                        : (w[j / 2] & ~(0xFFFEu << at)) | (0x8000u << at);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The words of N values. One branch for all of them: one for each group kept the groups'
// instructions apart (1834 x 512 x 11208 with kept values 55 us, 61 us).
template <bool RELATIVE, int N>
__device__ __forceinline__ void encode_groups_as(const float (&v)[N], uint32_t (&w)[N / 2]) {
  uint32_t m[N / 8], most = 0;
#pragma unroll
  for (int q = 0; q < N / 8; ++q) {
    m[q] = largest_bits(&v[8 * q]);
    most = max(most, m[q]);
  }
  const auto put = [&](int q, const uint4& u) {
    w[4 * q] = u.x;
    w[4 * q + 1] = u.y;
    w[4 * q + 2] = u.z;
    w[4 * q + 3] = u.w;
  };
  if (most < kInfBits) {
#pragma unroll
    for (int q = 0; q < N / 8; ++q)
      put(q, RELATIVE ? group_words_relative(&v[8 * q], m[q]) : group_words(&v[8 * q], m[q]));
  } else {
#pragma unroll
    for (int q = 0; q < N / 8; ++q) put(q, group_words_any<RELATIVE>(&v[8 * q]));
  }
}
template <int N>
__device__ __forceinline__ void encode_groups(bool relative, const float (&v)[N],
                                              uint32_t (&w)[N / 2]) {
  if (relative)
    encode_groups_as<true>(v, w);
  else
    encode_groups_as<false>(v, w);
}
// v, or NaN where the word in the upper half of w says so.
__device__ __forceinline__ float kept_number(uint32_t w, float v) {
  return (w >> 17) == 0x4000u ? __uint_as_float(0x7FFFFFFFu) : v;
}
__device__ __forceinline__ void decode_group_relative(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t eb = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) eb |= (((w[i] >> 14) & 1u) | ((w[i] >> 29) & 2u)) << (2 * i);
  const float scale = __uint_as_float(eb << 23);  // 2^(eb - 127)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = w[i] & 0xBFFFBFFFu;
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const float nan = __uint_as_float(0x7FFFFFFFu);
    v[2 * i] = (h & 0x3FFFu) == 0x3FFFu ? nan : 2.f * f.x * scale;
    v[2 * i + 1] = ((h >> 16) & 0x3FFFu) == 0x3FFFu ? nan : 2.f * f.y * scale;
  }
}
__device__ __forceinline__ void decode_group(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t eb = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) eb |= ((w[i] & 1u) | ((w[i] >> 15) & 2u)) << (2 * i);
  const float inv = __uint_as_float((eb - 13u) << 23) * (16384.f / 16383.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = static_cast<uint32_t>(static_cast<int32_t>(w[i] << 16) >> 17);
    const uint32_t hi = static_cast<uint32_t>(static_cast<int32_t>(w[i]) >> 17);
    v[2 * i] = kept_number(w[i] << 16, (__uint_as_float(0x4B400000u + lo) - kRound) * inv);
    v[2 * i + 1] = kept_number(w[i], (__uint_as_float(0x4B400000u + hi) - kRound) * inv);
  }
}

// --------------------------------------------------------- signs of relu's inputs
// relu's slope jumps at 0, so there the sign of a sum is the whole gradient. The tensor core
// drops the low bits of its running sum at every step of 16 products (off by 1.9e-5 of the sums'
// size after 16384 of them; 1.5e-6 with fp32 adds that round): one element in a million came
// out on the wrong side of 0, which put fp16 gradients of 5942 x 6456 x 1408 0.0023 of their
// size from 64 bits, where 32-bit sums are 0.0005 from them. A forward that keeps relu's
// slopes therefore takes the sign of a sum that is no further from 0 than its own error from
// the products once more, added in fp32. (Its value is that of the tensor core all the same.)
//
// The error: 2^-24 of the largest sum for each step, of this row's sums and of this column's. A
// warp that still has more than kMaxAgain such sums takes them as they are: they are no accident
// then, and each costs K products of one warp.
constexpr int kMaxAgain = 4;
__device__ __forceinline__ float sum_error(float largest, int K) {
  return largest * (static_cast<float>(K / 16 + 8) * 0x1p-24f);
}

template <int N>
__device__ __forceinline__ float largest_of(const float (&v)[N]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < N; j += 2) m = fmax3(m, fabsf(v[j]), fabsf(v[j + 1]));
  return m;
}
// Bit j: z[j] is not 0 but within the error of a sum of K products in this row.
template <int N>
__device__ __forceinline__ uint32_t near_zero(const float (&z)[N], float largest, int K) {
  const float off = sum_error(largest, K);
  float least = off;
#pragma unroll
  for (int j = 0; j < N; j += 2) least = fmin3(least, fabsf(z[j]), fabsf(z[j + 1]));
  uint32_t near = 0;
  if (least < off) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (fabsf(z[j]) < off && z[j] != 0.f) near |= 1u << j;
  }
  return near;
}
// Clears the bits of sums that are small as all of their column are, whose error is as much
// smaller. By the whole warp, a row to a lane.
__device__ __forceinline__ void near_zero_of_column(const float (&z)[32], int K, uint32_t& near) {
  const uint32_t columns = __reduce_or_sync(0xffffffffu, near);
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (((columns >> j) & 1u) == 0) continue;
    const float size = fabsf(z[j]);
    const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(size)));
    if (size >= sum_error(most, K)) near &= ~(1u << j);
  }
}
struct SignArgs {
  const uint16_t *x, *W;  // [M, ld_x]; [N, K]
  const uint16_t* bias;   // or null
  int64_t ld_x;
  int K;
};
// Bit j: the sum of this lane's row and column col + j is above 0, for the bits of `near`, which
// is cleared where there are too many. By the whole warp.
__device__ __forceinline__ uint32_t signs_again(const SignArgs& a, bool f16, int row, int col,
                                                uint32_t& near, int lane) {
  uint32_t above = 0;
  if (__reduce_add_sync(0xffffffffu, __popc(near)) > kMaxAgain) near = 0;
  uint32_t left = near;
  for (unsigned todo = __ballot_sync(0xffffffffu, left != 0); todo != 0;
       todo = __ballot_sync(0xffffffffu, left != 0)) {
    const int src = __ffs(static_cast<int>(todo)) - 1;
    const int j = __ffs(static_cast<int>(__shfl_sync(0xffffffffu, left, src))) - 1;
    const int r = __shfl_sync(0xffffffffu, row, src), c = __shfl_sync(0xffffffffu, col, src) + j;
    const uint16_t* x = a.x + static_cast<size_t>(r) * a.ld_x;
    const uint16_t* w = a.W + static_cast<size_t>(c) * a.K;
    float s[4] = {};
#pragma unroll 2
    for (int k = lane * 8; k < a.K; k += 256) {
      const uint4 xv = *reinterpret_cast<const uint4*>(x + k);
      const uint4 wv = *reinterpret_cast<const uint4*>(w + k);
      const uint32_t p[4] = {xv.x, xv.y, xv.z, xv.w}, q[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] = fmaf(unpack_16(p[e] & 0xFFFFu, f16), unpack_16(q[e] & 0xFFFFu, f16), s[e]);
        s[e] = fmaf(unpack_16(p[e] >> 16, f16), unpack_16(q[e] >> 16, f16), s[e]);
      }
    }
    float z = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (a.bias) z += unpack_16(a.bias[c], f16);
    if (lane == src) {
      left &= left - 1;
      if (z > 0.f) above |= 1u << j;
    }
  }
  return above;
}
// The codes of relu's slopes, with those of `near` as `above` says.
template <int N>
__device__ __forceinline__ void put_signs(uint32_t near, uint32_t above, uint32_t (&w)[N]) {
#pragma unroll
  for (int j = 0; j < 2 * N; ++j)
    if ((near >> j) & 1u)
      w[j / 2] = __byte_perm(w[j / 2], ((above >> j) & 1u) ? 0xA000u : 0x2000u,
                             (j & 1) ? 0x5410 : 0x3254);
}

// What a forward keeps, as a compile-time constant: the loops over a tile's columns are made for
// each, so that one's registers and branches do not slow another down. The arguments' `keep`: 0
// nothing, 1 the fixed form, 2 the relative one.
enum Keep : int { kKeepNone = 0, kKeepFixed = 1, kKeepRelative = 2, kKeepSigns = 3 };
template <class Fn>
__device__ __forceinline__ void with_keep(int keep, int act, Fn f) {
  if (keep == 0)
    f(std::integral_constant<int, kKeepNone>());
  else if (act == kActRelu)
    f(std::integral_constant<int, kKeepSigns>());  // the slopes 0 and 1 are the same in both forms
  else if (keep == 2)
    f(std::integral_constant<int, kKeepRelative>());
  else
    f(std::integral_constant<int, kKeepFixed>());
}

// A 16-bit [rows, cols] output: through a TMA store map of 32 x 32 boxes where
// its rows start on 16-byte boundaries (all but the linear layer's always do), else by
// plain stores.
struct Out16 {
  CUtensorMap map;
  uint16_t* ptr;
  int64_t ld;
  int use_map;
};

// A row's 32 values (this lane's) of a 32 x 32 16-bit block, two to a word.
__device__ __forceinline__ void pack_32(const float (&v)[32], bool fp16, uint32_t (&w)[16]) {
  if (fp16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_f16x2(v[2 * j], v[2 * j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
  }
}

// As tma_block_16 (epilogues.cuh: the box and its swizzle), through the two buffers
// of the warp's staging.
__device__ __forceinline__ void staged_block_16(const CUtensorMap* map, int x, int y,
                                                const uint32_t (&w)[16], Staging& st, int lane) {
  if (lane == 0) bulk_wait_group_read1();
  __syncwarp();
  uint4* stage = reinterpret_cast<uint4*>(st.buf + st.turn * 2048);
  st.turn ^= 1;
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

// A warp's 32 x 32 block of 16-bit values through its staging memory, between rows that lie
// one to a lane and global rows off the 16-byte boundaries. There half a warp takes a
// row, a word of two columns to a lane: 64 bytes of a row at a time, where a lane to a
// row touched 32 rows with every access (2691 x 504 x 7098 with bias and gelu 191 us, 54 us;
// 7104 columns take 41 us).
struct RowBlock {
  uint32_t* words;  // 16 words a row, the 64-byte swizzle of staged_block_16
  // One buffer of the staging, when no bulk store reads it or writes to it any more.
  __device__ __forceinline__ RowBlock(Staging& st, int lane) {
    if (lane == 0) bulk_wait_group_read0();
    __syncwarp();
    words = reinterpret_cast<uint32_t*>(st.buf + st.turn * 2048);
    st.turn ^= 1;
  }
  __device__ __forceinline__ uint4* chunk(int row, int q) const {
    return reinterpret_cast<uint4*>(words) + row * 4 + (q ^ ((row >> 1) & 3));
  }
  __device__ __forceinline__ uint32_t* word(int row, int j) const {
    return words + row * 16 + (((j >> 2) ^ ((row >> 1) & 3)) << 2) + (j & 3);
  }
};
// Words of two columns of p with pitch ld lie on 4-byte boundaries (columns from an even one).
__device__ __forceinline__ bool on_words(const uint16_t* p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) >> 1 | static_cast<uintptr_t>(ld)) & 1) == 0;
}
__device__ __forceinline__ void store_rows(uint16_t* p, int64_t ld, int rows, int cols, int row0,
                                           int col0, const uint32_t (&w)[16], Staging& st,
                                           int lane) {
  const RowBlock b(st, lane);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *b.chunk(lane, q) = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  __syncwarp();
  const bool pairs = on_words(p, ld);
  const int j = lane & 15, n = cols - col0 - 2 * j;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = 2 * i + (lane >> 4);
    if (row0 + r >= rows || n <= 0) continue;
    const uint32_t v = *b.word(r, j);
    uint16_t* to = p + static_cast<size_t>(row0 + r) * ld + col0 + 2 * j;
    if (pairs && n >= 2) {
      *reinterpret_cast<uint32_t*>(to) = v;
    } else {
      to[0] = static_cast<uint16_t>(v);
      if (n >= 2) to[1] = static_cast<uint16_t>(v >> 16);
    }
  }
  __syncwarp();
}
// v += the block of p, zeros outside it.
__device__ __forceinline__ void add_rows(const uint16_t* p, int64_t ld, int rows, int cols,
                                         int row0, int col0, bool fp16, float (&v)[32],
                                         Staging& st, int lane) {
  const RowBlock b(st, lane);
  const bool pairs = on_words(p, ld);
  const int j = lane & 15, n = cols - col0 - 2 * j;
  uint32_t in[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = 2 * i + (lane >> 4);
    in[i] = 0u;
    if (row0 + r >= rows || n <= 0) continue;
    const uint16_t* from = p + static_cast<size_t>(row0 + r) * ld + col0 + 2 * j;
    if (pairs && n >= 2)
      in[i] = *reinterpret_cast<const uint32_t*>(from);
    else
      in[i] = from[0] | (n >= 2 ? static_cast<uint32_t>(from[1]) << 16 : 0u);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) *b.word(2 * i + (lane >> 4), j) = in[i];
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 u = *b.chunk(lane, q);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[8 * q + 2 * e] += unpack_16(w[e] & 0xFFFFu, fp16);
      v[8 * q + 2 * e + 1] += unpack_16(w[e] >> 16, fp16);
    }
  }
  __syncwarp();
}

// One row (this lane's) of a warp's 32 x 32 block at (row0, col0) inside the output, whose
// rows and columns beyond its own are clipped.
__device__ __forceinline__ void put_words(const Out16& o, int rows, int cols, int row0, int col0,
                                          const uint32_t (&w)[16], Staging& st, int lane) {
  if (o.use_map)
    staged_block_16(&o.map, col0, row0, w, st, lane);
  else
    store_rows(o.ptr, o.ld, rows, cols, row0, col0, w, st, lane);
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

// v[j] += src[j] for the first ncol of a row's 32 columns (FULL: all); src at a 16-byte
// boundary.
template <bool F16, bool FULL>
__device__ __forceinline__ void add_cols(const uint16_t* src, int ncol, float (&v)[32]) {
  uint4 u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    u[q] = make_uint4(0u, 0u, 0u, 0u);
    if (FULL || 8 * q + 8 <= ncol) {
      u[q] = reinterpret_cast<const uint4*>(src)[q];
    } else if (8 * q < ncol) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (8 * q + j < ncol) w[j >> 1] |= static_cast<uint32_t>(src[8 * q + j]) << (16 * (j & 1));
      u[q] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
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
__device__ __forceinline__ void add_row_16(const uint16_t* src, int ncol, bool fp16,
                                           float (&v)[32]) {
  if (ncol >= 32) {
    if (fp16)
      add_cols<true, true>(src, ncol, v);
    else
      add_cols<false, true>(src, ncol, v);
  } else if (fp16) {
    add_cols<true, false>(src, ncol, v);
  } else {
    add_cols<false, false>(src, ncol, v);
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
  int act, fp16;
  int keep;              // also write the slopes; 2: in the relative form
  int M, N;
  SignArgs sign;
  Out16 y, slope;
};

struct LinearEpi {
  static constexpr bool kAMN = false, kBMN = false;
  static constexpr OperandPlan kPlan = kOneEach;
  using Args = LinearArgs;
  template <class Acc>
  __device__ static void tile(const Args& a, const PairArgs&, int, int row0, int col_base, int lane,
                              const Acc& acc, Staging& st, const TileSlice& sl) {
    with_keep(a.keep, a.act, [&](auto keep) {
      tile_as<decltype(keep)::value>(a, row0, col_base, lane, acc, st, sl);
    });
  }
  template <int KEEP, class Acc>
  __device__ __forceinline__ static void tile_as(const Args& a, int row0, int col_base, int lane,
                                                 const Acc& acc, Staging& st,
                                                 const TileSlice& sl) {
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
      float largest = 0.f;
      if constexpr (KEEP == kKeepSigns) largest = largest_of(v);
      if (a.bias) add_row_16(a.bias + col0, a.N - col0, f16, v);
      if constexpr (KEEP == kKeepNone) {
        act_all(a.act, v);
      } else {
        uint32_t w[16];
        if constexpr (KEEP == kKeepSigns) {
          uint32_t near = row < a.M ? near_zero(v, largest, a.sign.K) : 0u, above = 0;
          if (a.N - col0 < 32) near &= (1u << (a.N - col0)) - 1u;
          const bool any = __any_sync(0xffffffffu, near != 0);
          if (any) {
            near_zero_of_column(v, a.sign.K, near);
            above = signs_again(a.sign, f16, row, col0, near, lane);
          }
          act_keep_slopes<kActRelu, false>(v, w);
          if (any) put_signs(near, above, w);
        } else {
          with_act(a.act, [&](auto act) {
            act_keep_slopes<decltype(act)::value, KEEP == kKeepRelative>(v, w);
          });
        }
        put_words(a.slope, a.M, a.N, row0, col0, w, st, lane);
      }
      if (a.res) {
        if (a.res_vec == 0)
          add_rows(a.res, a.ld_res, a.M, a.N, row0, col0, f16, v, st, lane);
        else if (row < a.M)
          add_row_16(a.res + static_cast<size_t>(row) * a.ld_res + col0, a.N - col0, f16, v);
      }
      uint32_t w[16];
      pack_32(v, f16, w);
      put_words(a.y, a.M, a.N, row0, col0, w, st, lane);
    }
  }
};

// ---------------------------------------------------------- gated: forward
struct GatedArgs {
  int act, fp16;
  int keep;  // also write a(g) and u a'(g); 2: in the relative form
  int M, F;
  SignArgs sign;
  Out16 h, val, cross;
};

struct GatedEpi {
  static constexpr bool kAMN = false, kBMN = false;
  static constexpr OperandPlan kPlan = kTwoB;
  using Args = GatedArgs;
  template <class Acc>
  __device__ static void tile(const Args& a, const PairArgs&, int, int row0, int col_base, int lane,
                              const Acc& acc, Staging& st, const TileSlice& sl) {
    with_keep(a.keep, a.act, [&](auto keep) {
      tile_as<decltype(keep)::value>(a, row0, col_base, lane, acc, st, sl);
    });
  }
  template <int KEEP, class Acc>
  __device__ __forceinline__ static void tile_as(const Args& a, int row0, int col_base, int lane,
                                                 const Acc& acc, Staging& st,
                                                 const TileSlice& sl) {
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
      if constexpr (KEEP == kKeepNone) {
        act_all(a.act, g);
      } else {
        float x[32];  // u a'(g)
        if constexpr (KEEP == kKeepSigns) {
          uint32_t near = row0 + lane < a.M ? near_zero(g, largest_of(g), a.sign.K) : 0u, above = 0;
          if (a.F - col0 < 32) near &= (1u << (a.F - col0)) - 1u;
          const bool any = __any_sync(0xffffffffu, near != 0);
          if (any) {
            near_zero_of_column(g, a.sign.K, near);
            above = signs_again(a.sign, f16, row0 + lane, col0, near, lane);
          }
          act_cross(kActRelu, g, u, x);
          if (any) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if ((near >> j) & 1u) x[j] = ((above >> j) & 1u) ? u[j] : 0.f;
          }
        } else {
          act_cross(a.act, g, u, x);
        }
        uint32_t w[16];
        const auto encode_as = [&](const float (&v)[32], uint32_t (&out)[16]) {
          if constexpr (KEEP == kKeepSigns)  // of either form
            encode_groups(a.keep == 2, v, out);
          else
            encode_groups_as<KEEP == kKeepRelative>(v, out);
        };
        encode_as(g, w);
        staged_block_16(&a.val.map, col0, row0, w, st, lane);
        encode_as(x, w);
        staged_block_16(&a.cross.map, col0, row0, w, st, lane);
      }
#pragma unroll
      for (int j = 0; j < 32; j += 2)
        f32x2_split(fmul2(f32x2(g[j], g[j + 1]), f32x2(u[j], u[j + 1])), g[j], g[j + 1]);
      uint32_t w[16];
      pack_32(g, f16, w);
      staged_block_16(&a.h.map, col0, row0, w, st, lane);
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
      uint32_t w[16];
      pack_32(v, a.fp16 != 0, w);
      staged_block_16(&a.dx.map, col0, row0, w, st, lane);
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
      if (a.out16) {
        uint32_t w[16];
        pack_32(v, a.fp16 != 0, w);
        staged_block_16(out, col0, row0, w, st, lane);
      } else {
        tma_block_f32(out, col0, row0, v, st.buf, lane);
      }
    }
  }
};

}  // namespace flce
