// Host-side checks shared by the operators on the residual stream.
#pragma once
#include <cmath>
#include <cstdint>

#include "../../include/flce.h"
#include "stream_ops.cuh"

namespace flce {

inline bool float_type_ok(int32_t t) { return t >= FLCE_DTYPE_BF16 && t <= FLCE_DTYPE_FP32; }
// The residual stream is of the operands' type or fp32.
inline bool wider_ok(int32_t t, int32_t of) { return t == of || t == FLCE_DTYPE_FP32; }
inline bool aligned_to(const void* p, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}
inline int64_t pitch_of(int64_t ld, int64_t dense) { return ld == 0 ? dense : ld; }
inline bool pitch_ok(int64_t ld, int64_t dense) { return ld == 0 || ld >= dense; }
// Whether all rows start on 16-byte boundaries; null pointers do.
inline bool rows16(const void* p, int64_t ld, int64_t rows, int type) {
  return !p || (aligned_to(p, 16) && (rows <= 1 || ld * type_size(type) % 16 == 0));
}

flce_status_t check_norm(const flce_rms_norm_params_t* p);  // rms_norm.cu

// p in [0, 1] as 16 bits.
inline bool make_dropout(double p, int64_t seed, int64_t offset, const int64_t* seed_at, Dropout* d) {
  if (!(p >= 0.0) || !(p <= 1.0)) return false;
  d->threshold = static_cast<uint32_t>(std::floor(p * 65536.0 + 0.5));
  d->scale = d->threshold >= 65536u ? 0.f : 65536.f / static_cast<float>(65536u - d->threshold);
  d->seed = static_cast<uint64_t>(seed);
  d->offset = static_cast<uint64_t>(offset);
  d->seed_at = seed_at;
  return true;
}

}  // namespace flce
