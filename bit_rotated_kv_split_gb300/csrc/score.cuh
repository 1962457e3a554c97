// Device side of the score's form (scale, cap, distance bias, window),
// shared by the 4-bit decode and the prompt attention.
#pragma once

#include <cfloat>

#include "int4.h"

namespace oscar {

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap tanh(x scale / cap) in log2 units for a raw dot product x.  tanh(y) =
// sign(y) (1 - 2 / (1 + e^(2 |y|))), whose absolute error is a few 2^-24: a
// softmax needs its scores to an absolute error, and the approximate tanh
// instruction (2^-11 of the value) would leave one of 0.02 at a cap of 50.
__device__ __forceinline__ float capped(float x, const ScoreParams& s) {
  const float e = exp2_fast(fabsf(x) * s.cap_in);   // inf for a large score: tanh = 1
  return copysignf(s.cap_log2 - 2.f * s.cap_log2 * rcp_fast(1.f + e), x);
}

template <bool Cap>
__device__ __forceinline__ float score_of(float x, const ScoreParams& s) {
  return Cap ? capped(x, s) : x * s.scale_log2;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

}  // namespace oscar
