// Device side of the score's form (scale, cap, distance bias, window),
// shared by the decodes over paged layers and the prompt attention.
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

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The capped score cap tanh(x scale / cap), in log2 units, of a raw dot product x.
// A softmax needs its scores to an absolute error and the cap may be far above them,
// so the error is a few 2^-24 of the score itself, whatever the cap.  With
// w = x cap_in = 2 log2 e x scale / cap:
//   |w| <= log2 e (scores up to about half the cap): x P(w^2), P of degree 4 fitted at
//     the Chebyshev points of its interval (6e-8 of the value in fp32);
//   above: sign(x) cap (1 - 2 / (1 + 2^|w|)), off by a few 2^-24 of the cap.
// (The approximate tanh instruction, 2^-11 of the value, would leave 0.02 at a cap
// of 50; by powers and reciprocals alone a cap of 1e6 left 0.1.)
__device__ __forceinline__ bool cap_is_near(float x, const ScoreParams& s) { return !(fabsf(x) * s.cap_in > kLog2e); }
__device__ __forceinline__ float capped_near(float x, const ScoreParams& s) {
  const float w = x * s.cap_in, u = w * w;
  float r = s.cap_near[4];
#pragma unroll
  for (int k = 3; k >= 0; --k) r = fmaf(r, u, s.cap_near[k]);
  return x * r;
}
__device__ __forceinline__ float capped_far(float x, const ScoreParams& s) {
  const float e = exp2_fast(fabsf(x) * s.cap_in);   // inf for a large score: tanh = 1
  return copysignf(s.cap_log2 - 2.f * s.cap_log2 * rcp_fast(1.f + e), x);
}
// Either, by the score itself (a NaN stays one).  Both are worked out: as a branch for
// each score the choice took four times as long as the two forms.
__device__ __forceinline__ float capped_pick(float x, float near, const ScoreParams& s) {
  float r;
  asm("{\n\t.reg .pred p;\n\tsetp.gt.f32 p, %3, %4;\n\tselp.f32 %0, %1, %2, p;\n\t}"
      : "=f"(r)
      : "f"(capped_far(x, s)), "f"(near), "f"(fabsf(x) * s.cap_in), "f"(kLog2e));
  return r;
}
__device__ __forceinline__ float capped(float x, const ScoreParams& s) { return capped_pick(x, capped_near(x, s), s); }

}  // namespace oscar
