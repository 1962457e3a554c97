// Helpers of the decodes over paged layers: their products, reductions over a
// product's rows and columns, the exponent of a scale, and what takes a dot product
// of scaled queries back.
#pragma once

#include <cfloat>
#include <cstdint>

#include <algorithm>

#include "int4.h"
#include "ptx.cuh"

namespace oscar {

// D += A (16x16 f16, row) * B (16x8 f16, col); free for the compiler to move.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float max_over_quad(float v) {   // over the 4 lanes of a row
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float sum_over_quad(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ float max_over_rows(float v) {   // over the 8 lanes of a column pair
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float sum_over_rows(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// 2^ve with ve in [-14, 16] is at least a scale of this size (fp16 bits) and any smaller one
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  return min(max(((__float_as_int(half2_to_float2(bits).x) >> 23) & 255) - 126, -14), 16);
}

// A query head with a largest channel in [2^(ex - 127), 2^(ex - 126)), 14 <= ex <= 254 (every
// finite bf16), is held times 2^(141 - ex) beside codes times 2^-24, so its dot products are
// to be multiplied by 2^(ex - 117), which may pass fp32's end.  With a cap they are taken
// to s.unit of themselves, and capped() has constants to match (in_units).  Without
// one the score's scale is in the factor too, and where that passes fp32's end only a dot
// product of 0 gives a score within bounds: it is to stay 0.
// (A scale of 2^100 would take the constants past fp32's end; scores of large queries are
// far beyond any cap then.)
__device__ __forceinline__ float unscale_of(int ex, const ScoreParams& s) {
  const float f = pow2i(ex - 128);
  return fminf(s.cap_log2 != 0.f ? f * (2048.f * s.unit) : f * s.scale_log2 * 2048.f, FLT_MAX);
}
inline ScoreParams in_units(ScoreParams s) {
  s.unit = s.scale_log2 < 0x1p100f ? 0x1p-11f : 1.f;
  s.cap_in = std::min(s.cap_in / s.unit, FLT_MAX);   // (past it only with a cap that is next to nothing)
  for (float& c : s.cap_near) c /= s.unit;
  return s;
}

}  // namespace oscar
