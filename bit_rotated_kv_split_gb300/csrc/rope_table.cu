// Table of rotation angles: cosines and sines of position x frequency.
//
// The angle is held as a 64-bit fraction of a turn, which wraps by itself: the
// angle of any position is one integer product, and the next of a thread's
// positions one addition, without rounding beyond that of one position's turn to 2^-64
// (at position 2^40 it makes 2^-25 of a turn).  The nearest quarter turn is taken off in
// integers; what is left, at most an eighth of a turn (pi / 4), goes to fp32 with 24
// bits whatever its size, and sine and cosine are their Taylor polynomials there (to
// x^9 and x^10; the next terms are below 2e-9 and 2e-10).
//
// Bound by its writes: 4 bytes a value and about 14 instructions.
#include <cuda_runtime.h>

#include <algorithm>

#include "int8.h"
#include "kernels.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace oscar {
namespace {

constexpr int kTableThreads = 256;

// (sin, cos) of the turns a and b (64-bit fractions), times magnitude.
__device__ __forceinline__ void sincos2(uint64_t a, uint64_t b, float magnitude, float2* sine, float2* cosine) {
  const uint32_t ha = uint32_t(a >> 32) + 0x20000000u, hb = uint32_t(b >> 32) + 0x20000000u;
  const int ra = int(ha & 0x3FFFFFFFu) - 0x20000000, rb = int(hb & 0x3FFFFFFFu) - 0x20000000;
  // 2^32 of a turn to radians
  constexpr float kLow = 2.3283064365386963e-10f, kRad = 1.4629180792671596e-9f;
  float2 x = fma2(make_float2(__uint2float_rn(uint32_t(a)), __uint2float_rn(uint32_t(b))), twice(kLow),
                  make_float2(__int2float_rn(ra), __int2float_rn(rb)));
  x = mul2(x, twice(kRad));
  const float2 u = mul2(x, x);
  float2 s = fma2(u, twice(2.7557319e-6f), twice(-1.9841270e-4f));   // 1/9!, -1/7!
  s = fma2(s, u, twice(8.3333333e-3f));
  s = fma2(s, u, twice(-0.16666667f));
  s = fma2(mul2(s, u), x, x);
  float2 c = fma2(u, twice(-2.7557319e-7f), twice(2.4801587e-5f));   // -1/10!, 1/8!
  c = fma2(c, u, twice(-1.3888889e-3f));
  c = fma2(c, u, twice(4.1666667e-2f));
  c = fma2(c, u, twice(-0.5f));
  c = fma2(c, u, twice(1.f));
  // quarter q: (s, c), (c, -s), (-s, -c), (-c, s)
  const uint32_t qa = ha >> 30, qb = hb >> 30;
  float2 ss = make_float2(qa & 1 ? c.x : s.x, qb & 1 ? c.y : s.y), cc = make_float2(qa & 1 ? s.x : c.x, qb & 1 ? s.y : c.y);
  ss = make_float2(__uint_as_float(__float_as_uint(ss.x) ^ ((qa & 2) << 30)), __uint_as_float(__float_as_uint(ss.y) ^ ((qb & 2) << 30)));
  cc = make_float2(__uint_as_float(__float_as_uint(cc.x) ^ (((qa + 1) & 2) << 30)), __uint_as_float(__float_as_uint(cc.y) ^ (((qb + 1) & 2) << 30)));
  *sine = mul2(ss, twice(magnitude));
  *cosine = mul2(cc, twice(magnitude));
}

// A thread has four pairs of every `stride`-th position.
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lanes = p.pairs / 4;            // threads of a position
  const int64_t thread = int64_t(blockIdx.x) * kTableThreads + threadIdx.x;
  const int64_t stride = int64_t(gridDim.x) * kTableThreads / lanes;
  int64_t i = thread / lanes;
  if (i >= stride) return;
  const int g = 4 * int(thread - i * lanes);
  uint64_t at[4], step[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    at[k] = p.turn[g + k] * uint64_t(p.first + i);
    step[k] = p.turn[g + k] * uint64_t(stride);
  }
  for (; i < p.n; i += stride) {
    float4 s, c;
    float2 s0, c0;
    sincos2(at[0], at[1], p.magnitude, &s0, &c0);
    s.x = s0.x, s.y = s0.y, c.x = c0.x, c.y = c0.y;
    sincos2(at[2], at[3], p.magnitude, &s0, &c0);
    s.z = s0.x, s.w = s0.y, c.z = c0.x, c.w = c0.y;
    float4* row = reinterpret_cast<float4*>(p.cos_sin + i * 2 * p.pairs + g);
    row[0] = c;
    row[p.pairs / 4] = s;
#pragma unroll
    for (int k = 0; k < 4; ++k) at[k] += step[k];
  }
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams& p, cudaStream_t stream) {
  const int64_t threads = p.n * (p.pairs / 4);
  const int64_t blocks = std::min<int64_t>((threads + kTableThreads - 1) / kTableThreads, 152 * 8);
  return launch_pdl(rope_table_kernel, dim3(unsigned(blocks)), dim3(kTableThreads), 0, stream, p);
}

}  // namespace oscar
