// Device helpers of the kernels that work on rows of bf16 heads, a lane to an
// octet of adjacent channels: packed arithmetic, the group's extremes, angles,
// and how many of a token's heads a warp takes.
#pragma once

#include <cstdint>

#include <algorithm>

#include "int4.h"
#include "oscar.h"
#include "ptx.cuh"
#include "score.cuh"

namespace oscar {

constexpr int kRowThreads = 128;

__device__ __forceinline__ void unpack_bf16x8(const uint4& u, float (&x)[8]) {
  x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(u.z), x[5] = bf16_hi(u.z), x[6] = bf16_lo(u.w), x[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
  return make_uint4(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]), pack_bf162(x[4], x[5]), pack_bf162(x[6], x[7]));
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {   // a NaN wins
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 bf16_pair(uint32_t u) { return make_float2(bf16_lo(u), bf16_hi(u)); }

// a - b >= 0, to odd: where 24 bits do not hold it, the last one is set.  A quotient of it
// is then not taken for a tie of fewer bits that the exact one only comes near to.
__device__ __forceinline__ float sub_odd(float a, float b) {
  const float lo = __fsub_rz(a, b), hi = __fsub_ru(a, b);   // (a - a is +0 in both)
  return __uint_as_float(__float_as_uint(lo) | (lo != hi ? 1u : 0u));
}

__device__ __forceinline__ void flag(int32_t* dev_status, int bit) {
  if (dev_status) atomicOr(dev_status, bit);
}

// The block of (req, pos), KV head 0, or nullptr (skip) for a padding row, a
// place outside the table or a page outside the pool.
__device__ __forceinline__ uint8_t* block_of_token(const PagedCache& c, int block_bytes, int req, int pos,
                                                   bool report) {
  if (req == -1) return nullptr;
  if (req < 0 || req >= c.batch || pos < 0 || pos / kPageTokens >= c.max_pages) {
    if (report) flag(c.dev_status, OSCAR_DEV_LENGTH);
    return nullptr;
  }
  const int page = c.page_table[int64_t(req) * c.max_pages + pos / kPageTokens];
  if (page < 0 || page >= c.n_pages) {
    if (report) flag(c.dev_status, OSCAR_DEV_PAGE_BOUNDS);
    return nullptr;
  }
  return c.pages + int64_t(page) * c.n_kv * block_bytes;
}

__device__ __forceinline__ void load8(float (&x)[8], const float* p, int n) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (4 * i < n) {
      const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
}

// Slots of a token for one warp: as many as leave the GPU 24 warps an SM.  A
// token's place and angles are then read once, not once a slot.
inline int slots_of(int n, int slots) {
  return int(std::min<int64_t>(slots, std::max<int64_t>(1, int64_t(n) * slots / (152 * 24))));
}

inline cudaError_t grid_of(int64_t warps, unsigned* blocks) {
  const int64_t b = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
  if (b < 1 || b > 0x7fffffff) return cudaErrorInvalidValue;
  *blocks = unsigned(b);
  return cudaSuccess;
}

}  // namespace oscar
