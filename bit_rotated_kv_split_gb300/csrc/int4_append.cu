// 4-bit layers: position rotation and append (rope_append_kernel), and the
// way back (gather_kernel).
//
// One lane holds an octet of adjacent channels (16 bytes of bf16), d / 8
// lanes a row, so a warp holds 32 / (d / 8) rows at a time.  A rotation pair
// (i, i + rot / 2) sits in the same place of two lanes and comes by shuffle;
// an interleaved pair sits in one lane.  A quantisation group is 4, 8 or 16
// lanes: its extremes come by shuffles, and a lane's 8 codes are one 32-bit
// word of K or two 16-bit halves of V.  A slot is the rows a warp handles at
// once: q heads, then k heads, then v heads of one token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "int4.h"
#include "kernels.h"
#include "oscar.h"
#include "ptx.cuh"

namespace oscar {
namespace {

constexpr int kAppendThreads = 128;

__device__ __forceinline__ void unpack_bf16x8(const uint4& u, float (&x)[8]) {
  x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(u.z), x[5] = bf16_hi(u.z), x[6] = bf16_lo(u.w), x[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
  return make_uint4(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]), pack_bf162(x[4], x[5]), pack_bf162(x[6], x[7]));
}

// x c + y s, so that its rounding to bf16 is that of the exact value.  The
// fp32 result is within e of it; where e spans a rounding border of bf16
// (about one value in 2^12) the sum is formed in 64 bits, whose products are
// exact and whose sum is rounded at 2^-53.
__device__ __forceinline__ float rotate_exact(float x, float c, float y, float s) {
  const float t = y * s;
  const float r = fmaf(x, c, t);
  const float e = (fabsf(t) + fabsf(r)) * 1.1920929e-7f;
  const uint32_t both = pack_bf162(r - e, r + e);
  if ((both & 0xFFFFu) != (both >> 16)) return float(fma(double(x), double(c), double(y) * double(s)));
  return r;
}

// Codes of the 8 values of this lane (x - zero over scale, to nearest even,
// 0 .. 15) in a group of `lanes` lanes; *pair = (scale, zero) as fp16 bits.
__device__ __forceinline__ uint32_t quantise8(float (&x)[8], float tau, int lanes, uint32_t* pair) {
  float lo = tau, hi = -tau;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = fminf(fmaxf(x[i], -tau), tau);   // (a NaN becomes -tau)
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
  for (int m = 1; m < lanes; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  const __half sh = __float2half_rn(__fdiv_rn(hi - lo, 15.f)), zh = __float2half_rn(lo);
  const float s = __half2float(sh), z = __half2float(zh);
  *pair = uint32_t(__half_as_ushort(sh)) | (uint32_t(__half_as_ushort(zh)) << 16);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = s > 0.f ? rintf(__fdiv_rn(x[i] - z, s)) : 0.f;
    word |= uint32_t(fminf(fmaxf(u, 0.f), 15.f)) << (4 * i);
  }
  return word;
}

__device__ __forceinline__ void flag(int32_t* dev_status, int bit) {
  if (dev_status) atomicOr(dev_status, bit);
}

// The block of (req, pos), KV head 0, or nullptr (skip) for a padding row, a
// place outside the table or a page outside the pool.
__device__ __forceinline__ uint8_t* token_block(const Int4Cache& c, int req, int pos, bool report) {
  if (req == -1) return nullptr;
  if (req < 0 || req >= c.batch || pos < 0 || pos / kInt4Page >= c.max_pages) {
    if (report) flag(c.dev_status, OSCAR_DEV_LENGTH);
    return nullptr;
  }
  const int page = c.page_table[int64_t(req) * c.max_pages + pos / kInt4Page];
  if (page < 0 || page >= c.n_pages) {
    if (report) flag(c.dev_status, OSCAR_DEV_PAGE_BOUNDS);
    return nullptr;
  }
  return c.pages + int64_t(page) * c.n_kv * int4_block_bytes(c.d, c.ng_k, c.ng_v);
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) rope_append_kernel(const AppendParams p, int slots_per_warp) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, o = lane % kLanes, sub = lane / kLanes;
  const int sq = (p.c.n_q + kRows - 1) / kRows, sk = (p.c.n_kv + kRows - 1) / kRows;
  const int first_q = p.q ? 0 : sq, slots = sq + 2 * sk - first_q;
  const int warps_per_token = (slots + slots_per_warp - 1) / slots_per_warp;
  const int64_t w = (int64_t(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
  const int64_t i = w / warps_per_token;
  if (i >= p.n) return;
  const int part = int(w % warps_per_token);
  const int pos = p.dst_pos[i];
  const bool report = part == 0 && lane == 0;
  uint8_t* base = token_block(p.c, p.dst_req[i], pos, report);
  if (!base) return;
  const int slot = pos % kInt4Page;
  // this lane's angles: octet o of a half-split head turns with o mod h, h =
  // rot / 16; an interleaved octet has the 4 angles 4 o ..
  const int h = p.rot / 16;
  const bool turns = o < 2 * h;
  float cs[8], sn[8];
  int partner = lane;
  if (p.rot) {
    const int64_t at = p.rope_pos ? p.rope_pos[i] : pos;
    if (at < 0 || at >= p.n_positions) {
      if (report) flag(p.c.dev_status, OSCAR_DEV_LENGTH);
      return;
    }
    const float* row = p.cos_sin + at * p.rot;
    if (turns && !p.interleaved) {
      const int j = o < h ? o : o - h;
      partner = o < h ? lane + h : lane - h;
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] = row[8 * j + e], sn[e] = row[8 * (h + j) + e];
    } else if (turns) {
#pragma unroll
      for (int e = 0; e < 4; ++e) cs[e] = row[4 * o + e], sn[e] = row[8 * h + 4 * o + e];
    }
  }
  const int end = min(slots, (part + 1) * slots_per_warp);
  for (int t = part * slots_per_warp; t < end; ++t) {
    const int s = t + first_q;
    const int kind = s < sq ? 0 : s < sq + sk ? 1 : 2;   // q, k, v
    const int head = (s - (kind == 0 ? 0 : kind == 1 ? sq : sq + sk)) * kRows + sub;
    const bool valid = head < (kind == 0 ? p.c.n_q : p.c.n_kv);
    const uint16_t* src = kind == 0 ? p.q + i * p.q_stride : kind == 1 ? p.k + i * p.k_stride : p.v + i * p.v_stride;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (valid) raw = *reinterpret_cast<const uint4*>(src + int64_t(head) * D + 8 * o);
    float x[8];
    unpack_bf16x8(raw, x);
    if (kind < 2 && p.rot) {
      if (!p.interleaved) {
        uint4 other;
        other.x = __shfl_sync(0xffffffffu, raw.x, partner);
        other.y = __shfl_sync(0xffffffffu, raw.y, partner);
        other.z = __shfl_sync(0xffffffffu, raw.z, partner);
        other.w = __shfl_sync(0xffffffffu, raw.w, partner);
        float y[8];
        unpack_bf16x8(other, y);
        if (turns) {
          const float sign = o < h ? -1.f : 1.f;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[e] = kind == 0 ? fmaf(x[e], cs[e], y[e] * (sign * sn[e])) : rotate_exact(x[e], cs[e], y[e], sign * sn[e]);
        }
      } else if (turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x[2 * e], b = x[2 * e + 1];
          x[2 * e] = kind == 0 ? fmaf(a, cs[e], b * -sn[e]) : rotate_exact(a, cs[e], b, -sn[e]);
          x[2 * e + 1] = kind == 0 ? fmaf(a, sn[e], b * cs[e]) : rotate_exact(a, sn[e], b, cs[e]);
        }
      }
      raw = pack_bf16x8(x);
      if (kind == 1) unpack_bf16x8(raw, x);   // the codes are those of the rounded row
    }
    if (kind < 2) {
      uint16_t* out = kind == 0 ? p.q_out : p.k_out;
      if (out && valid) *reinterpret_cast<uint4*>(out + (i * (kind == 0 ? p.c.n_q : p.c.n_kv) + head) * D + 8 * o) = raw;
    }
    if (kind == 0) continue;
    const int ng_k = p.c.ng_k, ng_v = p.c.ng_v;
    const int lanes = kLanes / (kind == 1 ? ng_k : ng_v);
    uint32_t pair;
    const uint32_t word = quantise8(x, kind == 1 ? p.tau_k : p.tau_v, lanes, &pair);
    if (!valid) continue;
    uint8_t* block = base + int64_t(head) * int4_block_bytes(D, ng_k, ng_v);
    if (kind == 1) {
      *reinterpret_cast<uint32_t*>(block + int4_k_word(D, slot, o)) = word;
    } else {
      *reinterpret_cast<uint16_t*>(block + int4_v_half(D, slot, 2 * o)) = uint16_t(word);
      *reinterpret_cast<uint16_t*>(block + int4_v_half(D, slot, 2 * o + 1)) = uint16_t(word >> 16);
    }
    if (o % lanes == 0)
      *reinterpret_cast<uint32_t*>(block + int4_pair(D, ng_k, ng_v, slot, (kind == 1 ? 0 : ng_k) + o / lanes)) = pair;
  }
}

// One warp per (token, kRows KV heads): K, then V.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) gather_kernel(const GatherParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, o = lane % kLanes, sub = lane / kLanes;
  const int per_token = (p.c.n_kv + kRows - 1) / kRows;
  const int64_t w = (int64_t(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
  const int64_t i = w / per_token;
  if (i >= p.n) return;
  const int head = int(w % per_token) * kRows + sub;
  const int pos = p.src_pos[i];
  const uint8_t* base = token_block(p.c, p.src_req[i], pos, lane == 0 && w % per_token == 0);
  if (!base || head >= p.c.n_kv) return;
  const int slot = pos % kInt4Page, ng_k = p.c.ng_k, ng_v = p.c.ng_v;
  const uint8_t* block = base + int64_t(head) * int4_block_bytes(D, ng_k, ng_v);
  const uint32_t kw = *reinterpret_cast<const uint32_t*>(block + int4_k_word(D, slot, o));
  const uint32_t vw = uint32_t(*reinterpret_cast<const uint16_t*>(block + int4_v_half(D, slot, 2 * o))) |
                      (uint32_t(*reinterpret_cast<const uint16_t*>(block + int4_v_half(D, slot, 2 * o + 1))) << 16);
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int q = kind == 0 ? o * ng_k / kLanes : ng_k + o * ng_v / kLanes;
    const float2 sz = half2_to_float2(*reinterpret_cast<const uint32_t*>(block + int4_pair(D, ng_k, ng_v, slot, q)));
    const uint32_t word = kind == 0 ? kw : vw;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(float((word >> (4 * e)) & 15u), sz.x, sz.y);
    uint16_t* out = kind == 0 ? p.k_out + i * p.k_stride : p.v_out + i * p.v_stride;
    *reinterpret_cast<uint4*>(out + int64_t(head) * D + 8 * o) = pack_bf16x8(x);
  }
}

cudaError_t grid_of(int64_t warps, unsigned* blocks) {
  const int64_t b = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  if (b < 1 || b > 0x7fffffff) return cudaErrorInvalidValue;
  *blocks = unsigned(b);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_rope_append_int4(const AppendParams& p, cudaStream_t stream) {
  const int rows = 32 / (p.c.d / 8);
  const int slots = (p.q ? (p.c.n_q + rows - 1) / rows : 0) + 2 * ((p.c.n_kv + rows - 1) / rows);
  const int slots_per_warp = 1;
  unsigned blocks = 0;
  const cudaError_t e = grid_of(int64_t(p.n) * ((slots + slots_per_warp - 1) / slots_per_warp), &blocks);
  if (e != cudaSuccess) return e;
  return p.c.d == 128 ? launch_pdl(rope_append_kernel<128>, dim3(blocks), dim3(kAppendThreads), 0, stream, p, slots_per_warp)
                      : launch_pdl(rope_append_kernel<64>, dim3(blocks), dim3(kAppendThreads), 0, stream, p, slots_per_warp);
}

cudaError_t launch_gather_int4(const GatherParams& p, cudaStream_t stream) {
  const int rows = 32 / (p.c.d / 8);
  unsigned blocks = 0;
  const cudaError_t e = grid_of(int64_t(p.n) * ((p.c.n_kv + rows - 1) / rows), &blocks);
  if (e != cudaSuccess) return e;
  return p.c.d == 128 ? launch_pdl(gather_kernel<128>, dim3(blocks), dim3(kAppendThreads), 0, stream, p)
                      : launch_pdl(gather_kernel<64>, dim3(blocks), dim3(kAppendThreads), 0, stream, p);
}

}  // namespace oscar
