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
//
// Measured: 30,186 tokens of 32/8 heads x 128 appended in 136 us (710 MB read and
// written: 5.2 TB/s, 78 % of a plain copy's rate), bound by instruction issue (67 %)
// and by the latency of each token's place and angles; without the rotation it
// takes 32 us less, without the quantisation 13.  65,521 tokens read back in 57 us
// (5.9 TB/s, 89 %).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>

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

__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// Codes of the 8 bf16 values u of this lane (x - zero over scale, to nearest
// even, 0 .. 15) in a group of `lanes` lanes; *pair = (scale, zero), fp16 bits.
// Scales and codes are those of exact differences.
//
// The group's extremes are taken on packed bf16 (max x, max -x).  rint(t / s)
// is taken as rint(t / s by an approximate reciprocal) and checked: where the
// remainder t - k s (one fma) comes within 1e-6 of half a step (t's own rounding, 2^-24
// of at most 15.5 steps, is below that), the quotients are divided out.
// (With a division for every value the kernel had a third more instructions.)
__device__ __forceinline__ uint32_t quantise8(const uint4& u, float tau, int lanes, uint32_t* pair) {
  uint32_t hi2 = max_bf16x2(max_bf16x2(u.x, u.y), max_bf16x2(u.z, u.w));
  uint32_t lo2 = max_bf16x2(max_bf16x2(u.x ^ 0x80008000u, u.y ^ 0x80008000u),
                            max_bf16x2(u.z ^ 0x80008000u, u.w ^ 0x80008000u));
  uint32_t ends = max_bf16x2(prmt(hi2, lo2, 0x5410), prmt(hi2, lo2, 0x7632));   // (max x, max -x)
  for (int m = 1; m < lanes; m <<= 1) ends = max_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, m));
  float hi = bf16_lo(ends), lo = -bf16_hi(ends);
  float x[8];
  unpack_bf16x8(u, x);
  const bool clamped = !(hi <= tau && lo >= -tau);
  if (clamped) {                          // or a NaN, which becomes -tau
    hi = -tau, lo = tau;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = fminf(fmaxf(x[i], -tau), tau);
      hi = fmaxf(hi, x[i]);
      lo = fminf(lo, x[i]);
    }
    // (the whole group is here: the test is the group's)
    const uint32_t group = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1) << (threadIdx.x & 31 & ~(lanes - 1));
    for (int m = 1; m < lanes; m <<= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(group, hi, m));
      lo = fminf(lo, __shfl_xor_sync(group, lo, m));
    }
  }
  // (a range of two bf16 numbers comes near a tie of a normal scale only where 24 bits hold it)
  float range = hi - lo;
  if (clamped || range < 1e-3f) range = sub_odd(hi, lo);
  const __half sh = __float2half_rn(__fdiv_rn(range, 15.f)), zh = __float2half_rn(lo);
  const float s = __half2float(sh), z = __half2float(zh);
  *pair = uint32_t(__half_as_ushort(sh)) | (uint32_t(__half_as_ushort(zh)) << 16);
  const float inv = rcp_fast(s), top = 15.f * s, half = s * 0.499999f;
  constexpr float kRound = 12582912.f;   // 1.5 2^23: the sum's low bits are the rounded integer
  uint32_t word = 0;
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = fminf(fmaxf(x[i] - z, 0.f), top), k = fmaf(t, inv, kRound);
    near = near | (fabsf(fmaf(kRound - k, s, t)) >= half);
    word += (__float_as_uint(k) - 0x4B400000u) << (4 * i);
  }
  if (!(s > 0.f)) return 0;
  if (near) {
    word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = fminf(fmaxf(sub_odd(x[i], z), 0.f), top);
      word |= uint32_t(rintf(__fdiv_rn(t, s))) << (4 * i);
    }
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

// What a lane needs to turn an octet: octet o of a half-split head turns with
// o mod h, h = rot / 16, and takes its partner's channels from `partner`; an
// interleaved octet has the 4 angles 4 o ..
struct Turn {
  float c[8], s[8];   // s carries the sign of this half
  int partner;
  bool on;
};

// Values 2 i, 2 i + 1 of the turned octet are a c + b s.
template <bool Interleaved>
__device__ __forceinline__ void operands(const Turn& t, uint32_t x, uint32_t y, int i, float2* a, float2* c, float2* b,
                                         float2* s) {
  const float2 u = bf16_pair(x);
  if (!Interleaved) {
    *a = u;
    *b = bf16_pair(y);
    *c = make_float2(t.c[2 * i], t.c[2 * i + 1]);
    *s = make_float2(t.s[2 * i], t.s[2 * i + 1]);
  } else {
    *a = twice(u.x);
    *b = twice(u.y);
    *c = make_float2(t.c[i], t.s[i]);
    *s = make_float2(-t.s[i], t.c[i]);
  }
}

// Rotates the octet held in `raw`; whole warps call it.  Exact: the rounding to
// bf16 is that of the exact value's fp32.  The fp32 result r is within e of it;
// where r - e and r + e round apart (about one value in 2^13) the pair is formed
// in 64 bits, whose products are exact and whose sums are rounded at 2^-53.
template <bool Exact, bool Interleaved>
__device__ __forceinline__ void rotate8(uint4& raw, const Turn& t) {
  uint4 other = make_uint4(0, 0, 0, 0);
  if (!Interleaved) {
    other.x = __shfl_sync(0xffffffffu, raw.x, t.partner);
    other.y = __shfl_sync(0xffffffffu, raw.y, t.partner);
    other.z = __shfl_sync(0xffffffffu, raw.z, t.partner);
    other.w = __shfl_sync(0xffffffffu, raw.w, t.partner);
  }
  if (!t.on) return;
  const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w}, y[4] = {other.x, other.y, other.z, other.w};
  uint32_t out[4], apart[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 a, b, c, s;
    operands<Interleaved>(t, x[i], y[i], i, &a, &c, &b, &s);
    const float2 bs = mul2(b, s), r = fma2(a, c, bs);
    if (Exact) {
      // (twice the two roundings: 2^-23 of each, and at least the last place of a subnormal sum)
      const float2 e = add2(make_float2(fabsf(bs.x) + fabsf(r.x), fabsf(bs.y) + fabsf(r.y)), twice(FLT_MIN));
      const float2 lo = fma2(e, twice(-1.1920929e-7f), r), hi = fma2(e, twice(1.1920929e-7f), r);
      out[i] = pack_bf162(lo.x, lo.y);
      apart[i] = out[i] ^ pack_bf162(hi.x, hi.y);
    } else {
      out[i] = pack_bf162(r.x, r.y);
    }
  }
  if (Exact && (apart[0] | apart[1] | apart[2] | apart[3])) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (apart[i]) {
        float2 a, b, c, s;
        operands<Interleaved>(t, x[i], y[i], i, &a, &c, &b, &s);
        out[i] = pack_bf162(float(fma(double(a.x), double(c.x), double(b.x) * double(s.x))),
                            float(fma(double(a.y), double(c.y), double(b.y) * double(s.y))));
      }
  }
  raw = make_uint4(out[0], out[1], out[2], out[3]);
}

__device__ __forceinline__ void load8(float (&x)[8], const float* p, int n) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (4 * i < n) {
      const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
}

// One warp takes `slots_per_warp` slots of one token: its q heads four slots at
// a time, whose loads are in flight together, then k and v heads with the next
// slot's load ahead of the present one's work.
template <int D, bool Interleaved>
__global__ void __launch_bounds__(kAppendThreads, 7)
    rope_append_kernel(const __grid_constant__ AppendParams p, int slots_per_warp) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = 4;
  const int lane = threadIdx.x & 31, o = lane % kLanes, sub = lane / kLanes;
  const int sq = p.q ? (p.c.n_q + kRows - 1) / kRows : 0, sk = (p.c.n_kv + kRows - 1) / kRows;
  const int slots = sq + 2 * sk, warps_per_token = (slots + slots_per_warp - 1) / slots_per_warp;
  const int64_t w = (int64_t(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
  const int64_t i = w / warps_per_token;
  if (i >= p.n) return;
  const int part = int(w - i * warps_per_token);
  const int pos = p.dst_pos[i];
  const bool report = part == 0 && lane == 0;
  uint8_t* base = token_block(p.c, p.dst_req[i], pos, report);
  if (!base) return;
  const int slot = pos % kInt4Page;
  Turn turn;
  const int h = p.rot / 16;
  turn.on = o < 2 * h;
  turn.partner = lane;
  if (p.rot) {
    const int64_t at = p.rope_pos ? p.rope_pos[i] : pos;
    if (at < 0 || at >= p.n_positions) {
      if (report) flag(p.c.dev_status, OSCAR_DEV_LENGTH);
      return;
    }
    const float* row = p.cos_sin + at * p.rot;
    if (turn.on && !Interleaved) {
      const int j = o < h ? o : o - h;
      turn.partner = o < h ? lane + h : lane - h;
      load8(turn.c, row + 8 * j, 8);
      load8(turn.s, row + 8 * (h + j), 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) turn.s[e] = o < h ? -turn.s[e] : turn.s[e];
    } else if (turn.on) {
      load8(turn.c, row + 4 * o, 4);
      load8(turn.s, row + 8 * h + 4 * o, 4);
    }
  }
  const int begin = part * slots_per_warp, end = min(slots, begin + slots_per_warp);
  // q
  const int end_q = min(end, sq);
  const uint16_t* src = p.q + i * p.q_stride + sub * D + 8 * o;
  uint16_t* dst = p.q_out + (i * p.c.n_q + sub) * D + 8 * o;
  for (int s0 = begin; s0 < end_q; s0 += kBatch) {
    uint4 raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      raw[u] = make_uint4(0, 0, 0, 0);
      if (s0 + u < end_q && (s0 + u) * kRows + sub < p.c.n_q)
        raw[u] = *reinterpret_cast<const uint4*>(src + (s0 + u) * (kRows * D));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (s0 + u >= end_q) break;
      if (p.rot) rotate8<false, Interleaved>(raw[u], turn);
      if ((s0 + u) * kRows + sub < p.c.n_q) *reinterpret_cast<uint4*>(dst + (s0 + u) * (kRows * D)) = raw[u];
    }
  }
  // k, then v
  const int ng_k = p.c.ng_k, ng_v = p.c.ng_v, block_bytes = int4_block_bytes(D, ng_k, ng_v);
  auto load = [&](int s) {
    uint4 r = make_uint4(0, 0, 0, 0);
    const bool is_v = s >= sk;
    const int head = (is_v ? s - sk : s) * kRows + sub;
    const uint16_t* x = is_v ? p.v + i * p.v_stride : p.k + i * p.k_stride;
    if (s < end - sq && head < p.c.n_kv) r = *reinterpret_cast<const uint4*>(x + head * D + 8 * o);
    return r;
  };
  int s = max(0, begin - sq);
  uint4 next = load(s);
#pragma unroll 1
  for (; s < end - sq; ++s) {
    uint4 raw = next;
    next = load(s + 1);
    const bool is_v = s >= sk;
    const int head = (is_v ? s - sk : s) * kRows + sub;
    const bool valid = head < p.c.n_kv;
    if (!is_v) {
      if (p.rot) rotate8<true, Interleaved>(raw, turn);
      if (p.k_out && valid) *reinterpret_cast<uint4*>(p.k_out + (i * p.c.n_kv + head) * D + 8 * o) = raw;
    }
    const int lanes = kLanes >> ((is_v ? ng_v : ng_k) >> 1);   // 1, 2 or 4 groups
    uint32_t pair;
    const uint32_t word = quantise8(raw, is_v ? p.tau_v : p.tau_k, lanes, &pair);   // of the rounded row
    if (!valid) continue;
    uint8_t* block = base + int64_t(head) * block_bytes;
    if (!is_v) {
      *reinterpret_cast<uint32_t*>(block + int4_k_word(D, slot, o)) = word;
    } else {
      *reinterpret_cast<uint16_t*>(block + int4_v_half(D, slot, 2 * o)) = uint16_t(word);
      *reinterpret_cast<uint16_t*>(block + int4_v_half(D, slot, 2 * o + 1)) = uint16_t(word >> 16);
    }
    if ((o & (lanes - 1)) == 0)
      *reinterpret_cast<uint32_t*>(block + int4_pair(D, ng_k, ng_v, slot, is_v ? ng_k + o * ng_v / kLanes : o * ng_k / kLanes)) = pair;
  }
}

// zero + scale * code of the 8 codes of a word, as bf16.  Codes become halves
// by a mask (1024 + c is 0x6400 | c) and an exact subtraction: an integer
// conversion for each would keep the special function unit busy for longer than
// the loads take.
__device__ __forceinline__ uint4 values8(uint32_t word, uint32_t pair) {
  const float2 sz = half2_to_float2(pair);
  const __half2 k1024 = __floats2half2_rn(1024.f, 1024.f);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {           // nibbles i and i + 4
    uint32_t h;
    asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(h) : "r"(word >> (4 * i)));
    const float2 c = __half22float2(__hsub2(*reinterpret_cast<__half2*>(&h), k1024));
    x[i] = fmaf(c.x, sz.x, sz.y);
    x[i + 4] = fmaf(c.y, sz.x, sz.y);
  }
  return pack_bf16x8(x);
}

// A warp takes `slots_per_warp` slots (the KV heads that it holds at a time) of
// one token, or all slots of `tokens` tokens, whose places its lanes look up at
// once (position, page, block: one behind the other, they take longer than a
// token's rows do); the next slot's loads are ahead of the present one's work.
template <int D>
__global__ void __launch_bounds__(kAppendThreads)
    gather_kernel(const __grid_constant__ GatherParams p, int slots_per_warp, int tokens) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, o = lane % kLanes, sub = lane / kLanes;
  const int slots = (p.c.n_kv + kRows - 1) / kRows, warps_per_token = (slots + slots_per_warp - 1) / slots_per_warp;
  const int64_t w = (int64_t(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
  const int64_t i0 = w / warps_per_token * tokens;
  if (i0 >= p.n) return;
  const int part = int(w % warps_per_token), count = int(min(int64_t(tokens), p.n - i0));
  uint64_t mine = 0;                      // lane t: token t's block and slot (blocks are 64-byte aligned)
  if (lane < count) {
    const int pos = p.src_pos[i0 + lane];
    const uint8_t* base = token_block(p.c, p.src_req[i0 + lane], pos, part == 0);
    if (base) mine = reinterpret_cast<uint64_t>(base) | uint64_t(pos % kInt4Page);
  }
  const int ng_k = p.c.ng_k, ng_v = p.c.ng_v, block_bytes = int4_block_bytes(D, ng_k, ng_v);
  const int begin = part * slots_per_warp, end = min(slots, begin + slots_per_warp);
  const int kp_at = int4_pair(D, ng_k, ng_v, 0, o * ng_k / kLanes), vp_at = int4_pair(D, ng_k, ng_v, 0, ng_k + o * ng_v / kLanes);
  constexpr int kSecond = int4_v_half(D, 0, 1) - int4_v_half(D, 0, 0);   // from quad 2 o to 2 o + 1
  struct Raw {
    uint32_t k, v0, v1, kp, vp;
  };
  int t_next = 0, s_next = begin;         // the next slot to ask for
  bool ok_next = false;                   // it is there
  auto load = [&]() {
    Raw r{};
    const uint64_t at = __shfl_sync(0xffffffffu, mine, min(t_next, 31));
    const int head = s_next * kRows + sub, slot = int(at & 15);
    ok_next = t_next < count && at != 0 && head < p.c.n_kv;
    if (ok_next) {
      const uint8_t* block = reinterpret_cast<const uint8_t*>(at & ~uint64_t(15)) + int64_t(head) * block_bytes;
      const int pair = slot * 4 * (ng_k + ng_v);
      r.k = *reinterpret_cast<const uint32_t*>(block + int4_k_word(D, slot, o));
      r.v0 = *reinterpret_cast<const uint16_t*>(block + int4_v_half(D, slot, 2 * o));
      r.v1 = *reinterpret_cast<const uint16_t*>(block + int4_v_half(D, slot, 2 * o) + kSecond);
      r.kp = *reinterpret_cast<const uint32_t*>(block + kp_at + pair);
      r.vp = *reinterpret_cast<const uint32_t*>(block + vp_at + pair);
    }
    if (++s_next == end) s_next = begin, ++t_next;
    return r;
  };
  Raw next = load();
#pragma unroll 1
  for (int t = 0; t < count; ++t) {
    uint16_t* k_out = p.k_out + (i0 + t) * p.k_stride + sub * D + 8 * o;
    uint16_t* v_out = p.v_out + (i0 + t) * p.v_stride + sub * D + 8 * o;
#pragma unroll 2
    for (int s = begin; s < end; ++s) {
      const Raw r = next;
      const bool ok = ok_next;
      next = load();
      if (!ok) continue;
      *reinterpret_cast<uint4*>(k_out + s * (kRows * D)) = values8(r.k, r.kp);
      *reinterpret_cast<uint4*>(v_out + s * (kRows * D)) = values8(r.v0 | (r.v1 << 16), r.vp);
    }
  }
}

// Slots of a token for one warp: as many as leave the GPU 24 warps an SM.  A
// token's place and angles are then read once, not once a slot.
int slots_of(int n, int slots) {
  return int(std::min<int64_t>(slots, std::max<int64_t>(1, int64_t(n) * slots / (152 * 24))));
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
  const int slots_per_warp = slots_of(p.n, slots);
  unsigned blocks = 0;
  const cudaError_t e = grid_of(int64_t(p.n) * ((slots + slots_per_warp - 1) / slots_per_warp), &blocks);
  if (e != cudaSuccess) return e;
  auto* kernel = p.c.d == 128 ? (p.interleaved ? rope_append_kernel<128, true> : rope_append_kernel<128, false>)
                              : (p.interleaved ? rope_append_kernel<64, true> : rope_append_kernel<64, false>);
  return launch_pdl(kernel, dim3(blocks), dim3(kAppendThreads), 0, stream, p, slots_per_warp);
}

cudaError_t launch_gather_int4(const GatherParams& p, cudaStream_t stream) {
  const int rows = 32 / (p.c.d / 8), slots = (p.c.n_kv + rows - 1) / rows;
  const int slots_per_warp = slots_of(p.n, slots);
  // up to 4 tokens a warp, where that leaves the GPU 24 warps an SM (64k tokens:
  // 73 us with one, 57 with 4, 64 with 8)
  const int tokens = slots_per_warp == slots ? std::min(4, std::max(1, p.n / (152 * 24))) : 1;
  unsigned blocks = 0;
  const cudaError_t e = grid_of((int64_t(p.n) + tokens - 1) / tokens * ((slots + slots_per_warp - 1) / slots_per_warp), &blocks);
  if (e != cudaSuccess) return e;
  auto* kernel = p.c.d == 128 ? gather_kernel<128> : gather_kernel<64>;
  return launch_pdl(kernel, dim3(blocks), dim3(kAppendThreads), 0, stream, p, slots_per_warp, tokens);
}

}  // namespace oscar
