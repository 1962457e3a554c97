// Rows of attention heads: norm and rotation of q and k (norm_rope), the same
// with k and v quantised to 8 bits into pages (rope_append_int8), and cached rows
// back as bf16 (gather_int8).
//
// Norm, rotation, quantisation: a lane holds two octets of channels (16 bytes of bf16
// each) that turn with one another, d / 16 lanes a row, so a warp holds 32 / (d / 16)
// rows at a time (a slot).  With r the row's 1 / sqrt(mean x^2 + eps), w the weights and
// (c, s) a pair's angle, a rotated channel is r (own C + other S): C = c w_own, S = -+ s
// w_other.  C and S belong to a lane and a token, so every head of the token takes two
// products a channel.  (With an octet a lane and its partner by shuffle, every channel
// was unpacked twice and every row reduced by twice the lanes: 30k tokens appended in 157
// us where two octets a lane took 149, before the steps that follow.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "int8.h"
#include "kernels.h"
#include "oscar.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace oscar {
namespace {

// Lane i's octets of a row, e0 and e1, and their angles.
template <bool Interleaved>
struct Angles {
  int e0, e1;
  bool on0, on1;      // they turn (in halves: with one another)
  const float* row;   // of cos_sin, at the first angle of e0
  int half;           // to the sines
  __device__ __forceinline__ Angles(const RopeParams& r, int i) {
    const int h = r.rot / 16;               // octets of a half
    on0 = Interleaved ? 2 * i < 2 * h : i < h;
    on1 = Interleaved ? 2 * i + 1 < 2 * h : on0;
    e0 = Interleaved || !on0 ? 2 * i : i;
    e1 = Interleaved || !on0 ? 2 * i + 1 : i + h;
    half = r.rot / 2;
    row = nullptr;
  }
  __device__ __forceinline__ void turn_to(const RopeParams& r, int64_t at) {
    if (on0) row = r.cos_sin + at * r.rot + (Interleaved ? 4 : 8) * e0;
  }
};

// C and S of the lane's octets; w: the norm's weights or NULL.
struct Factors {
  float2 c0[4], s0[4], c1[4], s1[4];
};
template <bool Interleaved>
__device__ __forceinline__ void factors_of(Factors* f, const Angles<Interleaved>& a, const uint16_t* w) {
  float w0[8], w1[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w0[e] = w1[e] = 1.f;
  if (w) {
    unpack_bf16x8(*reinterpret_cast<const uint4*>(w + 8 * a.e0), w0);
    unpack_bf16x8(*reinterpret_cast<const uint4*>(w + 8 * a.e1), w1);
  }
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
  if (Interleaved) {                        // pairs 0 .. 3 of e0, then of e1
    if (a.on0) load8(c, a.row, 4), load8(s, a.row + a.half, 4);
    if (a.on1) {
      const float4 u = *reinterpret_cast<const float4*>(a.row + 4), v = *reinterpret_cast<const float4*>(a.row + a.half + 4);
      c[4] = u.x, c[5] = u.y, c[6] = u.z, c[7] = u.w;
      s[4] = v.x, s[5] = v.y, s[6] = v.z, s[7] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f->c0[i] = make_float2(c[i] * w0[2 * i], c[i] * w0[2 * i + 1]);
      f->s0[i] = make_float2(-s[i] * w0[2 * i + 1], s[i] * w0[2 * i]);
      f->c1[i] = make_float2(c[4 + i] * w1[2 * i], c[4 + i] * w1[2 * i + 1]);
      f->s1[i] = make_float2(-s[4 + i] * w1[2 * i + 1], s[4 + i] * w1[2 * i]);
    }
  } else {
    if (a.on0) load8(c, a.row, 8), load8(s, a.row + a.half, 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f->c0[i] = make_float2(c[2 * i] * w0[2 * i], c[2 * i + 1] * w0[2 * i + 1]);
      f->s0[i] = make_float2(-s[2 * i] * w1[2 * i], -s[2 * i + 1] * w1[2 * i + 1]);
      f->c1[i] = make_float2(c[2 * i] * w1[2 * i], c[2 * i + 1] * w1[2 * i + 1]);
      f->s1[i] = make_float2(s[2 * i] * w0[2 * i], s[2 * i + 1] * w0[2 * i + 1]);
    }
  }
}

struct Octets {
  uint4 u0, u1;
};

// The mean of a row's squares, and eps; whole warps call it.
template <int D>
__device__ __forceinline__ float mean_square(const Octets& x, float eps) {
  const uint32_t u[4] = {x.u0.x, x.u0.y, x.u0.z, x.u0.w}, v[4] = {x.u1.x, x.u1.y, x.u1.z, x.u1.w};
  float2 sum = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = bf16_pair(u[i]), q = bf16_pair(v[i]);
    sum = fma2(p, p, sum);
    sum1 = fma2(q, q, sum1);
  }
  sum = add2(sum, sum1);
  float all = sum.x + sum.y;
#pragma unroll
  for (int m = 1; m < D / 16; m <<= 1) all += __shfl_xor_sync(0xffffffffu, all, m);
  return fmaf(all, 1.f / D, eps);
}

// Below this a mean may have lost squares below fp32's end (which takes an eps as small).
constexpr float kSmallMean = 0x1p-90f;

// Multiplies the octets of the rows with such a mean by 2^80, exactly; the rows' means then.
// Zeros without an eps are to stay zeros.  Whole warps call it.
template <int D>
__device__ __forceinline__ float raise(Octets& x, float mean, float eps) {
  const float up = mean < kSmallMean ? 0x1p80f : 1.f;
  auto times = [&](uint32_t& w) {
    const float2 p = bf16_pair(w);
    w = pack_bf162(p.x * up, p.y * up);
  };
  times(x.u0.x), times(x.u0.y), times(x.u0.z), times(x.u0.w);
  times(x.u1.x), times(x.u1.y), times(x.u1.z), times(x.u1.w);
  mean = mean_square<D>(x, eps * up * up);
  return mean == 0.f ? INFINITY : mean;
}

// Norms (where `norm`) and rotates the octets held in x; whole warps call it.
// fp32 throughout: the sum of squares in a fixed order, one rounding to bf16.
// Small: eps is below kSmallMean.  (For every eps in one kernel, the test and the second
// sum of squares cost the append 1 to 3 % and the rotation 4.)
template <int D, bool Interleaved, bool Small>
__device__ __forceinline__ void turn16(Octets& x, const Factors& f, const Angles<Interleaved>& a, bool norm, float eps) {
  float r = 1.f;
  if (norm) {
    float mean = mean_square<D>(x, eps);
    if (Small && __any_sync(0xffffffffu, mean < kSmallMean)) mean = raise<D>(x, mean, eps);
    r = rsqrtf(mean);
  }
  const uint32_t u[4] = {x.u0.x, x.u0.y, x.u0.z, x.u0.w}, v[4] = {x.u1.x, x.u1.y, x.u1.z, x.u1.w};
  uint32_t out0[4], out1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = bf16_pair(u[i]), q = bf16_pair(v[i]);
    float2 y = mul2(p, f.c0[i]), z = mul2(q, f.c1[i]);
    // (a channel that stays takes nothing of a partner that may be infinite)
    if (a.on0) y = fma2(Interleaved ? make_float2(p.y, p.x) : q, f.s0[i], y);
    if (a.on1) z = fma2(Interleaved ? make_float2(q.y, q.x) : p, f.s1[i], z);
    y = mul2(y, twice(r)), z = mul2(z, twice(r));
    out0[i] = pack_bf162(y.x, y.y);
    out1[i] = pack_bf162(z.x, z.y);
  }
  x.u0 = make_uint4(out0[0], out0[1], out0[2], out0[3]);
  x.u1 = make_uint4(out1[0], out1[1], out1[2], out1[3]);
}

// (max x, max -x) of the 8 bf16 values of u
__device__ __forceinline__ uint32_t ends8(const uint4& u) {
  const uint32_t hi2 = max_bf16x2(max_bf16x2(u.x, u.y), max_bf16x2(u.z, u.w));
  const uint32_t lo2 = max_bf16x2(max_bf16x2(u.x ^ 0x80008000u, u.y ^ 0x80008000u),
                                  max_bf16x2(u.z ^ 0x80008000u, u.w ^ 0x80008000u));
  return max_bf16x2(prmt(hi2, lo2, 0x5410), prmt(hi2, lo2, 0x7632));
}

// A row's scale and zero, of which this lane holds the 16 bf16 values u, over `Lanes`
// lanes: zero = the least value, rounded down to fp16; scale = (greatest - zero) / 255,
// rounded up, so that no value lies outside the codes.
//
// The extremes are taken on packed bf16.  The scale is a product with 1/255 rounded up,
// and one fp16 less where that still reaches the greatest value (255 s has 19 bits,
// exact in fp32).
struct RowScale {
  float s, z;
  uint32_t pair;      // (s, z), fp16 bits
  bool clamped;       // some of its values lie beyond tau
};
template <int Lanes>
__device__ __forceinline__ RowScale scale_of(const Octets& u, float tau) {
  uint32_t ends = max_bf16x2(ends8(u.u0), ends8(u.u1));
#pragma unroll
  for (int m = 1; m < Lanes; m <<= 1) ends = max_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, m));
  float hi = bf16_lo(ends), lo = -bf16_hi(ends);
  RowScale r;
  r.clamped = !(hi <= tau && lo >= -tau);   // or a NaN, which becomes -tau; the test is the row's
  if (r.clamped) {
    const uint32_t w[8] = {u.u0.x, u.u0.y, u.u0.z, u.u0.w, u.u1.x, u.u1.y, u.u1.z, u.u1.w};
    hi = -tau, lo = tau;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = bf16_pair(w[i]);
      const float y0 = fminf(fmaxf(x.x, -tau), tau), y1 = fminf(fmaxf(x.y, -tau), tau);
      hi = fmaxf(hi, fmaxf(y0, y1));
      lo = fminf(lo, fminf(y0, y1));
    }
    const uint32_t row = ((1u << Lanes) - 1) << (threadIdx.x & 31 & ~(Lanes - 1));
#pragma unroll
    for (int m = 1; m < Lanes; m <<= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(row, hi, m));
      lo = fminf(lo, __shfl_xor_sync(row, lo, m));
    }
  }
  const __half zh = __float2half_rd(lo);
  r.z = __half2float(zh);
  const float range = __fsub_ru(hi, r.z);
  uint32_t sh = __half_as_ushort(__float2half_ru(__fmul_ru(range, 0x1.010102p-8f)));   // (just above 1 / 255)
  if (sh && 255.f * __half2float(__ushort_as_half(uint16_t(sh - 1))) >= range) --sh;
  r.s = __half2float(__ushort_as_half(uint16_t(sh)));
  r.pair = sh | (uint32_t(__half_as_ushort(zh)) << 16);
  return r;
}

// The codes of an octet: (x - zero) / scale to nearest even, of exact differences and
// quotients.  *held: zero + scale code, rounded to fp32 and that to bf16.
//
// A quotient is taken by an approximate reciprocal and checked: its error is below
// 255 (2^-22 + 2^-24) < 1e-4 of a step, and where the remainder t - k s (one fma) comes
// within 2e-4 of half a step it is divided out.  (An octet at a time: with the row's
// sixteen values at once the kernel spilled more; so it spills 8 bytes, for heads of 128 in
// halves alone.)
__device__ __forceinline__ uint2 encode8(const uint4& u, const RowScale& r, float tau, uint4* held) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float2 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = bf16_pair(w[i]);
  if (r.clamped)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = make_float2(fminf(fmaxf(x[i].x, -tau), tau), fminf(fmaxf(x[i].y, -tau), tau));
  constexpr float kRound = 12582912.f;   // 1.5 2^23: the sum's low byte is the rounded integer
  const float2 inv = twice(rcp_fast(r.s));
  float2 k[4];
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = add2(x[i], twice(-r.z));
    k[i] = fma2(t, inv, twice(kRound));
    const float2 rest = fma2(fma2(k[i], twice(-1.f), twice(kRound)), twice(r.s), t);
    off = fmaxf(off, fmaxf(fabsf(rest.x), fabsf(rest.y)));
  }
  if (!(r.s > 0.f)) {                     // a constant row that fp16 holds
#pragma unroll
    for (int i = 0; i < 4; ++i) k[i] = twice(kRound);
  } else if (off >= r.s * 0.4998f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      k[i] = make_float2(kRound + rintf(__fdiv_rn(sub_odd(x[i].x, r.z), r.s)), kRound + rintf(__fdiv_rn(sub_odd(x[i].y, r.z), r.s)));
  }
  uint32_t b[4], v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = fma2(fma2(k[i], twice(-1.f), twice(kRound)), twice(-r.s), twice(r.z));
    v[i] = pack_bf162(y.x, y.y);
    b[i] = prmt(__float_as_uint(k[i].x), __float_as_uint(k[i].y), 0x0040);
  }
  *held = make_uint4(v[0], v[1], v[2], v[3]);
  return make_uint2(prmt(b[0], b[1], 0x5410), prmt(b[2], b[3], 0x5410));
}

// One warp takes `slots_per_warp` slots of one token: its q heads two slots at a
// time, then its k and v heads, the next loads ahead of the present work and the first
// ones ahead of the token's place.
//
// Bound by issue and by the bytes that the warps keep in flight (30k tokens appended, 821
// MB: 145 us, 5.6 TB/s, 83 % of a plain copy's rate, issue 62 %; the
// quantisation costs some 19 us of it; normed and rotated only, 634 MB: 97 us, 96 %).  Set
// aside, each measured on the append when it took 149: rows by bulk copies into rings
// that run ahead over several tokens (176: more instructions a row), k and v rows side
// by side (151, spilled), q rows and k, v rows in CTAs of their own (157), four or six CTAs
// an SM (153, 150), a value's two octets' codes in one store (145).
template <int D, bool Interleaved, bool Append, bool Small>
__global__ void __launch_bounds__(kRowThreads, 5)
    head_rows_kernel(const __grid_constant__ HeadRowsParams p, int slots_per_warp) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kBatch = 2;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, li = lane % kLanes;
  const int sq = p.q ? (p.c.n_q + kRows - 1) / kRows : 0, sk = p.k ? (p.c.n_kv + kRows - 1) / kRows : 0;
  const int slots = sq + sk * (Append ? 2 : 1), warps_per_token = (slots + slots_per_warp - 1) / slots_per_warp;
  const int64_t w = (int64_t(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
  const int64_t i = w / warps_per_token;
  if (i >= p.n) return;
  const int part = int(w - i * warps_per_token), begin = part * slots_per_warp, end = min(slots, begin + slots_per_warp);
  Angles<Interleaved> a(p.rope, li);
  const int e0 = a.e0, e1 = a.e1;

  // The lane's octets of slot s (zeros from slot `to` and past the last head).  Rows are read
  // and written once, so both are marked for early eviction (rotation 101 us without, 98 with).
  auto load = [&](const uint16_t* row, int s, int to, int heads) {
    Octets x;
    x.u0 = x.u1 = make_uint4(0, 0, 0, 0);
    const int head = s * kRows + sub;
    if (s < to && head < heads) {
      x.u0 = __ldcs(reinterpret_cast<const uint4*>(row + head * D + 8 * e0));
      x.u1 = __ldcs(reinterpret_cast<const uint4*>(row + head * D + 8 * e1));
    }
    return x;
  };
  auto store = [&](uint16_t* row, int head, const Octets& x) {
    __stcs(reinterpret_cast<uint4*>(row + head * D + 8 * e0), x.u0);
    __stcs(reinterpret_cast<uint4*>(row + head * D + 8 * e1), x.u1);
  };
  const uint16_t* q_row = p.q + i * p.q_stride;
  const uint16_t* k_row = p.k + i * p.k_stride;
  const int end_q = min(end, sq);
  Octets first[kBatch];
  if (begin < sq)
#pragma unroll
    for (int u = 0; u < kBatch; ++u) first[u] = load(q_row, begin + u, end_q, p.c.n_q);

  const bool report = part == 0 && lane == 0;
  uint8_t* base = nullptr;
  int64_t at = 0;
  int slot = 0;
  if (Append) {
    const int pos = p.dst_pos[i];
    base = block_of_token(p.c, int8_block_bytes(D), p.dst_req[i], pos, report);
    if (!base) return;
    slot = pos % kPageTokens;
    at = pos;
  }
  if (p.rope_pos) at = p.rope_pos[i];
  if (!Append && at == -1) return;         // a padding row
  if (p.rope.rot != 0 && (at < 0 || at >= p.rope.n_positions)) {
    if (report) flag(p.c.dev_status, OSCAR_DEV_LENGTH);
    return;
  }
  a.turn_to(p.rope, at);

  auto rows = [&](int from, int to, int heads, const uint16_t* src, uint16_t* dst, const uint16_t* weight, Octets (&next)[kBatch]) {
    Factors f;
    factors_of<Interleaved>(&f, a, weight);
#pragma unroll 1
    for (int s0 = from; s0 < to; s0 += kBatch) {
      Octets x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) x[u] = next[u], next[u] = load(src, s0 + kBatch + u, to, heads);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (s0 + u >= to) break;
        turn16<D, Interleaved, Small>(x[u], f, a, weight != nullptr, p.eps);
        const int head = (s0 + u) * kRows + sub;
        if (head < heads) store(dst, head, x[u]);
      }
    }
  };
  if (begin < sq) rows(begin, end_q, p.c.n_q, q_row, p.q_out + i * p.q_out_stride, p.q_weight, first);
  if (end <= sq) return;
  const int begin_k = max(begin - sq, 0), end_k = end - sq;   // among the slots of k (and v)
  if (!Append) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) first[u] = load(k_row, begin_k + u, end_k, p.c.n_kv);
    rows(begin_k, end_k, p.c.n_kv, k_row, p.k_out + i * p.k_out_stride, p.k_weight, first);
    return;
  }
  // (v does not turn: its octets lie side by side)
  const uint16_t* v_row = p.v + i * p.v_stride;
  const int64_t row = i * p.c.n_kv * D;
  auto load_kv = [&](int s) {
    if (s < sk) return load(k_row, s, end_k, p.c.n_kv);
    Octets x;
    x.u0 = x.u1 = make_uint4(0, 0, 0, 0);
    const int head = (s - sk) * kRows + sub;
    if (s < end_k && head < p.c.n_kv) {
      x.u0 = __ldcs(reinterpret_cast<const uint4*>(v_row + head * D + 16 * li));
      x.u1 = __ldcs(reinterpret_cast<const uint4*>(v_row + head * D + 16 * li) + 1);
    }
    return x;
  };
  Octets next = load_kv(begin_k);
  Factors f;
  factors_of<Interleaved>(&f, a, p.k_weight);
#pragma unroll 1
  for (int s = begin_k; s < end_k; ++s) {
    Octets x = next;
    next = load_kv(s + 1);
    const bool is_v = s >= sk;
    const int head = (is_v ? s - sk : s) * kRows + sub;
    const bool valid = head < p.c.n_kv;
    if (!is_v) {
      turn16<D, Interleaved, Small>(x, f, a, p.k_weight != nullptr, p.eps);
      if (p.k_out && valid) store(p.k_out + row, head, x);
    }
    const float tau = is_v ? p.tau_v : p.tau_k;
    const RowScale scale = scale_of<kLanes>(x, tau);   // of the rounded row
    if (!valid) continue;
    uint8_t* block = base + int64_t(head) * int8_block_bytes(D) + (is_v ? 16 * D : 0);
    uint16_t* out = is_v ? p.v_held : p.k_held;
    if (li == 0) *reinterpret_cast<uint32_t*>(block + int8_pairs(D, slot) + (is_v ? 4 - 16 * D : 0)) = scale.pair;
    const int o0 = is_v ? 2 * li : e0, o1 = is_v ? 2 * li + 1 : e1;
    uint4 held;
    *reinterpret_cast<uint2*>(block + int8_octet(D, slot, o0)) = encode8(x.u0, scale, tau, &held);
    if (out) __stcs(reinterpret_cast<uint4*>(out + row + head * D + 8 * o0), held);
    *reinterpret_cast<uint2*>(block + int8_octet(D, slot, o1)) = encode8(x.u1, scale, tau, &held);
    if (out) __stcs(reinterpret_cast<uint4*>(out + row + head * D + 8 * o1), held);
  }
}

// zero + scale * code of 8 codes, as bf16: a byte under the exponent of 2^23 is
// 2^23 + code, so no integer conversion (they are slow) is needed.
__device__ __forceinline__ uint4 values8(uint2 codes, uint32_t pair) {
  const float2 sz = half2_to_float2(pair), s = twice(sz.x), z = twice(sz.y), shift = twice(-8388608.f);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = i < 2 ? codes.x : codes.y;
    const float2 c = make_float2(__uint_as_float(prmt(word, 0x4B000000u, i & 1 ? 0x7542 : 0x7540)),
                                 __uint_as_float(prmt(word, 0x4B000000u, i & 1 ? 0x7543 : 0x7541)));
    const float2 v = fma2(add2(c, shift), s, z);
    out[i] = pack_bf162(v.x, v.y);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// A warp takes `slots_per_warp` slots (the KV heads that it holds at a time) of
// one token, or all slots of `tokens` tokens, whose places its lanes look up at
// once; the next slot's loads are ahead of the present one's work.
template <int D>
__global__ void __launch_bounds__(kRowThreads)
    gather_int8_kernel(const __grid_constant__ Gather8Params p, int slots_per_warp, int tokens) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, o = lane % kLanes, sub = lane / kLanes;
  const int slots = (p.c.n_kv + kRows - 1) / kRows, warps_per_token = (slots + slots_per_warp - 1) / slots_per_warp;
  const int64_t w = (int64_t(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
  const int64_t i0 = w / warps_per_token * tokens;
  if (i0 >= p.n) return;
  const int part = int(w % warps_per_token), count = int(min(int64_t(tokens), p.n - i0));
  uint64_t mine = 0;                      // lane t: token t's block and slot (blocks are 128-byte aligned)
  if (lane < count) {
    const int pos = p.src_pos[i0 + lane];
    const uint8_t* base = block_of_token(p.c, int8_block_bytes(D), p.src_req[i0 + lane], pos, part == 0);
    if (base) mine = reinterpret_cast<uint64_t>(base) | uint64_t(pos % kPageTokens);
  }
  const int begin = part * slots_per_warp, end = min(slots, begin + slots_per_warp);
  struct Raw {
    uint2 k, v, pairs;
  };
  int t_next = 0, s_next = begin;         // the next slot to ask for
  bool ok_next = false;                   // it is there
  auto load = [&]() {
    Raw r{};
    const uint64_t at = __shfl_sync(0xffffffffu, mine, min(t_next, 31));
    const int head = s_next * kRows + sub, slot = int(at & 15);
    ok_next = t_next < count && at != 0 && head < p.c.n_kv;
    if (ok_next) {
      const uint8_t* block = reinterpret_cast<const uint8_t*>(at & ~uint64_t(15)) + int64_t(head) * int8_block_bytes(D);
      const int octet = int8_octet(D, slot, o);
      r.k = *reinterpret_cast<const uint2*>(block + octet);
      r.v = *reinterpret_cast<const uint2*>(block + 16 * D + octet);
      r.pairs = *reinterpret_cast<const uint2*>(block + int8_pairs(D, slot));
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
      *reinterpret_cast<uint4*>(k_out + s * (kRows * D)) = values8(r.k, r.pairs.x);
      *reinterpret_cast<uint4*>(v_out + s * (kRows * D)) = values8(r.v, r.pairs.y);
    }
  }
}

template <bool Append>
cudaError_t launch_head_rows(const HeadRowsParams& p, cudaStream_t stream) {
  const int rows = 512 / p.c.d;           // of a slot
  const int slots = (p.q ? (p.c.n_q + rows - 1) / rows : 0) + (p.k ? (Append ? 2 : 1) * ((p.c.n_kv + rows - 1) / rows) : 0);
  const int slots_per_warp = slots_of(p.n, slots);
  unsigned blocks = 0;
  const cudaError_t e = grid_of(int64_t(p.n) * ((slots + slots_per_warp - 1) / slots_per_warp), &blocks);
  if (e != cudaSuccess) return e;
  auto launch = [&](auto* kernel) { return launch_pdl(kernel, dim3(blocks), dim3(kRowThreads), 0, stream, p, slots_per_warp); };
  const bool wide = p.c.d == 128, inter = p.rope.interleaved;
  if ((p.q_weight || p.k_weight) && p.eps < kSmallMean)
    return launch(wide ? (inter ? head_rows_kernel<128, true, Append, true> : head_rows_kernel<128, false, Append, true>)
                       : (inter ? head_rows_kernel<64, true, Append, true> : head_rows_kernel<64, false, Append, true>));
  return launch(wide ? (inter ? head_rows_kernel<128, true, Append, false> : head_rows_kernel<128, false, Append, false>)
                     : (inter ? head_rows_kernel<64, true, Append, false> : head_rows_kernel<64, false, Append, false>));
}

}  // namespace

cudaError_t launch_norm_rope(const HeadRowsParams& p, cudaStream_t stream) { return launch_head_rows<false>(p, stream); }
cudaError_t launch_rope_append_int8(const HeadRowsParams& p, cudaStream_t stream) { return launch_head_rows<true>(p, stream); }

cudaError_t launch_gather_int8(const Gather8Params& p, cudaStream_t stream) {
  const int rows = 32 / (p.c.d / 8), slots = (p.c.n_kv + rows - 1) / rows;
  const int slots_per_warp = slots_of(p.n, slots);
  // up to 4 tokens a warp, where that leaves the GPU 24 warps an SM
  const int tokens = slots_per_warp == slots ? std::min(4, std::max(1, p.n / (152 * 24))) : 1;
  unsigned blocks = 0;
  const cudaError_t e = grid_of((int64_t(p.n) + tokens - 1) / tokens * ((slots + slots_per_warp - 1) / slots_per_warp), &blocks);
  if (e != cudaSuccess) return e;
  auto* kernel = p.c.d == 128 ? gather_int8_kernel<128> : gather_int8_kernel<64>;
  return launch_pdl(kernel, dim3(blocks), dim3(kRowThreads), 0, stream, p, slots_per_warp, tokens);
}

}  // namespace oscar
