// Rows of attention heads: norm and rotation of q and k (norm_rope), the same
// with k and v quantised to 8 bits into pages (rope_append_int8), and cached rows
// back as bf16 (gather_int8).
//
// One lane holds an octet of adjacent channels (16 bytes of bf16), d / 8 lanes a
// row, so a warp holds 32 / (d / 8) rows at a time (a slot).  With r the row's
// 1 / sqrt(mean x^2 + eps), w the weights and (c, s) a pair's angle, a rotated
// channel is r (own C + other S): C = c w_own, S = -+ s w_other.  C and S belong to
// a lane and a token, so every head of the token takes two products a channel;
// `other` is the partner octet (by shuffle) or the octet's own pairs swapped.
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

// The block of (req, pos), KV head 0, or nullptr (skip) for a padding row, a
// place outside the table or a page outside the pool.
template <int D>
__device__ __forceinline__ uint8_t* token_block(const PagedCache& c, int req, int pos, bool report) {
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
  return c.pages + int64_t(page) * c.n_kv * int8_block_bytes(D);
}

// A lane's share of a token's angles: its octet turns (or is not part of a
// rotated pair), with its partner's channels from lane `partner`.
struct Angles {
  const float* row;   // of cos_sin, at this octet's first angle
  int half;           // to the sines
  int partner;
  bool on, first;     // rotated; the first of the two halves
};

template <bool Interleaved>
__device__ __forceinline__ Angles angles_of(const RopeParams& r, int64_t at, int o, int lane) {
  const int h = r.rot / 16;                 // octets of a half
  Angles a;
  a.on = o < 2 * h;
  a.first = o < h;
  a.partner = Interleaved || !a.on ? lane : a.first ? lane + h : lane - h;
  a.half = r.rot / 2;
  a.row = r.cos_sin + at * r.rot + (Interleaved ? 4 * o : 8 * (a.first ? o : o - h));
  return a;
}

// C and S of the lane's octet; w: the norm's weights or NULL.
struct Factors {
  float2 c[4], s[4];
};
template <int D, bool Interleaved>
__device__ __forceinline__ Factors factors_of(const Angles& a, const uint16_t* w, int o, int lane) {
  float own[8], other[8], c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) own[e] = other[e] = c[e] = 1.f, s[e] = 0.f;
  if (w) {
    unpack_bf16x8(*reinterpret_cast<const uint4*>(w + 8 * o), own);
    if (Interleaved) {
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = own[e ^ 1];
    } else {
      unpack_bf16x8(*reinterpret_cast<const uint4*>(w + 8 * (o + a.partner - lane)), other);
    }
  }
  if (a.on) {
    if (Interleaved) {
      float c4[8], s4[8];
      load8(c4, a.row, 4);
      load8(s4, a.row + a.half, 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = c4[e / 2], s[e] = e & 1 ? s4[e / 2] : -s4[e / 2];
    } else {
      load8(c, a.row, 8);
      load8(s, a.row + a.half, 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = a.first ? -s[e] : s[e];
    }
  }
  Factors f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.c[i] = make_float2(c[2 * i] * own[2 * i], c[2 * i + 1] * own[2 * i + 1]);
    f.s[i] = make_float2(s[2 * i] * other[2 * i], s[2 * i + 1] * other[2 * i + 1]);
  }
  return f;
}

// Norms (where `norm`) and rotates the octet held in `raw`; whole warps call it.
// fp32 throughout: the sum of squares in a fixed order, one rounding to bf16.
template <int D, bool Interleaved>
__device__ __forceinline__ void turn8(uint4& raw, const Factors& f, const Angles& a, bool rotate, bool norm, float eps) {
  const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t y[4];
  if (rotate) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = Interleaved ? __funnelshift_l(x[i], x[i], 16) : __shfl_sync(0xffffffffu, x[i], a.partner);
  }
  float r = 1.f;
  if (norm) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = bf16_pair(x[i]);
      sum = fma2(v, v, sum);
    }
    float all = sum.x + sum.y;
#pragma unroll
    for (int m = 1; m < D / 8; m <<= 1) all += __shfl_xor_sync(0xffffffffu, all, m);
    r = rsqrtf(fmaf(all, 1.f / D, eps));
  }
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 v = mul2(bf16_pair(x[i]), f.c[i]);
    if (rotate && a.on) v = fma2(bf16_pair(y[i]), f.s[i], v);   // (an infinite partner is none of an octet that stays)
    if (norm) v = mul2(v, twice(r));
    out[i] = pack_bf162(v.x, v.y);
  }
  raw = make_uint4(out[0], out[1], out[2], out[3]);
}

// Quantises the row of which this lane holds the 8 bf16 values u, over `Lanes`
// lanes: zero = the least value, rounded down to fp16; scale = (greatest - zero) /
// 255, rounded up, so that no value lies outside the codes; code = (x - zero) /
// scale to nearest even, of exact differences and quotients.  *pair = (scale, zero);
// held: zero + scale code, rounded to fp32 and that to bf16.
//
// The extremes are taken on packed bf16 (max x, max -x).  The scale is a product with
// 1/255 rounded up, and one fp16 less where that still reaches the greatest value (255 s
// has 19 bits, exact in fp32).  A quotient is taken by an approximate reciprocal
// and checked: its error is below 255 (2^-22 + 2^-24) < 1e-4 of a step, and where the
// remainder t - k s (one fma) comes within 2e-4 of half a step it is divided out.
template <int Lanes, bool Held>
__device__ __forceinline__ uint2 quantise8(const uint4& u, float tau, uint32_t* pair, uint4* held) {
  const uint32_t hi2 = max_bf16x2(max_bf16x2(u.x, u.y), max_bf16x2(u.z, u.w));
  const uint32_t lo2 = max_bf16x2(max_bf16x2(u.x ^ 0x80008000u, u.y ^ 0x80008000u),
                                  max_bf16x2(u.z ^ 0x80008000u, u.w ^ 0x80008000u));
  uint32_t ends = max_bf16x2(prmt(hi2, lo2, 0x5410), prmt(hi2, lo2, 0x7632));   // (max x, max -x)
#pragma unroll
  for (int m = 1; m < Lanes; m <<= 1) ends = max_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, m));
  float hi = bf16_lo(ends), lo = -bf16_hi(ends);
  float x[8];
  unpack_bf16x8(u, x);
  if (!(hi <= tau && lo >= -tau)) {       // beyond tau, or a NaN, which becomes -tau; the test is the row's
    hi = -tau, lo = tau;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = fminf(fmaxf(x[i], -tau), tau);
      hi = fmaxf(hi, x[i]);
      lo = fminf(lo, x[i]);
    }
    const uint32_t row = Lanes == 32 ? 0xffffffffu : ((1u << Lanes) - 1) << (threadIdx.x & 31 & ~(Lanes - 1));
#pragma unroll
    for (int m = 1; m < Lanes; m <<= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(row, hi, m));
      lo = fminf(lo, __shfl_xor_sync(row, lo, m));
    }
  }
  const __half zh = __float2half_rd(lo);
  const float z = __half2float(zh), range = __fsub_ru(hi, z);
  uint32_t sh = __half_as_ushort(__float2half_ru(__fmul_ru(range, 0x1.010102p-8f)));   // (just above 1 / 255)
  if (sh && 255.f * __half2float(__ushort_as_half(uint16_t(sh - 1))) >= range) --sh;
  const float s = __half2float(__ushort_as_half(uint16_t(sh)));
  *pair = sh | (uint32_t(__half_as_ushort(zh)) << 16);
  const float inv = rcp_fast(s), half = s * 0.4998f;
  constexpr float kRound = 12582912.f;   // 1.5 2^23: the sum's low byte is the rounded integer
  float k[8];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = x[i] - z;
    k[i] = fmaf(t, inv, kRound);
    near = near | (fabsf(fmaf(kRound - k[i], s, t)) >= half);
  }
  if (!(s > 0.f)) {                       // a constant row that fp16 holds
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = kRound;
  } else if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = kRound + rintf(__fdiv_rn(sub_odd(x[i], z), s));
  }
  if (Held) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(k[i] - kRound, s, z);
    *held = pack_bf16x8(v);
  }
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(k[i]);
  return make_uint2(prmt(prmt(b[0], b[1], 0x0040), prmt(b[2], b[3], 0x0040), 0x5410),
                    prmt(prmt(b[4], b[5], 0x0040), prmt(b[6], b[7], 0x0040), 0x5410));
}

// One warp takes `slots_per_warp` slots of one token: its q heads four slots at a
// time, whose loads are in flight together, then its k and v heads.
template <int D, bool Interleaved, bool Append>
__global__ void __launch_bounds__(kRowThreads, 7)
    head_rows_kernel(const __grid_constant__ HeadRowsParams p, int slots_per_warp) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = 4;
  const int lane = threadIdx.x & 31, o = lane % kLanes, sub = lane / kLanes;
  const int sq = p.q ? (p.c.n_q + kRows - 1) / kRows : 0, sk = p.k ? (p.c.n_kv + kRows - 1) / kRows : 0;
  const int slots = sq + sk * (Append ? 2 : 1), warps_per_token = (slots + slots_per_warp - 1) / slots_per_warp;
  const int64_t w = (int64_t(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
  const int64_t i = w / warps_per_token;
  if (i >= p.n) return;
  const int part = int(w - i * warps_per_token);
  const bool report = part == 0 && lane == 0;
  uint8_t* base = nullptr;
  int64_t at = 0;
  int slot = 0;
  if (Append) {
    const int pos = p.dst_pos[i];
    base = token_block<D>(p.c, p.dst_req[i], pos, report);
    if (!base) return;
    slot = pos % kPageTokens;
    at = pos;
  }
  const bool rotate = p.rope.rot != 0;
  if (rotate) {
    if (p.rope_pos) at = p.rope_pos[i];
    if (!Append && at == -1) return;       // a padding row
    if (at < 0 || at >= p.rope.n_positions) {
      if (report) flag(p.c.dev_status, OSCAR_DEV_LENGTH);
      return;
    }
  }
  const Angles a = angles_of<Interleaved>(p.rope, at, o, lane);
  const int begin = part * slots_per_warp, end = min(slots, begin + slots_per_warp);

  auto rows = [&](int from, int to, int heads, const uint16_t* src, uint16_t* dst, const uint16_t* weight) {
    const Factors f = factors_of<D, Interleaved>(a, weight, o, lane);
    src += sub * D + 8 * o;
    dst += sub * D + 8 * o;
#pragma unroll 1
    for (int s0 = from; s0 < to; s0 += kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        if (s0 + u < to && (s0 + u) * kRows + sub < heads)
          raw[u] = *reinterpret_cast<const uint4*>(src + (s0 + u) * (kRows * D));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (s0 + u >= to) break;
        turn8<D, Interleaved>(raw[u], f, a, rotate, weight != nullptr, p.eps);
        if ((s0 + u) * kRows + sub < heads) *reinterpret_cast<uint4*>(dst + (s0 + u) * (kRows * D)) = raw[u];
      }
    }
  };
  if (begin < sq) rows(begin, min(end, sq), p.c.n_q, p.q + i * p.q_stride, p.q_out + i * p.q_out_stride, p.q_weight);
  if (end <= sq) return;
  if (!Append) {
    rows(max(begin - sq, 0), end - sq, p.c.n_kv, p.k + i * p.k_stride, p.k_out + i * p.k_out_stride, p.k_weight);
    return;
  }
  // k, then v, with the next slot's load ahead of the present one's work
  const Factors f = factors_of<D, Interleaved>(a, p.k_weight, o, lane);
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
    const int64_t row = (i * p.c.n_kv + head) * D + 8 * o;
    if (!is_v) {
      turn8<D, Interleaved>(raw, f, a, rotate, p.k_weight != nullptr, p.eps);
      if (p.k_out && valid) *reinterpret_cast<uint4*>(p.k_out + row) = raw;
    }
    uint32_t pair;
    uint4 held;
    const uint2 codes = quantise8<kLanes, true>(raw, is_v ? p.tau_v : p.tau_k, &pair, &held);   // of the rounded row
    if (!valid) continue;
    uint8_t* block = base + int64_t(head) * int8_block_bytes(D);
    *reinterpret_cast<uint2*>(block + (is_v ? 16 * D : 0) + int8_octet(D, slot, o)) = codes;
    if (o == 0) *reinterpret_cast<uint32_t*>(block + int8_pairs(D, slot) + (is_v ? 4 : 0)) = pair;
    uint16_t* out = is_v ? p.v_held : p.k_held;
    if (out) *reinterpret_cast<uint4*>(out + row) = held;
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
    const uint8_t* base = token_block<D>(p.c, p.src_req[i0 + lane], pos, part == 0);
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
  const int rows = 32 / (p.c.d / 8);
  const int slots = (p.q ? (p.c.n_q + rows - 1) / rows : 0) + (p.k ? (Append ? 2 : 1) * ((p.c.n_kv + rows - 1) / rows) : 0);
  const int slots_per_warp = slots_of(p.n, slots);
  unsigned blocks = 0;
  const cudaError_t e = grid_of(int64_t(p.n) * ((slots + slots_per_warp - 1) / slots_per_warp), &blocks);
  if (e != cudaSuccess) return e;
  auto* kernel = p.c.d == 128 ? (p.rope.interleaved ? head_rows_kernel<128, true, Append> : head_rows_kernel<128, false, Append>)
                              : (p.rope.interleaved ? head_rows_kernel<64, true, Append> : head_rows_kernel<64, false, Append>);
  return launch_pdl(kernel, dim3(blocks), dim3(kRowThreads), 0, stream, p, slots_per_warp);
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
