// Decode attention over a 4-bit layer: one query token per request.
//
// The pages of all (request, KV head, up to 8 query heads) runs stand in one row,
// and each of 304 lasting CTAs (two per SM) takes an equal share of it: a ragged
// batch is as even as a uniform one, and only the first and the last run of a
// share can be incomplete.  Those leave their unnormalised sums in the workspace,
// and the last CTA of a run to finish joins its parts.  (A grid of short CTAs, each
// for 16 pages a warp, took 139 us where this takes 97, 28 ragged requests: a third
// of it went into the CTAs' first loads and last sums.)
//
// Bound by: chains before and after the scan.  Of 100k tokens x 8 KV heads (32 us; 109
// MB, 16 us at the measured copy rate), cold: shares 1.5 us, a warp's first page at
// 6 (11 at the latest), scans done at 24 to 28, the warps' joins at 26 to 29, the
// runs' last parts joined at 34.  16 short windowed requests (16 us): shares 1.3, first
// pages 5 to 10, scans 10 to 12, warps' joins 11 to 14, parts joined 17.  Within the
// scan no unit is full (ragged batch with a cap: issue 54 %, ALU 46 %, DRAM 51 %): a
// warp's step is one chain, with four warps a scheduler.  At 128 registers the kernels
// for 128 channels spill 160 to 330 bytes a thread.  Code outside the scan is kept small
// on purpose: run once a CTA, its instructions come from far (unrolled joins cost 8 us).
// Groups of 9 to 16 query heads copy and unpack every page twice (100k tokens: group 8
// 35 us, group 16 52).
//
// A warp takes every 8th pair of a run's pages with an online softmax of its own,
// so nothing in the scan waits for another warp.  The pages' blocks come by bulk
// copies into a ring of the warp's own, the next run's ahead of the present one's
// end.
//
// Per page, on the tensor cores with 16 tokens or 16 channels as the rows and
// 8 query heads as the columns:
//   S = K q:     A = the K codes as they are: a code c in the low bits of an fp16
//                is c 2^-24 exactly (and c 2^-20 one nibble higher), so one mask
//                turns a word into two operands.  q is scaled by a power of two per
//                head to just below fp16's end, which is exact for bf16.
//                x = sum over groups of s (sum c q) + z (sum q).
//   O += V^T P:  A = the V codes the same way, B = P s_V.
//   Z += (z_V; 1) P:  the zeros' share of O and the softmax's sum.
// P and P s_V are rounded to fp16 (2^-11 each; the bf16 output has 2^-8); all sums
// are fp32.  (e4m3 operands would need fewer masks, but their mma.sync is not
// native here: 38 us against 32 for 100k tokens.)
// The weights' reference is raised only when a score exceeds it by 2^8, and
// the values' scales are taken relative to a power of two above them, raised
// when a larger one comes: both by one vote for two pages.  Where a warp's scales lie
// more than 2^14 apart, its segment is scanned anew in fp32 (scan_wide).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "decode_math.cuh"
#include "kernels.h"
#include "oscar.h"
#include "page_walk.cuh"
#include "ptx.cuh"
#include "score.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kHeads = 8;             // query heads per CTA (MMA columns)
constexpr int kStages = 2;            // ring stages of a warp, each two pages
constexpr int kCtas = 152 * 2;        // CTAs the GPU holds at a time
constexpr int kMinShare = 4 * kWarps; // pages
// A run costs its CTA about as much as this many pages besides its own (the
// query, the warps' join): a run takes up so many more places in the row.  (28
// ragged requests x 8 KV heads: 105 us with 8, 97 with 32, 95 with 64, 100 with 128;
// 16 short ones: 19, 17, 17, 22.)
constexpr int kRunCost = 64;
// A run of no more pages is not split: it goes whole to the CTA whose share holds
// its first page.  (Joining parts takes about as long as scanning these.)
constexpr int kWhole = 64;
constexpr int kJoinHeads = 4;         // heads whose states are joined at a time
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;

// Workspace: a ticket for each CTA (of the run that goes on behind its share),
// then two partial states for each, of a run that began before its share and of one
// that begins in it: (m, l) and the sums.
constexpr size_t kOffMl = 4096, kOffO = kOffMl + size_t(kCtas) * 2 * kHeads * 8;

template <int D>
constexpr int join_bytes() {
  // the warps' states of kJoinHeads heads; or the parts' weights and 256 partial sums
  return std::max(kWarps * kJoinHeads * D * 4, (kCtas + 1) * kHeads * 4 + kThreads * 16);
}

// N consecutive 32-bit words at a multiple of N words.
template <int N>
__device__ __forceinline__ void lds_n(uint32_t (&v)[N], const uint8_t* p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(p)[i];
      v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 x = reinterpret_cast<const uint2*>(p)[i];
      v[2 * i] = x.x, v[2 * i + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

using Walk = PageWalk<kRunCost, kWhole>;
// a warp's first pair of a segment
__device__ __forceinline__ int place_of(const Segment& s, int warp) { return (warp - (s.at >> 1)) & (kWarps - 1); }

// Joins the warps' states of heads h0 .. of a segment, 4 channels a thread: to `out`, or
// to the workspace's partial state `slot` if that is not negative.
template <int D>
__device__ __forceinline__ void join_warps(const Int4DecodeParams& p, int hq0, int h0, int heads, int slot, int b,
                                           const float* buf, const float (&sm_m)[kWarps][kHeads],
                                           const float (&sm_l)[kWarps][kHeads]) {
  const int i = threadIdx.x, h = h0 + i / (D / 4);
  if (i >= kJoinHeads * (D / 4) || h >= heads) return;
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  float mx = -FLT_MAX, sum = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (sm_l[w][h] > 0.f) mx = fmaxf(mx, sm_m[w][h]);
#pragma unroll 4
  for (int w = 0; w < kWarps; ++w) {
    const float l = sm_l[w][h], f = l > 0.f ? exp2_fast(sm_m[w][h] - mx) : 0.f;
    const float4 x = reinterpret_cast<const float4*>(buf)[w * kJoinHeads * (D / 4) + i];
    sum = fmaf(f, l, sum);
    v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
  }
  if (slot < 0) {
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    reinterpret_cast<uint2*>(p.out + (int64_t(b) * p.c.n_q + hq0) * D)[h0 * (D / 4) + i] =
        make_uint2(pack_bf162(v.x * inv, v.y * inv), pack_bf162(v.z * inv, v.w * inv));
  } else {
    reinterpret_cast<float4*>(ws + kOffO)[(int64_t(slot) * kHeads + h0) * (D / 4) + i] = v;
    if (i % (D / 4) == 0) reinterpret_cast<float2*>(ws + kOffMl)[slot * kHeads + h] = make_float2(mx, sum);
  }
}

// Scales, relative to 2^ve, that fp16 holds with fewer bits: below 2^(ve - 14).
// `least`: a lane's least ones that are not 0, less 1, as fp16 bits.  Whole warps.
__device__ __forceinline__ bool scales_wide(int ve, uint32_t least) {
  const int e = ve - 14;
  const uint32_t from = e >= -14 ? uint32_t(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 1u;
  return __any_sync(0xffffffffu, (least & 0xFFFFu) < from - 1 || (least >> 16) < from - 1);
}

// Once more, in fp32 throughout, those segments of the CTA's share whose values' scales
// lie further apart within a warp's pages than products of fp16 numbers hold.  (A token
// far above the others may have no weight, and the others are not to lose bits for it.)
// Rare, and slower: with one such value in each KV head 100k tokens take 181 us, with one
// in every page 216 (32 without).  Run after all segments, where nothing else is live: a
// call within the loop over them cost 7 % of every decode, the products in bands of
// scales there had the loop spill.
//
// A warp takes the pages it had, kJoinHeads heads at a time.  Lanes t and t + 16 take
// half a row each of token t for the scores, then each lane D / 32 channels of all
// tokens.  States as the scan leaves them, with the weights' 2^7.
template <int D, int NGK, int NGV>
__device__ __noinline__ void scan_wide(const Int4DecodeParams& p, Walk walk, int sets, int halves, float* buf_all,
                                       float (&sm_m)[kWarps][kHeads], float (&sm_l)[kWarps][kHeads]) {
  constexpr int C = D / 32, kBlock = int4_block_bytes(D, NGK, NGV);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 15, half = lane >> 4, ch = C * lane;
  const int group = p.c.n_q / p.c.n_kv;
  float* buf = buf_all + warp * kJoinHeads * D;
  Segment cur;
  __syncthreads();                          // the scan's states have been read
  while (walk.next(p, sets, &cur)) {
    const int hk = cur.h / halves, set = cur.h % halves, in_set = min(kHeads, group - set * kHeads);
    const int lo = cur.lo + 2 * place_of(cur, warp);
    const int32_t* table = p.c.page_table + int64_t(cur.b) * p.c.max_pages;
    auto page_of = [&](int i) { return lo + (i >> 1) * 2 * kWarps + (i & 1); };
    auto block_of = [&](int page) -> const uint8_t* {
      const int id = page < cur.hi ? table[page] : -1;
      return id < 0 || id >= p.c.n_pages ? nullptr : p.c.pages + (int64_t(id) * p.c.n_kv + hk) * kBlock;
    };
    // the scan's own test, a pair of pages at a time
    uint32_t top = 0, least = 0xFFFFFFFFu;
#pragma unroll 1
    for (int i = 0; page_of(i) < cur.hi; i += 2) {
      const int j = page_of(i + half) * kPageTokens + t;
      const uint8_t* block = block_of(page_of(i + half));
      if (block && j >= cur.first && j < cur.len)
#pragma unroll
        for (int g = 0; g < NGV; ++g) {
          const uint32_t s = *reinterpret_cast<const uint16_t*>(block + int4_pair(D, NGK, NGV, t, NGK + g));
          top = max(top, s);
          least = min(least, (s - 1) & 0xFFFFu);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (!__syncthreads_or(scales_wide(scale_exponent(top), least | 0xFFFF0000u))) continue;

#pragma unroll 1
    for (int h0 = 0; h0 < in_set; h0 += kJoinHeads) {
      const int heads = min(kJoinHeads, in_set - h0), hq0 = hk * group + set * kHeads + h0;
      const uint16_t* q = p.q + cur.b * p.q_stride + int64_t(hq0) * D;
      float m[kJoinHeads], l[kJoinHeads], o[kJoinHeads][C], slope[kJoinHeads];
#pragma unroll
      for (int h = 0; h < kJoinHeads; ++h) {
        m[h] = -FLT_MAX, l[h] = 0.f;
        slope[h] = p.s.slopes && h < heads ? p.s.slopes[hq0 + h] * kLog2e : 0.f;
#pragma unroll
        for (int n = 0; n < C; ++n) o[h][n] = 0.f;
      }
#pragma unroll 1
      for (int i = 0; page_of(i) < cur.hi; ++i) {
        const uint8_t* block = block_of(page_of(i));
        if (!block) continue;
        uint32_t vc[8], vp[16];
#pragma unroll
        for (int a = 0; a < 8; ++a) vc[a] = *reinterpret_cast<const uint32_t*>(block + int4_v_half(D, 2 * a, ch / 4)) >> (4 * (ch % 4));
#pragma unroll
        for (int a = 0; a < 16; ++a) vp[a] = *reinterpret_cast<const uint32_t*>(block + int4_pair(D, NGK, NGV, a, NGK + ch * NGV / D));
        float x[kJoinHeads] = {};
#pragma unroll 2
        for (int e = half * (D / 16); e < (half + 1) * (D / 16); ++e) {      // octets
          const uint32_t kc = *reinterpret_cast<const uint32_t*>(block + int4_k_word(D, t, e));
          const float2 ks = half2_to_float2(*reinterpret_cast<const uint32_t*>(block + int4_pair(D, NGK, NGV, t, 8 * e * NGK / D)));
          float k[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) k[n] = fmaf(float((kc >> (4 * n)) & 15u), ks.x, ks.y);
#pragma unroll
          for (int h = 0; h < kJoinHeads; ++h)
            if (h < heads) {
              const uint4 u = *reinterpret_cast<const uint4*>(q + h * D + 8 * e);
              x[h] = fmaf(bf16_lo(u.x), k[0], fmaf(bf16_hi(u.x), k[1], fmaf(bf16_lo(u.y), k[2], fmaf(bf16_hi(u.y), k[3], x[h]))));
              x[h] = fmaf(bf16_lo(u.z), k[4], fmaf(bf16_hi(u.z), k[5], fmaf(bf16_lo(u.w), k[6], fmaf(bf16_hi(u.w), k[7], x[h]))));
            }
        }
        const int j = page_of(i) * kPageTokens + t;
#pragma unroll
        for (int h = 0; h < kJoinHeads; ++h) {
          float y = x[h] + __shfl_xor_sync(0xffffffffu, x[h], 16);
          y = p.s.cap_log2 != 0.f ? capped(y * p.s.unit, p.s) : y * p.s.scale_log2;
          y = j >= cur.first && j < cur.len ? fmaf(slope[h], float(j - (cur.len - 1)), y) : -INFINITY;
          float mn = fmaxf(m[h], y);
#pragma unroll
          for (int n = 8; n; n >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, n));
          const float f = exp2_fast(m[h] - mn), g = exp2_fast(y - mn);
          m[h] = mn;
          float sum = g;
#pragma unroll
          for (int n = 8; n; n >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, n);
          l[h] = fmaf(l[h], f, sum);
#pragma unroll
          for (int n = 0; n < C; ++n) o[h][n] *= f;
#pragma unroll
          for (int a = 0; a < 16; ++a) {
            const float w = __shfl_sync(0xffffffffu, g, a);
            const float2 vs = half2_to_float2(vp[a]);
#pragma unroll
            for (int n = 0; n < C; ++n)
              if (w != 0.f)                     // (a stale slot holds anything; a NaN stays one)
                o[h][n] = fmaf(w, fmaf(float((vc[a / 2] >> (16 * (a & 1) + 4 * n)) & 15u), vs.x, vs.y), o[h][n]);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < kJoinHeads; ++h)
        if (h < heads) {
#pragma unroll
          for (int n = 0; n < C; ++n) buf[h * D + ch + n] = 128.f * o[h][n];
          if (lane == 0) sm_m[warp][h0 + h] = m[h], sm_l[warp][h0 + h] = 128.f * l[h];
        }
      __syncthreads();
      const bool whole = cur.off == 0 && cur.hi - cur.lo == cur.pages;
      join_warps<D>(p, hk * group + set * kHeads, h0, in_set, whole ? -1 : 2 * int(blockIdx.x) + (cur.off == 0), cur.b, buf_all, sm_m, sm_l);
      __syncthreads();                      // the states have been read
    }
  }
}

// A run in more than one share: its place in the row, pages, request, first
// query head and their number.
struct Part {
  int run, pages, b, hq0, heads;
};

// Joins the parts of a run; the whole CTA, 4 channels a thread.  Where the heads
// leave threads over, each takes every n-th part.  (Small code: it runs once a
// CTA, when its instructions have to come from far.)
template <int D>
__device__ __noinline__ void join_parts(const Int4DecodeParams& p, const Part& r, int share, float* wt, float* sum_of) {
  const uint8_t* ws = static_cast<const uint8_t*>(p.workspace);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = r.heads;
  const int f = r.run / share, n = (r.run + r.pages - 1) / share - f + 1;
  auto slot_of = [&](int i) { return 2 * (f + i) + (i == 0); };
  // the first sums are asked for before their weights are worked out
  constexpr int kBatch = 10;
  const int units = heads * (D / 4), ways = kThreads / units, way = threadIdx.x / units, unit = threadIdx.x % units;
  const int h = unit / (D / 4);
  const float4* from = reinterpret_cast<const float4*>(ws + kOffO) + unit;
  auto load = [&](float4 (&x)[kBatch], int i) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) x[k] = __ldcg(from + slot_of(min(i + k * ways, n - 1)) * (kHeads * D / 4));
  };
  float4 x[kBatch];
  load(x, way);
  const float2* ml = reinterpret_cast<const float2*>(ws + kOffMl) + warp;
  if (warp < heads) {                     // warp h: head h
    float mx = -FLT_MAX, sum = 0.f;
#pragma unroll 2
    for (int i = lane; i < n; i += 32) {
      const float2 s = __ldcg(&ml[slot_of(i) * kHeads]);
      const float m = s.y > 0.f ? s.x : -FLT_MAX, mn = fmaxf(mx, m);
      sum = fmaf(exp2_fast(m - mn), s.y, sum * exp2_fast(mx - mn));
      mx = mn;
      wt[i * kHeads + warp] = m;
    }
    float all = mx;
#pragma unroll
    for (int i = 16; i; i >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, i));
    sum *= exp2_fast(mx - all);
#pragma unroll
    for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
#pragma unroll 1
    for (int i = lane; i < n; i += 32) wt[i * kHeads + warp] = exp2_fast(wt[i * kHeads + warp] - all);
    if (lane == 0) sum_of[warp] = sum;
  }
  __syncthreads();
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (way < ways)
#pragma unroll 1
    for (int i = way; i < n; i += kBatch * ways) {
      if (i != way) load(x, i);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float g = i + k * ways < n ? wt[(i + k * ways) * kHeads + h] : 0.f;
        v.x = fmaf(g, x[k].x, v.x), v.y = fmaf(g, x[k].y, v.y), v.z = fmaf(g, x[k].z, v.z), v.w = fmaf(g, x[k].w, v.w);
      }
    }
  float4* sums = reinterpret_cast<float4*>(wt + n * kHeads);
  sums[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < units) {
#pragma unroll 1
    for (int i = 1; i < ways; ++i) {
      const float4 y = sums[i * units + unit];
      v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
    }
    const float inv = sum_of[h] > 0.f ? 1.f / sum_of[h] : 0.f;
    reinterpret_cast<uint2*>(p.out + (int64_t(r.b) * p.c.n_q + r.hq0) * D)[unit] =
        make_uint2(pack_bf162(v.x * inv, v.y * inv), pack_bf162(v.z * inv, v.w * inv));
  }
}

// Formed: the scores have a cap or a distance bias.
template <int D, int NGK, int NGV, bool Formed>
__global__ void __launch_bounds__(kThreads, 2)
    decode_int4_kernel(const __grid_constant__ Int4DecodeParams p, int halves) {
  constexpr int W = D / 32, kBlock = int4_block_bytes(D, NGK, NGV), kPairs = 16 * D, NG = NGK + NGV;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
  __shared__ int sm_scan[kWarps];
  __shared__ Walk sm_walk, sm_walks[kWarps];
  __shared__ Segment sm_next[kWarps];
  __shared__ Part sm_part[2];
  __shared__ int sm_last[2], sm_wide;     // (a segment of this CTA has to be scanned by scan_wide)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  if (lane < kStages) mbar_init(&bars[warp][lane], 1);
  fence_mbar_init();
  __syncwarp();
  if (threadIdx.x == 0) sm_wide = 0;
  pdl_wait();
  pdl_launch_dependents();
  const Int4Cache& c = p.c;
  const int sets = c.n_kv * halves, group = c.n_q / c.n_kv;

  int share = 0;
  const bool any = begin_share<kThreads>(p, sets, kMinShare, sm_scan, &sm_walk, &share);
  // requests without a token
  for (int b = blockIdx.x; b < c.batch; b += gridDim.x)
    if (c.seq_len[b] <= 0 || c.max_len == 0)
      for (int i = threadIdx.x; i < c.n_q * D / 8; i += kThreads)
        reinterpret_cast<uint4*>(p.out + int64_t(b) * c.n_q * D)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  if (!any) return;

  // Each warp walks by itself; the next segment waits in shared memory.
  auto advance = [&]() {
    bool ok = false;
    if (lane == 0) ok = sm_walks[warp].next(p, sets, &sm_next[warp]);
    __syncwarp();
    return __shfl_sync(0xffffffffu, int(ok), 0) != 0;
  };
  if (lane == 0) sm_walks[warp] = sm_walk;
  if (!advance()) return;                 // (nothing but places of a run's cost; the same in all warps)
  Segment cur = sm_next[warp];
  __syncwarp();
  bool more = false;                      // sm_next holds another

  // The ring.  A warp's pairs of a segment begin with another warp each time,
  // so that short segments spread over the warps.  Lane i knows pairs 32 n + i
  // of the segment that is being brought in.
  uint8_t* ring = smem + warp * (kStages * 2 * kBlock);
  float* buf = reinterpret_cast<float*>(smem + kWarps * kStages * 2 * kBlock);
  uint64_t* wbars = bars[warp];
  // the segment being brought in: its pages from this warp's first, KV head, request, and pairs
  int in_lo, in_hi, in_hk, in_b, in_it = 0, in_n;
  auto turn_to = [&](const Segment& s) {
    in_lo = s.lo + 2 * place_of(s, warp);
    in_hi = s.hi;
    in_hk = s.h / halves;
    in_b = s.b;
    in_it = 0;
    in_n = max(0, (in_hi - in_lo + 2 * kWarps - 1) / (2 * kWarps));
  };
  turn_to(cur);
  bool in_next = false, dead = false;     // it is the next one, not cur
  int id[2] = {-1, -1}, st_in = 0, flying = 0;
  uint32_t ring_dead = 0;                 // bits 2 i, 2 i + 1: stage i's pages that are not there
  auto bring = [&]() {                    // one more pair; false if there is none to bring yet
    if (in_it == in_n) {
      if (in_next || !more || dead) return false;
      in_next = true;
      turn_to(sm_next[warp]);
      if (in_n == 0) return false;
    }
    if ((in_it & 31) == 0) {
      const int32_t* table = c.page_table + int64_t(in_b) * c.max_pages;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int page = in_lo + 2 * kWarps * (in_it + lane) + g;
        id[g] = page < in_hi ? table[page] : -1;
        if (page < in_hi && (id[g] < 0 || id[g] >= c.n_pages)) {
          if (c.dev_status) atomicOr(c.dev_status, OSCAR_DEV_PAGE_BOUNDS);
          id[g] = -1;
        }
      }
    }
    const int owner = in_it & 31;
    const uint32_t none = __shfl_sync(0xffffffffu, (id[0] < 0 ? 1u : 0u) | (id[1] < 0 ? 2u : 0u), owner);
    ring_dead = (ring_dead & ~(3u << (2 * st_in))) | (none << (2 * st_in));
    if (lane == owner) {
      uint8_t* to = ring + st_in * 2 * kBlock;
      uint64_t* bar = wbars + st_in;
      const int n = 2 - __popc(none);
      if (n)
        mbar_arrive_expect_tx(bar, n * kBlock);
      else
        mbar_arrive(bar);
#pragma unroll
      for (int g = 0; g < 2; ++g)
        if (id[g] >= 0) bulk_copy_g2s(to + g * kBlock, c.pages + (int64_t(id[g]) * c.n_kv + in_hk) * kBlock, kBlock, bar);
    }
    st_in ^= 1;
    ++in_it;
    ++flying;
    return true;
  };
  static_assert(kStages == 2, "st_in and st toggle");
  // column gid's query, asked for before the copies: behind them it came 4 us late
  uint4 uq[W];
  auto ask_q = [&](const Segment& s) {
    const int set = s.h % halves, head = s.h / halves * group + set * kHeads + gid;
    const uint16_t* row = p.q + s.b * p.q_stride + int64_t(head) * D + 8 * tig;
#pragma unroll
    for (int w = 0; w < W; ++w)
      uq[w] = gid < min(kHeads, group - set * kHeads) ? *reinterpret_cast<const uint4*>(row + 32 * w) : make_uint4(0, 0, 0, 0);
  };
  ask_q(cur);
  while (flying < kStages && bring()) {
  }
  more = advance();                       // (the first copies do not wait for it)
  while (flying < kStages && bring()) {
  }

  int st = 0;
  uint32_t parity = 0;
  int has_part = 0;                       // bits: of a run that began before this share, of one that goes on behind it
  while (true) {
    const int hk = cur.h / halves, set = cur.h % halves, heads = min(kHeads, group - set * kHeads);
    const int hq0 = hk * group + set * kHeads, lo = cur.lo + 2 * place_of(cur, warp);
    const int n_it = max(0, (cur.hi - lo + 2 * kWarps - 1) / (2 * kWarps));

    // Query operands of column gid: head hq0 + gid, scaled by 2^(141 - ex) so
    // that its largest channel is in [2^14, 2^15).
    uint32_t qb[2 * W][2];
    float qs[NGK][2], unscale[2], slope[2];
    {
      float q[W][8], top = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        q[w][0] = bf16_lo(uq[w].x), q[w][1] = bf16_hi(uq[w].x), q[w][2] = bf16_lo(uq[w].y), q[w][3] = bf16_hi(uq[w].y);
        q[w][4] = bf16_lo(uq[w].z), q[w][5] = bf16_hi(uq[w].z), q[w][6] = bf16_lo(uq[w].w), q[w][7] = bf16_hi(uq[w].w);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(q[w][i]));
      }
      top = max_over_quad(top);
      const int ex = min(max((__float_as_int(top) >> 23) & 255, 14), 254);
      const float up = pow2i(141 - ex);
      float sum[NGK];
#pragma unroll
      for (int g = 0; g < NGK; ++g) sum[g] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          q[w][i] *= up;
          sum[w * NGK / W] += q[w][i];
        }
        // k-step 2 w: nibbles (0, 4) and (1, 5); 2 w + 1: (2, 6) and (3, 7);
        // the odd ones are masked in place and stand for 16 c
        qb[2 * w][0] = pack_half2(q[w][0], q[w][4]);
        qb[2 * w][1] = pack_half2(q[w][1] * 0.0625f, q[w][5] * 0.0625f);
        qb[2 * w + 1][0] = pack_half2(q[w][2], q[w][6]);
        qb[2 * w + 1][1] = pack_half2(q[w][3] * 0.0625f, q[w][7] * 0.0625f);
      }
#pragma unroll
      for (int g = 0; g < NGK; ++g) {
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
        sum[g] *= 5.9604644775390625e-8f;   // 2^-24, as the codes carry
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {         // to the lanes of columns 2 tig, 2 tig + 1
        const int from_lane = 4 * (2 * tig + e);
#pragma unroll
        for (int g = 0; g < NGK; ++g) qs[g][e] = __shfl_sync(0xffffffffu, sum[g], from_lane);
        unscale[e] = unscale_of(__shfl_sync(0xffffffffu, ex, from_lane), p.s);
        slope[e] = Formed && p.s.slopes && 2 * tig + e < heads ? p.s.slopes[hq0 + 2 * tig + e] * kLog2e : 0.f;
      }
    }

    // x is in the dot product's own scale, or in log2 units where the score has a
    // form of its own; us takes it to log2 units, thr is m + 8 / us, off 7 - m us:
    // the weights are 2^(7 + t - m) <= 2^15.
    float us[2], thr[2], m[2] = {-FLT_MAX, -FLT_MAX}, off[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) us[e] = Formed ? 1.f : fmaxf(unscale[e], FLT_MIN), thr[e] = -FLT_MAX;
    // rows: channels 32 w + 4 gid + (0, 1 | 2, 3); of zl: g < NGV the zeros' sums
    // of group g, NGV the weights' sum.  Columns: heads 2 tig, 2 tig + 1.
    float o[2 * W][4], zl[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 2 * W; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    int ve = -14;                           // the V scales seen are at most 2^ve
    uint32_t vs_top = 0x0400u, vs_mul = 0x74007400u;   // 2^ve, and 2^-ve twice, in fp16
    uint32_t vs_least = 0xFFFFFFFFu;        // one below the least scale seen that is not 0, fp16 bits twice
    const uint32_t z_keep = gid < NGV ? 0xffffffffu : 0u, z_one = gid == NGV ? 0x3C003C00u : 0u;

    int tok = lo * kPageTokens;
    for (int it = 0; it < n_it && !dead; ++it) {
      if (!__all_sync(0xffffffffu, mbar_try_wait(wbars + st, parity)) &&
          !__all_sync(0xffffffffu, mbar_wait_bounded(wbars + st, parity, kDefaultWaitNs))) {
        // a copy did not land in time: nothing more is brought in, and what is in
        // flight is still waited for before its shared memory goes
        if (lane == 0 && c.dev_status) atomicOr(c.dev_status, OSCAR_DEV_TIMEOUT);
        dead = true;
        for (; flying > 0; --flying) {
          mbar_wait_bounded(wbars + st, parity, kDrainWaitNs);
          st ^= 1;
          parity ^= st == 0;
        }
        __syncwarp();
        break;
      }
      const uint8_t* blk = ring + st * 2 * kBlock;
      // S: rows gid and gid + 8 of each page are tokens, columns 2 tig and 2 tig + 1 heads
      float y[4][2];
#pragma unroll
      for (int g2 = 0; g2 < 2; ++g2) {
        const uint8_t* page = blk + g2 * kBlock;
        float acc[NGK][4];
#pragma unroll
        for (int g = 0; g < NGK; ++g) acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
        uint32_t k0[W], k1[W];
        lds_n(k0, page + gid * (D / 2) + tig * (4 * W));
        lds_n(k1, page + (gid + 8) * (D / 2) + tig * (4 * W));
#pragma unroll
        for (int w = 0; w < W; ++w) {
          mma(acc[w * NGK / W], k0[w] & kLow, k1[w] & kLow, k0[w] & kHigh, k1[w] & kHigh, qb[2 * w][0], qb[2 * w][1]);
          const uint32_t a = k0[w] >> 8, d = k1[w] >> 8;
          mma(acc[w * NGK / W], a & kLow, d & kLow, a & kHigh, d & kHigh, qb[2 * w + 1][0], qb[2 * w + 1][1]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* pr = page + kPairs + 4 * NG * (gid + 8 * r);
          uint32_t kw[NGK];
          if constexpr (NG % 4 == 0 && NGK % 4 == 0 || NG % 2 == 0 && NGK == 2 || NGK == 1) {
            lds_n(kw, pr);
          } else {
#pragma unroll
            for (int g = 0; g < NGK; ++g) kw[g] = reinterpret_cast<const uint32_t*>(pr)[g];
          }
#pragma unroll
          for (int g = 0; g < NGK; ++g) {
            const float2 sz = half2_to_float2(kw[g]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float z = g ? fmaf(sz.y, qs[g][e], y[2 * g2 + r][e]) : sz.y * qs[g][e];
              y[2 * g2 + r][e] = fmaf(sz.x, acc[g][2 * r + e], z);
            }
          }
        }
      }
      // the values' scales and zeros of tokens 8 i + 2 tig, + 1
      uint32_t vs[4][NGV], vz[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* pp = blk + (i >> 1) * kBlock + kPairs + 4 * NG * (8 * (i & 1) + 2 * tig);
        uint32_t pr[2 * NG];
        lds_n(pr, pp);
#pragma unroll
        for (int g = 0; g < NGV; ++g) vs[i][g] = prmt(pr[NGK + g], pr[NG + NGK + g], 0x5410);
        if constexpr (NGV == 1) {
          vz[i] = prmt(pr[NGK], pr[NG + NGK], 0x7632);
        } else {                            // group gid's, for the row that sums it
          const uint32_t* zp = reinterpret_cast<const uint32_t*>(pp) + NGK + (gid & (NGV - 1));
          vz[i] = prmt(zp[0], zp[NG], 0x7632);
        }
      }
      // lane i: token i's scales, two to a word (fp16 values >= 0 order as integers)
      uint32_t own[(NGV + 1) / 2];
      {
        const uint32_t* pp = reinterpret_cast<const uint32_t*>(blk + (lane >> 4) * kBlock + kPairs + 4 * NG * (lane & 15)) + NGK;
#pragma unroll
        for (int g = 0; g < (NGV + 1) / 2; ++g) own[g] = NGV == 1 ? pp[0] & 0xFFFFu : prmt(pp[2 * g], pp[2 * g + 1], 0x5410);
      }
      if (Formed) {
        float far = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) y[r][e] *= unscale[e], far = fmaxf(far, fabsf(y[r][e]));
        if (p.s.cap_log2 != 0.f) {
          // (the vote skips a form that no score here needs; each score's own is its own)
          if (__builtin_expect(__any_sync(0xffffffffu, !cap_is_near(far, p.s)), 0)) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int e = 0; e < 2; ++e) y[r][e] = capped(y[r][e], p.s);
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int e = 0; e < 2; ++e) y[r][e] = capped_near(y[r][e], p.s);
          }
        }
        if (p.s.slopes) {
          const float away = float(tok + gid - (cur.len - 1));
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) y[r][e] = fmaf(slope[e], away + float(8 * r), y[r][e]);
        }
      }
      const uint32_t gone = (ring_dead >> (2 * st)) & 3u;
      if (gone || tok < cur.first || tok + 2 * kPageTokens > cur.len) {
        // what a stale slot holds is anything
        const bool here = !((gone >> (lane >> 4)) & 1u) && tok + lane >= cur.first && tok + lane < cur.len;
#pragma unroll
        for (int g = 0; g < (NGV + 1) / 2; ++g) own[g] = here ? own[g] : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool out_of = (gone >> (i >> 1)) & 1u;
          const int j = tok + 8 * i + gid, j2 = tok + 8 * i + 2 * tig;
          if (out_of || j < cur.first || j >= cur.len) y[i][0] = y[i][1] = -INFINITY;
          uint32_t keep = 0;
          if (!out_of && j2 >= cur.first && j2 < cur.len) keep |= 0x0000FFFFu;
          if (!out_of && j2 + 1 >= cur.first && j2 + 1 < cur.len) keep |= 0xFFFF0000u;
          vz[i] &= keep;
#pragma unroll
          for (int g = 0; g < NGV; ++g) vs[i][g] &= keep;
        }
      }
      uint32_t smax = own[0];
      vs_least = __viaddmin_u16x2(own[0], 0xFFFFFFFFu, vs_least);
      if constexpr (NGV == 4) {
        smax = __vmaxu2(smax, own[1]);
        vs_least = __viaddmin_u16x2(own[1], 0xFFFFFFFFu, vs_least);
      }
      const float y0 = fmaxf(fmaxf(y[0][0], y[1][0]), fmaxf(y[2][0], y[3][0]));
      const float y1 = fmaxf(fmaxf(y[0][1], y[1][1]), fmaxf(y[2][1], y[3][1]));
      if (__any_sync(0xffffffffu, (y0 > thr[0]) | (y1 > thr[1]) | ((smax & 0xFFFFu) > vs_top) | ((smax >> 16) > vs_top))) {
        const int ne = max(ve, scale_exponent(__reduce_max_sync(0xffffffffu, max(smax & 0xFFFFu, smax >> 16))));
        const float fv = pow2i(ve - ne);
        ve = ne;
        vs_top = ve < 16 ? uint32_t(ve + 15) << 10 : 0xFFFFu;
        vs_mul = uint32_t(__half_as_ushort(__float2half_rn(pow2i(-ve)))) * 0x10001u;
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[e], max_over_rows(e ? y1 : y0));
          f[e] = exp2_fast((m[e] - mn) * us[e]);
          m[e] = mn;
          off[e] = 7.f - mn * us[e];
          thr[e] = mn + 8.f / us[e];
          zl[e] *= f[e];
          f[e] *= fv;
        }
#pragma unroll
        for (int t = 0; t < 2 * W; ++t) o[t][0] *= f[0], o[t][1] *= f[1], o[t][2] *= f[0], o[t][3] *= f[1];
      }
#pragma unroll
      for (int g2 = 0; g2 < 2; ++g2) {
        uint32_t pw[2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
          pw[r] = movmatrix_trans(pack_half2(exp2_fast(fmaf(y[2 * g2 + r][0], us[0], off[0])),
                                             exp2_fast(fmaf(y[2 * g2 + r][1], us[1], off[1]))));
        mma(zl, (vz[2 * g2] & z_keep) | z_one, 0u, (vz[2 * g2 + 1] & z_keep) | z_one, 0u, pw[0], pw[1]);
        // O: rows are channels; depth = tokens 2 tig, 2 tig + 1 (and + 8)
        const uint8_t* page = blk + g2 * kBlock;
        uint32_t v0[W], v1[W];
        lds_n(v0, page + 8 * D + (8 * tig + gid) * (4 * W));
        lds_n(v1, page + 8 * D + (8 * (tig + 4) + gid) * (4 * W));
#pragma unroll
        for (int g = 0; g < NGV; ++g) {
          const uint32_t s0 = mul_half2(pw[0], mul_half2(vs[2 * g2][g], vs_mul));
          const uint32_t s1 = mul_half2(pw[1], mul_half2(vs[2 * g2 + 1][g], vs_mul));
#pragma unroll
          for (int w = g * W / NGV; w < (g + 1) * W / NGV; ++w) {
            mma(o[2 * w], v0[w] & kLow, v0[w] & kHigh, v1[w] & kLow, v1[w] & kHigh, s0, s1);
            const uint32_t a = v0[w] >> 8, d = v1[w] >> 8;
            mma(o[2 * w + 1], a & kLow, a & kHigh, d & kLow, d & kHigh, s0, s1);
          }
        }
      }
      __syncwarp();                         // the stage has been read
      --flying;
      bring();
      tok += 2 * kWarps * kPageTokens;
      st ^= 1;
      parity ^= st == 0;
    }

    if (more) ask_q(sm_next[warp]);
    // The warps' states of this segment, kJoinHeads heads at a time.  (All with
    // the weights' 2^7; a warp without a token has l = 0, whatever its m.)
    const float un = pow2i(24 + ve);        // 2^24 of the codes, 2^ve of the scales
    float z[NGV][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float l = __shfl_sync(0xffffffffu, zl[e], 4 * NGV + tig);
      if (gid == 0) sm_m[warp][2 * tig + e] = m[e] * us[e], sm_l[warp][2 * tig + e] = l;
#pragma unroll
      for (int g = 0; g < NGV; ++g) z[g][e] = __shfl_sync(0xffffffffu, zl[e], 4 * g + tig);
    }
    if (scales_wide(ve, vs_least) && !dead) sm_wide = 1;
    const bool whole = cur.off == 0 && cur.hi - cur.lo == cur.pages;
    const int slot = 2 * blockIdx.x + (cur.off == 0);
    for (int h0 = 0; h0 < heads; h0 += kJoinHeads) {
      if (h0) __syncthreads();              // the heads before have been read
      if (2 * tig >= h0 && 2 * tig < h0 + kJoinHeads) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float zg = z[w * NGV / W][e];
            *reinterpret_cast<float4*>(buf + (warp * kJoinHeads + 2 * tig + e - h0) * D + 32 * w + 4 * gid) =
                make_float4(fmaf(o[2 * w][e], un, zg), fmaf(o[2 * w][2 + e], un * 0.0625f, zg),
                            fmaf(o[2 * w + 1][e], un, zg), fmaf(o[2 * w + 1][2 + e], un * 0.0625f, zg));
          }
      }
      __syncthreads();
      join_warps<D>(p, hq0, h0, heads, whole ? -1 : slot, cur.b, buf, sm_m, sm_l);
    }
    if (!whole && threadIdx.x == 0) sm_part[cur.off == 0] = {cur.at - cur.off, cur.pages, cur.b, hq0, heads};
    has_part |= whole ? 0 : 1 << (cur.off == 0);
    if (!more) break;
    __syncthreads();                        // the joined states have been read
    cur = sm_next[warp];
    __syncwarp();
    more = advance();
    in_next = false;
    if (dead) in_n = in_it;
    if (!dead)
      while (flying < kStages && bring()) {
      }
  }
  if (__builtin_expect(sm_wide, 0)) scan_wide<D, NGK, NGV>(p, sm_walk, sets, halves, buf, sm_m, sm_l);
  if (!has_part) return;

  // The runs that this CTA has a part of (the first of its share, the last, or
  // both): the last of a run's CTAs to come here joins its parts.
  __syncthreads();
  if (threadIdx.x < 2 && ((has_part >> threadIdx.x) & 1)) {
    const Part& r = sm_part[threadIdx.x];
    const int f = r.run / share;          // the run lies in the shares of CTAs f ..
    uint32_t* ticket = static_cast<uint32_t*>(p.workspace) + f;
    const bool last = atom_add_acq_rel_gpu(ticket, 1) == uint32_t((r.run + r.pages - 1) / share - f);
    if (last) *ticket = 0;                // ready for the next call
    sm_last[threadIdx.x] = last;
  }
  __syncthreads();
  for (int which = 0; which < 2; ++which)
    if (((has_part >> which) & 1) && sm_last[which]) {
      if (which) __syncthreads();
      join_parts<D>(p, sm_part[which], share, buf, sm_l[0]);
    }
}

template <int D, int NGK, int NGV, bool Formed>
cudaError_t launch(const Int4DecodeParams& p, cudaStream_t stream) {
  constexpr int bytes = kWarps * kStages * 2 * int4_block_bytes(D, NGK, NGV) + join_bytes<D>();
  const cudaError_t e = set_smem_limit<decode_int4_kernel<D, NGK, NGV, Formed>>(bytes);
  if (e != cudaSuccess) return e;
  const int halves = (p.c.n_q / p.c.n_kv + kHeads - 1) / kHeads;
  int64_t tokens = p.c.max_len;
  if (p.s.window) tokens = std::min<int64_t>(tokens, int64_t(p.s.window) + kPageTokens);
  const int64_t places = ((tokens + kPageTokens - 1) / kPageTokens + kRunCost) * p.c.batch * p.c.n_kv * halves;
  if (places > INT32_MAX) return cudaErrorNotSupported;
  const int64_t ctas = std::min<int64_t>(kCtas, (places + kMinShare - 1) / kMinShare);
  return launch_pdl(decode_int4_kernel<D, NGK, NGV, Formed>, dim3(unsigned(ctas)), dim3(kThreads), bytes, stream, p, halves);
}

template <int D, int NGK, int NGV>
cudaError_t launch_f(const Int4DecodeParams& p, cudaStream_t stream) {
  return p.s.cap_log2 != 0.f || p.s.slopes ? launch<D, NGK, NGV, true>(p, stream) : launch<D, NGK, NGV, false>(p, stream);
}

template <int D, int NGK>
cudaError_t launch_v(const Int4DecodeParams& p, cudaStream_t stream) {
  if (p.c.ng_v == 1) return launch_f<D, NGK, 1>(p, stream);
  if (p.c.ng_v == 2) return launch_f<D, NGK, 2>(p, stream);
  if constexpr (D == 128) return launch_f<D, NGK, 4>(p, stream);
  return cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_k(const Int4DecodeParams& p, cudaStream_t stream) {
  if (p.c.ng_k == 1) return launch_v<D, 1>(p, stream);
  if (p.c.ng_k == 2) return launch_v<D, 2>(p, stream);
  if constexpr (D == 128) return launch_v<D, 4>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

size_t int4_decode_workspace_bytes(const Int4Cache& c) { return kOffO + size_t(kCtas) * 2 * kHeads * c.d * 4; }

cudaError_t launch_decode_int4(const Int4DecodeParams& p, cudaStream_t stream) {
  Int4DecodeParams u = p;
  u.s = in_units(p.s);
  return p.c.d == 128 ? launch_k<128>(u, stream) : launch_k<64>(u, stream);
}

}  // namespace oscar
