// Decode attention over a 4-bit layer: one query token per request, split over
// the pages of its context and joined by the last CTA of each (request, KV
// head) to finish.
//
// A CTA of 8 warps takes one split of one (request, KV head, up to 8 query
// heads); a warp takes every 8th page of the split with an online softmax of
// its own, so nothing in the scan waits for another warp.  The pages' blocks
// come by bulk copies into a ring of the warp's own.
//
// Per page, on the tensor cores with 16 tokens or 16 channels as the rows and
// 8 query heads as the columns:
//   S = K q:   A = the K codes as they are: a code c in the low bits of an fp16
//              is c 2^-24 exactly (and c 2^-20 one nibble higher), so one mask
//              turns a word into two operands.  q is scaled by a power of two
//              per head to just below fp16's end, which is exact for bf16.
//              x = sum over groups of s (sum c q) + z (sum q).
//   O += P V:  A = the V codes the same way, B = p s_V in fp16; the zeros are
//              summed apart as p z_V in fp32.  The 11 bits of p s_V are the one
//              rounding below fp32 (bf16 output has 8).
// The weights' reference is raised only when a score exceeds it by 2^8, and
// the values' scales are taken relative to a power of two above them, raised
// when a larger one comes: both by one vote per page.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kernels.h"
#include "oscar.h"
#include "ptx.cuh"
#include "score.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 8;
constexpr int kHeads = 8;             // query heads per CTA (MMA columns)
constexpr int kSlots = 152 * 2;       // CTAs the GPU holds at a time
constexpr int kRounds = 24;           // rounds of them that a grid is split into, at most
// Merge tickets sit at the same place of the workspace whatever the call's
// sizes, so that calls of different batches share one: no call writes partial
// states where another keeps tickets.  A grid is split (2 splits or more) only
// below this many (request, head set) pairs.
constexpr int kTickets = 4096;
static_assert(kSlots * kRounds / 2 <= kTickets, "every split pair has a ticket");
constexpr int kMostSplits = 512;      // their weights fit the joining CTA's shared memory
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;

struct SplitPlan {
  int splits;          // per (request, head set), at most
  int halves;          // head sets per KV head
  size_t off_ml, off_o, bytes;
};

// Pages of a request are split so that the grid is a whole number of rounds
// of the CTAs that the GPU holds, each of at least 16 pages a warp where the
// context has them, and at least 4.
SplitPlan plan_splits(const Int4Cache& c, const ScoreParams& s) {
  SplitPlan r{};
  const int group = c.n_q / c.n_kv;
  r.halves = (group + kHeads - 1) / kHeads;
  int64_t tokens = c.max_len;
  if (s.window) tokens = std::min<int64_t>(tokens, int64_t(s.window) + kInt4Page);
  const int64_t pages = std::max<int64_t>(1, (tokens + kInt4Page - 1) / kInt4Page);
  const int64_t pairs = int64_t(c.batch) * c.n_kv * r.halves;
  const int64_t round = int64_t(kSlots) * kWarps * 16;
  const int64_t rounds = std::min<int64_t>(kRounds, std::max<int64_t>(1, (pairs * pages + round / 2) / round));
  const int64_t most = std::max<int64_t>(1, pages / (kWarps * 4));
  r.splits = int(std::min<int64_t>(std::min<int64_t>(most, kMostSplits), std::max<int64_t>(1, kSlots * rounds / pairs)));
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  r.off_ml = up(size_t(kTickets) * 4);
  r.off_o = r.off_ml + up(size_t(pairs) * r.splits * kHeads * 8);
  r.bytes = r.off_o + up(size_t(pairs) * r.splits * kHeads * c.d * 4);
  if (r.splits == 1) r.bytes = 256;   // nothing is kept there
  return r;
}

// N consecutive 32-bit words, by the widest loads that the alignment of N
// words times any index allows.
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

// D += A (16x16 f16, row) * B (16x8 f16, col); free for the compiler to move.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Ring stages of a warp, each two pages: three where two CTAs' rings fit an
// SM's shared memory, else two.
constexpr int stages_of(int block) { return 2 * kWarps * 2 * 3 * block <= 212 * 1024 ? 3 : 2; }

// Formed: the scores have a cap or a distance bias.
template <int D, int NGK, int NGV, bool Formed>
__global__ void __launch_bounds__(32 * kWarps, 2) decode_int4_kernel(const Int4DecodeParams p, const SplitPlan plan) {
  constexpr int W = D / 32, kBlock = int4_block_bytes(D, NGK, NGV), kPairs = 16 * D, kStages = stages_of(kBlock);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
  __shared__ int sm_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  if (lane < kStages) mbar_init(&bars[warp][lane], 1);
  fence_mbar_init();
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();
  const Int4Cache& c = p.c;
  const int b = blockIdx.z, hk = blockIdx.y / plan.halves, set = blockIdx.y % plan.halves;
  const int group = c.n_q / c.n_kv, heads = min(kHeads, group - set * kHeads);
  const int hq0 = hk * group + set * kHeads;
  int len = c.seq_len[b];
  if (len < 0 || len > c.max_len) {
    if (threadIdx.x == 0 && c.dev_status) atomicOr(c.dev_status, OSCAR_DEV_LENGTH);
    len = min(max(len, 0), c.max_len);
  }
  const int first = p.s.window ? max(0, len - p.s.window) : 0;
  const int page0 = first / kInt4Page, page1 = (len + kInt4Page - 1) / kInt4Page;
  // this request's own split: as many as its pages need of the grid's
  const int pages = page1 - page0, most = max(1, pages / (kWarps * 4));
  const int splits = min(plan.splits, most), split = blockIdx.x;
  if (split >= splits) return;
  const int begin = page0 + int(int64_t(pages) * split / splits), end = page0 + int(int64_t(pages) * (split + 1) / splits);
  // a warp takes every 8th pair of pages
  const int n_it = max(0, ((end - begin + 1) / 2 - warp + kWarps - 1) / kWarps);

  // Lane i knows pairs 32 n + i of the warp's and brings them.
  const int32_t* table = c.page_table + int64_t(b) * c.max_pages;
  uint8_t* ring = smem + warp * (kStages * 2 * kBlock);
  uint64_t* wbars = bars[warp];
  auto pages_of = [&](int i, int (&id)[2]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int at = begin + 2 * (warp + kWarps * i) + g;
      id[g] = i < n_it && at < end ? table[at] : -1;
      if (id[g] < 0 || id[g] >= c.n_pages) {
        if (i < n_it && at < end && c.dev_status) atomicOr(c.dev_status, OSCAR_DEV_PAGE_BOUNDS);
        id[g] = -1;
      }
    }
  };
  int id[2], id_next[2] = {-1, -1};
  pages_of(lane, id);
  uint32_t ring_dead = 0;                 // bits 2 i, 2 i + 1: stage i's pages that are not there
  int st_issue = 0;
  auto issue = [&](int it) {
    const int at = it & 31;
    if (at == 0) {
      if (it) id[0] = id_next[0], id[1] = id_next[1];
      pages_of(it + 32 + lane, id_next);
    }
    const uint32_t none = __shfl_sync(0xffffffffu, (id[0] < 0 ? 1u : 0u) | (id[1] < 0 ? 2u : 0u), at);
    ring_dead = (ring_dead & ~(3u << (2 * st_issue))) | (none << (2 * st_issue));
    if (lane == at) {
      uint8_t* to = ring + st_issue * 2 * kBlock;
      uint64_t* bar = wbars + st_issue;
      const int n = 2 - __popc(none);
      if (n)
        mbar_arrive_expect_tx(bar, n * kBlock);
      else
        mbar_arrive(bar);
#pragma unroll
      for (int g = 0; g < 2; ++g)
        if (id[g] >= 0) bulk_copy_g2s(to + g * kBlock, c.pages + (int64_t(id[g]) * c.n_kv + hk) * kBlock, kBlock, bar);
    }
    st_issue = st_issue + 1 == kStages ? 0 : st_issue + 1;
  };
  int issued = min(n_it, kStages);
  for (int i = 0; i < issued; ++i) issue(i);

  // Query operands of column gid: head hq0 + gid, scaled by 2^(141 - ex) so
  // that its largest channel is in [2^14, 2^15).
  uint32_t qb[2 * W][2];
  float qs[NGK][2], unscale[2], slope[2];
  {
    float q[W][8], top = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (gid < heads)
        u = *reinterpret_cast<const uint4*>(p.q + b * p.q_stride + int64_t(hq0 + gid) * D + 32 * w + 8 * tig);
      q[w][0] = bf16_lo(u.x), q[w][1] = bf16_hi(u.x), q[w][2] = bf16_lo(u.y), q[w][3] = bf16_hi(u.y);
      q[w][4] = bf16_lo(u.z), q[w][5] = bf16_hi(u.z), q[w][6] = bf16_lo(u.w), q[w][7] = bf16_hi(u.w);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(q[w][i]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int ex = min(max((__float_as_int(top) >> 23) & 255, 14), 243);
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
    const float un = pow2i(ex - 117);     // 2^24 / up
#pragma unroll
    for (int g = 0; g < NGK; ++g) {
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
      sum[g] *= 5.9604644775390625e-8f;   // 2^-24, as the codes carry
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {         // to the lanes of columns 2 tig, 2 tig + 1
      const int from = 4 * (2 * tig + e);
#pragma unroll
      for (int g = 0; g < NGK; ++g) qs[g][e] = __shfl_sync(0xffffffffu, sum[g], from);
      unscale[e] = __shfl_sync(0xffffffffu, un, from);
      if (p.s.cap_log2 == 0.f) unscale[e] *= p.s.scale_log2;   // (with a cap, capped() takes the scale)
      slope[e] = p.s.slopes && 2 * tig + e < heads ? p.s.slopes[hq0 + 2 * tig + e] * kLog2e : 0.f;
    }
  }
  const bool cap = p.s.cap_log2 != 0.f;

  // x is in the dot product's own scale, or in log2 units where the score has a
  // form of its own; us takes it to log2 units, thr is m + 8 / us.
  float us[2], thr[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) us[e] = Formed ? 1.f : fmaxf(unscale[e], FLT_MIN), thr[e] = -FLT_MAX;
  float o[2 * W][4], zs[NGV][2], m[2] = {-FLT_MAX, -FLT_MAX}, off[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
  int ve = -24;                           // the V scales seen are at most 2^ve
  float vs_top = pow2i(-24), vs_mul = pow2i(31);   // 2^(7 - ve): p s_V 2^(7 - ve) <= 2^15
#pragma unroll
  for (int t = 0; t < 2 * W; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
#pragma unroll
  for (int g = 0; g < NGV; ++g) zs[g][0] = zs[g][1] = 0.f;

  int it = 0, st = 0;
  uint32_t parity = 0;
  int tok = (begin + 2 * warp) * kInt4Page;
  for (; it < issued; ++it) {
    if (!__all_sync(0xffffffffu, mbar_try_wait(wbars + st, parity)) &&
        !__all_sync(0xffffffffu, mbar_wait_bounded(wbars + st, parity, kDefaultWaitNs)))
      break;
    const uint8_t* blk = ring + st * 2 * kBlock;
    // S: rows gid and gid + 8 of each page are tokens, columns 2 tig and 2 tig + 1 heads
    float y[4][2], vp[4][NGV][2];
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
        uint32_t pr[NGK + NGV];
        lds_n(pr, page + kPairs + 4 * (NGK + NGV) * (gid + 8 * r));
#pragma unroll
        for (int g = 0; g < NGK; ++g) {
          const float2 sz = half2_to_float2(pr[g]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float z = g ? fmaf(sz.y, qs[g][e], y[2 * g2 + r][e]) : sz.y * qs[g][e];
            y[2 * g2 + r][e] = fmaf(sz.x, acc[g][2 * r + e], z);
          }
        }
#pragma unroll
        for (int g = 0; g < NGV; ++g) {
          const float2 sz = half2_to_float2(pr[NGK + g]);
          vp[2 * g2 + r][g][0] = sz.x, vp[2 * g2 + r][g][1] = sz.y;
        }
      }
    }
    if (Formed) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = y[r][e] * unscale[e];
          y[r][e] = fmaf(slope[e], float(tok + gid + 8 * r - (len - 1)), cap ? capped(x, p.s) : x);
        }
    }
    const uint32_t gone = (ring_dead >> (2 * st)) & 3u;
    if (gone || tok < first || tok + 2 * kInt4Page > len) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = tok + gid + 8 * r;
        if (j < first || j >= len || ((gone >> (r >> 1)) & 1u)) {
          y[r][0] = y[r][1] = -INFINITY;
#pragma unroll
          for (int g = 0; g < NGV; ++g) vp[r][g][0] = vp[r][g][1] = 0.f;   // a stale slot may hold anything
        }
      }
    }
    bool grow = false;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      grow = grow | (y[r][0] > thr[0]) | (y[r][1] > thr[1]);
#pragma unroll
      for (int g = 0; g < NGV; ++g) grow = grow | (vp[r][g][0] > vs_top);
    }
    if (__any_sync(0xffffffffu, grow)) {
      float top = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int g = 0; g < NGV; ++g) top = fmaxf(top, vp[r][g][0]);
      top = max_over_rows(top);
      // 2^e >= top for the exponent e of top plus one
      const int ne = max(ve, ((__float_as_int(top) >> 23) & 255) - 126);
      const float fv = ne - ve < 126 ? pow2i(ve - ne) : 0.f;
      ve = ne;
      vs_top = pow2i(ve);
      vs_mul = pow2i(7 - ve);
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(m[e], max_over_rows(fmaxf(fmaxf(y[0][e], y[1][e]), fmaxf(y[2][e], y[3][e]))));
        f[e] = exp2_fast((m[e] - mn) * us[e]);
        m[e] = mn;
        off[e] = -mn * us[e];
        thr[e] = mn + 8.f / us[e];
        l[e] *= f[e];
#pragma unroll
        for (int g = 0; g < NGV; ++g) zs[g][e] *= f[e];
        f[e] *= fv;
      }
#pragma unroll
      for (int t = 0; t < 2 * W; ++t) o[t][0] *= f[0], o[t][1] *= f[1], o[t][2] *= f[0], o[t][3] *= f[1];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        y[r][e] = exp2_fast(fmaf(y[r][e], us[e], off[e]));
        l[e] += y[r][e];
#pragma unroll
        for (int g = 0; g < NGV; ++g) zs[g][e] = fmaf(y[r][e], vp[r][g][1], zs[g][e]);
      }
    // O: rows are channels; k = tokens 2 tig, 2 tig + 1 (and + 8)
#pragma unroll
    for (int g2 = 0; g2 < 2; ++g2) {
      const uint8_t* page = blk + g2 * kBlock;
      uint32_t v0[W], v1[W];
      lds_n(v0, page + 8 * D + (8 * tig + gid) * (4 * W));
      lds_n(v1, page + 8 * D + (8 * (tig + 4) + gid) * (4 * W));
#pragma unroll
      for (int g = 0; g < NGV; ++g) {
        const float s0 = vp[2 * g2][g][0] * vs_mul, s1 = vp[2 * g2 + 1][g][0] * vs_mul;
        const uint32_t b0 = movmatrix_trans(pack_half2(y[2 * g2][0] * s0, y[2 * g2][1] * s0));
        const uint32_t b1 = movmatrix_trans(pack_half2(y[2 * g2 + 1][0] * s1, y[2 * g2 + 1][1] * s1));
#pragma unroll
        for (int w = g * W / NGV; w < (g + 1) * W / NGV; ++w) {
          mma(o[2 * w], v0[w] & kLow, v0[w] & kHigh, v1[w] & kLow, v1[w] & kHigh, b0, b1);
          const uint32_t a = v0[w] >> 8, d = v1[w] >> 8;
          mma(o[2 * w + 1], a & kLow, a & kHigh, d & kLow, d & kHigh, b0, b1);
        }
      }
    }
    __syncwarp();                         // the stage has been read
    if (issued < n_it) issue(issued++);
    tok += 2 * kWarps * kInt4Page;
    if (++st == kStages) st = 0, parity ^= 1;
  }
  if (it < issued) {
    // a copy did not land in time: nothing more is issued, and what is in
    // flight is still waited for before its shared memory goes
    if (lane == 0 && c.dev_status) atomicOr(c.dev_status, OSCAR_DEV_TIMEOUT);
    for (int i = max(it, issued - kStages); i < issued; ++i)
      mbar_wait_bounded(wbars + i % kStages, (i / kStages) & 1, kDrainWaitNs);
    __syncwarp();
  }

  // the warps' states in shared memory, over the rings
  __syncthreads();
  float* buf = reinterpret_cast<float*>(smem);
  const float un = pow2i(17 + ve);        // 2^24 of the codes, 2^(ve - 7) of the scales
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int h = 2 * tig + e;
    const float lt = sum_over_rows(l[e]);
    float z[NGV];
#pragma unroll
    for (int g = 0; g < NGV; ++g) z[g] = sum_over_rows(zs[g][e]);
    if (gid == 0) sm_m[warp][h] = lt > 0.f ? m[e] * us[e] : -FLT_MAX, sm_l[warp][h] = lt;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float zg = z[w * NGV / W];
      float4 v = make_float4(fmaf(o[2 * w][e], un, zg), fmaf(o[2 * w][2 + e], un * 0.0625f, zg),
                             fmaf(o[2 * w + 1][e], un, zg), fmaf(o[2 * w + 1][2 + e], un * 0.0625f, zg));
      *reinterpret_cast<float4*>(buf + (warp * kHeads + h) * D + 32 * w + 4 * gid) = v;
    }
  }
  __syncthreads();
  // (the request, head set) pair's partial states
  const int64_t pair = (int64_t(b) * c.n_kv + hk) * plan.halves + set;
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  float2* ml = reinterpret_cast<float2*>(ws + plan.off_ml) + pair * plan.splits * kHeads;
  float* po = reinterpret_cast<float*>(ws + plan.off_o) + pair * plan.splits * kHeads * D;
  uint16_t* out = p.out + (int64_t(b) * c.n_q + hq0) * D;
  for (int i = threadIdx.x; i < heads * D; i += 32 * kWarps) {
    const int h = i / D, ch = i % D;
    float mx = sm_m[0][h], sum = 0.f, v = 0.f;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w][h]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2_fast(sm_m[w][h] - mx);
      sum = fmaf(f, sm_l[w][h], sum);
      v = fmaf(f, buf[(w * kHeads + h) * D + ch], v);
    }
    if (splits == 1) {
      out[i] = __bfloat16_as_ushort(__float2bfloat16_rn(sum > 0.f ? v / sum : 0.f));
    } else {
      po[(split * kHeads + h) * D + ch] = v;
      if (ch == 0) ml[split * kHeads + h] = make_float2(mx, sum);
    }
  }
  if (splits == 1) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t* ticket = reinterpret_cast<uint32_t*>(ws) + pair;
    sm_last = atom_add_acq_rel_gpu(ticket, 1) == uint32_t(splits - 1);
    if (sm_last) *ticket = 0;             // ready for the next call
  }
  __syncthreads();
  if (!sm_last) return;
  // The last CTA: the parts' weights in shared memory, then 4 channels a
  // thread; where the heads leave threads over, each takes every n-th part.
  float* wt = reinterpret_cast<float*>(smem);           // [split][head]
  for (int i = threadIdx.x; i < splits * kHeads; i += 32 * kWarps)
    wt[i] = (i % kHeads) < heads ? __ldcg(&ml[i]).x : -FLT_MAX;
  __syncthreads();
  {                                                     // warp h: head h
    float mx = -FLT_MAX, sum = 0.f;
    for (int s = lane; s < splits; s += 32) mx = fmaxf(mx, wt[s * kHeads + warp]);
#pragma unroll
    for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    for (int s = lane; s < splits; s += 32) {
      const float f = exp2_fast(wt[s * kHeads + warp] - mx);
      wt[s * kHeads + warp] = f;
      if (warp < heads) sum = fmaf(f, __ldcg(&ml[s * kHeads + warp]).y, sum);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (lane == 0) sm_l[0][warp] = sum;
  }
  __syncthreads();
  const int units = heads * (D / 4), parts = 32 * kWarps / units, part = threadIdx.x / units, unit = threadIdx.x % units;
  const int h = unit / (D / 4);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (part < parts) {
    const float4* from = reinterpret_cast<const float4*>(po) + unit;
#pragma unroll 8
    for (int s = part; s < splits; s += parts) {
      const float f = wt[s * kHeads + h];
      const float4 x = __ldcg(from + s * (kHeads * D / 4));
      v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
    }
  }
  float4* sums = reinterpret_cast<float4*>(wt + splits * kHeads);
  sums[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < units) {
    for (int i = 1; i < parts; ++i) {
      const float4 x = sums[i * units + unit];
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    const float inv = sm_l[0][h] > 0.f ? 1.f / sm_l[0][h] : 0.f;
    reinterpret_cast<uint2*>(out)[unit] = make_uint2(pack_bf162(v.x * inv, v.y * inv), pack_bf162(v.z * inv, v.w * inv));
  }
}

template <int D, int NGK, int NGV, bool Formed>
cudaError_t launch(const Int4DecodeParams& p, const SplitPlan& plan, cudaStream_t stream) {
  constexpr int block = int4_block_bytes(D, NGK, NGV), ring = kWarps * stages_of(block) * 2 * block;
  constexpr int join = kWarps * kHeads * D * 4, last = kMostSplits * kHeads * 4 + 32 * kWarps * 16;
  constexpr int bytes = std::max(ring, std::max(join, last));
  const cudaError_t e = set_smem_limit<decode_int4_kernel<D, NGK, NGV, Formed>>(bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(unsigned(plan.splits), unsigned(p.c.n_kv * plan.halves), unsigned(p.c.batch));
  return launch_pdl(decode_int4_kernel<D, NGK, NGV, Formed>, grid, dim3(32 * kWarps), bytes, stream, p, plan);
}

template <int D, int NGK, int NGV>
cudaError_t launch_f(const Int4DecodeParams& p, const SplitPlan& plan, cudaStream_t stream) {
  return p.s.cap_log2 != 0.f || p.s.slopes ? launch<D, NGK, NGV, true>(p, plan, stream)
                                           : launch<D, NGK, NGV, false>(p, plan, stream);
}

template <int D, int NGK>
cudaError_t launch_v(const Int4DecodeParams& p, const SplitPlan& plan, cudaStream_t stream) {
  if (p.c.ng_v == 1) return launch_f<D, NGK, 1>(p, plan, stream);
  if (p.c.ng_v == 2) return launch_f<D, NGK, 2>(p, plan, stream);
  if constexpr (D == 128) return launch_f<D, NGK, 4>(p, plan, stream);
  return cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_k(const Int4DecodeParams& p, const SplitPlan& plan, cudaStream_t stream) {
  if (p.c.ng_k == 1) return launch_v<D, 1>(p, plan, stream);
  if (p.c.ng_k == 2) return launch_v<D, 2>(p, plan, stream);
  if constexpr (D == 128) return launch_v<D, 4>(p, plan, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

size_t int4_decode_workspace_bytes(const Int4Cache& c, const ScoreParams&, cudaError_t* err) {
  *err = cudaSuccess;
  return plan_splits(c, ScoreParams{}).bytes;
}

cudaError_t launch_decode_int4(const Int4DecodeParams& p, cudaStream_t stream) {
  const SplitPlan plan = plan_splits(p.c, p.s);
  return p.c.d == 128 ? launch_k<128>(p, plan, stream) : launch_k<64>(p, plan, stream);
}

}  // namespace oscar
