// Decode attention over an 8-bit layer: one query token per request.
//
// The pages of all (request, KV head) runs stand in one row, and each of 304 lasting
// CTAs (two per SM) takes an equal share of it.  Only the first and the last run of a
// share can be incomplete: they leave their unnormalised sums in the workspace, and the
// last CTA of a run to finish joins its parts.
//
// Bound by HBM where it is long: 8 requests of 100k tokens (8 KV heads x 128, 1.69 GB)
// take 244 to 247 us, 6.85 TB/s, the rate of a plain copy.  One of them (211 MB, 31 us at that
// rate) takes 41.0: shares 1.2 us, first pages at 3 to 5, scans done at 31 to 34, warps'
// joins by 34.7, tickets by 35.6, last parts joined at 39 to 40.  28 ragged requests of
// 2k to 32k (654 MB, 96 us), scores capped: 109 us, their scans done over 20 us (the memory serves SMs
// unevenly by some 8 %, and the work is dealt out beforehand).
//
// A warp takes every 6th page (or pair of pages) of a run with an online softmax of its own, so
// nothing in the scan waits for another warp.  The pages' blocks come by bulk copies
// into a ring of the warp's own, the next run's ahead of the present one's end.
//
// Per page, on the tensor cores with 16 tokens or 16 channels as the rows and 8 query
// heads as the columns (heads as the rows took twice the products and accumulators):
//   S = K q:     A = the K codes: ldmatrix gives a lane 4 channels' bytes of a token, two
//                operand registers of one operation each: a byte c alone in an fp16 is
//                the subnormal c 2^-24, exactly.  q is scaled by a power of two per head
//                to just below fp16's end, exact for bf16 (the largest finite ones too).
//                x = scale (sum c q) + zero (sum q).
//   O += V^T P:  A = the V codes less 128, by ldmatrix with transposition; B = P scale_V.
//                (Without the subtraction, one operation more per operand, the sums
//                grow with the tokens and the tensor cores' truncated additions with
//                them: 100k tokens that cancel came out with a third of bf16's own error
//                on top.)  The zeros' share of O takes zero + 128 scale.
// P scale_V is formed in fp32 and split into two fp16 parts, in columns 4 to 7 where a
// group has at most 4 heads, else in products of its own, so that it keeps 22 bits: a
// code's range is a value's range, and an error of 2^-11 of it would show in the bf16
// output where values cancel.  The weights' sum and the zeros' share of O are summed in
// fp32 beside it.
// The weights' reference is raised only when a score exceeds it by 2^8, and the
// values' scales are taken relative to a power of two above them, raised when a larger
// one comes: both by one vote a page.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "decode_math.cuh"
#include "int8.h"
#include "kernels.h"
#include "oscar.h"
#include "page_walk.cuh"
#include "ptx.cuh"
#include "score.cuh"

namespace oscar {
namespace {

// Warps of a CTA and pages of a warp's ring, by the most query heads of a group.  Up to 8
// heads: 6 warps (168 registers, none spilled; a count that does not divide over the 4
// schedulers costs 10 %).  Two pages each, 101 KB in flight on an SM: with three or four
// 8 requests of 100k tokens took 262 and 269 us where two take 247.  16 heads: 4 warps,
// which spill nothing.
constexpr int warps_of(int G) { return G <= 8 ? 6 : 4; }
constexpr int stages_of(int G) { return G <= 8 ? 2 : 3; }
// Pages of a step of the scan (and of a ring's stage): about 4 KB.  (Heads of 64 with one
// page a step: 8 x 100k tokens 151 us, with two 135, 6.4 TB/s.)
constexpr int pages_of(int D) { return D == 64 ? 2 : 1; }
constexpr int kPerSm = 2;
constexpr int kCtas = 152 * kPerSm;   // CTAs the GPU holds at a time
constexpr int kHeads = 16;            // most query heads of a KV head
constexpr int kMinShare = 6;          // pages
// A run costs its CTA about as much as this many pages besides its own (the query, the
// warps' join).  (28 ragged requests x 8 KV heads: 115 us with 8, 112 with 16, 111 with 32;
// 64 of 1000 tokens: 33, 33, 32.)
constexpr int kRunCost = 32;
constexpr int kWhole = 18;            // a run of no more pages is not split
constexpr int join_heads(int G) { return G == 4 ? 4 : 8; }   // heads whose states are joined at a time
constexpr uint32_t kLow = 0x00FF00FFu;

using Walk = PageWalk<kRunCost, kWhole>;
// a warp's first step in a segment
template <int kWarps, int P>
__device__ __forceinline__ int place_of(const Segment& s, int warp) {
  const int i = warp - s.at / P % kWarps;
  return i < 0 ? i + kWarps : i;
}

// Workspace: a ticket for each CTA (of the run that goes on behind its share),
// then two partial states for each, of a run that began before its share and of one
// that begins in it: (m, l) and the sums.
constexpr size_t kOffMl = 4096, kOffO = kOffMl + size_t(kCtas) * 2 * kHeads * 8;

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&d)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t (&d)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
// bytes 0 and 2, bytes 1 and 3 of a word as two fp16 subnormals: c 2^-24
__device__ __forceinline__ uint32_t even(uint32_t w) { return w & kLow; }
__device__ __forceinline__ uint32_t odd(uint32_t w) { return prmt(w, 0u, 0x4341); }
// the same as signed integers, c - 128 (a byte under the exponent of 1024 is 1024 + c)
__device__ __forceinline__ uint32_t minus_1152(uint32_t w) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0x64806480u));
  return d;
}
__device__ __forceinline__ uint32_t even_signed(uint32_t w) { return minus_1152((w & kLow) | 0x64006400u); }
__device__ __forceinline__ uint32_t odd_signed(uint32_t w) { return minus_1152(prmt(w, 0x64646464u, 0x4341)); }

// The logarithm of the sum, from the reference in log2 units and the sum of 2^(7 + x - m).
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f ? (m + (log2f(l) - 7.f)) * kLn2 : l == 0.f ? -INFINITY : l; }

// Joins the warps' states of heads h0 .. of a segment, kJoin at the most, 4 channels a
// thread: to `out`, or to the workspace's partial state `slot` if that is not negative.
template <int D, int kWarps, int kJoin>
__device__ __forceinline__ void join_warps(const Int8DecodeParams& p, int hq0, int h0, int heads, int slot, int b,
                                           const float* buf, const float (&sm_m)[kWarps][kHeads],
                                           const float (&sm_l)[kWarps][kHeads]) {
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  for (int i = threadIdx.x; i < min(kJoin, heads - h0) * (D / 4); i += 32 * kWarps) {
    const int h = h0 + i / (D / 4);
    float mx = -FLT_MAX, sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (sm_l[w][h] > 0.f) mx = fmaxf(mx, sm_m[w][h]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float l = sm_l[w][h], f = l == 0.f ? 0.f : exp2_fast(sm_m[w][h] - mx);   // (a NaN stays one)
      const float4 x = reinterpret_cast<const float4*>(buf)[w * kJoin * (D / 4) + i];
      sum = fmaf(f, l, sum);
      v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
    }
    if (slot < 0) {
      const float inv = sum != 0.f ? __fdividef(1.f, sum) : 0.f;
      reinterpret_cast<uint2*>(p.out + (int64_t(b) * p.c.n_q + hq0) * D)[h0 * (D / 4) + i] =
          make_uint2(pack_bf162(v.x * inv, v.y * inv), pack_bf162(v.z * inv, v.w * inv));
      if (p.lse && i % (D / 4) == 0) p.lse[int64_t(b) * p.c.n_q + hq0 + h] = lse_of(mx, sum);
    } else {
      reinterpret_cast<float4*>(ws + kOffO)[(int64_t(slot) * kHeads + h0) * (D / 4) + i] = v;
      if (i % (D / 4) == 0) reinterpret_cast<float2*>(ws + kOffMl)[slot * kHeads + h] = make_float2(mx, sum);
    }
  }
}

// A run in more than one share: its place in the row, pages, request, first
// query head and their number.
struct Part {
  int run, pages, b, hq0, heads;
};

// Joins the parts of a run; the whole CTA, 4 channels a thread.  Where the heads
// leave threads over, each takes every n-th part; where there are more heads than
// threads for them, they come in turns.  Each round trip to L2 costs as much as five
// pages, so up to twenty parts are asked for at once, the first before their weights are
// known.  (100k tokens, 39 parts: 41.0 us; 41.8 with ten at once, 41.3 and 42.6 with bulk
// and with asynchronous copies of all of them to shared memory.)  The loads stand in the
// code once, which runs once a CTA and comes from far: three copies of them took 41.4.
template <int D, int kWarps>
__device__ __noinline__ void join_parts(const Int8DecodeParams& p, const Part& r, int share, float* wt, float* sum_of) {
  constexpr int kThreads = 32 * kWarps, kBatch = 20;
  const uint8_t* ws = static_cast<const uint8_t*>(p.workspace);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = r.heads;
  const int f = r.run / share, n = (r.run + r.pages - 1) / share - f + 1;
  auto slot_of = [&](int i) { return 2 * (f + i) + (i == 0); };
  const int units = heads * (D / 4), ways = max(1, kThreads / units);
  const int left = min(units, kThreads), way = threadIdx.x / left;
  int unit = threadIdx.x % left;
  float4* sums = reinterpret_cast<float4*>(wt + n * kHeads);
  bool ready = false;                       // the weights are there
#pragma unroll 1
  do {                                      // (more than one unit only where ways is 1)
    const float4* from = reinterpret_cast<const float4*>(ws + kOffO) + unit;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    int i = way;
#pragma unroll 1
    do {
      const int stop = way < ways ? n : 0;
      float4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + k * ways < stop) x[k] = __ldcg(from + slot_of(i + k * ways) * (kHeads * D / 4));
      }
      if (!ready) {
        const float2* ml = reinterpret_cast<const float2*>(ws + kOffMl);
#pragma unroll 1
        for (int h = warp; h < heads; h += kWarps) {
          float mx = -FLT_MAX, sum = 0.f;
#pragma unroll 1
          for (int j = lane; j < n; j += 32) {
            const float2 s = __ldcg(&ml[slot_of(j) * kHeads + h]);
            const float m = s.y == 0.f ? -FLT_MAX : s.x, mn = fmaxf(mx, m);
            sum = fmaf(exp2_fast(m - mn), s.y, sum * exp2_fast(mx - mn));
            mx = mn;
            wt[j * kHeads + h] = m;
          }
          float all = mx;
#pragma unroll
          for (int j = 16; j; j >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, j));
          sum *= exp2_fast(mx - all);
#pragma unroll
          for (int j = 16; j; j >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, j);
#pragma unroll 1
          for (int j = lane; j < n; j += 32) wt[j * kHeads + h] = exp2_fast(wt[j * kHeads + h] - all);
          if (lane == 0) {
            sum_of[h] = sum;
            if (p.lse) p.lse[int64_t(r.b) * p.c.n_q + r.hq0 + h] = lse_of(all, sum);
          }
        }
        __syncthreads();
        ready = true;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (i + k * ways >= stop) break;
        const float g = wt[(i + k * ways) * kHeads + unit / (D / 4)];
        v.x = fmaf(g, x[k].x, v.x), v.y = fmaf(g, x[k].y, v.y), v.z = fmaf(g, x[k].z, v.z), v.w = fmaf(g, x[k].w, v.w);
      }
      i += kBatch * ways;
    } while (i < n);
    if (ways > 1) {
      sums[threadIdx.x] = v;
      __syncthreads();
    }
    if (way == 0) {
#pragma unroll 1
      for (int j = 1; j < ways; ++j) {
        const float4 y = sums[j * units + unit];
        v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
      }
      const float sum = sum_of[unit / (D / 4)], inv = sum != 0.f ? __fdividef(1.f, sum) : 0.f;
      reinterpret_cast<uint2*>(p.out + (int64_t(r.b) * p.c.n_q + r.hq0) * D)[unit] =
          make_uint2(pack_bf162(v.x * inv, v.y * inv), pack_bf162(v.z * inv, v.w * inv));
    }
    unit += kThreads;
  } while (unit < units);
}

// G: the most query heads of a group (4, 8 or 16).  Formed: the scores have a cap or a
// distance bias.
template <int D, int G, bool Formed>
__global__ void __launch_bounds__(32 * warps_of(G), kPerSm) decode_int8_kernel(const __grid_constant__ Int8DecodeParams p) {
  constexpr int kWarps = warps_of(G), kThreads = 32 * kWarps, kStages = stages_of(G);
  constexpr int kBlock = int8_block_bytes(D), C = D / 16;   // chunks of 16 channels
  constexpr int P = pages_of(D), kJoin = join_heads(G);
  constexpr int R = G == 16 ? 2 : 1;                        // sets of 8 columns
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
  __shared__ int sm_scan[kWarps];
  __shared__ Walk sm_walk, sm_walks[kWarps];
  __shared__ Segment sm_next[kWarps];
  __shared__ Part sm_part[2];
  __shared__ int sm_last[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  if (lane < kStages) mbar_init(&bars[warp][lane], 1);
  fence_mbar_init();
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();
  const PagedCache& c = p.c;
  const int group = c.n_q / c.n_kv;

  int share = 0;
  const bool any = begin_share<kThreads>(p, c.n_kv, kMinShare, sm_scan, &sm_walk, &share);
  // requests without a token
  for (int b = blockIdx.x; b < c.batch; b += gridDim.x)
    if (c.seq_len[b] <= 0 || c.max_len == 0) {
      for (int i = threadIdx.x; i < c.n_q * D / 8; i += kThreads)
        reinterpret_cast<uint4*>(p.out + int64_t(b) * c.n_q * D)[i] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (int i = threadIdx.x; i < c.n_q; i += kThreads) p.lse[int64_t(b) * c.n_q + i] = -INFINITY;
    }
  __syncthreads();
  if (!any) return;

  // Each warp walks by itself; the next segment waits in shared memory.
  auto advance = [&]() {
    bool ok = false;
    if (lane == 0) ok = sm_walks[warp].next(p, c.n_kv, &sm_next[warp]);
    __syncwarp();
    return __shfl_sync(0xffffffffu, int(ok), 0) != 0;
  };
  if (lane == 0) sm_walks[warp] = sm_walk;
  if (!advance()) return;                 // (nothing but places of a run's cost; the same in all warps)
  Segment cur = sm_next[warp];
  __syncwarp();
  bool more = false;                      // sm_next holds another

  // The ring.  A warp's steps of a segment begin with another warp each time, so
  // that short segments spread over the warps.  Lane i knows the addresses of the pages of
  // step 32 n + i of the segment that is being brought in (0: the page is not there).
  uint8_t* ring = smem + warp * (kStages * P * kBlock);
  float* buf = reinterpret_cast<float*>(smem + kWarps * kStages * P * kBlock);
  uint64_t* wbars = bars[warp];
  // the segment being brought in: its pages from this warp's first, KV head, request, and steps
  int in_lo, in_hi, in_hk, in_b, in_it = 0, in_n;
  auto turn_to = [&](const Segment& s) {
    in_lo = s.lo + P * place_of<kWarps, P>(s, warp);
    in_hi = s.hi;
    in_hk = s.h;
    in_b = s.b;
    in_it = 0;
    in_n = max(0, (in_hi - in_lo + P * kWarps - 1) / (P * kWarps));
  };
  turn_to(cur);
  bool in_next = false, dead = false;     // it is the next one, not cur
  const uint8_t* src[P];
  int st_in = 0, flying = 0;
  uint32_t ring_dead = 0;                 // bits P i ..: stage i's pages that are not there
  auto bring = [&]() {                    // one more step's; false if there is none to bring yet
    if (in_it == in_n) {
      if (in_next || !more || dead) return false;
      in_next = true;
      turn_to(sm_next[warp]);
      if (in_n == 0) return false;
    }
    if ((in_it & 31) == 0) {
#pragma unroll
      for (int g = 0; g < P; ++g) {
        const int page = in_lo + P * kWarps * (in_it + lane) + g;
        src[g] = nullptr;
        if (page < in_hi) {
          const int id = c.page_table[int64_t(in_b) * c.max_pages + page];
          if (id >= 0 && id < c.n_pages)
            src[g] = c.pages + (int64_t(id) * c.n_kv + in_hk) * kBlock;
          else if (c.dev_status)
            atomicOr(c.dev_status, OSCAR_DEV_PAGE_BOUNDS);
        }
      }
    }
    const int owner = in_it & 31;
    uint32_t there = 0;
#pragma unroll
    for (int g = 0; g < P; ++g) there |= ((__ballot_sync(0xffffffffu, src[g] != nullptr) >> owner) & 1u) << g;
    ring_dead = (ring_dead & ~(((1u << P) - 1) << (P * st_in))) | ((~there & ((1u << P) - 1)) << (P * st_in));
    if (lane == owner) {
      uint64_t* bar = wbars + st_in;
      if (there)
        mbar_arrive_expect_tx(bar, __popc(there) * kBlock);
      else
        mbar_arrive(bar);
#pragma unroll
      for (int g = 0; g < P; ++g)
        if (src[g]) bulk_copy_g2s(ring + (st_in * P + g) * kBlock, src[g], kBlock, bar);
    }
    st_in = st_in + 1 == kStages ? 0 : st_in + 1;
    ++in_it;
    ++flying;
    return true;
  };
  // The query of column gid of each set, channels 16 i + 4 tig .. + 3, asked for before
  // the copies.  G = 4: columns 4 to 7 repeat columns 0 to 3.
  uint2 uq[R][C];
  auto ask_q = [&](const Segment& s) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int h = G == 4 ? gid & 3 : gid + 8 * r;
      const uint16_t* row = p.q + s.b * p.q_stride + int64_t(s.h * group + h) * D + 4 * tig;
#pragma unroll
      for (int i = 0; i < C; ++i) uq[r][i] = h < group ? *reinterpret_cast<const uint2*>(row + 16 * i) : make_uint2(0, 0);
    }
  };
  ask_q(cur);
  while (flying < kStages && bring()) {
  }
  more = advance();                       // (the first copies do not wait for it)
  while (flying < kStages && bring()) {
  }

  // Where this lane's rows of the ldmatrix loads lie in a page: matrices 0 .. 3 are
  // tokens 0 - 7 and 8 - 15 of chunk 2 i, then of chunk 2 i + 1; chunks 2 i further
  // on are an exclusive or with 32 i.
  const int lm_t = (lane & 7) + 8 * ((lane >> 3) & 1);
  const uint32_t lm = uint32_t(lm_t * D + 16 * ((lane >> 4) ^ int8_swizzle(D, lm_t)));
  const bool low_part = G == 4 && tig >= 2;

  int st = 0;
  uint32_t parity = 0;
  int has_part = 0;                       // bits: of a run that began before this share, of one that goes on behind it
  while (true) {
    const int hq0 = cur.h * group, lo = cur.lo + P * place_of<kWarps, P>(cur, warp);
    const int n_it = max(0, (cur.hi - lo + P * kWarps - 1) / (P * kWarps));

    // Query operands, scaled by 2^(141 - ex) so that a head's largest channel is in [2^14, 2^15).
    uint32_t qb[R][C][2];
    float qs[R][2], unscale[R][2], slope[R][2];   // of columns 2 tig, 2 tig + 1
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        top = fmaxf(top, fmaxf(fabsf(bf16_lo(uq[r][i].x)), fabsf(bf16_hi(uq[r][i].x))));
        top = fmaxf(top, fmaxf(fabsf(bf16_lo(uq[r][i].y)), fabsf(bf16_hi(uq[r][i].y))));
      }
      top = max_over_quad(top);
      const int ex = min(max((__float_as_int(top) >> 23) & 255, 14), 254);
      const float up = pow2i(141 - ex);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float q0 = bf16_lo(uq[r][i].x) * up, q1 = bf16_hi(uq[r][i].x) * up;
        const float q2 = bf16_lo(uq[r][i].y) * up, q3 = bf16_hi(uq[r][i].y) * up;
        sum += (q0 + q1) + (q2 + q3);
        qb[r][i][0] = pack_half2(q0, q2);
        qb[r][i][1] = pack_half2(q1, q3);
      }
      sum = sum_over_quad(sum) * 5.9604644775390625e-8f;     // 2^-24, as the codes carry
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 2 * tig + e, h = G == 4 ? col & 3 : col + 8 * r;
        qs[r][e] = __shfl_sync(0xffffffffu, sum, 4 * col);
        unscale[r][e] = unscale_of(__shfl_sync(0xffffffffu, ex, 4 * col), p.s);
        slope[r][e] = Formed && p.s.slopes && h < group ? p.s.slopes[hq0 + h] * kLog2e : 0.f;
      }
    }

    // x is in the dot product's own scale, or in log2 units where the score has a
    // form of its own; us takes it to log2 units, thr is m + 8 / us.  The weights are
    // 2^(7 + (x - m) us) <= 2^15 (the difference first: exact where it matters, however
    // far the scores).
    float us[R][2], thr[R][2], m[R][2], l[R][2], zs[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        us[r][e] = Formed ? 1.f : fmaxf(unscale[r][e], FLT_MIN);
        m[r][e] = thr[r][e] = -FLT_MAX;
        l[r][e] = zs[r][e] = 0.f;
      }
    // rows: channels 16 i + 2 gid (0, 1), + 1 (2, 3); columns 2 tig, 2 tig + 1
    float o[R][C][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < C; ++i) o[r][i][0] = o[r][i][1] = o[r][i][2] = o[r][i][3] = 0.f;
    int ve = -14;                           // the V scales seen are at most 2^ve
    uint32_t vs_top = 0x0400u;              // 2^ve in fp16
    float vs_mul = 16384.f;                 // 2^-ve

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
          st = st + 1 == kStages ? 0 : st + 1;
          parity ^= st == 0;
        }
        __syncwarp();
        break;
      }
      const uint32_t blk0 = smem_addr(ring + st * P * kBlock);
      // tokens 8 t + gid of the step: their values' scales and zeros, and the scores
      float vs[2 * P], vz[2 * P], y[R][2 * P][2];
      uint32_t vbits[2 * P];
#pragma unroll
      for (int g = 0; g < P; ++g) {
        const uint32_t blk = blk0 + g * kBlock, at = blk + lm;
        // S: rows gid and gid + 8 are tokens, columns heads; two chains of products
        float acc[R][2][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int u = 0; u < 2; ++u) acc[r][u][0] = acc[r][u][1] = acc[r][u][2] = acc[r][u][3] = 0.f;
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
          uint32_t k[4];
          ldmatrix_x4(k, at ^ (32 * i));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a0 = even(k[2 * u]), a1 = even(k[2 * u + 1]), a2 = odd(k[2 * u]), a3 = odd(k[2 * u + 1]);
#pragma unroll
            for (int r = 0; r < R; ++r) mma(acc[r][u], a0, a1, a2, a3, qb[r][2 * i + u][0], qb[r][2 * i + u][1]);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint2 w = lds64(blk + 32 * D + 8 * gid + 64 * t);
          const float2 k = half2_to_float2(w.x), v = half2_to_float2(w.y);
          vs[2 * g + t] = v.x;
          vz[2 * g + t] = fmaf(128.f, v.x, v.y);
          vbits[2 * g + t] = w.y & 0xFFFFu;
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              y[r][2 * g + t][e] = fmaf(k.x, acc[r][0][2 * t + e] + acc[r][1][2 * t + e], k.y * qs[r][e]);
        }
      }
      if (Formed) {
        float far = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < 2 * P; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) y[r][t][e] *= unscale[r][e], far = fmaxf(far, fabsf(y[r][t][e]));
        if (p.s.cap_log2 != 0.f) {
          // (the vote skips a form that no score here needs; each score's own is its own)
          if (__builtin_expect(__any_sync(0xffffffffu, !cap_is_near(far, p.s)), 0)) {
#pragma unroll
            for (int j = 0; j < 4 * P * R; ++j) {
              float& x = y[j / (4 * P)][(j >> 1) % (2 * P)][j & 1];
              x = capped(x, p.s);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4 * P * R; ++j) {
              float& x = y[j / (4 * P)][(j >> 1) % (2 * P)][j & 1];
              x = capped_near(x, p.s);
            }
          }
        }
        if (p.s.slopes) {
          const float away = float(tok + gid - (cur.len - 1));
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < 2 * P; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) y[r][t][e] = fmaf(slope[r][e], away + 8.f * t, y[r][t][e]);
        }
      }
      const uint32_t gone = (ring_dead >> (P * st)) & ((1u << P) - 1);
      if (gone || tok < cur.first || tok + P * kPageTokens > cur.len) {
        // what a stale slot holds is anything
#pragma unroll
        for (int t = 0; t < 2 * P; ++t) {
          const int at_tok = tok + 8 * t + gid;
          if (((gone >> (t >> 1)) & 1u) || at_tok < cur.first || at_tok >= cur.len) {
            vs[t] = vz[t] = 0.f;
            vbits[t] = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) y[r][t][0] = y[r][t][1] = -INFINITY;
          }
        }
      }
      uint32_t smax = max(vbits[0], vbits[1]);   // (fp16 values >= 0 order as integers)
      if (P == 2) smax = max(smax, max(vbits[2 * P - 2], vbits[2 * P - 1]));
      bool raise = smax > vs_top;
      float top[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[r][e] = fmaxf(y[r][0][e], y[r][1][e]);
          if (P == 2) top[r][e] = fmaxf(top[r][e], fmaxf(y[r][2 * P - 2][e], y[r][2 * P - 1][e]));
          raise = raise | (top[r][e] > thr[r][e]);
        }
      if (__any_sync(0xffffffffu, raise)) {
        const int ne = max(ve, scale_exponent(__reduce_max_sync(0xffffffffu, smax)));
        const float fv = pow2i(ve - ne);
        ve = ne;
        vs_top = ve < 16 ? uint32_t(ve + 15) << 10 : 0xFFFFu;
        vs_mul = pow2i(-ve);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m[r][e], max_over_rows(top[r][e]));
            f[e] = exp2_fast((m[r][e] - mn) * us[r][e]);
            m[r][e] = mn;
            thr[r][e] = mn + 8.f / us[r][e];
            l[r][e] *= f[e];
            zs[r][e] *= f[e];
            f[e] *= fv;
          }
#pragma unroll
          for (int i = 0; i < C; ++i) o[r][i][0] *= f[0], o[r][i][1] *= f[1], o[r][i][2] *= f[0], o[r][i][3] *= f[1];
        }
      }
#pragma unroll
      for (int g = 0; g < P; ++g) {
        // P's operands: the weights times the values' scales, in two parts
        uint32_t hi[R][2], part[R][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float s = vs[2 * g + t] * vs_mul;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = exp2_fast(fmaf(y[r][2 * g + t][e] - m[r][e], us[r][e], 7.f));
              l[r][e] += x;
              zs[r][e] = fmaf(x, vz[2 * g + t], zs[r][e]);
              w[e] = x * s;
            }
            const uint32_t h = pack_half2(w[0], w[1]);
            const float2 hf = half2_to_float2(h);
            const uint32_t rest = pack_half2(w[0] - hf.x, w[1] - hf.y);
            if (G == 4) {                   // (columns 4 to 7 take the second parts)
              hi[r][t] = movmatrix_trans(low_part ? rest : h);
            } else {
              hi[r][t] = movmatrix_trans(h);
              part[r][t] = movmatrix_trans(rest);
            }
          }
        }
        // O: rows are channels
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
          uint32_t v[4];
          ldmatrix_x4_t(v, (blk0 + g * kBlock + lm + 16 * D) ^ (32 * i));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a0 = even_signed(v[2 * u]), a1 = odd_signed(v[2 * u]);
            const uint32_t a2 = even_signed(v[2 * u + 1]), a3 = odd_signed(v[2 * u + 1]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              mma(o[r][2 * i + u], a0, a1, a2, a3, hi[r][0], hi[r][1]);
              if (G > 4) mma(o[r][2 * i + u], a0, a1, a2, a3, part[r][0], part[r][1]);
            }
          }
        }
      }
      __syncwarp();                         // the stage has been read
      --flying;
      bring();
      tok += P * kWarps * kPageTokens;
      st = st + 1 == kStages ? 0 : st + 1;
      parity ^= st == 0;
    }

    if (more) ask_q(sm_next[warp]);
    // The warps' states of this segment, kJoin heads at a time.  (All with
    // the weights' 2^7; a warp without a token has l = 0, whatever its m.)
    const float un = pow2i(ve);             // of the scales
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[r][e] = sum_over_rows(l[r][e]);
        zs[r][e] = sum_over_rows(zs[r][e]);
        if (gid == 0 && !low_part) sm_m[warp][8 * r + 2 * tig + e] = m[r][e] * us[r][e], sm_l[warp][8 * r + 2 * tig + e] = l[r][e];
      }
      if (G == 4)
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[r][i][j] += __shfl_xor_sync(0xffffffffu, o[r][i][j], 2);
    }
    const bool whole = cur.off == 0 && cur.hi - cur.lo == cur.pages;
    const int slot = 2 * blockIdx.x + (cur.off == 0);
    for (int h0 = 0; h0 < group; h0 += kJoin) {
      if (h0) __syncthreads();              // the heads before have been read
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int h = 8 * r + 2 * tig - h0;
        if (h >= 0 && h < kJoin && !low_part) {
          float2* to = reinterpret_cast<float2*>(buf + (warp * kJoin + h) * D + 2 * gid);
#pragma unroll
          for (int i = 0; i < C; ++i) {
            to[8 * i] = make_float2(fmaf(o[r][i][0], un, zs[r][0]), fmaf(o[r][i][2], un, zs[r][0]));
            to[8 * i + D / 2] = make_float2(fmaf(o[r][i][1], un, zs[r][1]), fmaf(o[r][i][3], un, zs[r][1]));
          }
        }
      }
      __syncthreads();
      join_warps<D, kWarps, kJoin>(p, hq0, h0, group, whole ? -1 : slot, cur.b, buf, sm_m, sm_l);
    }
    if (!whole && threadIdx.x == 0) sm_part[cur.off == 0] = {cur.at - cur.off, cur.pages, cur.b, hq0, group};
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
      join_parts<D, kWarps>(p, sm_part[which], share, reinterpret_cast<float*>(smem), sm_l[0]);   // (the ring is free)
    }
}

template <int D, int G, bool Formed>
cudaError_t launch(const Int8DecodeParams& p, cudaStream_t stream) {
  // the ring, and the warps' states of the heads that are joined at a time
  constexpr int bytes = warps_of(G) * (stages_of(G) * pages_of(D) * int8_block_bytes(D) + join_heads(G) * D * 4);
  static_assert((kCtas + 1) * kHeads * 4 + 32 * warps_of(G) * 16 <= bytes);   // the parts' weights and partial sums
  const cudaError_t e = set_smem_limit<decode_int8_kernel<D, G, Formed>>(bytes);
  if (e != cudaSuccess) return e;
  int64_t tokens = p.c.max_len;
  if (p.s.window) tokens = std::min<int64_t>(tokens, int64_t(p.s.window) + kPageTokens);
  const int64_t places = ((tokens + kPageTokens - 1) / kPageTokens + kRunCost) * p.c.batch * p.c.n_kv;
  if (places > INT32_MAX) return cudaErrorNotSupported;
  const int64_t ctas = std::min<int64_t>(kCtas, (places + kMinShare - 1) / kMinShare);
  return launch_pdl(decode_int8_kernel<D, G, Formed>, dim3(unsigned(ctas)), dim3(32 * warps_of(G)), bytes, stream, p);
}

template <int D, int G>
cudaError_t launch_f(const Int8DecodeParams& p, cudaStream_t stream) {
  return p.s.cap_log2 != 0.f || p.s.slopes ? launch<D, G, true>(p, stream) : launch<D, G, false>(p, stream);
}
template <int D>
cudaError_t launch_g(const Int8DecodeParams& p, cudaStream_t stream) {
  const int group = p.c.n_q / p.c.n_kv;
  return group <= 4 ? launch_f<D, 4>(p, stream) : group <= 8 ? launch_f<D, 8>(p, stream) : launch_f<D, 16>(p, stream);
}

}  // namespace

size_t int8_decode_workspace_bytes(const PagedCache& c) { return kOffO + size_t(kCtas) * 2 * kHeads * c.d * 4; }

cudaError_t launch_decode_int8(const Int8DecodeParams& p, cudaStream_t stream) {
  Int8DecodeParams u = p;
  u.s = in_units(p.s);
  return p.c.d == 128 ? launch_g<128>(u, stream) : launch_g<64>(u, stream);
}

}  // namespace oscar
