// Attention of packed prompts over bf16 rows, on the tensor cores (tcgen05).
//
// A CTA takes 2 x 128 query rows of one KV head: rows are (token, head) pairs
// of the query heads that read it (up to 16), so that short
// prompts fill the tiles and K and V are read once for those heads.  Keys come
// in tiles of 128.  One warp brings Q, K and V by TMA, one issues the MMAs, one
// clears what no row sees of V, and four for each of the two row tiles do the
// softmax, one thread a row.  Per key tile and row tile:
//   S = Q K^T   A and B in shared memory, the 128 x 128 result in TMEM;
//   P = 2^(S - m) in the thread's registers, written over S in TMEM as bf16 (the
//               one rounding below fp32: the tensor cores take 16-bit operands);
//   O += P V    A = P in TMEM, B = V as it lies in memory (MN-major), O in TMEM.
// While one row tile's softmax runs, the tensor cores work for the other.  The
// reference m of a row is raised only when a score exceeds it by 2^8: then its
// thread rescales O in TMEM after the last product is done (rare after the
// first tiles).  Tiles of keys that the mask rules out for all rows are not
// visited.  A few rows over many keys are split over the keys; the parts'
// unnormalised sums go to the workspace and a second kernel joins them.  Where the
// rows fit one tile, the two row tiles take alternate key tiles of a part, and
// are joined in the CTA before they go out (24 tokens on 32,000 keys: 36.7 us, with
// twice the parts for the second kernel 40.9).
//
// Measured: 8,192 causal tokens of 32/8 heads x 128 in 380 to 400 us, 1.37 to 1.45
// PFLOP/s (71 to 75 % of the burst rate of a large GEMM), bound by the chain S, softmax,
// P, O, which two row tiles cover only in part: of a step's 3,100 cycles the tensor
// cores work 2,000 (S 484 and P V 512 for each tile), a tile's softmax takes 1,300.  24
// tokens on 32,000 keys in 37 us (132 MB): 5.2 TB/s within the scan, then 4 us of first
// loads and 4 of the join.  The dual kernels spill 32 to 40 bytes a thread (with bias
// and cap at 64 channels 124), of the others one 12.  Slower: P handed over in halves
// (4 %), a second issuing warp (10 %), the maximum taken beside the powers (6 %).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "kernels.h"
#include "oscar.h"
#include "ptx.cuh"
#include "score.cuh"

namespace oscar {
namespace {

constexpr int kTile = 128;            // rows of a tile, of queries and of keys
constexpr int kPanel = kTile * 128;   // bytes of 128 rows of 64 channels
constexpr int kThreads = 384;         // three warpgroups: two of softmax, one of single warps
constexpr int kMmaWarp = 8, kLoadWarp = 9, kHoleWarp = 10;
constexpr int kSms = 152;
// tiles of K and V in flight or in use: a ring in the order K0 V0 K1 V1 ..
template <int D>
constexpr int kRing = D == 128 ? 5 : 10;

struct PromptPlan {
  int pack;        // query heads in a tile's rows: row = token * pack + head, 128 / pack tokens
  int sets;        // head sets
  int blocks;      // row blocks of the longest request
  int splits;      // parts of the keys
  int dual;        // 1: the rows fit one tile, and the row tiles take every other key tile of them
  size_t off_ml, off_o, bytes;
};

PromptPlan plan_prompt(const PromptParams& p) {
  PromptPlan r{};
  const int group = p.n_q / p.n_kv;
  // the heads of a KV head, or the largest divisor of their number up to 16: a tile
  // then has at most 11 rows to spare, and the split-off sets read K and V again
  for (r.pack = std::min(group, 16); group % r.pack; --r.pack) {
  }
  r.sets = p.n_q / r.pack;
  const int per_tile = kTile / r.pack;
  r.blocks = int((int64_t(p.max_q) + 2 * per_tile - 1) / (2 * per_tile));
  const int64_t ctas = int64_t(r.blocks) * r.sets * p.batch;
  const int64_t tiles = (int64_t(p.max_k) + kTile - 1) / kTile;
  r.splits = int(std::max<int64_t>(1, std::min<int64_t>(kSms / std::max<int64_t>(1, ctas), tiles / 4)));
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  r.dual = r.splits > 1 && p.max_q <= per_tile;
  if (r.splits > 1) {
    const size_t rows = size_t(ctas) * r.splits * (r.dual ? 1 : 2) * kTile;
    r.off_o = up(rows * 8);
    r.bytes = r.off_o + rows * p.d * 4;
  } else {
    r.bytes = 256;
  }
  return r;
}

// The rows of request b: first query and key row, clamped counts.
struct PromptSpan {
  int64_t q0, k0;
  int n_q, n_k, prefix;
};
__device__ __forceinline__ PromptSpan prompt_span(const PromptParams& p, int b, bool report) {
  PromptSpan r;
  const int64_t q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
  const bool bad = q0 < 0 || q1 < q0 || q1 > p.total_q || q1 - q0 > p.max_q || k0 < 0 || k1 < k0 || k1 > p.total_k ||
                   k1 - k0 > p.max_k;
  if (bad && report && p.dev_status) atomicOr(p.dev_status, OSCAR_DEV_LENGTH);
  r.q0 = min(max(q0, int64_t(0)), p.total_q);
  r.k0 = min(max(k0, int64_t(0)), p.total_k);
  r.n_q = int(min(max(min(q1, p.total_q) - r.q0, int64_t(0)), int64_t(p.max_q)));
  r.n_k = int(min(max(min(k1, p.total_k) - r.k0, int64_t(0)), int64_t(p.max_k)));
  r.prefix = p.prefix ? min(max(p.prefix[b], 0), r.n_k) : 0;
  return r;
}

struct Barriers {
  uint64_t q_full, full[10], empty[10], holed[3], s_full[2], p_full[2], o_done[2], fin;
  uint32_t tmem;
  int dead;
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

// capped_near of two scores; c holds its coefficients.  (By powers and reciprocals, two
// of the special function unit's instructions a score besides the softmax's one, a
// tile of 128 x 128 scores took twice as long.)
__device__ __forceinline__ float2 capped_near2(float2 x, float cap_in, const float (&c)[5]) {
  const float2 w = mul2(x, make_float2(cap_in, cap_in)), u = mul2(w, w);
  float2 r = make_float2(c[4], c[4]);
#pragma unroll
  for (int k = 3; k >= 0; --k) r = fma2(r, u, make_float2(c[k], c[k]));
  return mul2(x, r);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float row_max(const float (&s)[kTile]) {
  float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int i = 4; i < kTile - 4; i += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = max3(m[e], s[i + e], s[i + 4 + e]);
#pragma unroll
  for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], s[kTile - 4 + e]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// What the scores go through before the softmax.  (In a kernel for all forms the
// loop spills: 8k tokens without any took 406 us against 388; 4096 with a bias, in one
// for biases with and without a cap, 155 against 141.)
enum Form { kPlain, kCapped, kBiased, kBiasedCapped };   // kBiased: a distance bias

// Dual: one row tile, its key tiles to the two warpgroups in turn (PromptPlan's dual).
template <int D, Form kForm, bool Dual>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ PromptParams p, const PromptPlan plan, const __grid_constant__ CUtensorMap tq,
                  const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  constexpr int kPanels = D / 64, kTileBytes = kPanels * kPanel, kR = kRing<D>;
  constexpr uint32_t kIdescS = idesc_bf16_f32(kTile, kTile), kIdescO = idesc_bf16_f32_bmn(kTile, D);
  constexpr uint32_t kColO = 2 * kTile;          // TMEM columns: S0, S1, O0, O1
  extern __shared__ uint8_t raw[];
  __shared__ Barriers bar;
  uint8_t* sq = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  uint8_t* ring = sq + 2 * kTileBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();

  const int set = blockIdx.x % plan.sets, blk = plan.blocks - 1 - int(blockIdx.x / plan.sets);
  const int b = blockIdx.y, split = blockIdx.z;
  const PromptSpan sp = prompt_span(p, b, tid == 0 && blockIdx.x == 0 && split == 0);
  const int pack = plan.pack, per_tile = kTile / pack;   // tokens of a tile
  constexpr bool dual = Dual, kFormed = kForm != kPlain;
  constexpr bool kBias = kForm == kBiased || kForm == kBiasedCapped, kCap = kForm == kCapped || kForm == kBiasedCapped;
  const int tok0 = blk * 2 * per_tile;
  if (tok0 >= sp.n_q) return;
  const int hq0 = set * pack, hk = hq0 / (p.n_q / p.n_kv), shift = sp.n_k - sp.n_q;   // position = shift + token

  // key tiles that some row sees: the prefix's, then those from the window's
  // first to the last row's last; n[w]: as far as row tile w goes
  int n_pre = 0, from = 0, first = 0, n[2];   // first: the window's first key for the CTA's first row
  const int tiles = (sp.n_k + kTile - 1) / kTile;
  // (positions may be negative and the window any int: compared before they are subtracted)
  if (p.s.window && shift + tok0 >= p.s.window) first = shift + tok0 - p.s.window + 1;
  from = min(first / kTile, tiles);
  n_pre = min((sp.prefix + kTile - 1) / kTile, from);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int last = min(tok0 + (w + 1) * per_tile, sp.n_q) - 1;     // last token of the tile
    int to = tiles;
    if (p.causal) to = max((sp.prefix + kTile - 1) / kTile, (max(0, min(shift + last + 1, sp.n_k)) + kTile - 1) / kTile);
    n[w] = tok0 + w * per_tile < sp.n_q ? n_pre + max(0, to - from) : 0;
  }
  // this part of them
  const int all = max(n[0], n[1]);
  const int lo = int(int64_t(all) * split / plan.splits), hi = int(int64_t(all) * (split + 1) / plan.splits);
  const int n_all = hi - lo;
  n[0] = dual ? (n_all + 1) / 2 : max(0, min(n[0], hi) - lo);
  n[1] = dual ? n_all / 2 : max(0, min(n[1], hi) - lo);
  auto tile_of = [&](int j) { return j + lo < n_pre ? j + lo : j + lo - n_pre + from; };

  if (n_all > 0) {
    if (tid == 0) {
      mbar_init(&bar.q_full, 1);
      for (int i = 0; i < 3; ++i) mbar_init(&bar.holed[i], 1);
      mbar_init(&bar.fin, 1);
      for (int i = 0; i < kR; ++i) {
        mbar_init(&bar.full[i], 1);
        mbar_init(&bar.empty[i], 1);
      }
      for (int w = 0; w < 2; ++w) {
        mbar_init(&bar.s_full[w], 1);
        mbar_init(&bar.p_full[w], kTile);
        mbar_init(&bar.o_done[w], 1);
      }
      bar.dead = 0;
      fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc(&bar.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem = bar.tmem;
  volatile int* dead = &bar.dead;
  // False where a wait ran out: reported once, and every other wait of the CTA ends soon after.
  auto wait = [&](uint64_t* at, uint32_t parity) {
    if (mbar_try_wait(at, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_sleep(at, parity, 10000)) {
      if (*dead) return false;
      if (global_timer_ns() - t0 > kDefaultWaitNs) {
        *dead = 1;
        if (p.dev_status) atomicOr(p.dev_status, OSCAR_DEV_TIMEOUT);
        return false;
      }
    }
    return true;
  };
  // Rows of V that no row here sees may hold anything, and 0 times that is not
  // 0: a warp of its own clears them between the load and the product.  They are
  // the keys from the prefix's end to the window's first, in the list's entries
  // e_pre and e_win, and those behind the last key, in e_end.
  const int e_pre = first > sp.prefix && sp.prefix % kTile ? n_pre - 1 - lo : -1;
  const int e_win = first > sp.prefix && first % kTile ? n_pre - lo : -1;
  const int e_end = n_all > 0 && tile_of(n_all - 1) == tiles - 1 && sp.n_k % kTile ? n_all - 1 : -1;
  auto holes = [&](int j) { return j == e_pre || j == e_win || j == e_end; };

  // Registers: the launch's 168 a thread, 504 over the three warpgroups.  A
  // softmax thread holds a row's 128 scores; the issuing warp must not spill (at
  // 56 registers it did, and an 8k prompt took 7 % longer).
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == kLoadWarp && lane == 0 && n_all > 0) {
      const int tiles_q = !dual && tok0 + per_tile < sp.n_q ? 2 : 1;
      mbar_arrive_expect_tx(&bar.q_full, uint32_t(tiles_q * kPanels * pack * per_tile * 128));
      for (int w = 0; w < tiles_q; ++w)
        for (int c = 0; c < kPanels; ++c)
          tma_load_3d(sq + w * kTileBytes + c * kPanel, &tq, 64 * c, hq0, int(sp.q0) + tok0 + w * per_tile, &bar.q_full);
      int t = 0, st = 0, turn = 0, n_holed = 0;   // t = 2 j is K of step j, 2 j + 1 its V
      for (; t < 2 * n_all; ++t) {
        if (turn > 0 && !wait(&bar.empty[st], (turn - 1) & 1)) break;
        const int row = int(sp.k0) + tile_of(t >> 1) * kTile;
        uint64_t* at = (t & 1) && holes(t >> 1) ? &bar.holed[n_holed++] : &bar.full[st];
        mbar_arrive_expect_tx(at, kTileBytes);
        for (int c = 0; c < kPanels; ++c)
          tma_load_3d(ring + st * kTileBytes + c * kPanel, (t & 1) ? &tv : &tk, 64 * c, hk, row, at);
        if (++st == kR) st = 0, ++turn;
      }
      // what was issued has landed before the CTA's shared memory goes
      mbar_wait_bounded(&bar.q_full, 0, kDrainWaitNs);
      for (int i = 0; i < n_holed; ++i) mbar_wait_bounded(&bar.holed[i], 0, kDrainWaitNs);
      for (int i = max(0, t - kR); i < t; ++i)
        if (!((i & 1) && holes(i >> 1))) mbar_wait_bounded(&bar.full[i % kR], (i / kR) & 1, kDrainWaitNs);
    } else if (warp == kHoleWarp) {
      int n_holed = 0;
      for (int j = 0; j < n_all; ++j) {
        if (!holes(j)) continue;
        const int k0 = tile_of(j) * kTile, st = (2 * j + 1) % kR;
        if (!__all_sync(0xffffffffu, wait(&bar.holed[n_holed++], 0))) break;
        uint8_t* v = ring + st * kTileBytes;
        auto clear = [&](int a, int b) {     // rows a .. b - 1
          for (int i = a * 8 + lane; i < b * 8; i += 32)
#pragma unroll
            for (int c = 0; c < kPanels; ++c) *reinterpret_cast<uint4*>(v + c * kPanel + 16 * i) = make_uint4(0, 0, 0, 0);
        };
        clear(max(sp.prefix - k0, 0), min(first - k0, kTile));
        clear(max(sp.n_k - k0, 0), kTile);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.full[st]);
      }
    } else if (warp == kMmaWarp && n_all > 0) {
      // Step i of row tile w uses K and V of the list's entry i (dual: 2 i + w).
      // Per step and row tile: O += P V of this step, then S of the next, so
      // that the other row tile's softmax runs beside them.  The whole warp
      // walks through the steps and one thread issues: the MMAs' operands stay
      // in uniform registers (in a branch of one thread each MMA took three
      // times as long to issue as to run).
      const uint64_t dq = smem_desc_kmajor_sw128(smem_addr(sq)), dk = smem_desc_kmajor_sw128(smem_addr(ring));
      const uint64_t dv = smem_desc_mnmajor_sw128(smem_addr(ring), kPanel);
      auto arrived = [&](uint64_t* at, uint32_t parity) { return __all_sync(0xffffffffu, wait(at, parity)) != 0; };
      auto mma_s = [&](int w, int st) {
        const uint64_t a = dq + uint64_t(dual ? 0 : w * (kTileBytes >> 4)), bb = dk + uint64_t(st * (kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * (kPanel >> 4) + (kk % 4) * 2;
          umma_f16_ss(tmem + w * kTile, a + off, bb + off, kIdescS, kk > 0);
        }
        umma_commit(&bar.s_full[w]);
      };
      // ring places of K (of the step to come) and V, and the parities of their turns
      int ks[2], vs[2];
      uint32_t kp[2] = {0, 0}, vp[2] = {0, 0};
      bool ok = arrived(&bar.q_full, 0);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        ks[w] = dual ? 2 * w : 0;
        vs[w] = ks[w] + 1;
        if (ok && n[w] > 0) {
          ok = arrived(&bar.full[ks[w]], 0);
          if (ok && elect_one()) {
            mma_s(w, ks[w]);
            if (dual || w == 1 || n[1] == 0) umma_commit(&bar.empty[ks[w]]);
          }
          __syncwarp();
        }
      }
      const int stride = dual ? 4 : 2, rounds = max(n[0], n[1]);
      for (int i = 0; i < rounds && ok; ++i) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          ks[w] += stride;
          if (ks[w] >= kR) ks[w] -= kR, kp[w] ^= 1;
          if (ok && i < n[w]) {
            // K first, too: with P there the two products go out together.  (A
            // dual part is bound by its loads, and does not wait for K here.)
            const bool more = i + 1 < n[w];
            if (w == 0 || dual || i >= n[0]) ok = arrived(&bar.full[vs[w]], vp[w]);
            if (ok && more && !dual && (w == 0 || i + 1 >= n[0])) ok = arrived(&bar.full[ks[w]], kp[w]);
            ok = ok && arrived(&bar.p_full[w], i & 1);
            if (ok) {
              tc_fence_after();
              const uint64_t bb = dv + uint64_t(vs[w] * (kTileBytes >> 4));
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                  umma_f16_ts(tmem + kColO + w * D, tmem + w * kTile + 8 * kk, bb + 128 * kk, kIdescO, i > 0 || kk > 0);
                umma_commit(&bar.o_done[w]);
                // the last row tile to use a tile of keys lets it go
                if (dual || w == 1 || i >= n[1]) umma_commit(&bar.empty[vs[w]]);
                if (more && !dual) {
                  mma_s(w, ks[w]);
                  if (w == 1 || i + 1 >= n[1]) umma_commit(&bar.empty[ks[w]]);
                }
              }
              __syncwarp();
              if (more && dual) {
                ok = arrived(&bar.full[ks[w]], kp[w]);
                if (ok && elect_one()) {
                  mma_s(w, ks[w]);
                  umma_commit(&bar.empty[ks[w]]);
                }
                __syncwarp();
              }
            }
          }
          vs[w] += stride;
          if (vs[w] >= kR) vs[w] -= kR, vp[w] ^= 1;
        }
      }
      // every MMA issued is done before TMEM is given back
      if (elect_one()) umma_commit(&bar.fin);
      __syncwarp();
      mbar_wait_bounded(&bar.fin, 0, kDrainWaitNs);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int w = warp >> 2, row = tid & (kTile - 1);
    const int steps = w ? n[1] : n[0];     // (n[w] would put n, and with it the kernel, in local memory)
    const int tok = tok0 + (dual ? 0 : w * per_tile) + row / pack, head = hq0 + row % pack;
    // a query of this request (the rows to spare of a group that does not divide 128
    // are never written: they hold what an earlier CTA left there)
    const bool mine = row < pack * per_tile && tok < sp.n_q;
    const int pos = shift + tok;
    const int row_lo = p.s.window && pos >= p.s.window ? pos - p.s.window + 1 : 0;
    const int row_hi = p.causal ? min(pos + 1, sp.n_k) : sp.n_k;
    const float slope = kBias ? p.s.slopes[head] * kLog2e : 0.f;
    const float sc = kFormed ? 1.f : p.s.scale_log2;
    const float cap_in = p.s.cap_in;
    float near[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) near[k] = p.s.cap_near[k];
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + lanes + w * kTile, t_o = tmem + lanes + kColO + w * D;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < steps; ++j) {
      ok = wait(&bar.s_full[w], j & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float s[kTile];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, reinterpret_cast<uint32_t(&)[32]>(s[32 * c]));
      tc_wait_ld();
      const int k0 = tile_of(dual ? 2 * j + w : j) * kTile;
      if (kCap) {
        // The form is chosen for each score by itself, so that a row's bits are its own;
        // the votes skip the form that no score of theirs needs.
        auto far = [&](int a, int b) {
          float x = 0.f;
#pragma unroll
          for (int i = a; i < b; ++i) x = fmaxf(x, fabsf(s[i]));
          // (a NaN is not above either: both ways keep it)
          return __any_sync(0xffffffffu, mine && x * cap_in > kLog2e) != 0;
        };
        auto near_all = [&](int a, int b) {
#pragma unroll
          for (int i = a; i < b; i += 2) {
            const float2 t = capped_near2(make_float2(s[i], s[i + 1]), cap_in, near);
            s[i] = t.x;
            s[i + 1] = t.y;
          }
        };
        if (__builtin_expect(!far(0, kTile), 1)) {
          near_all(0, kTile);
        } else {
          // (32 keys at a time: the code for all of them at once spills)
#pragma unroll
          for (int c = 0; c < kTile; c += 32) {
            if (far(c, c + 32)) {
#pragma unroll
              for (int i = c; i < c + 32; i += 2) {
                const float2 t = capped_near2(make_float2(s[i], s[i + 1]), cap_in, near);
                s[i] = capped_pick(s[i], t.x, p.s);
                s[i + 1] = capped_pick(s[i + 1], t.y, p.s);
              }
            } else {
              near_all(c, c + 32);
            }
          }
        }
      }
      if (kBias) {
        const float away = float(pos - k0);
#pragma unroll
        for (int i = 0; i < kTile; ++i) s[i] = fmaf(-slope, fabsf(away - float(i)), kCap ? s[i] : s[i] * p.s.scale_log2);
      }
      const bool full = (k0 >= row_lo && k0 + kTile <= row_hi) || k0 + kTile <= sp.prefix;
      if (!__all_sync(0xffffffffu, full)) {
        // k0 + i in [row_lo, row_hi) or below the prefix
        const uint32_t width = uint32_t(max(0, row_hi - row_lo));
        const int a = k0 - row_lo, pre = sp.prefix - k0;
#pragma unroll
        for (int i = 0; i < kTile; ++i)
          if (uint32_t(a + i) >= width && i >= pre) s[i] = -INFINITY;
      }
      const float mt = row_max(s);
      // Each row raises its own reference (a factor of 1 changes no bit of the other
      // rows' O); rows to spare and other requests' rows, which may hold anything, have
      // no say.  (Nothing seen yet, nothing here: -inf - -inf is no growth.)
      const bool grows = mine && (mt - m) * sc > 8.f;
      if (__any_sync(0xffffffffu, grows)) {
        const float f = !grows ? 1.f : m == -INFINITY ? 0.f : exp2_fast((m - mt) * sc);
        m = grows ? mt : m;
        l *= f;
        if (j > 0) {
          ok = __all_sync(0xffffffffu, wait(&bar.o_done[w], (j - 1) & 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(t_o + 16 * c, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(t_o + 16 * c, o);
          }
        }
      }
      const float off = m == -INFINITY ? 0.f : -m * sc;
      float2 sum[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 e = fma2(make_float2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), make_float2(sc, sc), make_float2(off, off));
          e.x = exp2_fast(e.x);
          e.y = exp2_fast(e.y);
          sum[i & 1] = add2(sum[i & 1], e);
          pk[i] = pack_bf162(e.x, e.y);
        }
        tmem_st16(t_s + 16 * c, pk);
      }
      const float2 both = add2(sum[0], sum[1]);
      l = both.x + both.y;
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(&bar.p_full[w]);
    }
    if (ok && steps > 0) {
      ok = wait(&bar.o_done[w], (steps - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    const int64_t cta = (int64_t(b) * plan.blocks + blk) * plan.sets + set;
    if (plan.splits > 1) {
      // a part: each row's maximum (log2 units), sum and channels.  One without
      // keys, or without visible ones: l = 0, its channels are not read.
      uint8_t* ws = static_cast<uint8_t*>(p.workspace);
      const int64_t at = (cta * plan.splits + split) * (dual ? 1 : 2) * kTile + (dual ? 0 : w * kTile) + row;
      float* po = reinterpret_cast<float*>(ws + plan.off_o) + at * D;
      float2 ml = make_float2(m == -INFINITY ? 0.f : m * sc, ok ? l : 0.f);
      if (dual) {
        // Both warpgroups hold the same rows.  Each gives the other its half of
        // the channels, by way of the queries' place, and joins its own half.
        float4* xo = reinterpret_cast<float4*>(sq);
        float2* xml = reinterpret_cast<float2*>(ring);
        constexpr int kChunks = D / 8;                    // 4 channels each, of half a row
        auto chunk = [&](int half, int c) { return (half * kTile + row) * kChunks + (c ^ (row & (kChunks - 1))); };
        named_barrier(1, 2 * kTile);                      // the products are done: their operands' place is free
        if (ok && steps > 0) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            tmem_ld32(t_o + (1 - w) * (D / 2) + 32 * c, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<uint4*>(xo)[chunk(1 - w, 8 * c + i)] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        xml[w * kTile + row] = ml;
        named_barrier(1, 2 * kTile);
        const float2 other = xml[(1 - w) * kTile + row];
        const float top = other.y == 0.f ? ml.x : ml.y == 0.f ? other.x : fmaxf(ml.x, other.x);
        const float f = ml.y != 0.f ? exp2_fast(ml.x - top) : 0.f, g = other.y != 0.f ? exp2_fast(other.x - top) : 0.f;
        const bool read = ok && steps > 0;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[32];
          if (read) {
            tmem_ld32(t_o + w * (D / 2) + 32 * c, o);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4 x = make_float4(f * __uint_as_float(o[4 * i]), f * __uint_as_float(o[4 * i + 1]),
                                   f * __uint_as_float(o[4 * i + 2]), f * __uint_as_float(o[4 * i + 3]));
            if (other.y != 0.f) {
              const float4 y = xo[chunk(w, 8 * c + i)];
              x.x = fmaf(g, y.x, x.x), x.y = fmaf(g, y.y, x.y), x.z = fmaf(g, y.z, x.z), x.w = fmaf(g, y.w, x.w);
            }
            if (mine) reinterpret_cast<float4*>(po + w * (D / 2) + 32 * c)[i] = x;
          }
        }
        ml = make_float2(top, fmaf(f, ml.y, g * other.y));
        if (mine && w == 0) reinterpret_cast<float2*>(ws + plan.off_ml)[at] = ml;
      } else {
        if (mine) reinterpret_cast<float2*>(ws + plan.off_ml)[at] = ml;
        if (ok && steps > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(t_o + 32 * c, o);
            tc_wait_ld();
            if (mine)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<uint4*>(po + 32 * c)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
      }
    } else {
      const float inv = l != 0.f ? 1.f / l : 0.f;         // (a row with NaN scores stays NaN)
      uint16_t* out = p.out + ((sp.q0 + tok) * p.n_q + head) * D;
      if (mine && p.lse) p.lse[(sp.q0 + tok) * p.n_q + head] = l != 0.f ? (m * sc + log2f(l)) * kLn2 : -INFINITY;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (ok && steps > 0) {
          tmem_ld32(t_o + 32 * c, o);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (mine) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              q[e] = pack_bf162(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
            reinterpret_cast<uint4*>(out + 32 * c)[i] = make_uint4(q[0], q[1], q[2], q[3]);
          }
        }
      }
    }
    if (n_all > 0) tc_fence_before();
  }
  if (n_all > 0) {
    __syncthreads();
    if (warp == kMmaWarp) {
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  }
}

// Joins the parts of each row: one warp a row, 16 parts at a time, whose sums
// are asked for together with their maxima (a part that saw no key has written
// no sums: what is read there is not used).
template <int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptParams p, const PromptPlan plan, int rows) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kC = D / 32, kBatch = 16;
  const int lane = threadIdx.x & 31, row = (blockIdx.x % (rows / 8)) * 8 + (threadIdx.x >> 5);
  const int64_t cta = blockIdx.x / (rows / 8);
  const int set = int(cta % plan.sets), blk = int(cta / plan.sets % plan.blocks), b = int(cta / plan.sets / plan.blocks);
  const PromptSpan sp = prompt_span(p, b, false);
  const int per_tile = kTile / plan.pack, in_tile = row % kTile;
  const int tok = (blk * 2 + row / kTile) * per_tile + in_tile / plan.pack, head = set * plan.pack + in_tile % plan.pack;
  if (in_tile >= plan.pack * per_tile || tok >= sp.n_q) return;
  const uint8_t* ws = static_cast<const uint8_t*>(p.workspace);
  const int parts = plan.splits;
  const int64_t first = cta * parts * rows + row;    // parts are `rows` rows apart
  const float2* ml = reinterpret_cast<const float2*>(ws + plan.off_ml) + first;
  const float* po = reinterpret_cast<const float*>(ws + plan.off_o) + first * D + lane * kC;
  float mx = -INFINITY, sum = 0.f, o[kC] = {};
  for (int s0 = 0; s0 < parts; s0 += kBatch) {
    float v[kBatch][kC];
    float2 x = make_float2(0.f, 0.f);
    if (lane < kBatch && s0 + lane < parts) x = __ldcg(&ml[int64_t(s0 + lane) * rows]);
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const float* from = po + int64_t(min(s0 + s, parts - 1)) * rows * D;
      if constexpr (kC == 4) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(from));
        v[s][0] = u.x, v[s][1] = u.y, v[s][2] = u.z, v[s][3] = u.w;
      } else {
        const float2 u = __ldcg(reinterpret_cast<const float2*>(from));
        v[s][0] = u.x, v[s][1] = u.y;
      }
    }
    float top = x.y != 0.f ? x.x : -INFINITY;   // (a part whose sum is NaN counts)
#pragma unroll
    for (int i = 8; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    top = __shfl_sync(0xffffffffu, top, 0);
    if (top == -INFINITY) continue;          // the same in all lanes
    const float mn = fmaxf(mx, top), f = mx == -INFINITY ? 0.f : exp2_fast(mx - mn);
    mx = mn;
    const float g = x.y != 0.f ? exp2_fast(x.x - mn) : 0.f;
    sum = fmaf(g, x.y, sum * f);             // of this lane's parts
#pragma unroll
    for (int e = 0; e < kC; ++e) o[e] *= f;
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const float gs = __shfl_sync(0xffffffffu, g, s);
#pragma unroll
      for (int e = 0; e < kC; ++e) o[e] = gs > 0.f ? fmaf(gs, v[s][e], o[e]) : o[e];
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + ((sp.q0 + tok) * p.n_q + head) * D + kC * lane);
#pragma unroll
  for (int e = 0; e < kC / 2; ++e) out[e] = pack_bf162(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (p.lse && lane == 0) p.lse[(sp.q0 + tok) * p.n_q + head] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// rows [total][heads][d] bf16, `stride` elements apart, in boxes of 64 channels
bool encode_rows(CUtensorMap* map, const uint16_t* x, int d, int heads, int64_t total, int64_t stride, int box_heads,
                 int box_rows) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
      return false;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(std::max<int64_t>(1, total))};
  const cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(stride) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(x), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, Form kForm, bool Dual>
cudaError_t launch(const PromptParams& p, const PromptPlan& plan, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  const uint16_t* k = p.total_k ? p.k : p.q;   // no key, no load: the maps only have to be well-formed
  const uint16_t* v = p.total_k ? p.v : p.q;
  if (!encode_rows(&tq, p.q, D, p.n_q, p.total_q, p.q_stride, plan.pack, kTile / plan.pack) ||
      !encode_rows(&tk, k, D, p.n_kv, p.total_k, p.k_stride, 1, kTile) ||
      !encode_rows(&tv, v, D, p.n_kv, p.total_k, p.v_stride, 1, kTile))
    return cudaErrorInvalidValue;
  constexpr int bytes = 1024 + (2 + kRing<D>) * (D / 64) * kPanel;
  cudaError_t e = set_smem_limit<prompt_kernel<D, kForm, Dual>>(bytes);
  if (e != cudaSuccess) return e;
  const int64_t x = int64_t(plan.blocks) * plan.sets;
  const dim3 grid(unsigned(x), unsigned(p.batch), unsigned(plan.splits));
  e = launch_pdl(prompt_kernel<D, kForm, Dual>, grid, dim3(kThreads), bytes, stream, p, plan, tq, tk, tv);
  if (e != cudaSuccess || plan.splits == 1) return e;
  const int rows = Dual ? kTile : 2 * kTile;
  return launch_pdl(prompt_join_kernel<D>, dim3(unsigned(x * p.batch * (rows / 8))), dim3(256), 0, stream, p, plan, rows);
}

template <int D, Form kForm>
cudaError_t launch_f(const PromptParams& p, const PromptPlan& plan, cudaStream_t stream) {
  return plan.dual ? launch<D, kForm, true>(p, plan, stream) : launch<D, kForm, false>(p, plan, stream);
}

template <int D>
cudaError_t launch_d(const PromptParams& p, const PromptPlan& plan, cudaStream_t stream) {
  const bool cap = p.s.cap_log2 != 0.f;
  if (p.s.slopes) return cap ? launch_f<D, kBiasedCapped>(p, plan, stream) : launch_f<D, kBiased>(p, plan, stream);
  return cap ? launch_f<D, kCapped>(p, plan, stream) : launch_f<D, kPlain>(p, plan, stream);
}

}  // namespace

size_t prompt_workspace_bytes(const PromptParams& p) { return plan_prompt(p).bytes; }

cudaError_t launch_prompt(const PromptParams& p, cudaStream_t stream) {
  const PromptPlan plan = plan_prompt(p);
  // grid limits, of the join's grid too (32 CTAs for each of this one's)
  if (int64_t(plan.blocks) * plan.sets * p.batch > 0x7fffffff / 32) return cudaErrorNotSupported;
  return p.d == 128 ? launch_d<128>(p, plan, stream) : launch_d<64>(p, plan, stream);
}

}  // namespace oscar
