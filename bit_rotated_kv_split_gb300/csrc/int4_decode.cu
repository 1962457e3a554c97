// Decode attention over a 4-bit layer: one query token per request.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "oscar.h"
#include "ptx.cuh"
#include "score.cuh"

namespace oscar {
namespace {

constexpr int kDecodeWarps = 8;

// One CTA per (query head, request); a warp takes every kDecodeWarps-th
// token with an online softmax of its own, and the warps are joined in
// shared memory.  A lane holds D / 32 adjacent channels.
template <int D>
__global__ void __launch_bounds__(32 * kDecodeWarps) decode_int4_kernel(const Int4DecodeParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kC = D / 32;
  __shared__ float sm_m[kDecodeWarps], sm_l[kDecodeWarps], sm_o[kDecodeWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hq = blockIdx.x, b = blockIdx.y;
  const Int4Cache& c = p.c;
  const int hk = hq / (c.n_q / c.n_kv);
  int len = c.seq_len[b];
  if (len < 0 || len > c.max_len) {
    if (threadIdx.x == 0 && c.dev_status) atomicOr(c.dev_status, OSCAR_DEV_LENGTH);
    len = min(max(len, 0), c.max_len);
  }
  const int first = p.s.window ? max(0, len - p.s.window) : 0;
  const float slope = p.s.slopes ? p.s.slopes[hq] * kLog2e : 0.f;
  float q[kC], o[kC];
  for (int e = 0; e < kC; ++e) {
    q[e] = __uint_as_float(uint32_t(p.q[b * p.q_stride + hq * D + kC * lane + e]) << 16);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int64_t block_bytes = int4_block_bytes(D, c.ng_k, c.ng_v);
  for (int j = first + warp; j < len; j += kDecodeWarps) {
    const int page = c.page_table[int64_t(b) * c.max_pages + j / kInt4Page], t = j % kInt4Page;
    if (page < 0 || page >= c.n_pages) {
      if (lane == 0 && c.dev_status) atomicOr(c.dev_status, OSCAR_DEV_PAGE_BOUNDS);
      continue;
    }
    const uint8_t* block = c.pages + (int64_t(page) * c.n_kv + hk) * block_bytes;
    float x = 0.f, v[kC];
    for (int e = 0; e < kC; ++e) {
      const int ch = kC * lane + e;
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(block + int4_k_word(D, t, ch >> 3));
      const uint32_t vh = *reinterpret_cast<const uint16_t*>(block + int4_v_half(D, t, ch >> 2));
      const float2 sk = half2_to_float2(
          *reinterpret_cast<const uint32_t*>(block + int4_pair(D, c.ng_k, c.ng_v, t, ch * c.ng_k / D)));
      const float2 sv = half2_to_float2(
          *reinterpret_cast<const uint32_t*>(block + int4_pair(D, c.ng_k, c.ng_v, t, c.ng_k + ch * c.ng_v / D)));
      x = fmaf(q[e], fmaf(float((kw >> (4 * (ch & 7))) & 15u), sk.x, sk.y), x);
      v[e] = fmaf(float((vh >> (4 * (ch & 3))) & 15u), sv.x, sv.y);
    }
    for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    const float y = (p.s.cap_log2 != 0.f ? capped(x, p.s) : x * p.s.scale_log2) - slope * float(len - 1 - j);
    const float mn = fmaxf(m, y), f = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(y - mn);
    m = mn;
    l = l * f + w;
    for (int e = 0; e < kC; ++e) o[e] = fmaf(w, v[e], o[e] * f);
  }
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
  for (int e = 0; e < kC; ++e) sm_o[warp][kC * lane + e] = o[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float mx = -INFINITY, sum = 0.f, acc = 0.f;
    for (int w = 0; w < kDecodeWarps; ++w) mx = fmaxf(mx, sm_m[w]);
    for (int w = 0; w < kDecodeWarps; ++w) {
      const float f = sm_m[w] == -INFINITY ? 0.f : exp2f(sm_m[w] - mx);
      sum += f * sm_l[w];
      acc += f * sm_o[w][threadIdx.x];
    }
    p.out[(int64_t(b) * c.n_q + hq) * D + threadIdx.x] =
        __bfloat16_as_ushort(__float2bfloat16_rn(sum > 0.f ? acc / sum : 0.f));
  }
}

}  // namespace

size_t int4_decode_workspace_bytes(const Int4Cache&, const ScoreParams&, cudaError_t* err) {
  *err = cudaSuccess;
  return 256;
}

cudaError_t launch_decode_int4(const Int4DecodeParams& p, cudaStream_t stream) {
  const dim3 grid(unsigned(p.c.n_q), unsigned(p.c.batch));
  return p.c.d == 128 ? launch_pdl(decode_int4_kernel<128>, grid, dim3(32 * kDecodeWarps), 0, stream, p)
                      : launch_pdl(decode_int4_kernel<64>, grid, dim3(32 * kDecodeWarps), 0, stream, p);
}

}  // namespace oscar
