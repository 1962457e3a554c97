// Attention of packed prompts over bf16 rows.
#include <cuda_bf16.h>

#include "kernels.h"
#include "oscar.h"
#include "ptx.cuh"
#include "score.cuh"

namespace oscar {
namespace {

constexpr int kPromptWarps = 4;

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

// One warp per (query row, head), keys one after the other.
template <int D>
__global__ void __launch_bounds__(32 * kPromptWarps) prompt_kernel(const PromptParams p) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kC = D / 32;
  const int lane = threadIdx.x & 31, hq = blockIdx.y, b = blockIdx.z;
  const int r = blockIdx.x * kPromptWarps + (threadIdx.x >> 5);
  const PromptSpan sp = prompt_span(p, b, threadIdx.x == 0 && blockIdx.x == 0 && hq == 0);
  if (r >= sp.n_q) return;
  const int hk = hq / (p.n_q / p.n_kv), i = sp.n_k - sp.n_q + r;
  const float slope = p.s.slopes ? p.s.slopes[hq] * kLog2e : 0.f;
  float q[kC], o[kC];
  for (int e = 0; e < kC; ++e) {
    q[e] = __uint_as_float(uint32_t(p.q[(sp.q0 + r) * p.q_stride + hq * D + kC * lane + e]) << 16);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < sp.n_k; ++j) {
    const bool seen = j < sp.prefix || ((!p.causal || j <= i) && (!p.s.window || i - j < p.s.window));
    if (!seen) continue;
    float x = 0.f, v[kC];
    for (int e = 0; e < kC; ++e) {
      const int ch = hk * D + kC * lane + e;
      x = fmaf(q[e], __uint_as_float(uint32_t(p.k[(sp.k0 + j) * p.k_stride + ch]) << 16), x);
      v[e] = __uint_as_float(uint32_t(p.v[(sp.k0 + j) * p.v_stride + ch]) << 16);
    }
    for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    const float y = (p.s.cap_log2 != 0.f ? capped(x, p.s) : x * p.s.scale_log2) - slope * fabsf(float(i - j));
    const float mn = fmaxf(m, y), f = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(y - mn);
    m = mn;
    l = l * f + w;
    for (int e = 0; e < kC; ++e) o[e] = fmaf(w, v[e], o[e] * f);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int e = 0; e < kC; ++e)
    p.out[((sp.q0 + r) * p.n_q + hq) * D + kC * lane + e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * inv));
  if (p.lse && lane == 0) p.lse[(sp.q0 + r) * p.n_q + hq] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t prompt_workspace_bytes(const PromptParams&, cudaError_t* err) {
  *err = cudaSuccess;
  return 256;
}

cudaError_t launch_prompt(const PromptParams& p, cudaStream_t stream) {
  const dim3 grid(unsigned((p.max_q + kPromptWarps - 1) / kPromptWarps), unsigned(p.n_q), unsigned(p.batch));
  return p.d == 128 ? launch_pdl(prompt_kernel<128>, grid, dim3(32 * kPromptWarps), 0, stream, p)
                    : launch_pdl(prompt_kernel<64>, grid, dim3(32 * kPromptWarps), 0, stream, p);
}

}  // namespace oscar
