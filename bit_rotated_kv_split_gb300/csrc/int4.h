// Internal interface between the 4-bit layer's C-ABI functions (int4_api.cu)
// and its kernels (int4_append.cu, int4_decode.cu, prompt.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace oscar {

constexpr int kPageTokens = 16;

// Page block of one (page, KV head), d channels, ng_k / ng_v groups:
//   [0, 8 d)      K: slot t's d / 2 code bytes at t d / 2; channel 32 w + 8 u
//                 + n is nibble n of its 32-bit word W u + w, W = d / 32;
//   [8 d, 16 d)   V: channel 32 w + 4 u + n of slot t is nibble 4 (t % 2) + n
//                 of word (8 (t / 2) + u) W + w;
//   [16 d, ...)   slot t's K pairs, then its V pairs, fp16 (scale, zero).
__host__ __device__ constexpr int int4_block_bytes(int d, int ng_k, int ng_v) { return 16 * d + 64 * (ng_k + ng_v); }
// byte of the word that holds octet o (channels 8 o ..) of K slot t
__host__ __device__ constexpr int int4_k_word(int d, int t, int o) {
  return t * (d / 2) + 4 * ((d / 32) * (o & 3) + (o >> 2));
}
// byte of the 16-bit half that holds quad e (channels 4 e ..) of V slot t
__host__ __device__ constexpr int int4_v_half(int d, int t, int e) {
  return 8 * d + 4 * ((8 * (t >> 1) + (e & 7)) * (d / 32) + (e >> 3)) + 2 * (t & 1);
}
__host__ __device__ constexpr int int4_pair(int d, int ng_k, int ng_v, int t, int q) {
  return 16 * d + 4 * ((ng_k + ng_v) * t + q);
}

// The pages of a layer, whatever its codes' width.
struct PagedCache {
  uint8_t* pages;
  const int32_t* page_table;
  const int32_t* seq_len;
  int32_t* dev_status;
  int32_t batch, n_q, n_kv, d, max_pages, max_len;
  int64_t n_pages;
};

struct Int4Cache : PagedCache {
  int32_t ng_k, ng_v;
};

struct RopeParams {
  const float* cos_sin;
  int64_t n_positions;
  int32_t rot, interleaved;
};

// The score's form: log2 units throughout (t log2 e), so that the softmax is
// a power of two.  cap: t = cap2 tanh(x * scale / cap) with cap2 = cap log2 e.
struct ScoreParams {
  float scale_log2;    // scale log2 e (no cap)
  float cap_in;        // 2 scale / cap log2 e: e^(2 x scale / cap) = 2^(x cap_in)
  float cap_log2;      // cap log2 e; 0 = no cap
  float unit;          // the decodes: cap_in and cap_near are for dot products times this
  float cap_near[5];   // scores up to half the cap are x P((x cap_in)^2): P's coefficients
  int32_t window;      // 0 = none
  const float* slopes; // natural units; NULL = none
};

struct AppendParams {
  Int4Cache c;
  RopeParams rope;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *dst_req, *dst_pos, *rope_pos;
  int32_t n;
  uint16_t *q_out, *k_out;
  float tau_k, tau_v;
};
cudaError_t launch_rope_append_int4(const AppendParams& p, cudaStream_t stream);

struct GatherParams {
  Int4Cache c;
  const int32_t *src_req, *src_pos;
  int32_t n;
  uint16_t *k_out, *v_out;
  int64_t k_stride, v_stride;
};
cudaError_t launch_gather_int4(const GatherParams& p, cudaStream_t stream);

struct Int4DecodeParams {
  Int4Cache c;
  ScoreParams s;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  void* workspace;
};
size_t int4_decode_workspace_bytes(const Int4Cache& c);
cudaError_t launch_decode_int4(const Int4DecodeParams& p, cudaStream_t stream);

struct PromptParams {
  ScoreParams s;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *cu_q, *cu_k, *prefix;
  uint16_t* out;
  float* lse;
  int32_t* dev_status;
  void* workspace;
  int32_t batch, n_q, n_kv, d, max_q, max_k, causal;
  int64_t total_q, total_k;
};
size_t prompt_workspace_bytes(const PromptParams& p);
cudaError_t launch_prompt(const PromptParams& p, cudaStream_t stream);

}  // namespace oscar
