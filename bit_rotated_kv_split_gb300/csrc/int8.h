// Internal interface between the C-ABI functions of the 8-bit layer and of
// the rotations (int8_api.cu) and their kernels (head_rows.cu, int8_decode.cu,
// rope_table.cu).
#pragma once

#include "int4.h"

namespace oscar {

// Page block of one (page, KV head), d channels (64 or 128):
//   [0, 16 d)     K: slot t's d code bytes at t d, their 16-byte chunk c at the
//                 place of chunk c ^ int8_swizzle(d, t);
//   [16 d, 32 d)  V the same way;
//   [32 d, ...)   slot t's K scale, K zero, V scale, V zero, fp16, at 32 d + 8 t.
// The places of the chunks are such that 8 slots' chunks of the same channels lie
// in different shared-memory banks (ldmatrix reads them at once).
__host__ __device__ constexpr int int8_block_bytes(int d) { return 32 * d + 128; }
__host__ __device__ constexpr int int8_swizzle(int d, int t) { return d == 128 ? t & 7 : (t >> 1) & 3; }
// byte of octet o (channels 8 o ..) of K slot t (V: 16 d further on)
__host__ __device__ constexpr int int8_octet(int d, int t, int o) {
  return t * d + 16 * ((o >> 1) ^ int8_swizzle(d, t)) + 8 * (o & 1);
}
__host__ __device__ constexpr int int8_pairs(int d, int t) { return 32 * d + 8 * t; }

// Rows of query and key heads: normed, rotated and, where `c.pages` is given,
// quantised with the value heads into an 8-bit layer's pages.
struct HeadRowsParams {
  PagedCache c;                  // n_q, n_kv, d and dev_status always
  RopeParams rope;
  const uint16_t *q_weight, *k_weight;
  float eps;
  const uint16_t *q, *k, *v;     // v only with pages
  int64_t q_stride, k_stride, v_stride;
  const int32_t *dst_req, *dst_pos, *rope_pos;   // without pages: rope_pos alone
  int32_t n;
  uint16_t *q_out, *k_out, *k_held, *v_held;
  int64_t q_out_stride, k_out_stride;
  float tau_k, tau_v;
};
cudaError_t launch_norm_rope(const HeadRowsParams& p, cudaStream_t stream);
cudaError_t launch_rope_append_int8(const HeadRowsParams& p, cudaStream_t stream);

struct Gather8Params {
  PagedCache c;
  const int32_t *src_req, *src_pos;
  int32_t n;
  uint16_t *k_out, *v_out;
  int64_t k_stride, v_stride;
};
cudaError_t launch_gather_int8(const Gather8Params& p, cudaStream_t stream);

struct Int8DecodeParams {
  PagedCache c;
  ScoreParams s;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  float* lse;
  void* workspace;
};
size_t int8_decode_workspace_bytes(const PagedCache& c);
cudaError_t launch_decode_int8(const Int8DecodeParams& p, cudaStream_t stream);

// Angles are kept as 64-bit fractions of a turn: a position times the turn of
// one position wraps by itself.
constexpr int kMaxRopePairs = 64;
struct RopeTableParams {
  uint64_t turn[kMaxRopePairs];
  int32_t pairs;
  int64_t first, n;
  float magnitude;
  float* cos_sin;
};
cudaError_t launch_rope_table(const RopeTableParams& p, cudaStream_t stream);

}  // namespace oscar
