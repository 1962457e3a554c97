// C-ABI entry points of the 8-bit layers and of the rotations: host
// validation, then the launch.  A rejected call launches nothing.
#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "int8.h"
#include "kernels.h"
#include "oscar.h"
#include "trace.h"

using oscar::aligned;
using oscar::done;
using oscar::row_stride_ok;

namespace {

oscar_status check_norm(const oscar_head_norm* norm, oscar::HeadRowsParams* p) {
  if (!norm) return OSCAR_OK;
  if (!(norm->eps >= 0.f) || !std::isfinite(norm->eps) || norm->reserved != 0) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(norm->q_weight, 16) || !aligned(norm->k_weight, 16)) return OSCAR_ERR_ALIGNMENT;
  p->q_weight = norm->q_weight;
  p->k_weight = norm->k_weight;
  p->eps = norm->eps;
  return OSCAR_OK;
}

// written in place only where a row is its own output
bool in_place_ok(const uint16_t* x, int64_t stride, const uint16_t* out, int64_t out_stride) {
  return x != out || stride == out_stride;
}

// The fraction of a turn that a position adds at w radians, to the nearest 2^-64: w / 2 pi
// as a double and its rest, which together are good to about 2^-104 of it.
uint64_t turn_of(double w) {
  const double inv = 0.15915494309189535, rest = -9.839338337591243e-18;   // 1 / 2 pi
  const double t = w * inv, e = std::fma(w, inv, -t) + w * rest;
  // t < 1 (w <= 6): times 2^64 it fits, and splits exactly; |e| 2^64 is below 2^11
  const double whole = std::floor(t * 0x1p64);
  return uint64_t(whole) + uint64_t(std::llrint((t * 0x1p64 - whole) + e * 0x1p64));
}

}  // namespace

extern "C" oscar_status oscar_rope_table(const double* freq, int32_t rot_dim, double magnitude, int64_t first,
                                         int64_t n, float* cos_sin, void* stream) {
  OSCAR_TRACE_CALL();
  if (rot_dim < 16 || rot_dim > 2 * oscar::kMaxRopePairs || rot_dim % 16 || !freq || first < 0 || n < 0 ||
      first > (int64_t(1) << 40) || n > (int64_t(1) << 40) || !std::isfinite(float(magnitude)))
    return OSCAR_ERR_INVALID_ARG;
  oscar::RopeTableParams p{};
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!(freq[i] >= 0.) || !(freq[i] <= 6.)) return OSCAR_ERR_INVALID_ARG;
    p.turn[i] = turn_of(freq[i]);
  }
  if (n == 0) return OSCAR_OK;
  if (!cos_sin) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(cos_sin, 16)) return OSCAR_ERR_ALIGNMENT;
  p.pairs = rot_dim / 2;
  p.first = first;
  p.n = n;
  p.magnitude = float(magnitude);
  p.cos_sin = cos_sin;
  return done(oscar::launch_rope_table(p, static_cast<cudaStream_t>(stream)));
}

extern "C" oscar_status oscar_norm_rope(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                        const oscar_head_norm* norm, const oscar_rope_desc* rope, const uint16_t* q,
                                        int64_t q_stride, const uint16_t* k, int64_t k_stride, const int32_t* pos,
                                        int32_t n, uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out,
                                        int64_t k_out_stride, int32_t* dev_status, void* stream) {
  OSCAR_TRACE_CALL();
  if (n_q_heads < 1 || n_kv_heads < 1 || n_q_heads > 65535 || n_kv_heads > 65535 || (head_dim != 64 && head_dim != 128))
    return OSCAR_ERR_INVALID_ARG;
  oscar::HeadRowsParams p{};
  oscar_status st = check_norm(norm, &p);
  if (st != OSCAR_OK) return st;
  st = oscar::check_rope(rope, head_dim, &p.rope);
  if (st != OSCAR_OK) return st;
  if (n < 0) return OSCAR_ERR_INVALID_ARG;
  if (n == 0) return OSCAR_OK;
  if ((!q && !k) || (q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (p.rope.rot && !pos))
    return OSCAR_ERR_INVALID_ARG;
  if ((q && (!row_stride_ok(q_stride, n_q_heads, head_dim) || !row_stride_ok(q_out_stride, n_q_heads, head_dim))) ||
      (k && (!row_stride_ok(k_stride, n_kv_heads, head_dim) || !row_stride_ok(k_out_stride, n_kv_heads, head_dim))))
    return OSCAR_ERR_INVALID_ARG;
  if ((q && !in_place_ok(q, q_stride, q_out, q_out_stride)) || (k && !in_place_ok(k, k_stride, k_out, k_out_stride)) ||
      (q && k && (q_out == k || k_out == q || q_out == k_out)))
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(pos, 4) ||
      !aligned(dev_status, 4))
    return OSCAR_ERR_ALIGNMENT;
  p.c.n_q = n_q_heads;
  p.c.n_kv = n_kv_heads;
  p.c.d = head_dim;
  p.c.dev_status = dev_status;
  p.q = q;
  p.k = k;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.rope_pos = pos;
  p.n = n;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  return done(oscar::launch_norm_rope(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int64_t oscar_int8_block_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? oscar::int8_block_bytes(head_dim) : 0;
}

extern "C" oscar_status oscar_rope_append_int8(const oscar_int8_desc* desc, const oscar_head_norm* norm,
                                               const oscar_rope_desc* rope, const uint16_t* q, int64_t q_stride,
                                               const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                               const int32_t* dst_req, const int32_t* dst_pos, const int32_t* rope_pos,
                                               int32_t n, uint16_t* q_out, uint16_t* k_out, uint16_t* k_held,
                                               uint16_t* v_held, void* stream) {
  OSCAR_TRACE_CALL();
  oscar::HeadRowsParams p{};
  oscar_status st = oscar::check_pages(desc, true, &p.c);
  if (st != OSCAR_OK) return st;
  st = check_norm(norm, &p);
  if (st != OSCAR_OK) return st;
  st = oscar::check_rope(rope, desc->head_dim, &p.rope);
  if (st != OSCAR_OK) return st;
  if (n < 0) return OSCAR_ERR_INVALID_ARG;
  if (n == 0) return OSCAR_OK;
  if (!k || !v || !dst_req || !dst_pos || (q == nullptr) != (q_out == nullptr)) return OSCAR_ERR_INVALID_ARG;
  const int64_t q_row = int64_t(desc->n_q_heads) * desc->head_dim, k_row = int64_t(desc->n_kv_heads) * desc->head_dim;
  if ((q && !row_stride_ok(q_stride, desc->n_q_heads, desc->head_dim)) ||
      !row_stride_ok(k_stride, desc->n_kv_heads, desc->head_dim) ||
      !row_stride_ok(v_stride, desc->n_kv_heads, desc->head_dim))
    return OSCAR_ERR_INVALID_ARG;
  if ((q && !in_place_ok(q, q_stride, q_out, q_row)) || !in_place_ok(k, k_stride, k_out, k_row) ||
      !in_place_ok(k, k_stride, k_held, k_row) || !in_place_ok(v, v_stride, v_held, k_row))
    return OSCAR_ERR_INVALID_ARG;
  // no other two rows in one place: a row would be written before it is read, or twice
  const uint16_t *rows_in[3] = {q, k, v}, *rows_out[4] = {q_out, k_out, k_held, v_held};
  const bool may_share[4][3] = {{true, false, false}, {false, true, false}, {false, true, false}, {false, false, true}};
  for (int o = 0; o < 4; ++o)
    for (int x = 0; rows_out[o] && x < 4; ++x)
      if ((x < 3 && rows_out[o] == rows_in[x] && !may_share[o][x]) || (x != o && rows_out[o] == rows_out[x]))
        return OSCAR_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
      !aligned(k_held, 16) || !aligned(v_held, 16) || !aligned(dst_req, 4) || !aligned(dst_pos, 4) || !aligned(rope_pos, 4))
    return OSCAR_ERR_ALIGNMENT;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.dst_req = dst_req;
  p.dst_pos = dst_pos;
  p.rope_pos = rope_pos;
  p.n = n;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_out_stride = q_row;
  p.k_out_stride = k_row;
  p.k_held = k_held;
  p.v_held = v_held;
  p.tau_k = desc->tau_k;
  p.tau_v = desc->tau_v;
  return done(oscar::launch_rope_append_int8(p, static_cast<cudaStream_t>(stream)));
}

extern "C" oscar_status oscar_gather_int8(const oscar_int8_desc* desc, const int32_t* src_req, const int32_t* src_pos,
                                          int32_t n, uint16_t* k_out, int64_t k_stride, uint16_t* v_out,
                                          int64_t v_stride, void* stream) {
  OSCAR_TRACE_CALL();
  oscar::Gather8Params p{};
  const oscar_status st = oscar::check_pages(desc, true, &p.c);
  if (st != OSCAR_OK) return st;
  if (n < 0) return OSCAR_ERR_INVALID_ARG;
  if (n == 0) return OSCAR_OK;
  if (!src_req || !src_pos || !k_out || !v_out) return OSCAR_ERR_INVALID_ARG;
  if (!row_stride_ok(k_stride, desc->n_kv_heads, desc->head_dim) ||
      !row_stride_ok(v_stride, desc->n_kv_heads, desc->head_dim))
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(src_req, 4) || !aligned(src_pos, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return OSCAR_ERR_ALIGNMENT;
  if (k_out == v_out) return OSCAR_ERR_INVALID_ARG;   // each row would be written twice
  p.src_req = src_req;
  p.src_pos = src_pos;
  p.n = n;
  p.k_out = k_out;
  p.v_out = v_out;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  return done(oscar::launch_gather_int8(p, static_cast<cudaStream_t>(stream)));
}

extern "C" oscar_status oscar_decode_attention_int8(const oscar_int8_desc* desc, const oscar_score_desc* score,
                                                    const uint16_t* q, int64_t q_stride, uint16_t* out, float* lse,
                                                    void* workspace, size_t* workspace_bytes, void* stream) {
  OSCAR_TRACE_CALL();
  oscar::Int8DecodeParams p{};
  oscar_status st = oscar::check_pages(desc, true, &p.c);
  if (st != OSCAR_OK) return st;
  if (!desc->seq_len || !workspace_bytes) return OSCAR_ERR_INVALID_ARG;
  if (desc->n_q_heads / desc->n_kv_heads > 16) return OSCAR_ERR_UNSUPPORTED;
  // positions up to a few pages past the end are 32-bit numbers
  if (desc->max_len >= INT32_MAX - 511) return OSCAR_ERR_UNSUPPORTED;
  st = oscar::check_score(score, desc->head_dim, &p.s);
  if (st != OSCAR_OK) return st;
  const size_t need = oscar::int8_decode_workspace_bytes(p.c);
  if (!workspace) {
    *workspace_bytes = need;
    return OSCAR_OK;
  }
  if (*workspace_bytes < need) return OSCAR_ERR_WORKSPACE;
  if (!q || !out || !row_stride_ok(q_stride, desc->n_q_heads, desc->head_dim)) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return OSCAR_ERR_ALIGNMENT;
  p.q = q;
  p.q_stride = q_stride;
  p.out = out;
  p.lse = lse;
  p.workspace = workspace;
  return done(oscar::launch_decode_int8(p, static_cast<cudaStream_t>(stream)));
}
