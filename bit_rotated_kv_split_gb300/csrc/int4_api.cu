// C-ABI entry points of the 4-bit layers and of prompt attention: host
// validation, then the launch.  A rejected call launches nothing.
#include <cstdint>

#include "api_checks.h"
#include "int4.h"
#include "kernels.h"
#include "oscar.h"
#include "trace.h"

using oscar::aligned;
using oscar::check_heads;
using oscar::check_score;
using oscar::done;
using oscar::row_stride_ok;

namespace {

// groups per vector of d channels for a quantisation group size (0 = d); 0 if invalid
int groups(int32_t d, int32_t g) {
  if (d != 64 && d != 128) return 0;
  if (g == 0) g = d;
  return (g == 32 || g == 64 || g == 128) && g <= d ? d / g : 0;
}

oscar_status check_cache(const oscar_int4_desc* d, oscar::Int4Cache* c) {
  c->ng_k = d ? groups(d->head_dim, d->quant_group_k) : 0;
  c->ng_v = d ? groups(d->head_dim, d->quant_group_v) : 0;
  return oscar::check_pages(d, c->ng_k && c->ng_v, c);
}

}  // namespace

extern "C" int64_t oscar_int4_block_bytes(int32_t head_dim, int32_t quant_group_k, int32_t quant_group_v) {
  const int gk = groups(head_dim, quant_group_k), gv = groups(head_dim, quant_group_v);
  return gk && gv ? int64_t(oscar::int4_block_bytes(head_dim, gk, gv)) : 0;
}

extern "C" oscar_status oscar_rope_append_int4(const oscar_int4_desc* desc, const oscar_rope_desc* rope,
                                               const uint16_t* q, int64_t q_stride, const uint16_t* k,
                                               int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                               const int32_t* dst_req, const int32_t* dst_pos,
                                               const int32_t* rope_pos, int32_t n, uint16_t* q_out, uint16_t* k_out,
                                               void* stream) {
  OSCAR_TRACE_CALL();
  oscar::AppendParams p{};
  const oscar_status st = check_cache(desc, &p.c);
  if (st != OSCAR_OK) return st;
  const oscar_status rs = oscar::check_rope(rope, desc->head_dim, &p.rope);
  if (rs != OSCAR_OK) return rs;
  if (n < 0) return OSCAR_ERR_INVALID_ARG;
  if (n == 0) return OSCAR_OK;
  if (!k || !v || !dst_req || !dst_pos || (q == nullptr) != (q_out == nullptr)) return OSCAR_ERR_INVALID_ARG;
  if ((q && !row_stride_ok(q_stride, desc->n_q_heads, desc->head_dim)) ||
      !row_stride_ok(k_stride, desc->n_kv_heads, desc->head_dim) ||
      !row_stride_ok(v_stride, desc->n_kv_heads, desc->head_dim))
    return OSCAR_ERR_INVALID_ARG;
  // written in place only where the rows are the output's
  if ((q && q == q_out && q_stride != int64_t(desc->n_q_heads) * desc->head_dim) ||
      (k == k_out && k_stride != int64_t(desc->n_kv_heads) * desc->head_dim))
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
      !aligned(dst_req, 4) || !aligned(dst_pos, 4) || !aligned(rope_pos, 4))
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
  p.tau_k = desc->tau_k;
  p.tau_v = desc->tau_v;
  return done(oscar::launch_rope_append_int4(p, static_cast<cudaStream_t>(stream)));
}

extern "C" oscar_status oscar_gather_int4(const oscar_int4_desc* desc, const int32_t* src_req, const int32_t* src_pos,
                                          int32_t n, uint16_t* k_out, int64_t k_stride, uint16_t* v_out,
                                          int64_t v_stride, void* stream) {
  OSCAR_TRACE_CALL();
  oscar::GatherParams p{};
  const oscar_status st = check_cache(desc, &p.c);
  if (st != OSCAR_OK) return st;
  if (n < 0) return OSCAR_ERR_INVALID_ARG;
  if (n == 0) return OSCAR_OK;
  if (!src_req || !src_pos || !k_out || !v_out) return OSCAR_ERR_INVALID_ARG;
  if (!row_stride_ok(k_stride, desc->n_kv_heads, desc->head_dim) ||
      !row_stride_ok(v_stride, desc->n_kv_heads, desc->head_dim))
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(src_req, 4) || !aligned(src_pos, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return OSCAR_ERR_ALIGNMENT;
  p.src_req = src_req;
  p.src_pos = src_pos;
  p.n = n;
  p.k_out = k_out;
  p.v_out = v_out;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  return done(oscar::launch_gather_int4(p, static_cast<cudaStream_t>(stream)));
}

extern "C" oscar_status oscar_decode_attention_int4(const oscar_int4_desc* desc, const oscar_score_desc* score,
                                                    const uint16_t* q, int64_t q_stride, uint16_t* out,
                                                    void* workspace, size_t* workspace_bytes, void* stream) {
  OSCAR_TRACE_CALL();
  oscar::Int4DecodeParams p{};
  oscar_status st = check_cache(desc, &p.c);
  if (st != OSCAR_OK) return st;
  if (!desc->seq_len || !workspace_bytes) return OSCAR_ERR_INVALID_ARG;
  if (desc->n_q_heads / desc->n_kv_heads > 16) return OSCAR_ERR_UNSUPPORTED;
  // positions up to a few pages past the end are 32-bit numbers
  if (desc->max_len >= INT32_MAX - 511) return OSCAR_ERR_UNSUPPORTED;
  st = check_score(score, desc->head_dim, &p.s);
  if (st != OSCAR_OK) return st;
  const size_t need = oscar::int4_decode_workspace_bytes(p.c);
  if (!workspace) {
    *workspace_bytes = need;
    return OSCAR_OK;
  }
  if (*workspace_bytes < need) return OSCAR_ERR_WORKSPACE;
  if (!q || !out || !row_stride_ok(q_stride, desc->n_q_heads, desc->head_dim)) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(q, 16) || !aligned(out, 16)) return OSCAR_ERR_ALIGNMENT;
  p.q = q;
  p.q_stride = q_stride;
  p.out = out;
  p.workspace = workspace;
  return done(oscar::launch_decode_int4(p, static_cast<cudaStream_t>(stream)));
}

extern "C" oscar_status oscar_prompt_attention(const oscar_prompt_desc* desc, const oscar_score_desc* score,
                                               const uint16_t* q, int64_t q_stride, const uint16_t* k,
                                               int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                               const int32_t* cu_q, const int32_t* cu_k, const int32_t* prefix_len,
                                               uint16_t* out, float* lse, void* workspace, size_t* workspace_bytes,
                                               void* stream) {
  OSCAR_TRACE_CALL();
  if (!desc || !workspace_bytes) return OSCAR_ERR_INVALID_ARG;
  oscar_status st = check_heads(desc->batch, desc->n_q_heads, desc->n_kv_heads, desc->head_dim);
  if (st != OSCAR_OK) return st;
  if (desc->max_q < 0 || desc->max_k < 0 || desc->total_q < 0 || desc->total_k < 0 || desc->total_q > INT32_MAX ||
      desc->total_k > INT32_MAX || (desc->causal != 0 && desc->causal != 1) || desc->reserved != 0)
    return OSCAR_ERR_INVALID_ARG;
  oscar::PromptParams p{};
  st = check_score(score, desc->head_dim, &p.s);
  if (st != OSCAR_OK) return st;
  p.batch = desc->batch;
  p.n_q = desc->n_q_heads;
  p.n_kv = desc->n_kv_heads;
  p.d = desc->head_dim;
  p.max_q = desc->max_q;
  p.max_k = desc->max_k;
  p.causal = desc->causal;
  p.total_q = desc->total_q;
  p.total_k = desc->total_k;
  p.dev_status = desc->dev_status;
  const size_t need = oscar::prompt_workspace_bytes(p);
  if (!workspace) {
    *workspace_bytes = need;
    return OSCAR_OK;
  }
  if (*workspace_bytes < need) return OSCAR_ERR_WORKSPACE;
  if (!cu_q || !cu_k) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(prefix_len, 4) ||
      !aligned(desc->dev_status, 4))
    return OSCAR_ERR_ALIGNMENT;
  if (desc->max_q == 0 || desc->total_q == 0) return OSCAR_OK;   // no query at all
  if (!q || !out || (desc->total_k > 0 && (!k || !v))) return OSCAR_ERR_INVALID_ARG;
  if (!row_stride_ok(q_stride, desc->n_q_heads, desc->head_dim) ||
      !row_stride_ok(k_stride, desc->n_kv_heads, desc->head_dim) ||
      !row_stride_ok(v_stride, desc->n_kv_heads, desc->head_dim))
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return OSCAR_ERR_ALIGNMENT;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.prefix = prefix_len;
  p.out = out;
  p.lse = lse;
  p.workspace = workspace;
  return done(oscar::launch_prompt(p, static_cast<cudaStream_t>(stream)));
}
