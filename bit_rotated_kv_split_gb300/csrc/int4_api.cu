// C-ABI entry points of the 4-bit layers and of prompt attention: host
// validation, then the launch.  A rejected call launches nothing.
#include <cmath>
#include <cstdint>

#include "int4.h"
#include "kernels.h"
#include "oscar.h"
#include "trace.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// groups per vector of d channels for a quantisation group size (0 = d); 0 if invalid
int groups(int32_t d, int32_t g) {
  if (d != 64 && d != 128) return 0;
  if (g == 0) g = d;
  return (g == 32 || g == 64 || g == 128) && g <= d ? d / g : 0;
}

oscar_status check_heads(int32_t batch, int32_t n_q, int32_t n_kv, int32_t d) {
  if (batch < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv || (d != 64 && d != 128)) return OSCAR_ERR_INVALID_ARG;
  // grid dimensions
  return batch > 65535 || n_q > 65535 ? OSCAR_ERR_UNSUPPORTED : OSCAR_OK;
}

oscar_status check_cache(const oscar_int4_desc* d, oscar::Int4Cache* c) {
  if (!d) return OSCAR_ERR_INVALID_ARG;
  const oscar_status st = check_heads(d->batch, d->n_q_heads, d->n_kv_heads, d->head_dim);
  if (st != OSCAR_OK) return st;
  if (d->max_pages_per_seq < 1 || d->n_pages < 1 || d->n_pages > INT32_MAX) return OSCAR_ERR_INVALID_ARG;
  if (d->max_len < 0 || int64_t(d->max_len) > int64_t(d->max_pages_per_seq) * oscar::kInt4Page)
    return OSCAR_ERR_INVALID_ARG;
  if (!(d->tau_k > 0.f) || !(d->tau_v > 0.f) || !(d->tau_k <= 65504.f) || !(d->tau_v <= 65504.f))
    return OSCAR_ERR_INVALID_ARG;
  const int gk = groups(d->head_dim, d->quant_group_k), gv = groups(d->head_dim, d->quant_group_v);
  if (!gk || !gv || !d->pages || !d->page_table) return OSCAR_ERR_INVALID_ARG;
  if (!aligned(d->pages, 128) || !aligned(d->page_table, 4) || !aligned(d->seq_len, 4) || !aligned(d->dev_status, 4))
    return OSCAR_ERR_ALIGNMENT;
  c->pages = d->pages;
  c->page_table = d->page_table;
  c->seq_len = d->seq_len;
  c->dev_status = d->dev_status;
  c->batch = d->batch;
  c->n_q = d->n_q_heads;
  c->n_kv = d->n_kv_heads;
  c->d = d->head_dim;
  c->max_pages = d->max_pages_per_seq;
  c->max_len = d->max_len;
  c->n_pages = d->n_pages;
  c->ng_k = gk;
  c->ng_v = gv;
  return OSCAR_OK;
}

oscar_status check_score(const oscar_score_desc* d, int32_t head_dim, oscar::ScoreParams* s) {
  const oscar_score_desc none{};
  if (!d) d = &none;
  if (!(d->scale >= 0.f) || !std::isfinite(d->scale) || !(d->softcap >= 0.f) || !std::isfinite(d->softcap) ||
      d->window < 0 || d->reserved != 0)
    return OSCAR_ERR_INVALID_ARG;
  if (!aligned(d->slopes, 4)) return OSCAR_ERR_ALIGNMENT;
  const double log2e = 1.4426950408889634;
  const double scale = d->scale > 0.f ? double(d->scale) : 1.0 / std::sqrt(double(head_dim));
  s->scale_log2 = float(scale * log2e);
  s->cap_in = d->softcap > 0.f ? float(2.0 * scale / double(d->softcap) * log2e) : 0.f;
  s->cap_log2 = float(double(d->softcap) * log2e);
  // tanh(y) = y P(y^2) for |y| <= 1 / 2, and y = x cap_in ln 2 / 2
  const double tanh_near[5] = {1., -0x1.5554a6p-2, 0x1.10e47ap-3, -0x1.b2167ep-5, 0x1.18d7e8p-6};
  double unit = scale * log2e;
  for (int k = 0; k < 5; ++k, unit /= 4. * log2e * log2e) s->cap_near[k] = float(tanh_near[k] * unit);
  if (!std::isnormal(s->scale_log2) || !std::isfinite(s->cap_in) || !std::isfinite(2.f * s->cap_log2))
    return OSCAR_ERR_INVALID_ARG;
  s->window = d->window;
  s->slopes = d->slopes;
  return OSCAR_OK;
}

// rows of `heads` heads of d bf16, `stride` elements apart
bool row_stride_ok(int64_t stride, int64_t heads, int32_t d) { return stride >= heads * d && stride % 8 == 0; }

oscar_status done(cudaError_t e) {
  return e == cudaSuccess ? OSCAR_OK : e == cudaErrorNotSupported ? OSCAR_ERR_UNSUPPORTED : OSCAR_ERR_CUDA;
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
  if (rope) {
    if (rope->rot_dim < 0 || rope->rot_dim > desc->head_dim || rope->rot_dim % 16 ||
        (rope->interleaved != 0 && rope->interleaved != 1))
      return OSCAR_ERR_INVALID_ARG;
    if (rope->rot_dim > 0) {
      if (!rope->cos_sin || rope->n_positions < 1) return OSCAR_ERR_INVALID_ARG;
      if (!aligned(rope->cos_sin, 16)) return OSCAR_ERR_ALIGNMENT;
    }
    p.cos_sin = rope->cos_sin;
    p.n_positions = rope->n_positions;
    p.rot = rope->rot_dim;
    p.interleaved = rope->interleaved;
  }
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
