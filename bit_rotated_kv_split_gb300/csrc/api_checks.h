// Host checks that the entry points of the 4-bit and 8-bit layers, the
// rotations and the prompt attention share.
#pragma once

#include <cmath>
#include <cstdint>

#include "int4.h"
#include "oscar.h"

namespace oscar {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline oscar_status check_heads(int32_t batch, int32_t n_q, int32_t n_kv, int32_t d) {
  if (batch < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv || (d != 64 && d != 128)) return OSCAR_ERR_INVALID_ARG;
  // grid dimensions
  return batch > 65535 || n_q > 65535 ? OSCAR_ERR_UNSUPPORTED : OSCAR_OK;
}

// The pages of a 4-bit or 8-bit layer's descriptor; groups_ok: its quantisation groups are valid.
template <class Desc>
oscar_status check_pages(const Desc* d, bool groups_ok, PagedCache* c) {
  if (!d) return OSCAR_ERR_INVALID_ARG;
  const oscar_status st = check_heads(d->batch, d->n_q_heads, d->n_kv_heads, d->head_dim);
  if (st != OSCAR_OK) return st;
  if (d->max_pages_per_seq < 1 || d->n_pages < 1 || d->n_pages > INT32_MAX) return OSCAR_ERR_INVALID_ARG;
  if (d->max_len < 0 || int64_t(d->max_len) > int64_t(d->max_pages_per_seq) * kPageTokens) return OSCAR_ERR_INVALID_ARG;
  if (!(d->tau_k > 0.f) || !(d->tau_v > 0.f) || !(d->tau_k <= 65504.f) || !(d->tau_v <= 65504.f))
    return OSCAR_ERR_INVALID_ARG;
  if (!groups_ok || !d->pages || !d->page_table) return OSCAR_ERR_INVALID_ARG;
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
  return OSCAR_OK;
}

inline oscar_status check_rope(const oscar_rope_desc* rope, int32_t head_dim, RopeParams* p) {
  if (!rope) return OSCAR_OK;
  if (rope->rot_dim < 0 || rope->rot_dim > head_dim || rope->rot_dim % 16 ||
      (rope->interleaved != 0 && rope->interleaved != 1))
    return OSCAR_ERR_INVALID_ARG;
  if (rope->rot_dim > 0) {
    if (!rope->cos_sin || rope->n_positions < 1) return OSCAR_ERR_INVALID_ARG;
    if (!aligned(rope->cos_sin, 16)) return OSCAR_ERR_ALIGNMENT;
  }
  p->cos_sin = rope->cos_sin;
  p->n_positions = rope->n_positions;
  p->rot = rope->rot_dim;
  p->interleaved = rope->interleaved;
  return OSCAR_OK;
}

inline oscar_status check_score(const oscar_score_desc* d, int32_t head_dim, ScoreParams* s) {
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
inline bool row_stride_ok(int64_t stride, int64_t heads, int32_t d) { return stride >= heads * d && stride % 8 == 0; }

inline oscar_status done(cudaError_t e) {
  return e == cudaSuccess ? OSCAR_OK : e == cudaErrorNotSupported ? OSCAR_ERR_UNSUPPORTED : OSCAR_ERR_CUDA;
}

}  // namespace oscar
