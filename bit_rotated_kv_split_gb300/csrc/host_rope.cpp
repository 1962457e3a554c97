// Frequencies of rotary positions, plain or scaled for contexts longer than
// the trained one (host, float64).
#include <cmath>
#include <cstdint>

#include "oscar.h"
#include "trace.h"

namespace {

constexpr double kPi = 3.14159265358979323846;

double clamp01(double x) { return x < 0. ? 0. : x > 1. ? 1. : x; }

}  // namespace

extern "C" oscar_status oscar_rope_frequencies(int32_t rot_dim, double theta, const oscar_rope_scaling* scaling,
                                               double* freq_out, double* magnitude_out) {
  OSCAR_TRACE_CALL();
  if (rot_dim < 16 || rot_dim > OSCAR_HEAD_DIM || rot_dim % 16 || !(theta > 1.) || !std::isfinite(theta) || !freq_out)
    return OSCAR_ERR_INVALID_ARG;
  oscar_rope_scaling s{};
  if (scaling) s = *scaling;
  if (s.kind < OSCAR_ROPE_PLAIN || s.kind > OSCAR_ROPE_BY_TURNS || s.reserved != 0) return OSCAR_ERR_INVALID_ARG;
  if (s.kind != OSCAR_ROPE_PLAIN && (!(s.factor >= 1.) || !std::isfinite(s.factor))) return OSCAR_ERR_INVALID_ARG;
  const bool parts = s.kind == OSCAR_ROPE_BY_INDEX || s.kind == OSCAR_ROPE_BY_TURNS;
  if (parts) {
    if (s.turns_low == 0. && s.turns_high == 0.) s.turns_low = 1., s.turns_high = s.kind == OSCAR_ROPE_BY_INDEX ? 32. : 4.;
    if (!(s.original_len >= 1.) || !std::isfinite(s.original_len) || !(s.turns_low > 0.) || !(s.turns_high > s.turns_low) ||
        !std::isfinite(s.turns_high))
      return OSCAR_ERR_INVALID_ARG;
  }
  const int pairs = rot_dim / 2;
  if (s.kind == OSCAR_ROPE_BASE) {
    theta *= std::pow(s.factor, double(rot_dim) / (rot_dim - 2));
    if (!std::isfinite(theta)) return OSCAR_ERR_INVALID_ARG;
  }
  double lo = 0., hi = 0.;
  if (s.kind == OSCAR_ROPE_BY_INDEX) {
    // the index of the pair that makes r turns over the trained context
    const auto at = [&](double r) { return rot_dim * std::log(s.original_len / (r * 2. * kPi)) / (2. * std::log(theta)); };
    lo = std::fmax(std::floor(at(s.turns_high)), 0.);
    hi = std::fmin(std::ceil(at(s.turns_low)), rot_dim - 1.);
  }
  for (int i = 0; i < pairs; ++i) {
    const double w = std::pow(theta, -2. * i / rot_dim);
    double keep = 1.;                       // of the plain frequency; the rest is slowed by the factor
    if (s.kind == OSCAR_ROPE_LINEAR) keep = 0.;
    if (s.kind == OSCAR_ROPE_BY_INDEX) keep = 1. - clamp01((i - lo) / std::fmax(hi - lo, 1e-3));
    if (s.kind == OSCAR_ROPE_BY_TURNS)
      keep = clamp01((s.original_len * w / (2. * kPi) - s.turns_low) / (s.turns_high - s.turns_low));
    freq_out[i] = s.kind == OSCAR_ROPE_PLAIN || s.kind == OSCAR_ROPE_BASE ? w : w * keep + w / s.factor * (1. - keep);
  }
  if (magnitude_out) *magnitude_out = s.kind == OSCAR_ROPE_BY_INDEX ? 0.1 * std::log(s.factor) + 1. : 1.;
  return OSCAR_OK;
}
