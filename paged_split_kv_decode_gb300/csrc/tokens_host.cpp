// Host side of a step with several new tokens a request: scaled rotary frequencies and
// the plan of the attention (which token rows and which pages belong to a request).
#include <algorithm>
#include <cmath>

#include "psd_internal.h"

using namespace psd;

namespace {
constexpr double kPi = 3.14159265358979323846;
double clamp01(double x) { return x < 0.0 ? 0.0 : (x > 1.0 ? 1.0 : x); }
}  // namespace

extern "C" psd_status psd_rope_frequencies(const psd_rope_scaling *a, double *inv_freq, double *magnitude) {
  clear_error();
  if (!a || !inv_freq || !magnitude) return fail(PSD_ERR_INVALID_ARG, "psd_rope_frequencies: NULL");
  const int r = a->rot_dim;
  if (r < 2 || r % 2 || r > 512)
    return fail(PSD_ERR_INVALID_ARG, "psd_rope_frequencies: rot_dim %d must be even, in [2, 512]", r);
  if (!(a->base > 1.0) || !std::isfinite(a->base))
    return fail(PSD_ERR_INVALID_ARG, "psd_rope_frequencies: base must be finite and > 1");
  if (a->kind < PSD_ROPE_PLAIN || a->kind > PSD_ROPE_BANDS)
    return fail(PSD_ERR_INVALID_ARG, "psd_rope_frequencies: kind %d", a->kind);
  if (a->kind != PSD_ROPE_PLAIN && (!(a->factor > 0.0) || !std::isfinite(a->factor)))
    return fail(PSD_ERR_INVALID_ARG, "psd_rope_frequencies: factor must be finite and > 0");
  const bool mix = a->kind == PSD_ROPE_YARN || a->kind == PSD_ROPE_BANDS;
  if (mix && (a->original_max_position < 1 || !(a->low > 0.0) || !(a->high > a->low) || !std::isfinite(a->high)))
    return fail(PSD_ERR_INVALID_ARG, "psd_rope_frequencies: need original_max_position > 0 and 0 < low < high");
  if (a->kind == PSD_ROPE_NTK && r == 2)
    return fail(PSD_ERR_INVALID_ARG, "psd_rope_frequencies: NTK scaling needs rot_dim > 2");
  const double base = a->kind == PSD_ROPE_NTK ? a->base * std::pow(a->factor, r / (r - 2.0)) : a->base;
  double lo = 0.0, span = 1.0;
  if (a->kind == PSD_ROPE_YARN) {
    auto dim = [&](double turns) {
      return r * std::log(a->original_max_position / (turns * 2.0 * kPi)) / (2.0 * std::log(a->base));
    };
    lo = std::max(std::floor(dim(a->high)), 0.0);
    span = std::max(std::min(std::ceil(dim(a->low)), r - 1.0) - lo, 0.001);
  }
  for (int i = 0; i < r / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / r);
    double keep = 1.0;  // share of the unscaled frequency
    if (a->kind == PSD_ROPE_LINEAR) keep = 0.0;
    if (a->kind == PSD_ROPE_YARN) keep = 1.0 - clamp01((i - lo) / span);
    if (a->kind == PSD_ROPE_BANDS)
      keep = clamp01((a->original_max_position * f / (2.0 * kPi) - a->low) / (a->high - a->low));
    const bool scaled = mix || a->kind == PSD_ROPE_LINEAR;
    inv_freq[i] = scaled ? f * keep + f / a->factor * (1.0 - keep) : f;
  }
  *magnitude = a->kind == PSD_ROPE_YARN && a->factor > 1.0 ? 0.1 * std::log(a->factor) + 1.0 : 1.0;
  return PSD_OK;
}

extern "C" psd_status psd_plan_multi_token(const psd_page_table *host, const int32_t *q_indptr,
                                           psd_multi_token_plan *plan) {
  clear_error();
  if (!plan || !q_indptr) return fail(PSD_ERR_INVALID_ARG, "psd_plan_multi_token: NULL");
  const psd_status st = validate_table(host, -1);
  if (st != PSD_OK) return st;
  const int32_t B = host->batch;
  if (B > plan->batch_capacity || (B > 0 && !plan->requests))
    return fail(PSD_ERR_INVALID_ARG, "psd_plan_multi_token: capacity %d < batch %d", plan->batch_capacity, B);
  if (q_indptr[0] != 0) return fail(PSD_ERR_INVALID_ARG, "psd_plan_multi_token: q_indptr[0] != 0");
  int32_t most = 0;
  for (int32_t b = 0; b < B; ++b) {
    const int64_t len =
        int64_t(host->page_indptr[b + 1] - host->page_indptr[b] - 1) * host->page_size + host->last_page_len[b];
    const int64_t n = int64_t(q_indptr[b + 1]) - q_indptr[b];
    if (n < 0 || n > len)
      return fail(PSD_ERR_INVALID_ARG, "psd_plan_multi_token: request %d has %lld new tokens of %lld", b, (long long)n,
                  (long long)len);
    if (len > kMaxKvLen) return fail(PSD_ERR_INVALID_ARG, "psd_plan_multi_token: request %d too long", b);
    plan->requests[b] = psd_token_request{q_indptr[b], int32_t(n), host->page_indptr[b], int32_t(len)};
    most = std::max(most, int32_t(n));
  }
  plan->batch = B;
  plan->page_size = host->page_size;
  plan->num_tokens = q_indptr[B];
  plan->max_new = most;
  return PSD_OK;
}
