// What the kernels that append tokens share: their parameters, the place of a token in the paged cache, the
// angles of its rotation (append_tokens.cu says how they are made), and the checks of their arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "context.h"
#include "device.cuh"
#include "kernels.h"

namespace psd {

constexpr int kMaxPairs = 256;  // rot_dim / 2

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *q_indptr, *kv_len, *positions, *page_indptr, *page_indices;
  void *k_pool, *v_pool;
  int32_t *fault;
  int64_t num_page_indices, num_pages;
  int T, B, Hq, Hkv, D, Dv, rot_col, rot, neox, page_size, fp8;
  float k_scale, v_scale, magnitude;
};
struct Turns {
  uint64_t f[kMaxPairs];  // turns per position, 64-bit fixed point
};

// Saturating round-to-nearest-even E4M3 code of v (NaN gives the NaN code).
__device__ __forceinline__ uint8_t e4m3_of(float v) {
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(v));
  return uint8_t(two & 0xFF);
}

// The request that owns token row t: the largest b with q_indptr[b] <= t, found by the
// warp 32 entries at a time (two rounds of loads for 1024 requests).
__device__ __forceinline__ int request_of(const int32_t *q_indptr, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool below = i < n && __ldg(q_indptr + lo + i) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, below));
    const int skip = c > 0 ? (c - 1) * step : 0;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}

struct Place {
  int pos;      // rotation position; negative: leave the token untouched
  int64_t slot; // pool row, or -1
};

// Every lane of a warp returns the same.  Faults are raised by the caller's thread 0.
__device__ __forceinline__ Place place_of(const AppendParams &p, int t, uint32_t &faults) {
  Place x{-1, -1};
  faults = 0;
  if (t >= __ldg(p.q_indptr + p.B)) return x;  // behind the last request
  const int b = request_of(p.q_indptr, p.B, t);
  const int end = __ldg(p.q_indptr + b + 1);
  const int at = __ldg(p.kv_len + b) - (end - t);  // index in the request
  const int first = __ldg(p.page_indptr + b), last = __ldg(p.page_indptr + b + 1);
  x.pos = p.positions ? __ldg(p.positions + t) : at;
  if (t < __ldg(p.q_indptr + b) || t >= end || x.pos < 0) {
    faults = PSD_FAULT_RANGE;
    x.pos = -1;
    return x;
  }
  const int64_t page = int64_t(first) + at / p.page_size;
  int id = -1;
  if (at >= 0 && first >= 0 && page < last && page < p.num_page_indices) id = __ldg(p.page_indices + page);
  if (id < 0 || int64_t(id) >= p.num_pages)
    faults = PSD_FAULT_PAGE_ID;
  else
    x.slot = int64_t(id) * p.page_size + at % p.page_size;
  return x;
}

// cos and sin (times the magnitude) of pos * F turns.
__device__ __forceinline__ float2 turn(uint64_t F, int pos, float magnitude) {
  const int64_t frac = int64_t(F * uint64_t(uint32_t(pos)));  // turns * 2^64, in [-1/2, 1/2)
  const float half_turns = __ll2float_rn(frac) * 0x1p-63f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}

inline AppendParams append_params(const psd_append_args *a) {
  AppendParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a->q);
  p.k = static_cast<const __nv_bfloat16 *>(a->k);
  p.v = static_cast<const __nv_bfloat16 *>(a->v);
  p.q_out = static_cast<__nv_bfloat16 *>(a->q_out);
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.q_indptr = a->q_indptr;
  p.kv_len = a->kv_len;
  p.positions = a->positions;
  p.page_indptr = a->page_indptr;
  p.page_indices = a->page_indices;
  p.k_pool = a->k_pool;
  p.v_pool = a->v_pool;
  p.fault = a->fault_dev;
  p.num_page_indices = a->num_page_indices;
  p.num_pages = a->num_pages;
  p.T = a->num_tokens;
  p.B = a->batch;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.D = a->D;
  p.Dv = a->Dv;
  p.rot_col = a->rot_col;
  p.rot = a->rot_dim;
  p.neox = a->neox;
  p.page_size = a->page_size;
  p.fp8 = a->kv_dtype == PSD_FP8_E4M3;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.magnitude = float(a->magnitude);
  return p;
}
inline Turns append_turns(const psd_append_args *a) {
  Turns turns = {};
  for (int i = 0; i < a->rot_dim / 2; ++i) {
    // the fraction of a turn a position adds, in [0, 1): 2^64 times it is an integer's
    // worth of 53 significant bits, exact in the conversion
    const double f = a->inv_freq[i] * (0.5 / 3.14159265358979323846);
    turns.f[i] = uint64_t(std::ldexp(f - std::floor(f), 64));
  }
  return turns;
}

// *none: the call has nothing to do.
inline psd_status check_append(const char *what, const psd_append_args *a, bool *none) {
  *none = false;
  if (a->num_tokens < 0 || a->batch < 0 || a->Hq < 0 || a->Hkv < 1 || a->D < 1 || a->Dv < 0)
    return fail(PSD_ERR_INVALID_ARG, "%s: bad sizes", what);
  *none = a->num_tokens == 0 || a->batch == 0;  // nothing is read or written
  if (*none) return PSD_OK;
  if (a->rot_dim < 2 || a->rot_dim % 2 || a->rot_dim > 2 * kMaxPairs || a->rot_col < 0 ||
      int64_t(a->rot_col) + a->rot_dim > a->D)
    return fail(PSD_ERR_INVALID_ARG, "%s: rotated columns [%d, %d + %d) of %d (rot_dim even, in [2, 512])", what,
                a->rot_col, a->rot_col, a->rot_dim, a->D);
  if ((a->Hq > 0) != (a->q != nullptr) || (a->Hq > 0) != (a->q_out != nullptr) ||
      (a->Dv > 0) != (a->v != nullptr) || (a->Dv > 0) != (a->v_pool != nullptr))
    return fail(PSD_ERR_INVALID_ARG, "%s: q / q_out / v / v_pool must be given exactly when their width > 0", what);
  if (!a->k || !a->k_pool || !a->inv_freq || !a->q_indptr || !a->kv_len || !a->page_indptr || !a->page_indices ||
      !a->fault_dev)
    return fail(PSD_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if (a->q_stride < int64_t(a->Hq) * a->D || a->k_stride < int64_t(a->Hkv) * a->D ||
      a->v_stride < int64_t(a->Hkv) * a->Dv)
    return fail(PSD_ERR_INVALID_ARG, "%s: a token stride is shorter than its token", what);
  if (a->q == a->q_out && a->Hq > 0 && a->q_stride != int64_t(a->Hq) * a->D)
    return fail(PSD_ERR_INVALID_ARG, "%s: q_out may be q only when q is contiguous", what);
  if (a->page_size < 1 || a->num_pages < 0 || a->num_page_indices < 0)
    return fail(PSD_ERR_INVALID_ARG, "%s: bad pool or table sizes", what);
  if (int64_t(a->Hkv) * a->D > 0x7fffffffLL / 2 || int64_t(a->Hq) * a->D > 0x7fffffffLL / 2 ||
      int64_t(a->Hkv) * a->Dv > 0x7fffffffLL / 2)
    return fail(PSD_ERR_INVALID_ARG, "%s: heads * dim too large", what);
  if (a->kv_dtype != PSD_BF16 && a->kv_dtype != PSD_FP8_E4M3)
    return fail(PSD_ERR_INVALID_ARG, "%s: kv_dtype %d", what, a->kv_dtype);
  if (a->kv_dtype == PSD_FP8_E4M3 &&
      !(std::isfinite(a->k_scale) && a->k_scale > 0.f && std::isfinite(a->v_scale) && a->v_scale > 0.f))
    return fail(PSD_ERR_INVALID_ARG, "%s: fp8 scales must be finite and > 0", what);
  if (!std::isfinite(float(a->magnitude)))
    return fail(PSD_ERR_INVALID_ARG, "%s: magnitude must be finite in f32", what);
  for (int i = 0; i < a->rot_dim / 2; ++i)
    if (!(a->inv_freq[i] >= 0.0) || !std::isfinite(a->inv_freq[i]))
      return fail(PSD_ERR_INVALID_ARG, "%s: inv_freq[%d] must be finite and >= 0", what, i);
  return PSD_OK;
}

}  // namespace psd
