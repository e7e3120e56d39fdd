// Verification of drafted tokens (the contract is in include/psd.h).
//
// Mathematics.  With draft d drawn from q, accepting with probability min(1, p(d)/q(d))
// and drawing from max(p - q, 0) after a refusal leaves the outcome distributed as p.
// Acceptance compares u q(d) < p(d): the product of two f32 numbers is exact in 64 bits.
// The draw wants the least v with C_v > u C: a border decided by sums of up to 2^17
// numbers, so the sums are taken exactly, in 64-bit fixed point with 58 fraction bits
// (a probability below 2^-34 loses bits under 2^-58, at most 2^-41 in all over 2^17
// entries; the sums stay below 2^63 up to a row total of 16).  Integer sums
// do not depend on their order, so the split over threads cannot change a token.
#include <cuda_runtime.h>

#include "context.h"
#include "device.cuh"
#include "kernels.h"

namespace psd {

namespace {

struct VerifyParams {
  const float *target, *draft;
  int64_t target_stride, draft_stride;
  const int32_t *tokens, *indptr;
  const float *uniforms;
  int32_t *accepted, *out;
  int32_t *fault;
  int B, num_drafts, V;
};

// A probability in 58-bit fixed point, cut: 0 for NaN and what is not positive, 2^58 from 1 on.
__device__ __forceinline__ uint64_t fix58(float x) {
  if (!(x > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(fminf(x, 1.f));
  const int e = int(bits >> 23);                                   // 2^(e - 127)
  const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);    // 24 bits
  const int sh = (e ? e : 1) - 127 - 23 + 58;                      // <= 35
  return sh >= 0 ? m << sh : (sh > -24 ? m >> -sh : 0);
}
__device__ __forceinline__ uint64_t weight(float p, float q) {
  const uint64_t a = fix58(p), b = fix58(q);
  return a > b ? a - b : 0;
}
// floor(u * total): the least v with C_v > u * total is the least with C_v > this.
__device__ __forceinline__ uint64_t share_of(float u, uint64_t total) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return total;
  const uint32_t bits = __float_as_uint(u);
  const int e = int(bits >> 23);
  const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int sh = 150 - (e ? e : 1);  // u = m 2^-sh, sh in [24, 149]
  const uint64_t hi = __umul64hi(m, total), lo = m * total;
  if (sh < 64) return (hi << (64 - sh)) | (lo >> sh);
  return sh < 128 ? hi >> (sh - 64) : 0;
}

// Inclusive sum over the block's threads in thread order; `tmp` holds a sum per warp.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t *tmp, uint64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
  for (int w = 0; w < int(blockDim.x >> 5); ++w) {
    if (w < warp) before += tmp[w];
    total += tmp[w];
  }
  __syncthreads();
  return x + before;
}

// One CTA per request: the accepted drafts, then two passes over the chosen row.
__global__ void __launch_bounds__(1024) verify_drafts_kernel(const VerifyParams p) {
  __shared__ uint64_t tmp[32];
  __shared__ int first_refused, found;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int d0 = p.indptr[b], d1 = p.indptr[b + 1];
  if (d0 < 0 || d1 < d0 || d1 > p.num_drafts) {
    if (tid == 0) atomicOr(p.fault, PSD_FAULT_RANGE);
    return;
  }
  const int K = d1 - d0, R = d0 + b;
  if (tid == 0) first_refused = K, found = p.V;
  __syncthreads();
  for (int j = tid; j < K; j += blockDim.x) {
    const int d = p.tokens[d0 + j];
    const bool inside = d >= 0 && d < p.V;
    bool ok = false;
    if (inside) {
      const double q = p.draft ? double(p.draft[(d0 + j) * p.draft_stride + d]) : 1.0;
      ok = double(p.uniforms[R + j]) * q < double(p.target[(R + j) * p.target_stride + d]);
    }
    if (!ok) atomicMin(&first_refused, j);
  }
  __syncthreads();
  const int a = first_refused;
  const float *prow = p.target + (R + a) * p.target_stride;
  const float *qrow = nullptr;
  int hot = -1;  // the refused token of a draft without probabilities
  if (a < K) {
    const int d = p.tokens[d0 + a];
    if (d < 0 || d >= p.V) {
      if (tid == 0) atomicOr(p.fault, PSD_FAULT_RANGE);
    } else if (p.draft) {
      qrow = p.draft + (d0 + a) * p.draft_stride;
    } else {
      hot = d;
    }
  }
  uint64_t total = 0;
  for (int pass = 0; pass < 2 && total == 0; ++pass) {
    if (pass == 1) qrow = nullptr, hot = -1;  // p <= q everywhere: draw from p
    uint64_t sum = 0;
    for (int v = tid; v < p.V; v += blockDim.x)
      if (v != hot) sum += weight(prow[v], qrow ? qrow[v] : 0.f);
    block_scan(sum, tmp, total);
  }
  const uint64_t want = share_of(p.uniforms[R + K], total);
  uint64_t before = 0;
  for (int v0 = 0; v0 < p.V && total; v0 += blockDim.x) {
    const int v = v0 + tid;
    const uint64_t w = v < p.V && v != hot ? weight(prow[v], qrow ? qrow[v] : 0.f) : 0;
    uint64_t here;
    const uint64_t c = before + block_scan(w, tmp, here);
    // u >= 1 (outside the contract): the last entry with a weight
    if (w && (c > want || (want >= total && c == total))) atomicMin(&found, v);
    before += here;
    if (before > want || before == total) break;
  }
  __syncthreads();
  for (int j = tid; j <= K; j += blockDim.x)
    p.out[R + j] = j < a ? p.tokens[d0 + j] : (j == a && total ? found : -1);
  if (tid == 0) {
    p.accepted[b] = a;
    if (!total) atomicOr(p.fault, PSD_FAULT_RANGE);
  }
}

}  // namespace
}  // namespace psd

using namespace psd;

extern "C" psd_status verify_drafts(psd_ctx *ctx, const psd_verify_args *a, psd_stream_t stream) {
  clear_error();
  if (!ctx || !a) return fail(PSD_ERR_INVALID_ARG, "verify_drafts: NULL");
  if (a->batch < 0 || a->num_drafts < 0 || a->vocab < 1 || (a->batch == 0 && a->num_drafts > 0))
    return fail(PSD_ERR_INVALID_ARG, "verify_drafts: batch %d, num_drafts %d, vocab %d", a->batch, a->num_drafts,
                a->vocab);
  if (int64_t(a->batch) + a->num_drafts > 0x7fffffffLL) return fail(PSD_ERR_INVALID_ARG, "verify_drafts: too many rows");
  if (a->batch == 0) return PSD_OK;
  if (!a->target_probs || !a->draft_indptr || !a->uniforms || !a->num_accepted || !a->out_tokens || !a->fault_dev ||
      (a->num_drafts > 0 && !a->draft_tokens))
    return fail(PSD_ERR_INVALID_ARG, "verify_drafts: NULL pointer");
  if (a->target_stride < a->vocab || (a->draft_probs && a->draft_stride < a->vocab))
    return fail(PSD_ERR_INVALID_ARG, "verify_drafts: a row stride is shorter than vocab");
  DeviceGuard g(ctx->dev.device);
  VerifyParams p{a->target_probs, a->draft_probs, a->target_stride, a->draft_stride, a->draft_tokens, a->draft_indptr,
                 a->uniforms, a->num_accepted, a->out_tokens, a->fault_dev, a->batch, a->num_drafts, a->vocab};
  verify_drafts_kernel<<<a->batch, 1024, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "verify_drafts launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}
