// Attention of several new tokens a request over the paged cache (the contract is in
// include/psd.h): the entry point, and the CUDA-core kernel for the shapes that the
// tcgen05 kernel does not take.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "context.h"
#include "device.cuh"
#include "multi_token.h"

namespace psd {

namespace {

constexpr int kMaxDim = 256;
constexpr int kWarps = 4;

// Eight consecutive pool elements from element `at` on.
template <bool FP8>
__device__ __forceinline__ void load8(const void *pool, int64_t at, float (&x)[8]) {
  if constexpr (FP8) {
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(pool) + at));
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e4m3x2_to_float2((u[i >> 1] >> (16 * (i & 1))) & 0xffffu);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(pool) + at));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(u[i]);
      x[2 * i + 1] = bf16_hi(u[i]);
    }
  }
}

// One CTA per (new token, query head).  Warp w takes the keys 32 w .. 32 w + 31 of every
// 128: a lane scores one key, then the lanes share out V's columns, 8 each, key by key
// (a key with no weight, hidden ones among them, is not read).  The warps' states
// (m, l, O) join in shared memory.  Everything in f32.  It reads a KV head's cache once per query
// head and token, where the tensor-core kernel reads it once per 128 rows: it is here for
// head dims and page sizes that the latter does not take.
template <bool FP8>
__global__ void __launch_bounds__(kWarps * 32)
    step_general_kernel(const StepParams p, const __grid_constant__ StepRequests req) {
  __shared__ __align__(16) float qs[kMaxDim];
  __shared__ float part[kWarps][kMaxDim], ms[kWarps], ls[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = req.r[0].token0 + blockIdx.x, h = blockIdx.y;
  int b = 0;
  for (int n = p.B; n > 1;) {  // the last request with token0 <= t
    const int mid = n / 2;
    if (req.r[b + mid].token0 <= t) b += mid, n -= mid;
    else n = mid;
  }
  const psd_token_request r = req.r[b];
  const int i = t - r.token0, start = r.kv_len - r.num_new, D = p.D;
  const uint64_t tree = p.tree ? p.tree[t] & (r.num_new < 64 ? (uint64_t(1) << r.num_new) - 1 : ~uint64_t(0)) : 0;
  const int n_keys = p.tree ? r.kv_len : start + i + 1;
  for (int d = threadIdx.x; d < D; d += blockDim.x)
    qs[d] = __bfloat162float(p.q[t * p.q_stride + int64_t(h) * D + d]) * p.q_scale;
  __syncthreads();
  const int kv = h / p.G;
  float o[8] = {}, m = neg_inf(), l = 0.f;
  for (int j0 = 32 * warp; j0 < n_keys; j0 += 32 * kWarps) {
    const int j = j0 + lane;
    bool seen = j < n_keys;
    if (p.tree && seen && j >= start) seen = (tree >> (j - start)) & 1;
    int64_t row = 0;
    if (j < n_keys) {
      const int id = __ldg(p.page_indices + r.page_off + j / p.page_size);
      if (id < 0 || int64_t(id) >= p.num_pages) {
        raise_fault(p.fault, PSD_FAULT_PAGE_ID);
        seen = false;
      } else {
        row = (int64_t(id) * p.page_size + j % p.page_size) * p.Hkv + kv;
      }
    }
    float s = neg_inf();
    if (seen) {
      float acc = 0.f;
      for (int d = 0; d < D; d += 8) {
        float x[8];
        load8<FP8>(p.k_pool, row * D + d, x);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc = fmaf(qs[d + c], x[c], acc);
      }
      s = acc;
    }
    float top = s;
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float m_new = fmaxf(m, top);
    const float base = m_new == neg_inf() ? 0.f : m_new;
    const float alpha = ex2(m - base);
    const float w = ex2(s - base);
    float sum = w;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * alpha + sum;
    m = m_new;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] *= alpha;
    const uint32_t weighed = __ballot_sync(0xffffffffu, seen);
    for (int k = 0; k < 32; ++k) {
      if (!(weighed >> k & 1)) continue;
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const int64_t rk = __shfl_sync(0xffffffffu, row, k);
      if (8 * lane < D) {
        float x[8];
        load8<FP8>(p.v_pool, rk * D + 8 * lane, x);
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = fmaf(wk, x[c], o[c]);
      }
    }
  }
  if (8 * lane < D)
#pragma unroll
    for (int c = 0; c < 8; ++c) part[warp][8 * lane + c] = o[c];
  if (lane == 0) ms[warp] = m, ls[warp] = l;
  __syncthreads();
  float top = ms[0];
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, ms[w]);
  const float base = top == neg_inf() ? 0.f : top;
  float scale[kWarps], sum = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    scale[w] = ex2(ms[w] - base);
    sum += ls[w] * scale[w];
  }
  const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
  const int64_t out = int64_t(t) * p.Hq + h;
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x = fmaf(part[w][d], scale[w], x);
    x *= inv;
    if (p.out_f32) static_cast<float *>(p.o)[out * D + d] = x;
    else static_cast<__nv_bfloat16 *>(p.o)[out * D + d] = __float2bfloat16_rn(x);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[out] = sum == 0.f ? neg_inf() : top + log2f(sum);
}

}  // namespace

psd_status launch_step_general(const StepParams &p, const StepRequests &req, const DeviceInfo &, cudaStream_t s) {
  const int64_t tokens = int64_t(req.r[p.B - 1].token0) + req.r[p.B - 1].num_new - req.r[0].token0;
  const dim3 grid(unsigned(tokens), unsigned(p.Hq));
  if (p.fp8) step_general_kernel<true><<<grid, kWarps * 32, 0, s>>>(p, req);
  else step_general_kernel<false><<<grid, kWarps * 32, 0, s>>>(p, req);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "multi_token_decode launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}

}  // namespace psd

using namespace psd;

extern "C" size_t psd_multi_token_workspace_bytes(const psd_ctx *ctx, int32_t D) {
  if (!ctx || D < 1) return 0;
  // the fault word, then the partial rows of the tensor-core kernel's CTAs, one per SM
  return 256 + (D == 64 || D == 128 ? 4 * step_tc_place(ctx->dev.num_sms, D, nullptr).floats : 0);
}

extern "C" psd_status multi_token_decode(psd_ctx *ctx, const psd_multi_token_args *a, const psd_multi_token_plan *plan,
                                         void *o, float *lse, void *workspace, size_t workspace_bytes,
                                         psd_stream_t stream) {
  clear_error();
  if (!ctx || !a || !plan || !workspace) return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: NULL");
  if (plan->batch < 0 || plan->num_tokens < 0 || a->num_tokens < plan->num_tokens)
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: %d token rows, the plan has %d", a->num_tokens,
                plan->num_tokens);
  if (a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv)
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: need Hq %% Hkv == 0 (Hq %d, Hkv %d)", a->Hq, a->Hkv);
  if (a->D < 8 || a->D % 8) return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: D %d must be a positive multiple of 8", a->D);
  if (a->D > kMaxDim) return fail(PSD_ERR_UNSUPPORTED, "multi_token_decode: head dim %d > %d", a->D, kMaxDim);
  if (a->Hq > 65535) return fail(PSD_ERR_UNSUPPORTED, "multi_token_decode: Hq %d", a->Hq);
  if (a->page_size < 1 || a->page_size != plan->page_size || a->num_pages < 1 || a->num_pages > 0x7fffffffLL ||
      a->num_page_indices < 0)
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: page_size %d (plan %d) / num_pages / num_page_indices",
                a->page_size, plan->page_size);
  if (a->kv_dtype != PSD_BF16 && a->kv_dtype != PSD_FP8_E4M3)
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: kv_dtype %d", a->kv_dtype);
  const bool fp8 = a->kv_dtype == PSD_FP8_E4M3;
  if (!std::isfinite(a->sm_scale) || (fp8 && (!std::isfinite(a->k_scale) || !std::isfinite(a->v_scale))))
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: scales must be finite");
  if (a->q_stride < int64_t(a->Hq) * a->D || a->q_stride % 8)
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: q_stride must be a multiple of 8 and >= Hq * D");
  if (a->tree_mask && plan->max_new > 64)
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: a tree mask holds 64 new tokens a request, the plan has %d",
                plan->max_new);
  if (plan->batch == 0 || plan->num_tokens == 0) return PSD_OK;
  if (!plan->requests || !a->q || !a->k_pool || !a->v_pool || !a->page_indices_dev || !o)
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: NULL pointer");
  if (!aligned16(a->q) || !aligned16(a->k_pool) || !aligned16(a->v_pool) || !aligned16(o) || !aligned16(workspace))
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: q / pools / o / workspace must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(a->tree_mask) & 7u) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: tree_mask / lse alignment");
  const size_t need = psd_multi_token_workspace_bytes(ctx, a->D);
  if (workspace_bytes < need)
    return fail(PSD_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", workspace_bytes, need);
  int64_t row = 0;
  for (int32_t b = 0; b < plan->batch; ++b) {
    const psd_token_request &r = plan->requests[b];
    if (r.token0 != row || r.num_new < 0 || r.kv_len < 1 || r.num_new > r.kv_len || r.page_off < 0 ||
        (a->tree_mask && r.num_new > 64) ||
        int64_t(r.page_off) + (int64_t(r.kv_len) + a->page_size - 1) / a->page_size > a->num_page_indices)
      return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: request %d of the plan", b);
    row += r.num_new;
  }
  if (row != plan->num_tokens) return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: the plan's token rows");

  DeviceGuard g(ctx->dev.device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  StepParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a->q);
  p.k_pool = a->k_pool;
  p.v_pool = a->v_pool;
  p.page_indices = a->page_indices_dev;
  p.tree = a->tree_mask;
  p.o = o;
  p.lse = lse;
  p.fault = next_fault(ctx, workspace);
  p.q_stride = a->q_stride;
  p.num_pages = a->num_pages;
  p.num_tokens = a->num_tokens;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.G = a->Hq / a->Hkv;
  p.D = a->D;
  p.page_size = a->page_size;
  p.fp8 = fp8;
  p.out_f32 = a->out_f32 != 0;
  p.q_scale = a->sm_scale * 1.4426950408889634f * (fp8 ? a->k_scale : 1.f);
  p.v_scale = fp8 ? a->v_scale : 1.f;
  const StepPlace place =
      step_tc_place(ctx->dev.num_sms, a->D, reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + 256));
  StepRequests req;
  const bool tensor = step_tc_supports(p);
  for (int32_t b0 = 0; b0 < plan->batch;) {
    // up to kStepRequests requests that have new tokens
    p.B = 0;
    for (; b0 < plan->batch && p.B < kStepRequests; ++b0)  // (the others' rows are none)
      if (plan->requests[b0].num_new > 0) req.r[p.B++] = plan->requests[b0];
    if (p.B == 0) break;
    const psd_status st =
        tensor ? launch_step_tc(p, req, place, ctx->dev, s) : launch_step_general(p, req, ctx->dev, s);
    if (st != PSD_OK) return st;
  }
  return PSD_OK;
}
