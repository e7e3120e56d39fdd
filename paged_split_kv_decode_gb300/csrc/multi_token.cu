// Attention of several new tokens a request over the paged cache (the contract is in
// include/psd.h): the entry point, and the CUDA-core kernel for the shapes that the
// tcgen05 kernel does not take.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "context.h"
#include "device.cuh"
#include "multi_token.h"

namespace psd {

namespace {

constexpr int kMaxDim = 256;
constexpr int kWarps = 4, kGroupRows = 8;

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

// Row groups of a launch: request b's rows (its new tokens, G query heads of a KV head each, token
// by token) in groups of kGroupRows, from group first[b] on.
struct GeneralRequests {
  StepRequests req;
  int32_t first[kStepRequests];
  float *part_o;    // [groups][Hkv][splits][kGroupRows][D], with more than one split
  float *part_lse;  // [groups][Hkv][splits][kGroupRows]
};

// The request of row group x.
__device__ __forceinline__ int request_of(const GeneralRequests &g, int B, int x) {
  int b = 0;
  for (int n = B; n > 1;) {  // the last request with first <= x
    const int mid = n / 2;
    if (g.first[b + mid] <= x) b += mid, n -= mid;
    else n = mid;
  }
  return b;
}

// One CTA per (row group, KV head, split of the keys), in f32 on CUDA cores.  A warp takes every
// fourth tile of 32 keys: a lane scores one key against the group's rows, so that K is read once
// for kGroupRows rows; then the lanes share out V's columns, 8 each, and KG keys at a time (a key
// that no row sees is not read).  The warps' states (m, l, O) join in shared memory, the
// splits' in general_join_kernel.  It takes the head dims, page sizes and scales that the
// tensor-core kernel does not: pages of 5 tokens, 32 requests of 5 tokens over 512 to 4096 keys
// of 8 heads of 128, 555 us (the other kernel, pages of 16: 54); head dim 256, 3 single tokens over
// 20000 to 65536 keys, 510 us at 2.5 TB/s.  What bounds it is the latency of each lane's own key row
// and the row's queries from shared memory.  (A CTA a token and query head, K read anew for each,
// took 1450 and 7360 us.)
template <bool FP8, int KG>
__global__ void __launch_bounds__(kWarps * 32, 4)
    step_general_kernel(const StepParams p, const __grid_constant__ GeneralRequests g) {
  constexpr int R = kGroupRows, kLanes = 32 / KG;  // lanes that share out a row of V
  __shared__ __align__(16) float qs[R][kMaxDim], weights[kWarps][32][R], part[kWarps][R][8 * kLanes];
  __shared__ float ms[kWarps][R], ls[kWarps][R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kv = blockIdx.y, D = p.D;
  const int b = request_of(g, p.B, blockIdx.x);
  const psd_token_request r = g.req.r[b];
  const int row0 = (int(blockIdx.x) - g.first[b]) * R, start = r.kv_len - r.num_new;
  const int64_t rows = int64_t(r.num_new) * p.G;  // the request's, of this KV head
  const int last = int(min(int64_t(row0) + R, rows) - 1) / p.G;
  const int n_keys = p.tree ? r.kv_len : start + last + 1;  // some row of the group sees
  for (int x = threadIdx.x; x < R * D; x += blockDim.x) {
    const int rr = x / D, d = x - rr * D, i = (row0 + rr) / p.G, h = kv * p.G + (row0 + rr) % p.G;
    qs[rr][d] = row0 + rr < rows ? __bfloat162float(p.q[int64_t(r.token0 + i) * p.q_stride + int64_t(h) * D + d]) * p.q_scale : 0.f;
  }
  __syncthreads();
  // What each row sees: keys before `seen`, and in a tree those whose bit is set from `start` on.
  int seen[R];
  uint64_t tree[R];
#pragma unroll
  for (int rr = 0; rr < R; ++rr) {
    const int i = (row0 + rr) / p.G;
    const bool live = row0 + rr < rows;
    tree[rr] = p.tree && live ? p.tree[r.token0 + i] & (r.num_new < 64 ? (uint64_t(1) << r.num_new) - 1 : ~uint64_t(0)) : 0;
    seen[rr] = !live ? 0 : p.tree ? start : start + i + 1;
  }
  const int group = lane / kLanes, col = 8 * (lane % kLanes);
  float2 o[R][4];
  float m[R], l[R];  // l: this lane's keys
#pragma unroll
  for (int rr = 0; rr < R; ++rr) {
    m[rr] = neg_inf(), l[rr] = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[rr][c] = make_float2(0.f, 0.f);
  }
  const int64_t tiles = (int64_t(n_keys) + 31) / 32;
  const int t_end = int(tiles * (blockIdx.z + 1) / gridDim.z);
  for (int t = int(tiles * blockIdx.z / gridDim.z) + warp; t < t_end; t += kWarps) {
    const int j = 32 * t + lane;
    bool there = j < n_keys;
    int64_t row = 0;
    if (there) {
      const int id = __ldg(p.page_indices + r.page_off + j / p.page_size);
      if (id < 0 || int64_t(id) >= p.num_pages) {
        raise_fault(p.fault, PSD_FAULT_PAGE_ID);
        there = false;
      } else {
        row = (int64_t(id) * p.page_size + j % p.page_size) * p.Hkv + kv;
      }
    }
    float2 acc[R];
#pragma unroll
    for (int rr = 0; rr < R; ++rr) acc[rr] = make_float2(0.f, 0.f);
    if (there) {
#pragma unroll 2
      for (int d = 0; d < D; d += 8) {
        float x[8];
        load8<FP8>(p.k_pool, row * D + d, x);
#pragma unroll
        for (int rr = 0; rr < R; ++rr)
#pragma unroll
          for (int c = 0; c < 8; c += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(&qs[rr][d + c]);
            acc[rr] = __ffma2_rn(make_float2(q.x, q.y), make_float2(x[c], x[c + 1]), acc[rr]);
            acc[rr] = __ffma2_rn(make_float2(q.z, q.w), make_float2(x[c + 2], x[c + 3]), acc[rr]);
          }
      }
    }
    float w[R];
    bool any = false;
#pragma unroll
    for (int rr = 0; rr < R; ++rr) {
      const bool sees = there && (j < seen[rr] || (j >= start && j - start < 64 && (tree[rr] >> ((j - start) & 63) & 1)));
      any |= sees;
      const float s = sees ? acc[rr].x + acc[rr].y : neg_inf();
      float top = s;
#pragma unroll
      for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      if (top > m[rr]) {
        const float alpha = ex2(m[rr] - top);
        m[rr] = top;
        l[rr] *= alpha;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[rr][c].x *= alpha, o[rr][c].y *= alpha;
      }
      w[rr] = sees ? ex2(s - (m[rr] == neg_inf() ? 0.f : m[rr])) : 0.f;
      l[rr] += w[rr];
    }
    const uint32_t weighed = __ballot_sync(0xffffffffu, any);
#pragma unroll
    for (int rr = 0; rr < R; rr += 4)
      *reinterpret_cast<float4 *>(&weights[warp][lane][rr]) = make_float4(w[rr], w[rr + 1], w[rr + 2], w[rr + 3]);
    __syncwarp();
#pragma unroll 4
    for (int k0 = 0; k0 < 32; k0 += KG) {
      const int k = k0 + group;
      const int64_t rk = __shfl_sync(0xffffffffu, row, k);
      if (col < D && (weighed >> k & 1)) {
        float x[8];
        load8<FP8>(p.v_pool, rk * D + col, x);
#pragma unroll
        for (int rr = 0; rr < R; rr += 4) {
          const float4 y = *reinterpret_cast<const float4 *>(&weights[warp][k][rr]);
          const float wk[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              o[rr + i][c] = __ffma2_rn(make_float2(wk[i], wk[i]), make_float2(x[2 * c], x[2 * c + 1]), o[rr + i][c]);
        }
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int rr = 0; rr < R; ++rr) {
#pragma unroll
    for (int x = 16; x; x >>= 1) l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], x);
#pragma unroll
    for (int x = kLanes; x < 32; x <<= 1)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        o[rr][c].x += __shfl_xor_sync(0xffffffffu, o[rr][c].x, x);
        o[rr][c].y += __shfl_xor_sync(0xffffffffu, o[rr][c].y, x);
      }
    if (group == 0)
#pragma unroll
      for (int c = 0; c < 4; ++c) *reinterpret_cast<float2 *>(&part[warp][rr][col + 2 * c]) = o[rr][c];
    if (lane == 0) ms[warp][rr] = m[rr], ls[warp][rr] = l[rr];
  }
  __syncthreads();
  const int64_t piece = (int64_t(blockIdx.x) * gridDim.y + kv) * gridDim.z + blockIdx.z;
  for (int x = threadIdx.x; x < R * D; x += blockDim.x) {
    const int rr = x / D, d = x - rr * D;
    if (row0 + rr >= rows) break;
    float top = ms[0][rr];
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, ms[w][rr]);
    const float base = top == neg_inf() ? 0.f : top;
    float sum = 0.f, y = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float scale = ex2(ms[w][rr] - base);
      sum += ls[w][rr] * scale;
      y = fmaf(part[w][rr][d], scale, y);
    }
    y *= sum == 0.f ? 0.f : p.v_scale / sum;
    const float lse = sum == 0.f ? neg_inf() : top + log2f(sum);
    if (gridDim.z > 1) {
      g.part_o[(piece * R + rr) * D + d] = y;
      if (d == 0) g.part_lse[piece * R + rr] = lse;
      continue;
    }
    const int i = (row0 + rr) / p.G;
    const int64_t out = int64_t(r.token0 + i) * p.Hq + kv * p.G + (row0 + rr) % p.G;
    if (p.out_f32) static_cast<float *>(p.o)[out * D + d] = y;
    else static_cast<__nv_bfloat16 *>(p.o)[out * D + d] = __float2bfloat16_rn(y);
    if (d == 0 && p.lse) p.lse[out] = lse;
  }
}

// Joins the splits of a row group, in key order: a thread per (row, column).
__global__ void __launch_bounds__(256) general_join_kernel(const StepParams p, const __grid_constant__ GeneralRequests g, int splits) {
  constexpr int R = kGroupRows;
  const int b = request_of(g, p.B, blockIdx.x), kv = blockIdx.y, D = p.D;
  const psd_token_request r = g.req.r[b];
  const int row0 = (int(blockIdx.x) - g.first[b]) * R;
  const int64_t piece = (int64_t(blockIdx.x) * gridDim.y + kv) * splits;
  for (int x = threadIdx.x; x < R * D; x += blockDim.x) {
    const int rr = x / D, d = x - rr * D;
    if (row0 + rr >= int64_t(r.num_new) * p.G) break;
    float m = neg_inf();
    for (int z = 0; z < splits; ++z) m = fmaxf(m, g.part_lse[(piece + z) * R + rr]);
    const float from = m == neg_inf() ? 0.f : m;
    float sum = 0.f, y = 0.f;
#pragma unroll 4
    for (int z = 0; z < splits; ++z) {
      const float s = g.part_lse[(piece + z) * R + rr], w = ex2(s - from);
      const float v = g.part_o[((piece + z) * R + rr) * D + d];
      sum += w;
      y = s == neg_inf() ? y : fmaf(w, v, y);
    }
    y *= sum == 0.f ? 0.f : 1.f / sum;
    const int i = (row0 + rr) / p.G;
    const int64_t out = int64_t(r.token0 + i) * p.Hq + kv * p.G + (row0 + rr) % p.G;
    if (p.out_f32) static_cast<float *>(p.o)[out * D + d] = y;
    else static_cast<__nv_bfloat16 *>(p.o)[out * D + d] = __float2bfloat16_rn(y);
    if (d == 0 && p.lse) p.lse[out] = sum == 0.f ? neg_inf() : m + log2f(sum);
  }
}

// Pieces a launch may leave in the workspace.
int64_t general_pieces(int sms) { return 16 * int64_t(sms); }

}  // namespace

psd_status launch_step_general(const StepParams &p, const StepRequests &req, float *base, const DeviceInfo &dev,
                               cudaStream_t s) {
  GeneralRequests g;
  std::memcpy(g.req.r, req.r, sizeof(psd_token_request) * size_t(p.B));
  int64_t groups = 0;
  int longest = 0;
  for (int b = 0; b < p.B; ++b) {
    if (groups > 0x7fffffffLL || int64_t(req.r[b].num_new) * p.G > 0x7fffffffLL)
      return fail(PSD_ERR_UNSUPPORTED, "multi_token_decode: more than 2^31 query rows in one launch");
    g.first[b] = int32_t(groups);
    groups += (int64_t(req.r[b].num_new) * p.G + kGroupRows - 1) / kGroupRows;
    longest = std::max(longest, req.r[b].kv_len);
  }
  if (groups > 0x7fffffffLL) return fail(PSD_ERR_UNSUPPORTED, "multi_token_decode: more than 2^31 query rows in one launch");
  // Four CTAs an SM fit.  With fewer units than that the keys are split to make as many, and up to
  // eight an SM in three, since lengths differ, no finer than a tile a warp.  3 single tokens over
  // 20000 to 65536 keys: 510 us, against 590 with 16 an SM and 7360 unsplit; 32 requests of 5 tokens
  // over 512 to 4096 keys: 555 us against 700 unsplit.
  const int64_t units = groups * p.Hkv, sms = dev.num_sms;
  const int64_t want = std::min(std::max<int64_t>(3, 4 * sms / units), general_pieces(dev.num_sms) / units);
  const int splits = units < 8 * sms ? int(std::max<int64_t>(1, std::min<int64_t>(want, (longest + 127) / 128))) : 1;
  g.part_o = base;
  g.part_lse = base + general_pieces(dev.num_sms) * kGroupRows * p.D;
  const dim3 grid(unsigned(groups), unsigned(p.Hkv), unsigned(splits));
  auto go = [&](auto fp8, auto kg) {
    step_general_kernel<decltype(fp8)::value, decltype(kg)::value><<<grid, kWarps * 32, 0, s>>>(p, g);
  };
  auto by_dim = [&](auto fp8) {
    if (p.D <= 64) go(fp8, std::integral_constant<int, 4>{});
    else if (p.D <= 128) go(fp8, std::integral_constant<int, 2>{});
    else go(fp8, std::integral_constant<int, 1>{});
  };
  if (p.fp8) by_dim(std::true_type{});
  else by_dim(std::false_type{});
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && splits > 1) {
    general_join_kernel<<<dim3(unsigned(groups), unsigned(p.Hkv)), 256, 0, s>>>(p, g, splits);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "multi_token_decode launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}

}  // namespace psd

using namespace psd;

extern "C" size_t psd_multi_token_workspace_bytes(const psd_ctx *ctx, int32_t D) {
  if (!ctx || D < 1) return 0;
  // the fault word, then the partial rows of the tensor-core kernel's CTAs, one per SM, or the
  // other kernel's pieces
  const size_t general = size_t(general_pieces(ctx->dev.num_sms)) * kGroupRows * (size_t(D) + 1);
  return 256 + 4 * (D == 64 || D == 128 ? std::max(general, step_tc_place(ctx->dev.num_sms, D, nullptr).floats) : general);
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
  const float q_scale = a->sm_scale * 1.4426950408889634f * (fp8 ? a->k_scale : 1.f);
  if (!std::isfinite(a->sm_scale) || (fp8 && (!std::isfinite(a->k_scale) || !std::isfinite(a->v_scale))) ||
      !std::isfinite(q_scale))
    return fail(PSD_ERR_INVALID_ARG, "multi_token_decode: scales and sm_scale * log2(e) * k_scale must be finite");
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
    if (r.token0 != row || r.num_new < 0 || r.kv_len < 1 || r.kv_len > kMaxKvLen || r.num_new > r.kv_len ||
        r.page_off < 0 || (a->tree_mask && r.num_new > 64) ||
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
  p.fault = next_fault(ctx, workspace, s);
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
  p.q_scale = q_scale;
  p.v_scale = fp8 ? a->v_scale : 1.f;
  float *const base = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + 256);
  const StepPlace place = step_tc_place(ctx->dev.num_sms, a->D, base);
  StepRequests req;
  const bool tensor = step_tc_supports(p);
  for (int32_t b0 = 0; b0 < plan->batch;) {
    // up to kStepRequests requests that have new tokens
    p.B = 0;
    for (; b0 < plan->batch && p.B < kStepRequests; ++b0)  // (the others' rows are none)
      if (plan->requests[b0].num_new > 0) req.r[p.B++] = plan->requests[b0];
    if (p.B == 0) break;
    const psd_status st =
        tensor ? launch_step_tc(p, req, place, ctx->dev, s) : launch_step_general(p, req, base, ctx->dev, s);
    if (st != PSD_OK) return st;
  }
  return PSD_OK;
}
