// Verification of drafted tokens (the contract is in include/psd.h).
//
// Mathematics.  With draft d drawn from q, accepting with probability min(1, p(d)/q(d))
// and drawing from max(p - q, 0) after a refusal leaves the outcome distributed as p.
// Acceptance compares u q(d) < p(d): the product of two f32 numbers is exact in 64 bits.
// The draw wants the least v with C_v > u C: a border decided by sums of many thousand
// numbers, so the weights are summed as integers, multiples of 2^-46.  Integer sums do not depend
// on their order, so the split over threads cannot change a token.  64 bits hold sums below
// 2^18; larger ones (rows that are no probabilities) stay at the largest number, in any order
// too, and are reported as a row without weights is.  A weight is rounded to that unit once:
// weights from 2^-23 on (1.2e-7) are exact, the error of a row's sum is about 1e-12.
//
// The weight of an entry with p > q, in f32 operations: d = p - q rounded, and its error e =
// (p - d) - q, exact since p >= q >= 0; d's multiples of 2^-23 are the low bits of d + 1
// (whose unit in the last place is 2^-23), what that leaves, r, is exact too, and the
// multiples of 2^-46 in r and e are the low bits of their sums with 1.5 * 2^-23.  18
// instructions an entry; shifting the two significands into place as 64-bit integers took
// 41 and bounded the kernel (128 requests: 36 us against 29).
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

// Low words of sums of weights: the weight is high * 2^-23 + low * 2^-46.
struct Acc {
  uint32_t high = 0, low = 0;  // modulo 2^32, the added constants' bits included
  __device__ __forceinline__ void level(float d, float e) {
    constexpr float kOne = 1.f, kSmall = 1.5f * 0x1p-23f;
    const float t = d + kOne;
    const float r = d - (t - kOne);
    high += __float_as_uint(t);
    low += __float_as_uint(r + kSmall) + __float_as_uint(e + kSmall);
  }
  __device__ __forceinline__ void level(float d) {  // e = 0
    constexpr float kOne = 1.f, kSmall = 1.5f * 0x1p-23f;
    const float t = d + kOne;
    high += __float_as_uint(t);
    low += __float_as_uint(d - (t - kOne) + kSmall);
  }
  // max(p - q, 0); p and q are taken as 0 where NaN or negative, as 1 from 1 on
  __device__ __forceinline__ void add(float p, float q) {
    p = __saturatef(p);
    q = __saturatef(q);
    const float d = p - q, e = (p - d) - q;
    const bool some = p > q;
    level(some ? d : 0.f, some ? e : 0.f);
  }
  __device__ __forceinline__ void add(float p) { level(__saturatef(p)); }
  // The sum of n weights added with a q each (two low words) or without: n <= 128.
  __device__ __forceinline__ uint64_t value(int n, bool with_q) const {
    const uint32_t h = high - uint32_t(n) * 0x3f800000u;
    const int32_t l = int32_t(low - uint32_t(with_q ? 2 * n : n) * 0x34400000u);
    return (uint64_t(h) << 23) + uint64_t(int64_t(l));
  }
};
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

constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr int kDeepCtas = 4;   // CTAs an SM of the form for few CTAs
constexpr int kMaxSums = 1023; // sums a CTA keeps of its part of a row; 256 kMaxSums < 2^18
constexpr uint64_t kFull = ~uint64_t(0);  // 2^18 or more

__device__ __forceinline__ uint64_t add_sums(uint64_t x, uint64_t y) { return x + y < x ? kFull : x + y; }

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t x) {  // inclusive, in lane order
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint64_t peer_load(const uint64_t *mine, int rank) {
  uint32_t at;
  uint64_t x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(at) : "memory");
  return x;
}

// The row that the next token is drawn from: weights max(p - q, 0).
struct Row {
  const float *p, *q;  // q NULL: p alone
  int hot;             // a token of weight 0, or -1
  __device__ __forceinline__ uint64_t at(int v) const {
    Acc x;
    if (q) x.add(__ldg(p + v), __ldg(q + v));
    else x.add(v == hot ? 0.f : __ldg(p + v));
    return x.value(1, q != nullptr);
  }
};

// One cluster per request.  Every CTA finds the accepted drafts for itself (a gather of
// K values of p and q); then the CTAs share out the chosen row, a stretch each: a warp sums
// blocks of `step` entries, keeping each block's sum, so that the row is read once, and
// the CTA that holds the crossing looks only at the block where it lies again.
// The work is the row's bytes: 8 V with a refusal, 4 V without; 8 CTAs a request put
// enough loads in flight from one request on.  4 requests of 32000 words take 13-14 us, nearly all of
// it the chain (offsets, drafts, their p and q, the row, two cluster barriers, the block again);
// 128 requests of 98305 words with sampled drafts 31 us (101 MB: the chain, then 5 TB/s).
// U blocks of a warp are on their way at once: two where all CTAs fit at four an SM, one at seven
// an SM else.  48 requests of 131072 words 15.1 us against 16.7 with one (17 against 19 sampled),
// 128 requests of 98305 words in 1024 CTAs 38 us with two against 29.7: a second wave.
template <int U>
__global__ void __launch_bounds__(kVerifyThreads, U == 1 ? 7 : kDeepCtas) verify_drafts_kernel(const VerifyParams p, int ctas) {
  __shared__ uint64_t sums[kMaxSums], warps[kVerifyWarps], mine;
  __shared__ int first_refused;
  const int b = blockIdx.x / ctas, rank = blockIdx.x - b * ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int d0 = __ldg(p.indptr + b), d1 = __ldg(p.indptr + b + 1);
  if (d0 < 0 || d1 < d0 || d1 > p.num_drafts) {  // the whole cluster leaves
    if (rank == 0 && tid == 0) atomicOr(p.fault, PSD_FAULT_RANGE);
    return;
  }
  const int K = d1 - d0, R = d0 + b;
  if (tid == 0) first_refused = K;
  __syncthreads();
  for (int j = tid; j < K; j += kVerifyThreads) {
    const int d = __ldg(p.tokens + d0 + j);
    bool ok = false;
    if (d >= 0 && d < p.V) {
      const double q = p.draft ? double(__ldg(p.draft + (d0 + j) * p.draft_stride + d)) : 1.0;
      ok = double(__ldg(p.uniforms + R + j)) * q < double(__ldg(p.target + (R + j) * p.target_stride + d));
    }
    if (!ok) atomicMin(&first_refused, j);
  }
  const float u = __ldg(p.uniforms + R + K);
  __syncthreads();
  const int a = first_refused;
  Row row{p.target + (R + a) * p.target_stride, nullptr, -1};
  bool outside = false;
  if (a < K) {
    const int d = __ldg(p.tokens + d0 + a);
    outside = d < 0 || d >= p.V;
    if (!outside && p.draft) row.q = p.draft + (d0 + a) * p.draft_stride;
    if (!outside && !p.draft) row.hot = d;
  }
  // This CTA's entries [v0, v1), in blocks of `step` (a multiple of 256).  The sum of a block, of up
  // to 131328 entries, fits 64 bits, and with blocks of 256 that of all of them does.
  const int part = (p.V + ctas - 1) / ctas;
  const int v0 = min(rank * part, p.V), v1 = min(v0 + part, p.V);
  const int step = 256 * ((part + 256 * kMaxSums - 1) / (256 * kMaxSums));
  const int blocks = (v1 - v0 + step - 1) / step;
  uint64_t total = 0, before = 0;
  for (int pass = 0; pass < 2 && total == 0; ++pass) {
    if (pass == 1) {  // p <= q everywhere: draw from p
      row.q = nullptr, row.hot = -1;
      cluster_sync();  // the peers have read `mine`
    }
    uint64_t own = 0;
    for (int k = warp; k < blocks; k += kVerifyWarps) {
      if constexpr (U > 1) {
        const int at = v0 + k * 256 + lane;
        if (step == 256 && v0 + (k + (U - 1) * kVerifyWarps + 1) * 256 <= v1) {  // U whole blocks of the warp
          float pv[U][8], qv[U][8];
#pragma unroll
          for (int n = 0; n < U; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) pv[n][i] = __ldg(row.p + at + n * kVerifyWarps * 256 + 32 * i);
          if (row.q)
#pragma unroll
            for (int n = 0; n < U; ++n)
#pragma unroll
              for (int i = 0; i < 8; ++i) qv[n][i] = __ldg(row.q + at + n * kVerifyWarps * 256 + 32 * i);
#pragma unroll
          for (int n = 0; n < U; ++n) {
            Acc s;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (row.q) s.add(pv[n][i], qv[n][i]);
              else s.add(row.hot - at == n * kVerifyWarps * 256 + 32 * i ? 0.f : pv[n][i]);
            }
            const uint64_t x = warp_sum(s.value(8, row.q != nullptr));
            if (lane == 0) sums[k + n * kVerifyWarps] = x;
            own += x;
          }
          k += (U - 1) * kVerifyWarps;
          continue;
        }
      }
      const int lo = v0 + k * step, hi = min(lo + step, v1);
      uint64_t x = 0;
      for (int c = lo; c < hi; c += 256) {
        if (c + 256 <= hi) {
          float pv[8], qv[8];
          Acc s;
#pragma unroll
          for (int i = 0; i < 8; ++i) pv[i] = __ldg(row.p + c + 32 * i + lane);
          if (row.q) {
#pragma unroll
            for (int i = 0; i < 8; ++i) qv[i] = __ldg(row.q + c + 32 * i + lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) s.add(pv[i], qv[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) s.add(row.hot - c - lane == 32 * i ? 0.f : pv[i]);
          }
          x += s.value(8, row.q != nullptr);
        } else {
          for (int v = c + lane; v < hi; v += 32) x += row.at(v);
        }
      }
      x = warp_sum(x);
      if (lane == 0) sums[k] = x;
      own += x;
    }
    if (lane == 0) warps[warp] = own;
    __syncthreads();
    if (step == 256) {
      if (tid == 0) {
        uint64_t x = 0;
        for (int w = 0; w < kVerifyWarps; ++w) x += warps[w];
        mine = x;
      }
    } else if (warp == 0) {
      uint64_t x = 0;
      for (int k = lane; k < blocks; k += 32) x = add_sums(x, sums[k]);
#pragma unroll
      for (int d = 16; d; d >>= 1) x = add_sums(x, __shfl_xor_sync(0xffffffffu, x, d));
      if (lane == 0) mine = x;
    }
    cluster_sync();
    total = before = 0;
    for (int c = 0; c < ctas; ++c) {
      const uint64_t x = peer_load(&mine, c);
      if (c < rank) before = add_sums(before, x);
      total = add_sums(total, x);
    }
  }
  if (total == kFull) total = 0;  // no token's
  const uint64_t own = mine;
  uint64_t want = share_of(u, total);
  if (want >= total && total) want = total - 1;  // u >= 1 (outside the contract): the last entry with a weight
  if (warp == 0 && total && before <= want && want < before + own) {
    // the block, then the entry, at which the running sum passes `want`
    want -= before;
    int k0 = 0;
    uint64_t run = 0;
    for (;; k0 += 32) {
      const uint64_t x = warp_scan(k0 + lane < blocks ? sums[k0 + lane] : 0);
      const uint32_t past = __ballot_sync(0xffffffffu, run + x > want);
      const int f = past ? __ffs(past) - 1 : 32;
      if (f > 0) {
        const uint64_t y = __shfl_sync(0xffffffffu, x, f - 1);
        run += y;
      }
      if (past || k0 + 32 >= blocks) {
        k0 += f;
        break;
      }
    }
    const int lo = v0 + k0 * step, hi = min(lo + step, v1);
    bool done = false;
    for (int c = lo; c < hi && !done; c += 256) {
      uint64_t w[8];  // all on their way before the first is needed
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int v = c + 32 * i + lane;
        w[i] = v < hi ? row.at(v) : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t x = warp_scan(w[i]);
        const uint32_t past = __ballot_sync(0xffffffffu, run + x > want);
        if (past && !done) {
          if (lane == 0) p.out[R + a] = c + 32 * i + __ffs(past) - 1;
          done = true;
        }
        run += __shfl_sync(0xffffffffu, x, 31);
      }
    }
  }
  if (rank == 0) {
    for (int j = tid; j <= K; j += kVerifyThreads)
      if (j != a || !total) p.out[R + j] = j < a ? __ldg(p.tokens + d0 + j) : -1;
    if (tid == 0) {
      p.accepted[b] = a;
      if (outside || !total) atomicOr(p.fault, PSD_FAULT_RANGE);
    }
  }
  cluster_sync();  // a peer may still read `mine`
}

}  // namespace
}  // namespace psd

using namespace psd;

extern "C" psd_status verify_drafts(psd_ctx *ctx, const psd_verify_args *a, psd_stream_t stream) {
  clear_error();
  if (!ctx || !a) return fail(PSD_ERR_INVALID_ARG, "verify_drafts: NULL");
  if (a->batch < 0 || a->num_drafts < 0 || a->vocab < 1 || a->vocab > (1 << 30) || (a->batch == 0 && a->num_drafts > 0))
    return fail(PSD_ERR_INVALID_ARG, "verify_drafts: batch %d, num_drafts %d, vocab %d", a->batch, a->num_drafts,
                a->vocab);
  if (int64_t(a->batch) + a->num_drafts > 0x7fffffffLL) return fail(PSD_ERR_INVALID_ARG, "verify_drafts: too many rows");
  if (a->batch == 0) return PSD_OK;
  if (a->batch > 0x7fffffff / 8) return fail(PSD_ERR_UNSUPPORTED, "verify_drafts: batch %d", a->batch);
  if (!a->target_probs || !a->draft_indptr || !a->uniforms || !a->num_accepted || !a->out_tokens || !a->fault_dev ||
      (a->num_drafts > 0 && !a->draft_tokens))
    return fail(PSD_ERR_INVALID_ARG, "verify_drafts: NULL pointer");
  if (a->target_stride < a->vocab || (a->draft_probs && a->draft_stride < a->vocab))
    return fail(PSD_ERR_INVALID_ARG, "verify_drafts: a row stride is shorter than vocab");
  DeviceGuard g(ctx->dev.device);
  VerifyParams p{a->target_probs, a->draft_probs, a->target_stride, a->draft_stride, a->draft_tokens, a->draft_indptr,
                 a->uniforms, a->num_accepted, a->out_tokens, a->fault_dev, a->batch, a->num_drafts, a->vocab};
  // 2048 entries or more a CTA, 8 CTAs (the portable cluster) at most
  int ctas = 1;
  while (ctas < 8 && a->vocab > 2048 * ctas) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a->batch) * unsigned(ctas));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool few = int64_t(a->batch) * ctas <= int64_t(kDeepCtas) * ctx->dev.num_sms;  // all on the SMs at once
  const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, verify_drafts_kernel<2>, p, ctas)
                            : cudaLaunchKernelEx(&cfg, verify_drafts_kernel<1>, p, ctas);
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "verify_drafts launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}
