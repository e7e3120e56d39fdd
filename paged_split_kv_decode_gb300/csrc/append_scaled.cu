// append_tokens into a cache of 8-bit blocks with a scale each (the contract is in include/psd.h).
//
// Mathematics.  The scale of a block is the least power of two that brings its largest magnitude within e4m3's
// 448 = 1.75 2^8: with A = f 2^E, f in [1, 2), that is 2^(E - 8), or 2^(E - 7) where f > 1.75, read off A's bits.
// x 2^-k is exact in f32, so a code is rounded once.  A block that holds older tokens keeps its scale or takes a
// larger one; older codes then go down by a power of two, which rounds only what falls below 2^-6.
//
// A CTA has some tokens, and K, V or the queries of them: it rotates their queries, or it writes the blocks whose first new
// token is one of them, the tokens of such a block behind its own included.  So every block has one writer, whatever the lengths,
// without a list of blocks and without atomics on scales.  A warp takes one block of one head's K or V, D / 16 lanes a
// token, and keeps the rotated values between finding the scale and writing the codes (blocks of 16 tokens up to 128
// columns; larger ones are read and rotated twice).
#include <algorithm>
#include <atomic>

#include "append.cuh"
#include "block_scales.cuh"

namespace psd {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kLeast = 95;  // 2^-32
constexpr int kMaxBlock = 64, kMany = 16;

struct ScaledParams {
  AppendParams a;
  uint8_t *k_scales, *v_scales;
  int block;
};

// A token of the CTA.
struct Token {
  int pos;       // rotation position; negative: left as it is
  int count;     // tokens of the block from this one on, if it is the block's first new one, else 0
  int older;     // tokens of the block before this one
  int64_t slot;  // pool row, or -1
};

// Token t0 + lane of a warp's, for the lanes below `own`: the warp finds the first one's request, and the lanes walk on from
// there.  (A search for each token, two a warp one after the other, took twice the time of these dependent loads.)
__device__ __forceinline__ Token locate(const ScaledParams &s, int t0, int own, uint32_t &faults) {
  const AppendParams &p = s.a;
  Token x{-1, 0, 0, -1};
  faults = 0;
  const int t = t0 + int(threadIdx.x & 31), all = __ldg(p.q_indptr + p.B);
  int b = request_of(p.q_indptr, p.B, t0);
  if (t >= t0 + own || t >= p.T || t >= all) return x;  // not the CTA's, or behind the last request
  while (b + 1 < p.B && __ldg(p.q_indptr + b + 1) <= t) ++b;
  const int begin = __ldg(p.q_indptr + b), end = __ldg(p.q_indptr + b + 1);
  const int at = __ldg(p.kv_len + b) - (end - t);  // index in the request
  const int first = __ldg(p.page_indptr + b), last = __ldg(p.page_indptr + b + 1);
  if (t < begin || t >= end) {
    faults = PSD_FAULT_RANGE;
    return x;
  }
  x.pos = p.positions ? __ldg(p.positions + t) : at;
  if (x.pos < 0) faults = PSD_FAULT_RANGE, x.pos = -1;
  const int64_t page = int64_t(first) + at / p.page_size;
  int id = -1;
  if (at >= 0 && first >= 0 && page < last && page < p.num_page_indices) id = __ldg(p.page_indices + page);
  if (id < 0 || int64_t(id) >= p.num_pages) {
    if (x.pos >= 0) faults |= PSD_FAULT_PAGE_ID;
    return x;
  }
  x.slot = int64_t(id) * p.page_size + at % p.page_size;
  x.older = at % s.block;
  // the first of the block: its request's first token, or the block's
  if (t == begin || x.older == 0) x.count = min(s.block - x.older, min(end, p.T) - t);  // (no row behind the last that is there)
  return x;
}

__device__ __forceinline__ void prefetch_l2(const void *at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at) : "memory"); }

struct F8 {
  float v[8];
};
__device__ __forceinline__ uint4 load_raw(const __nv_bfloat16 *src) { return __ldg(reinterpret_cast<const uint4 *>(src)); }
__device__ __forceinline__ F8 unpack(const uint4 &w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  F8 f;
#pragma unroll
  for (int k = 0; k < 4; ++k) f.v[2 * k] = bf16_lo(u[k]), f.v[2 * k + 1] = bf16_hi(u[k]);
  return f;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *dst, const F8 &f) {
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(f.v[2 * k], f.v[2 * k + 1]);
    u[k] = *reinterpret_cast<const uint32_t *>(&x);
  }
  *reinterpret_cast<uint4 *>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ uint2 codes8(const F8 &f, float by) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f.v[4 * k + 1] * by), "f"(f.v[4 * k] * by));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f.v[4 * k + 3] * by), "f"(f.v[4 * k + 2] * by));
    w[k] = uint32_t(lo) | (uint32_t(hi) << 16);
  }
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ F8 values8(const uint2 &w) {
  F8 f;
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = e4m3x2_to_float2((u[i >> 1] >> (16 * (i & 1))) & 0xffffu);
    f.v[2 * i] = y.x, f.v[2 * i + 1] = y.y;
  }
  return f;
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN operands lose, as in fmaxf
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The least e with top <= 448 2^(e - 127), top >= 0 finite.
__device__ __forceinline__ int scale_of(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = int(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
  return max(e, kLeast);
}

// A token's angles in shared memory: cosines, sines, `half` each.  Pair 8 g + e lies at (e / 4) (half / 2) + 4 g + e % 4, so
// that neighbouring groups' four values lie side by side.
__device__ __forceinline__ int angle_at(int pair, int half) { return (pair & 4 ? half / 2 : 0) + (pair >> 3) * 4 + (pair & 3); }
// cos and sin of pos * F turns, of which 32 bits behind the point are kept (1.5e-9 rad), times the magnitude.
__device__ __forceinline__ float2 short_turn(uint64_t F, int pos, float magnitude) {
  const int frac = int(uint32_t((F * uint64_t(uint32_t(pos))) >> 32));
  float s, c;
  sincospif(__int2float_rn(frac) * 0x1p-31f, &s, &c);
  return make_float2(c * magnitude, s * magnitude);
}
// Rotates eight pairs, group g, in place: a and b are the two runs of its columns, c and s the token's cosines and sines.
template <bool NEOX>
__device__ __forceinline__ void rotate(F8 &a, F8 &b, const float *c, const float *s, int g, int half) {
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    const int at = (k ? half / 2 : 0) + 4 * g;
    const float4 cc = *reinterpret_cast<const float4 *>(c + at), ss = *reinterpret_cast<const float4 *>(s + at);
    const float c4[4] = {cc.x, cc.y, cc.z, cc.w}, s4[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float &x = NEOX ? a.v[k + i] : k ? b.v[2 * i] : a.v[2 * i], &y = NEOX ? b.v[k + i] : k ? b.v[2 * i + 1] : a.v[2 * i + 1];
      const float u = x * c4[i] - y * s4[i];
      y = y * c4[i] + x * s4[i];
      x = u;
    }
  }
}

// KIND: all in one launch, K and V alone, or the queries alone, whose CTAs have more room without the others' code.
enum { kAllParts, kBlocks, kQueries };
template <int NT, bool NEOX, int KIND>
__global__ void __launch_bounds__(kThreads, KIND == kQueries ? 5 : 2) append_scaled_kernel(const ScaledParams s, const __grid_constant__ Turns turns) {
  extern __shared__ __align__(16) float table[];  // cosines [tokens][half], then sines
  __shared__ Token tokens[NT];
  __shared__ int pos[NT + kMaxBlock];
  __shared__ int n_table, n_starts, starts[NT];  // tokens whose angles are needed; tokens that begin their block
  const AppendParams &p = s.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = p.rot / 2;
  const int groups = half / 8, far = NEOX ? half : 8;  // groups of 8 pairs; their second run of 8 columns is `far` behind
  // CTAs of K (0) and V (1) in turn, NT tokens each, then those of the queries (2), NQ each.
  constexpr int NQ = NT < 2 ? NT : 2;
  const int kv_ctas = KIND == kQueries ? 0 : 2 * ((p.T + NT - 1) / NT), cta = blockIdx.x;
  if (KIND == kQueries) dependents_may_launch();  // K and V are another launch's
  const int part = KIND == kQueries || (KIND == kAllParts && cta >= kv_ctas) ? 2 : cta & 1, own = part == 2 ? NQ : NT;
  const int t0 = part == 2 ? (cta - kv_ctas) * NQ : cta / 2 * NT;

  // Queries: a thread has the same group of pairs, or run that is not rotated, of all tokens, which are on their way before
  // their places are known.
  const int rest = (p.D - p.rot) / 8, per_head = groups + rest;
  uint4 qa[NQ], qb[NQ];
  int job = tid, q_col = 0;
  bool q_turned = false;
  auto enter = [&]() {  // the thread's job: its column in a token's heads
    const int h = job / per_head, g = job - h * per_head;
    q_turned = g < groups;
    int col = q_turned ? p.rot_col + (NEOX ? 8 * g : 16 * g) : 8 * (g - groups);
    if (!q_turned && col >= p.rot_col) col += p.rot;
    q_col = h * p.D + col;
  };
  auto fetch_q = [&]() {
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (t0 + q < p.T) {
        const __nv_bfloat16 *at = p.q + (t0 + q) * p.q_stride + q_col;
        qa[q] = load_raw(at);
        if (q_turned) qb[q] = load_raw(at + far);
      }
  };
  if (part == 2) {
    if (job < p.Hq * per_head) {
      enter();
      fetch_q();
    }
  } else {  // the rows of K or V, as far as the CTA's own tokens go, to the second-level cache
    const int lines = ((part ? p.Dv : p.D) * p.Hkv * 2 + 127) / 128;
    for (int i = tid; i < NT * lines; i += kThreads)
      if (t0 + i / lines < p.T)
        prefetch_l2(reinterpret_cast<const uint8_t *>(part ? p.v + (t0 + i / lines) * p.v_stride : p.k + (t0 + i / lines) * p.k_stride) +
                    i % lines * 128);
  }
  if (warp == 0) {
    static_assert(NT <= 32, "a lane a token");
    uint32_t faults;
    const Token x = locate(s, t0, own, faults);
    if (lane < own) tokens[lane] = x;
    faults = __reduce_or_sync(0xffffffffu, faults);
    if (faults && lane == 0 && part == 0) atomicOr(p.fault, int32_t(faults));
    __syncwarp();
    // the tokens whose angles are needed: its own, and those of its last block behind them
    const bool begins = x.slot >= 0 && x.count > 0;
    const uint32_t who = __ballot_sync(0xffffffffu, begins);
    const int most = part == 2 ? own : __reduce_max_sync(0xffffffffu, begins ? max(own, lane + x.count) : own);
    for (int n = lane; n < most; n += 32) {
      if (n < own) {
        pos[n] = tokens[n].pos;
      } else {  // of the request of the last block that starts here
        int at = -1;
        if (p.positions) {
          at = __ldg(p.positions + t0 + n);
        } else {
          const int i = 31 - __clz(who);
          if (tokens[i].count > n - i) at = tokens[i].pos + (n - i);
        }
        pos[n] = max(at, -1);
      }
    }
    if (begins) starts[__popc(who & ((1u << lane) - 1u))] = lane;
    if (lane == 0) n_table = most, n_starts = __popc(who);
  }
  __syncthreads();
  const int nt = n_table;
  float *cosine = table, *sine = table + nt * half;
  const int from = part == 2 || n_starts == 0 ? 0 : starts[0];  // (tokens before the first block's begin are another CTA's)
  for (int i = from * half + tid; part != 1 && (part == 2 || n_starts > 0) && i < nt * half; i += kThreads) {
    const int n = i / half, k = i - n * half;
    const float2 cs = pos[n] >= 0 ? short_turn(turns.f[k], pos[n], p.magnitude) : make_float2(0.f, 0.f);
    cosine[n * half + angle_at(k, half)] = cs.x;
    sine[n * half + angle_at(k, half)] = cs.y;
  }
  __syncthreads();

  // ---- blocks: K of head h, or V of it.  A lane has two runs of 8 columns of a token, up to kPasses tokens at once.
  constexpr int kPasses = 4;
  const bool is_v = part == 1;
  const int W = is_v ? p.Dv : p.D;
  for (int u = warp; part < 2 && u < n_starts * p.Hkv; u += kWarps) {
    const int start = u / p.Hkv, h = u - start * p.Hkv, n = starts[start];
    const Token x = tokens[n];
    const int lanes = (W + 15) / 16, a_pass = 32 / lanes;  // lanes a token, tokens a pass
    const int mine = lane / lanes, k = lane - mine * lanes;
    const bool turned = !is_v && k < groups;
    // the columns of the two runs (the second may not be there): a group of pairs, or two runs that are not rotated
    int ca = turned ? p.rot_col + (NEOX ? 8 * k : 16 * k) : 16 * k - (is_v ? 0 : p.rot), cb = turned ? ca + far : ca + 8;
    if (!is_v && !turned) {
      if (ca >= p.rot_col) ca += p.rot;
      if (cb >= p.rot_col) cb += p.rot;
    }
    const bool there_b = cb < W;
    const __nv_bfloat16 *src = is_v ? p.v + int64_t(h) * W : p.k + int64_t(h) * W;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    bool any = false;  // of the tokens is appended
    for (int i = lane; i < x.count; i += 32) any |= pos[n + i] >= 0;
    if (!__any_sync(0xffffffffu, any)) continue;
    const int passes = (x.count + a_pass - 1) / a_pass;
    F8 a[kPasses], b[kPasses];
    uint32_t valid = 0;  // passes of those at hand that have a token for this lane
    auto fetch = [&](int pass0) {
      valid = 0;
      const __nv_bfloat16 *at = src + (t0 + n + pass0 * a_pass + mine) * stride;
      uint4 wa[kPasses], wb[kPasses];
#pragma unroll
      for (int q = 0; q < kPasses; ++q) {
        const int i = (pass0 + q) * a_pass + mine;
        wa[q] = wb[q] = make_uint4(0u, 0u, 0u, 0u);
        if (mine < a_pass && i < x.count && pos[n + i] >= 0) {
          valid |= 1u << q;
          wa[q] = load_raw(at + ca);
          if (there_b) wb[q] = load_raw(at + cb);
        }
        at += a_pass * stride;
      }
#pragma unroll
      for (int q = 0; q < kPasses; ++q) {
        a[q] = unpack(wa[q]), b[q] = unpack(wb[q]);
        const int i = (n + (pass0 + q) * a_pass + mine) * half;
        if (turned && (valid >> q & 1)) rotate<NEOX>(a[q], b[q], cosine + i, sine + i, k, half);
      }
    };
    float top = 0.f;
    // (NaN loses; infinities are looked for again, and left out, where there are any)
    auto larger = [&](const F8 &f, bool finite) {
      if (!finite) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) top = max3(top, fabsf(f.v[i]), fabsf(f.v[i + 1]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (fabsf(f.v[i]) != __int_as_float(0x7f800000)) top = fmaxf(top, fabsf(f.v[i]));
      }
    };
#pragma unroll 1
    for (bool finite = false;; finite = true) {
#pragma unroll 1
      for (int pass0 = 0; pass0 < passes; pass0 += kPasses) {
        if (!finite || passes > kPasses) fetch(pass0);
#pragma unroll
        for (int q = 0; q < kPasses; ++q) {
          larger(a[q], finite);
          larger(b[q], finite);
        }
      }
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      if (top < __int_as_float(0x7f800000)) break;
      top = 0.f;
    }
    const int64_t first = x.slot - x.older;              // the block's first row
    uint8_t *scale = (is_v ? s.v_scales : s.k_scales) + first / s.block * p.Hkv + h;
    uint8_t *pool = static_cast<uint8_t *>(is_v ? p.v_pool : p.k_pool) + (first * p.Hkv + h) * W;
    const int64_t pool_stride = int64_t(p.Hkv) * W;
    int e = scale_of(top);
    if (x.older > 0) {
      const int had = *scale;
      if (e > had) {
        const float down = ex2(float(had - e));          // (0 below 2^-126)
        for (int i = mine; mine < a_pass && i < x.older; i += a_pass) {
          uint2 *at = reinterpret_cast<uint2 *>(pool + i * pool_stride + ca);
          *at = codes8(values8(*at), down);
          if (there_b) {
            at = reinterpret_cast<uint2 *>(pool + i * pool_stride + cb);
            *at = codes8(values8(*at), down);
          }
        }
      }
      e = max(e, had);
    }
    __syncwarp();
    if (lane == 0) *scale = uint8_t(e);
    const float by = __uint_as_float(uint32_t(254 - min(e, 253)) << 23);
#pragma unroll 1
    for (int pass0 = 0; pass0 < passes; pass0 += kPasses) {
      if (passes > kPasses) fetch(pass0);                // (otherwise they are there)
      uint8_t *at = pool + (x.older + pass0 * a_pass + mine) * pool_stride;
#pragma unroll
      for (int q = 0; q < kPasses; ++q) {
        if (valid >> q & 1) {
          *reinterpret_cast<uint2 *>(at + ca) = codes8(a[q], by);
          if (there_b) *reinterpret_cast<uint2 *>(at + cb) = codes8(b[q], by);
        }
        at += a_pass * pool_stride;
      }
    }
  }

  // ---- queries.  (q_out may be q: both runs of a group are read before either is written.)
  if (KIND == kBlocks) wait_for_prior_grid();  // what waits for this launch waits for the queries' too
  while (KIND != kBlocks && part == 2 && job < p.Hq * per_head) {
    const int g = job % per_head;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (pos[q] < 0) continue;
      __nv_bfloat16 *to = p.q_out + int64_t(t0 + q) * p.Hq * p.D + q_col;
      if (q_turned) {
        F8 x = unpack(qa[q]), y = unpack(qb[q]);
        rotate<NEOX>(x, y, cosine + q * half, sine + q * half, g, half);
        store8(to, x);
        store8(to + far, y);
      } else {
        *reinterpret_cast<uint4 *>(to) = qa[q];
      }
    }
    job += kThreads;
    if (job < p.Hq * per_head) {
      enter();
      fetch_q();
    }
  }
}

template <int NT, bool NEOX, int KIND>
psd_status launch(const ScaledParams &p, const Turns &turns, const DeviceInfo &dev, cudaStream_t s) {
  constexpr int NQ = NT < 2 ? NT : 2;
  const size_t shared = size_t(KIND == kQueries ? NQ : NT + p.block - 1) * size_t(p.a.rot) * 4;
  const int64_t kv_ctas = 2 * ((int64_t(p.a.T) - 1) / NT + 1), q_ctas = (int64_t(p.a.T) - 1) / NQ + 1;
  const int64_t ctas = KIND == kQueries ? q_ctas : KIND == kBlocks || p.a.Hq == 0 ? kv_ctas : kv_ctas + q_ctas;
  if (ctas > 0x7fffffffLL) return fail(PSD_ERR_UNSUPPORTED, "append_tokens_scaled: %d tokens", p.a.T);
  auto kern = append_scaled_kernel<NT, NEOX, KIND>;
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = dev.device < 64 ? uint64_t(1) << dev.device : 0;
  cudaError_t e = cudaSuccess;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (NT + kMaxBlock - 1) * kMaxPairs * 4);
    if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = KIND == kBlocks && p.a.Hq > 0 ? 1 : 0;  // K and V start while the queries end, and wait for that at their end
  e = cudaLaunchKernelEx(&cfg, kern, p, turns);
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "append_tokens_scaled launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}

template <bool NEOX>
psd_status launch_all(const ScaledParams &p, const Turns &turns, const DeviceInfo &dev, cudaStream_t s) {
  // One launch while its CTAs fit on the SMs at once.
  if (p.a.T <= 2 * dev.num_sms) return launch<1, NEOX, kAllParts>(p, turns, dev, s);
  const psd_status st = p.a.Hq ? launch<kMany, NEOX, kQueries>(p, turns, dev, s) : PSD_OK;
  return st != PSD_OK ? st : launch<kMany, NEOX, kBlocks>(p, turns, dev, s);
}

}  // namespace

psd_status check_scales(const char *what, const psd_block_scales *scales, int32_t page_size, int32_t kv_dtype, float k_scale,
                        float v_scale) {
  if (!scales) return fail(PSD_ERR_INVALID_ARG, "%s: NULL scales", what);
  if (scales->block != 16 && scales->block != 32 && scales->block != 64)
    return fail(PSD_ERR_INVALID_ARG, "%s: blocks of 16, 32 or 64 tokens, not %d", what, scales->block);
  if (page_size < 1 || page_size % scales->block)
    return fail(PSD_ERR_INVALID_ARG, "%s: page_size %d is no multiple of the block, %d", what, page_size, scales->block);
  if (kv_dtype != PSD_FP8_E4M3) return fail(PSD_ERR_INVALID_ARG, "%s: scaled blocks are e4m3 (kv_dtype %d)", what, kv_dtype);
  if (k_scale != 1.f || v_scale != 1.f)
    return fail(PSD_ERR_INVALID_ARG, "%s: k_scale and v_scale must be 1 beside the blocks' scales", what);
  return PSD_OK;
}

}  // namespace psd

using namespace psd;

extern "C" psd_status append_tokens_scaled(psd_ctx *ctx, const psd_append_args *a, const psd_block_scales *scales,
                                           psd_stream_t stream) {
  clear_error();
  if (!ctx || !a) return fail(PSD_ERR_INVALID_ARG, "append_tokens_scaled: NULL");
  bool none;
  psd_status st = check_append("append_tokens_scaled", a, &none);
  if (st != PSD_OK) return st;
  st = check_scales("append_tokens_scaled", scales, a->page_size, a->kv_dtype, a->k_scale, a->v_scale);
  if (st != PSD_OK || none) return st;
  if (!scales->k || !scales->v) return fail(PSD_ERR_INVALID_ARG, "append_tokens_scaled: NULL scales");
  auto fits = [](const void *ptr, int64_t stride) { return aligned16(ptr) && stride % 8 == 0; };
  if (a->D % 8 || a->D > 256 || a->Dv < 8 || a->Dv % 8 || a->Dv > 256 || a->rot_dim % 16 || a->rot_col % 8)
    return fail(PSD_ERR_UNSUPPORTED, "append_tokens_scaled: D %d and Dv %d multiples of 8 up to 256, rot_dim %d of 16, rot_col %d of 8",
                a->D, a->Dv, a->rot_dim, a->rot_col);
  if (!fits(a->q, a->Hq ? a->q_stride : 0) || !fits(a->k, a->k_stride) || !fits(a->v, a->v_stride) || !aligned16(a->q_out) ||
      !aligned16(a->k_pool) || !aligned16(a->v_pool))
    return fail(PSD_ERR_UNSUPPORTED, "append_tokens_scaled: tensors must be 16-byte aligned, strides multiples of 8");
  DeviceGuard g(ctx->dev.device);
  ScaledParams p;
  p.a = append_params(a);
  p.k_scales = scales->k;
  p.v_scales = scales->v;
  p.block = scales->block;
  const Turns turns = append_turns(a);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a->neox ? launch_all<true>(p, turns, ctx->dev, s) : launch_all<false>(p, turns, ctx->dev, s);
}
