// append_tokens into a cache of 8-bit blocks with a scale each (the contract is in include/psd.h).
//
// Mathematics.  The scale of a block is the least power of two that brings its largest magnitude within e4m3's
// 448 = 1.75 2^8: with A = f 2^E, f in [1, 2), that is 2^(E - 8), or 2^(E - 7) where f > 1.75, read off A's bits.
// x 2^-k is exact in f32, so a code is rounded once.  A block that holds older tokens keeps its scale or takes a
// larger one; older codes then go down by a power of two, which rounds only what falls below 2^-6.
//
// A CTA has NT tokens: it rotates their queries, and it writes the blocks whose first new token is one of them,
// the tokens of such a block behind its own NT included.  So every block has one writer, whatever the lengths,
// without a list of blocks and without atomics on scales.  A warp takes one block of one head's K or V: D / 8
// lanes a token.
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

__device__ __forceinline__ Token locate(const ScaledParams &s, int t, uint32_t &faults) {
  const AppendParams &p = s.a;
  Token x{-1, 0, 0, -1};
  faults = 0;
  if (t >= __ldg(p.q_indptr + p.B)) return x;  // behind the last request
  const int b = request_of(p.q_indptr, p.B, t);
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
  if (t == begin || x.older == 0) x.count = min(s.block - x.older, end - t);
  return x;
}

struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 load8(const __nv_bfloat16 *src) {
  const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src));
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
// The least e with top <= 448 2^(e - 127), top >= 0 finite.
__device__ __forceinline__ int scale_of(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = int(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
  return max(e, kLeast);
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 4) append_scaled_kernel(const ScaledParams s, const __grid_constant__ Turns turns) {
  extern __shared__ __align__(16) float table[];  // cosines [tokens][half], then sines
  __shared__ Token tokens[NT];
  __shared__ int pos[NT + kMaxBlock];
  __shared__ int n_table;
  const AppendParams &p = s.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t0 = blockIdx.x * NT;
  const int half = p.rot / 2;
  for (int n = warp; n < NT; n += kWarps) {
    uint32_t faults = 0;
    Token x{-1, 0, 0, -1};
    if (t0 + n < p.T) x = locate(s, t0 + n, faults);
    if (lane == 0) {
      tokens[n] = x;
      if (faults) atomicOr(p.fault, int32_t(faults));
    }
  }
  __syncthreads();
  if (warp == 0) {
    // the tokens whose angles are needed: its own, and those of its last block behind them
    int most = NT;
    for (int n = lane; n < NT; n += 32)
      if (tokens[n].slot >= 0) most = max(most, n + tokens[n].count);
    most = __reduce_max_sync(0xffffffffu, most);
    for (int n = lane; n < most; n += 32) {
      if (n < NT) {
        pos[n] = tokens[n].pos;
      } else {  // of the request of the last block that starts here
        int at = -1;
        if (p.positions) {
          at = __ldg(p.positions + t0 + n);
        } else {
          for (int i = NT - 1; i >= 0; --i)
            if (tokens[i].count > n - i) {
              at = tokens[i].pos + (n - i);
              break;
            }
        }
        pos[n] = max(at, -1);
      }
    }
    if (lane == 0) n_table = most;
  }
  __syncthreads();
  const int nt = n_table;
  float *cosine = table, *sine = table + nt * half;
  for (int i = tid; i < nt * half; i += kThreads) {
    const int n = i / half, k = i - n * half;
    const float2 cs = pos[n] >= 0 ? turn(turns.f[k], pos[n], p.magnitude) : make_float2(0.f, 0.f);
    cosine[i] = cs.x;
    sine[i] = cs.y;
  }
  __syncthreads();

  // ---- blocks: K of head h, or V of it
  const int units = NT * 2 * p.Hkv;
  for (int u = warp; u < units; u += kWarps) {
    const int n = u / (2 * p.Hkv), r = u - n * 2 * p.Hkv;
    const Token x = tokens[n];
    if (x.slot < 0 || x.count == 0) continue;
    const bool is_v = r >= p.Hkv;
    const int h = is_v ? r - p.Hkv : r, W = is_v ? p.Dv : p.D;
    const int lanes = W / 8, a_pass = 32 / lanes;        // lanes a token, tokens a pass
    const int mine = lane / lanes, col = 8 * (lane - mine * lanes);
    const bool working = mine < a_pass;
    const __nv_bfloat16 *src = is_v ? p.v + int64_t(h) * W : p.k + int64_t(h) * W;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const int i0 = col - p.rot_col;                      // of the rotated columns
    const bool turned = !is_v && i0 >= 0 && i0 < p.rot;
    // Columns col .. col + 7 of token n + i.
    auto value = [&](int i) {
      const __nv_bfloat16 *at = src + (t0 + n + i) * stride;
      F8 f = load8(at + col);
      if (!turned) return f;
      const float *c = cosine + (n + i) * half, *sn = sine + (n + i) * half;
      if (p.neox) {
        const bool low = i0 < half;
        const int k0 = low ? i0 : i0 - half;
        const F8 g = load8(at + (low ? col + half : col - half));
#pragma unroll
        for (int k = 0; k < 8; ++k) f.v[k] = low ? f.v[k] * c[k0 + k] - g.v[k] * sn[k0 + k] : f.v[k] * c[k0 + k] + g.v[k] * sn[k0 + k];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = f.v[2 * k], b = f.v[2 * k + 1], cc = c[i0 / 2 + k], ss = sn[i0 / 2 + k];
          f.v[2 * k] = a * cc - b * ss;
          f.v[2 * k + 1] = b * cc + a * ss;
        }
      }
      return f;
    };
    bool any = false;  // of the tokens is appended
    for (int i = lane; i < x.count; i += 32) any |= pos[n + i] >= 0;
    if (!__any_sync(0xffffffffu, any)) continue;
    float top = 0.f;
    for (int i = mine; working && i < x.count; i += a_pass) {
      if (pos[n + i] < 0) continue;
      const F8 f = value(i);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float m = fabsf(f.v[k]);
        if (m < __int_as_float(0x7f800000)) top = fmaxf(top, m);
      }
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    const int64_t first = x.slot - x.older;              // the block's first row
    uint8_t *scale = (is_v ? s.v_scales : s.k_scales) + first / s.block * p.Hkv + h;
    uint8_t *pool = static_cast<uint8_t *>(is_v ? p.v_pool : p.k_pool) + (first * p.Hkv + h) * W + col;
    int e = scale_of(top);
    if (x.older > 0) {
      const int had = *scale;
      if (e > had) {
        const float down = ex2(float(had - e));          // (0 below 2^-126)
        for (int i = mine; working && i < x.older; i += a_pass) {
          uint2 *at = reinterpret_cast<uint2 *>(pool + int64_t(i) * p.Hkv * W);
          *at = codes8(values8(*at), down);
        }
      }
      e = max(e, had);
    }
    __syncwarp();
    if (lane == 0) *scale = uint8_t(e);
    const float by = __uint_as_float(uint32_t(254 - min(e, 253)) << 23);
    for (int i = mine; working && i < x.count; i += a_pass) {
      if (pos[n + i] < 0) continue;
      *reinterpret_cast<uint2 *>(pool + int64_t(x.older + i) * p.Hkv * W) = codes8(value(i), by);
    }
  }

  // ---- queries: both runs of 8 columns of a group of pairs (q_out may be q), then the rest
  const int groups = half / 8, rest = (p.D - p.rot) / 8, far = p.neox ? half : 8;
  const int per_head = groups + rest, per_token = p.Hq * per_head;
  for (int j = tid; j < NT * per_token; j += kThreads) {
    const int n = j / per_token, m = j - n * per_token, h = m / per_head, g = m - h * per_head;
    if (pos[n] < 0) continue;
    const __nv_bfloat16 *src = p.q + (t0 + n) * p.q_stride + int64_t(h) * p.D;
    __nv_bfloat16 *dst = p.q_out + (int64_t(t0 + n) * p.Hq + h) * p.D;
    if (g >= groups) {
      int col = 8 * (g - groups);
      if (col >= p.rot_col) col += p.rot;
      *reinterpret_cast<uint4 *>(dst + col) = *reinterpret_cast<const uint4 *>(src + col);
      continue;
    }
    const int col = p.rot_col + (p.neox ? 8 * g : 16 * g);
    const float *c = cosine + n * half + 8 * g, *sn = sine + n * half + 8 * g;
    F8 a = load8(src + col), b = load8(src + col + far);
    if (p.neox) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = a.v[k], y = b.v[k];
        a.v[k] = x * c[k] - y * sn[k];
        b.v[k] = y * c[k] + x * sn[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = a.v[2 * k], y = a.v[2 * k + 1], z = b.v[2 * k], w = b.v[2 * k + 1];
        a.v[2 * k] = x * c[k] - y * sn[k];
        a.v[2 * k + 1] = y * c[k] + x * sn[k];
        b.v[2 * k] = z * c[k + 4] - w * sn[k + 4];
        b.v[2 * k + 1] = w * c[k + 4] + z * sn[k + 4];
      }
    }
    store8(dst + col, a);
    store8(dst + col + far, b);
  }
}

template <int NT>
psd_status launch(const ScaledParams &p, const Turns &turns, const DeviceInfo &dev, cudaStream_t s) {
  const size_t shared = size_t(NT + p.block - 1) * size_t(p.a.rot) * 4;
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = dev.device < 64 ? uint64_t(1) << dev.device : 0;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(append_scaled_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (NT + kMaxBlock - 1) * kMaxPairs * 4);
    if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    ready.fetch_or(bit, std::memory_order_release);
  }
  append_scaled_kernel<NT><<<(p.a.T - 1) / NT + 1, kThreads, shared, s>>>(p, turns);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "append_tokens_scaled launch: %s", cudaGetErrorString(e));
  return PSD_OK;
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
  return a->num_tokens <= 4 * ctx->dev.num_sms ? launch<1>(p, turns, ctx->dev, s) : launch<kMany>(p, turns, ctx->dev, s);
}
