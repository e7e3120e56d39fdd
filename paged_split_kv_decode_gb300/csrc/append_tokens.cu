// Rotation and append of several new tokens a request: queries and keys rotated by their
// positions, K and V rows written to the pages the device page table names.
//
// Angles.  a = pos * f must be right modulo one turn at far positions, where an f32
// product has lost it (pos 1e6 at f = 1: ulp 2^-4 rad).  The host gives each frequency as
// a fraction of a turn in 64-bit fixed point, F = f / (2 pi) * 2^64 mod 2^64, and the
// kernel multiplies in integers: pos * F wraps at whole turns by itself, and its top bits
// read as a signed number are the angle in (-1/2, 1/2] turns.  F carries the 53 bits of f,
// so the angle is off by at most pos * f * 2^-53 (1e-10 rad at pos 1e6), and the f32
// sine and cosine of it by their own rounding.  No table is read: a cos/sin table of
// 128 K positions and 64 frequencies is 64 MB, and each token would read 512 B of it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "append.cuh"

namespace psd {

namespace {

constexpr int kCtasPerSm = 5;   // of the 16-byte form: 48 registers a thread

__device__ __forceinline__ void put(void *pool, int64_t at, float v, bool fp8, float scale) {
  if (fp8)
    static_cast<uint8_t *>(pool)[at] = e4m3_of(__fdiv_rn(v, scale));
  else
    static_cast<__nv_bfloat16 *>(pool)[at] = __float2bfloat16_rn(v);
}

// One CTA per token, element by element: any width, stride and alignment.
// (8502 tokens, 32 query and 8 KV heads of 128, 20 columns rotated: 157 us, 1.3 TB/s; issue bounds it.)
__global__ void __launch_bounds__(256)
    append_tokens_kernel(const AppendParams p, const __grid_constant__ Turns turns) {
  __shared__ float2 cs[kMaxPairs];
  const int t = blockIdx.x;
  uint32_t faults;
  const Place x = place_of(p, t, faults);
  if (faults && threadIdx.x == 0) atomicOr(p.fault, int32_t(faults));
  if (x.pos < 0) return;
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < half; i += blockDim.x) cs[i] = turn(turns.f[i], x.pos, p.magnitude);
  __syncthreads();
  // One rotated or copied column pair; the first element of pair i of a head of width D.
  // Columns outside the rotation are visited singly as (d, d).
  const int units = half + (p.D - p.rot);
  auto head = [&](const __nv_bfloat16 *src, int u, int &a, int &b, float &xo, float &yo) {
    if (u < half) {
      a = p.rot_col + (p.neox ? u : 2 * u);
      b = p.rot_col + (p.neox ? u + half : 2 * u + 1);
      const float xi = __bfloat162float(src[a]), yi = __bfloat162float(src[b]);
      xo = xi * cs[u].x - yi * cs[u].y;
      yo = yi * cs[u].x + xi * cs[u].y;
    } else {
      a = u - half;
      if (a >= p.rot_col) a += p.rot;
      b = a;
      xo = yo = __bfloat162float(src[a]);
    }
  };
  for (int j = threadIdx.x; j < p.Hq * units; j += blockDim.x) {
    const int h = j / units;
    int a, b;
    float xo, yo;
    head(p.q + t * p.q_stride + int64_t(h) * p.D, j - h * units, a, b, xo, yo);
    __nv_bfloat16 *dst = p.q_out + (int64_t(t) * p.Hq + h) * p.D;
    dst[a] = __float2bfloat16_rn(xo);
    dst[b] = __float2bfloat16_rn(yo);
  }
  if (x.slot < 0) return;
  for (int j = threadIdx.x; j < p.Hkv * units; j += blockDim.x) {
    const int h = j / units;
    int a, b;
    float xo, yo;
    head(p.k + t * p.k_stride + int64_t(h) * p.D, j - h * units, a, b, xo, yo);
    const int64_t row = (x.slot * p.Hkv + h) * p.D;
    put(p.k_pool, row + a, xo, p.fp8 != 0, p.k_scale);
    put(p.k_pool, row + b, yo, p.fp8 != 0, p.k_scale);
  }
  const int nv = p.Hkv * p.Dv;
  for (int j = threadIdx.x; j < nv; j += blockDim.x)
    put(p.v_pool, x.slot * nv + j, __bfloat162float(p.v[t * p.v_stride + j]), p.fp8 != 0, p.v_scale);
}

// ------------------------------------------------------------------ 16-byte form
// NT consecutive tokens per CTA, 8 pairs or 8 columns a thread and access.  A thread takes
// the same columns of all NT tokens, so that index arithmetic is paid once and NT loads
// are in flight; the first queries are on their way while the places and angles are found.
// Keys start at the threads that the queries' last round left idle, copies after those: the
// phases of a CTA overlap (9800 tokens 42.9 us against 47.5 with each phase from thread 0 on, and
// with 64 of 128 columns rotated and fp8 pools 49.5 against 68.5).
// 32 query and 8 KV heads of 128, cold caches: one token 7 us (a chain of dependent loads:
// lengths, page id, frequencies, rows), 160 tokens into fp8 pools 9 us, 10784 tokens 48 us (265 MB at
// 5.5 TB/s, writes and reads mixed).
struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 unpack8(uint4 w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  F8 f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f.v[2 * k] = bf16_lo(u[k]);
    f.v[2 * k + 1] = bf16_hi(u[k]);
  }
  return f;
}
__device__ __forceinline__ uint4 pack8(const F8 &f) {
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __nv_bfloat162 x = __floats2bfloat162_rn(f.v[2 * k], f.v[2 * k + 1]);
    u[k] = *reinterpret_cast<uint32_t *>(&x);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
// Eight values at element `at` of a pool.
__device__ __forceinline__ void put8(void *pool, int64_t at, const F8 &f, bool fp8, float scale) {
  if (!fp8) {
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(pool) + at) = pack8(f);
    return;
  }
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(__fdiv_rn(f.v[4 * k + 1], scale)), "f"(__fdiv_rn(f.v[4 * k], scale)));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(__fdiv_rn(f.v[4 * k + 3], scale)), "f"(__fdiv_rn(f.v[4 * k + 2], scale)));
    w[k] = uint32_t(lo) | (uint32_t(hi) << 16);
  }
  *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(pool) + at) = make_uint2(w[0], w[1]);
}

template <int NT>
__global__ void __launch_bounds__(256, kCtasPerSm)
    append_tokens_vec_kernel(const AppendParams p, const __grid_constant__ Turns turns) {
  __shared__ __align__(16) float cosine[NT][kMaxPairs], sine[NT][kMaxPairs];
  __shared__ Place places[NT];
  const int t0 = blockIdx.x * NT, tid = threadIdx.x;
  const int half = p.rot / 2, groups = half / 8;          // 8-pair groups of a head
  const int rest = (p.D - p.rot) / 8;                     // 8-column chunks outside the rotation
  const bool neox = p.neox != 0, fp8 = p.fp8 != 0;
  // Group g of a head: its two runs of 8 columns start at a and a + far.
  const int far = neox ? half : 8;
  auto column = [&](int g) { return p.rot_col + (neox ? 8 * g : 16 * g); };
  auto load = [&](uint4 (&x)[NT][2], const __nv_bfloat16 *src, int64_t stride, int col) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 *at = reinterpret_cast<const uint4 *>(src + (t0 + n) * stride + col);
      if (t0 + n < p.T) {
        x[n][0] = *at;
        x[n][1] = *reinterpret_cast<const uint4 *>(src + (t0 + n) * stride + col + far);
      }
    }
  };
  // Rotates token n's group g in place: f0 and f1 are its two runs.
  auto rotate = [&](int n, int g, F8 &f0, F8 &f1) {
    float c[8], s[8];
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      *reinterpret_cast<float4 *>(c + k) = *reinterpret_cast<const float4 *>(&cosine[n][8 * g + k]);
      *reinterpret_cast<float4 *>(s + k) = *reinterpret_cast<const float4 *>(&sine[n][8 * g + k]);
    }
    if (neox) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = f0.v[k], y = f1.v[k];
        f0.v[k] = x * c[k] - y * s[k];
        f1.v[k] = y * c[k] + x * s[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = f0.v[2 * k], y = f0.v[2 * k + 1], z = f1.v[2 * k], w = f1.v[2 * k + 1];
        f0.v[2 * k] = x * c[k] - y * s[k];
        f0.v[2 * k + 1] = y * c[k] + x * s[k];
        f1.v[2 * k] = z * c[k + 4] - w * s[k + 4];
        f1.v[2 * k + 1] = w * c[k + 4] + z * s[k + 4];
      }
    }
  };

  const int nq = p.Hq * groups;
  uint4 x[NT][2];
  int j = tid, h = j / groups, col = column(j - h * groups);
  if (j < nq) load(x, p.q + int64_t(h) * p.D, p.q_stride, col);
  for (int n = tid >> 5; n < NT; n += 8) {                 // a warp per token
    uint32_t faults = 0;
    Place at{-1, -1};
    if (t0 + n < p.T) at = place_of(p, t0 + n, faults);
    if ((tid & 31) == 0) {
      places[n] = at;
      if (faults) atomicOr(p.fault, int32_t(faults));
    }
  }
  __syncthreads();
  for (int i = tid; i < NT * half; i += 256) {
    const int n = i / half, k = i - n * half;
    const float2 cs = places[n].pos >= 0 ? turn(turns.f[k], places[n].pos, p.magnitude) : make_float2(0.f, 0.f);
    cosine[n][k] = cs.x;
    sine[n][k] = cs.y;
  }
  __syncthreads();
  // ---- queries
  while (j < nq) {
    const int g = j - h * groups;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (places[n].pos < 0) continue;
      F8 f0 = unpack8(x[n][0]), f1 = unpack8(x[n][1]);
      rotate(n, g, f0, f1);
      __nv_bfloat16 *dst = p.q_out + (int64_t(t0 + n) * p.Hq + h) * p.D + col;
      *reinterpret_cast<uint4 *>(dst) = pack8(f0);
      *reinterpret_cast<uint4 *>(dst + far) = pack8(f1);
    }
    j += 256;
    if (j >= nq) break;
    h = j / groups;
    col = column(j - h * groups);
    load(x, p.q + int64_t(h) * p.D, p.q_stride, col);
  }
  // ---- keys
  const int nk = p.Hkv * groups;
  for (j = (tid - nq) & 255; j < nk; j += 256) {  // the threads the queries left idle first
    h = j / groups;
    const int g = j - h * groups;
    col = column(g);
    load(x, p.k + int64_t(h) * p.D, p.k_stride, col);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const Place at = places[n];
      if (at.pos < 0 || at.slot < 0) continue;
      F8 f0 = unpack8(x[n][0]), f1 = unpack8(x[n][1]);
      rotate(n, g, f0, f1);
      const int64_t dst = (at.slot * p.Hkv + h) * p.D + col;
      put8(p.k_pool, dst, f0, fp8, p.k_scale);
      put8(p.k_pool, dst + far, f1, fp8, p.k_scale);
    }
  }
  // ---- columns outside the rotation, and V
  const int cq = p.Hq * rest, ck = p.Hkv * rest, cv = p.Hkv * p.Dv / 8;
  for (j = (tid - nq - nk) & 255; j < cq + ck + cv; j += 256) {
    const bool is_q = j < cq, is_k = !is_q && j < cq + ck;
    const int i = is_q ? j : is_k ? j - cq : j - cq - ck;
    int64_t off;  // in the token's heads
    if (is_q || is_k) {
      h = i / rest;
      col = 8 * (i - h * rest);
      if (col >= p.rot_col) col += p.rot;
      off = int64_t(h) * p.D + col;
    } else {
      off = 8 * int64_t(i);
    }
    const __nv_bfloat16 *src = (is_q ? p.q : is_k ? p.k : p.v) + off;
    const int64_t stride = is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride;
    uint4 y[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (t0 + n < p.T) y[n] = *reinterpret_cast<const uint4 *>(src + (t0 + n) * stride);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const Place at = places[n];
      if (at.pos < 0) continue;
      if (is_q) *reinterpret_cast<uint4 *>(p.q_out + int64_t(t0 + n) * p.Hq * p.D + off) = y[n];
      else if (at.slot < 0) continue;
      else if (is_k) put8(p.k_pool, at.slot * p.Hkv * p.D + off, unpack8(y[n]), fp8, p.k_scale);
      else put8(p.v_pool, at.slot * p.Hkv * p.Dv + off, unpack8(y[n]), fp8, p.v_scale);
    }
  }
}

}  // namespace

static psd_status launch_append_tokens(const psd_append_args *a, int sms, cudaStream_t s) {
  const AppendParams p = append_params(a);
  const Turns turns = append_turns(a);
  auto fits = [](const void *ptr, int64_t stride) { return aligned16(ptr) && stride % 8 == 0; };
  const bool vec = a->rot_dim % 16 == 0 && a->rot_col % 8 == 0 && a->D % 8 == 0 && a->Dv % 8 == 0 &&
                   fits(a->q, a->Hq ? a->q_stride : 0) && fits(a->k, a->k_stride) && fits(a->v, a->Dv ? a->v_stride : 0) &&
                   aligned16(a->q_out) && aligned16(a->k_pool) && aligned16(a->v_pool);
  // One token a CTA while all of them fit on the SMs at once, two beyond: 608 tokens 7.6 us against 8.2,
  // 1218 tokens 10.7 against 9.3, 9800 tokens 47.8 against 42.9 (four: 46.8; registers).
  constexpr int kMany = 2;
  if (!vec) append_tokens_kernel<<<a->num_tokens, 256, 0, s>>>(p, turns);
  else if (a->num_tokens <= kCtasPerSm * sms) append_tokens_vec_kernel<1><<<a->num_tokens, 256, 0, s>>>(p, turns);
  else append_tokens_vec_kernel<kMany><<<(a->num_tokens - 1) / kMany + 1, 256, 0, s>>>(p, turns);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "append_tokens launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}

}  // namespace psd

using namespace psd;

extern "C" psd_status append_tokens(psd_ctx *ctx, const psd_append_args *a, psd_stream_t stream) {
  clear_error();
  if (!ctx || !a) return fail(PSD_ERR_INVALID_ARG, "append_tokens: NULL");
  bool none;
  const psd_status st = check_append("append_tokens", a, &none);
  if (st != PSD_OK || none) return st;
  DeviceGuard g(ctx->dev.device);
  return launch_append_tokens(a, ctx->dev.num_sms, reinterpret_cast<cudaStream_t>(stream));
}
