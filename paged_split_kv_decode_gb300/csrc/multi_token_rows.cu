// Attention of few rows (a request's new tokens times the G query heads of a KV head, at most 32) over a cache of
// 8-bit blocks with a scale each: single tokens and short drafts, where reading the cache is all the work.
//
// Mathematics.  S^T = K Q^T and O^T += V^T P^T, keys and columns as the rows of mma.sync m16n8k16 (f16, f32 sums),
// query rows as its 8 columns: 8 rows fill an MMA, where S = Q K^T would take 16.  e4m3 codes become f16 exactly.
// Which columns a lane takes is free as long as Q and K agree, so each lane's 16 bytes of a key are its operands as
// they lie: no shuffles, no transposition of K; V's bytes are paired by one permute for four codes.
//   K's scale 2^a multiplies the scores of its block's 16 keys.  V's 2^b goes into P: P' = P 2^(b - r), r the largest b
// so far (O follows when r grows), so that P' <= P and f16 holds it to 2^-12 of itself down to b = r - 21 and
// beyond that to 2^-32 of the row's largest; the sum l is of P.  The row maximum follows lazily, as in the
// tensor-core kernel for many rows: P <= 2^15, and O and l are rescaled only when it grows by more than 2^8.
// f32 outputs take P' as two f16 terms (2^-22).
//
// Bytes: a key's row of a head is 64 or 128 bytes, and a step of a warp is 16 keys.  Each lane copies (cp.async) the
// very bytes that it will use into its own slots of a ring and reads only those: a warp's ring needs no barrier.
// Three steps of 4 KB a warp, 16 warps an SM, are 192 KB on their way; DRAM at its full rate wants about 50.
//
// Split: the steps of all units (request, KV head) lie on one line, and each CTA takes a stretch of it that costs the
// same; its eight warps take a unit's steps in turn and join their O through shared memory.  A unit that a stretch's
// bound cuts leaves normalised pieces, which a second kernel joins in key order.  Nothing is added atomically.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "device.cuh"
#include "multi_token.h"

namespace psd {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kStep = 16;        // keys
constexpr int kMaxCtas = 384;
constexpr float kLazy = 8.f, kBias = 7.f;  // log2 units: P's top is 2^7, and grows to 2^15 at most
constexpr int kUnitCost = 12;    // of a unit beside its steps, in steps

template <int D, int NT>
struct Lay {
  static constexpr int kCtasPerSm = NT <= 2 ? 2 : 1;
  static constexpr int kStages = NT <= 2 ? 3 : 6;
  static constexpr uint32_t kStageBytes = 2 * kStep * D;
  static constexpr uint32_t kOffMeta = kWarps * kStages * kStageBytes;  // a stage's scales: two words and a shift
  static constexpr uint32_t kOffStats = kOffMeta + kWarps * kStages * 16;
  static constexpr uint32_t kOffRef = kOffStats + kWarps * 8 * NT * 8;
  static constexpr uint32_t kOffQ = kOffRef + kWarps * 4;               // NT > 1: Q as operands
  static constexpr uint32_t kOffJoin = kOffQ + (NT > 1 ? NT * (D / 16) * 32 * 8 : 0);
  static constexpr uint32_t kSmem = kOffJoin + kWarps * 8 * 32 * 4;
  static_assert(kCtasPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory");
};

struct RowsParams {
  const __nv_bfloat16 *q;
  const uint8_t *k_pool, *v_pool, *k_scales, *v_scales;
  const int32_t *page_indices;
  const uint64_t *tree;
  void *o;
  float *lse;
  float *part_o, *part_lse;  // [CTAs][2][rows of a unit][D], and without D
  FaultRef fault;
  int64_t q_stride, num_pages, num_scales;
  int Hq, Hkv, G, page_size, shift, out_f32;
  float q_scale;
};
struct Start {
  uint16_t b, kv;  // request, KV head
  int32_t j;       // first step of the unit
  int32_t steps;   // of the stretch
};
struct RowsRequests {
  psd_token_request r[kStepRequests];
  Start start[kMaxCtas];
};

// A stretch's part of one unit.
struct Segment {
  int b, kv, s0, s1, n;
  bool first;
};
struct Walk {
  const RowsRequests &req;
  int left, b, kv, j, heads;
  bool first = true;
  __device__ Walk(const RowsRequests &r, int Hkv) : req(r), heads(Hkv) {
    const Start &s = req.start[blockIdx.x];
    left = s.steps, b = s.b, kv = s.kv, j = s.j;
  }
  __device__ bool next(Segment &g) {
    if (left == 0) return false;
    g.b = b, g.kv = kv, g.s0 = j, g.first = first;
    g.n = (req.r[b].kv_len + kStep - 1) / kStep;
    g.s1 = min(g.n, j + left);
    left -= g.s1 - g.s0;
    first = false;
    j = 0;
    if (++kv == heads) kv = 0, ++b;
    return true;
  }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, uint32_t bytes) {  // the rest reads as 0
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four codes to two pairs of f16.
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <int D, int NT, int TERMS>
__global__ void __launch_bounds__(kThreads, Lay<D, NT>::kCtasPerSm)
    rows_kernel(const RowsParams p, const __grid_constant__ RowsRequests req) {
  using L = Lay<D, NT>;
  constexpr int NS = L::kStages, kHalves = D / 64, kMmas = D / 16;  // MMAs of S for 16 keys; of O as many
  extern __shared__ __align__(128) uint8_t sm[];
  dependents_may_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(sm) + warp * NS * L::kStageBytes;
  const uint8_t *ring_at = sm + warp * NS * L::kStageBytes;
  const uint32_t meta = smem_u32(sm) + L::kOffMeta + warp * NS * 16;
  const int64_t row_bytes = int64_t(p.Hkv) * D;  // between a head's rows of neighbouring slots
  uint32_t bad = 0;

  // ------------------------------------------------------------------------------ copies
  // The steps to be copied run NS - 1 ahead of those worked on, across the units' ends.
  Walk ahead(req, p.Hkv);
  Segment from;
  bool more = ahead.next(from);
  int at = more ? from.s0 + warp : 0;
  int ids = -1, ids_at = -1;  // page ids of 32 of the warp's steps, one a lane, from step ids_at on
  auto issue = [&](int stage) {
    while (more && at >= from.s1) {
      more = ahead.next(from);
      at = from.s0 + warp;
      ids_at = -1;
    }
    if (more) {
      const psd_token_request &r = req.r[from.b];
      if (ids_at < 0 || at >= ids_at + 32 * kWarps) {
        ids_at = at;
        const int mine = at + lane * kWarps;
        ids = mine < from.s1 ? __ldg(p.page_indices + r.page_off + mine * kStep / p.page_size) : 0;
        if (ids < 0 || int64_t(ids) >= p.num_pages) {
          bad |= PSD_FAULT_PAGE_ID;
          ids = -1;
        }
      }
      const int id = __shfl_sync(0xffffffffu, ids, (at - ids_at) / kWarps);
      const uint32_t dst = ring + stage * L::kStageBytes;
      // a page that is not there: its step is left out (a shift of 32 says so)
      uint32_t shift = 32;
      if (id >= 0) {
        const int64_t slot = int64_t(id) * p.page_size + at * kStep % p.page_size;
        const int64_t base = slot * row_bytes + int64_t(from.kv) * D;
        const uint8_t *k = p.k_pool + base, *v = p.v_pool + base;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            copy16(dst + (t * kHalves + h) * 512 + lane * 16, k + (g + 8 * t) * row_bytes + 64 * h + 16 * c);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int key = 2 * c + (t & 1) + 8 * (t >> 1);
          if constexpr (D == 128) copy16(dst + kStep * D + t * 512 + lane * 16, v + key * row_bytes + 16 * g);
          else copy8(dst + kStep * D + t * 256 + lane * 8, v + key * row_bytes + 8 * g);
        }
        const int64_t scale = (slot >> p.shift) * p.Hkv + from.kv, word = scale & ~int64_t(3);
        shift = uint32_t(scale & 3) * 8;
        if (lane < 2)
          copy4(meta + stage * 16 + 4 * lane, (lane ? p.v_scales : p.k_scales) + word, uint32_t(min(int64_t(4), p.num_scales - word)));
      }
      if (lane == 0) *reinterpret_cast<uint32_t *>(sm + L::kOffMeta + (warp * NS + stage) * 16 + 8) = shift;
      at += kWarps;
    }
    copies_end();
  };
  for (int s = 0; s < NS - 1; ++s) issue(s);

  // -------------------------------------------------------------------------------- units
  Walk walk(req, p.Hkv);
  Segment u;
  int stage = 0;
  while (walk.next(u)) {
    const psd_token_request r = req.r[u.b];
    const int start = r.kv_len - r.num_new, rows = r.num_new * p.G;
    const bool has_tree = p.tree != nullptr;
    // Q of row g of each tile, times the power of two that puts its top in [2^14, 2^15): exact but for
    // elements 2^-31 below the top.
    [[maybe_unused]] uint32_t qf[NT == 1 ? kMmas : 1][2];
    float qs[NT][2];  // score factors of rows 2 c and 2 c + 1
    uint2 *q_at = reinterpret_cast<uint2 *>(sm + L::kOffQ) + lane;  // NT > 1: [tile][MMA][lane]
    if constexpr (NT > 1) __syncthreads();  // the unit before is done with it
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (NT > 1 && nt % kWarps != warp) continue;
      const int row = 8 * nt + g;
      uint4 w[kHalves][2];
      const bool live = row < rows;
      const __nv_bfloat16 *src = p.q + (int64_t(r.token0) + (live ? row / p.G : 0)) * p.q_stride +
                                 (int64_t(u.kv) * p.G + (live ? row % p.G : 0)) * D + 16 * c;
      float top = 0.f;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[h][i] = live ? __ldg(reinterpret_cast<const uint4 *>(src + 64 * h) + i) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t y[4] = {w[h][i].x, w[h][i].y, w[h][i].z, w[h][i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(bf16_lo(y[k])), fabsf(bf16_hi(y[k]))));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the factor on the scores stays a normal number
      const int most = min(100, int((__float_as_uint(p.q_scale) >> 23) & 255u) - 1);
      const int e = max(-114, min(most, 14 - (int(__float_as_uint(top) >> 23) - 127)));
      const float f = __uint_as_float(uint32_t(127 + e) << 23);
      const float back = p.q_scale * __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // columns 64 h + 16 c + 4 i .. + 3
          const uint4 &x = w[h][i >> 1];
          const uint32_t lo = i & 1 ? x.z : x.x, hi = i & 1 ? x.w : x.y;
          const uint32_t b0 = f16x2_bits(bf16_lo(lo) * f, bf16_hi(lo) * f), b1 = f16x2_bits(bf16_lo(hi) * f, bf16_hi(hi) * f);
          if constexpr (NT == 1) qf[4 * h + i][0] = b0, qf[4 * h + i][1] = b1;
          else q_at[(nt * kMmas + 4 * h + i) * 32] = make_uint2(b0, b1);
        }
      if constexpr (NT == 1) {
        qs[0][0] = __shfl_sync(0xffffffffu, back, 8 * c);
        qs[0][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
      } else if (c == 0) {
        reinterpret_cast<float *>(sm + L::kOffStats)[8 * nt + g] = back;  // (free until the unit's end)
      }
    }
    if constexpr (NT > 1) {
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) qs[nt][i] = reinterpret_cast<const float *>(sm + L::kOffStats)[8 * nt + 2 * c + i];
      __syncthreads();
    }
    // Keys before this one are seen by all rows.
    const int clear = has_tree ? start : start + 1;
    float m[NT][2], l[NT][2], o[NT][kMmas][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = neg_inf();
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < kMmas; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
    }
    int ref = 0;  // V's largest scale byte so far
    for (int s = u.s0 + warp; s < u.s1; s += kWarps) {
      copies_wait<NS - 2>();
      __syncwarp();  // the scales came through other lanes
      const uint4 scales = *reinterpret_cast<const uint4 *>(sm + L::kOffMeta + (warp * NS + stage) * 16);
      const uint8_t *src = ring_at + stage * L::kStageBytes;
      if (scales.z < 32) {
        const uint32_t ke = (scales.x >> scales.z) & 255u, ve = (scales.y >> scales.z) & 255u;
        const float ks = scale_value(ke);
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const uint4 a = *reinterpret_cast<const uint4 *>(src + h * 512 + lane * 16);
          const uint4 b = *reinterpret_cast<const uint4 *>(src + (kHalves + h) * 512 + lane * 16);
          const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t f[4];
            widen(wa[i], f[0], f[2]);
            widen(wb[i], f[1], f[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (NT == 1) {
                mma(sc[nt], f, qf[4 * h + i][0], qf[4 * h + i][1]);
              } else {
                const uint2 b2 = q_at[(nt * kMmas + 4 * h + i) * 32];
                mma(sc[nt], f, b2.x, b2.y);
              }
            }
          }
        }
        const int j0 = s * kStep;
        const bool masked = j0 + kStep > clear;
        if (ve == 255 && ref == 0) ref = 127;  // (what it will be multiplied by must not be 0)
        if (ve > uint32_t(ref) && ve < 255) {  // the same in all lanes
          const float down = ref == 0 ? 0.f : ex2(float(ref) - float(ve));  // (O holds nothing yet, or is 0)
          ref = int(ve);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < kMmas; ++j)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[nt][j][x] *= down;
        }
        const float vf = ve == 255 ? scale_value(255) : ex2(float(ve) - float(ref));
        uint32_t pb[NT][TERMS][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float f0 = qs[nt][0] * ks, f1 = qs[nt][1] * ks;
          float z[4] = {sc[nt][0] * f0, sc[nt][1] * f1, sc[nt][2] * f0, sc[nt][3] * f1};
          if (masked) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int j = j0 + g + 8 * (x >> 1), row = 8 * nt + 2 * c + (x & 1);
              bool sees = row < rows && j < r.kv_len;
              if (sees && j >= start) {
                const int tok = row / p.G;
                sees = has_tree ? j - start < 64 && (__ldg(reinterpret_cast<const unsigned long long *>(p.tree) + r.token0 + tok) >> (j - start) & 1)
                                : j <= start + tok;
              }
              if (!sees) z[x] = neg_inf();
            }
          }
          const bool grow = fmaxf(z[0], z[2]) > m[nt][0] + (kBias + kLazy) || fmaxf(z[1], z[3]) > m[nt][1] + (kBias + kLazy);
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float top = fmaxf(z[i], z[2 + i]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              if (top > m[nt][i] + (kBias + kLazy)) {
                const float to = top - kBias, alpha = ex2(m[nt][i] - to);
                m[nt][i] = to;
                l[nt][i] *= alpha;
#pragma unroll
                for (int j = 0; j < kMmas; ++j) o[nt][j][i] *= alpha, o[nt][j][2 + i] *= alpha;
              }
            }
          }
          const float n0 = m[nt][0] == neg_inf() ? 0.f : m[nt][0], n1 = m[nt][1] == neg_inf() ? 0.f : m[nt][1];
          float e[4] = {ex2(z[0] - n0), ex2(z[1] - n1), ex2(z[2] - n0), ex2(z[3] - n1)};
          l[nt][0] += e[0] + e[2];
          l[nt][1] += e[1] + e[3];
#pragma unroll
          for (int x = 0; x < 4; ++x) e[x] = masked && e[x] == 0.f ? 0.f : e[x] * vf;  // (0 beside a scale of NaN: hidden)
#pragma unroll
          for (int y = 0; y < TERMS; ++y) {
            const uint32_t w0 = f16x2_bits(e[0], e[1]), w1 = f16x2_bits(e[2], e[3]);
            pb[nt][y][0] = transpose8(w0);
            pb[nt][y][1] = transpose8(w1);
            if (y + 1 < TERMS) {
              const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w0)), b = __half22float2(*reinterpret_cast<const __half2 *>(&w1));
              e[0] -= a.x, e[1] -= a.y, e[2] -= b.x, e[3] -= b.y;
            }
          }
        }
        // V: four keys a lane, D / 8 columns of each
        constexpr int kWords = D / 32;
        uint32_t v[4][kWords];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(src + kStep * D + t * 512 + lane * 16);
            v[t][0] = w.x, v[t][1] = w.y, v[t][2] = w.z, v[t][3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(src + kStep * D + t * 256 + lane * 8);
            v[t][0] = w.x, v[t][1] = w.y;
          }
        }
        if (j0 + kStep > r.kv_len) {  // slots behind the last token may hold anything, NaN included
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (j0 + 2 * c + (t & 1) + 8 * (t >> 1) >= r.kv_len)
#pragma unroll
              for (int i = 0; i < kWords; ++i) v[t][i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5140), a1 = __byte_perm(v[2][i], v[3][i], 0x5140);
          const uint32_t b0 = __byte_perm(v[0][i], v[1][i], 0x7362), b1 = __byte_perm(v[2][i], v[3][i], 0x7362);
          uint32_t f[4], h[4];
          widen(a0, f[0], f[1]);
          widen(a1, f[2], f[3]);
          widen(b0, h[0], h[1]);
          widen(b1, h[2], h[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < TERMS; ++y) {
              mma(o[nt][2 * i], f, pb[nt][y][0], pb[nt][y][1]);
              mma(o[nt][2 * i + 1], h, pb[nt][y][0], pb[nt][y][1]);
            }
        }
      }
      issue(stage ? stage - 1 : NS - 1);  // the stage before this one
      if (++stage == NS) stage = 0;
    }

    // ------------------------------------------------------------------------ the unit's end
    // Lane (g, c) holds columns D / 8 g .. of rows 2 c and 2 c + 1.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], x);
    float2 *stats = reinterpret_cast<float2 *>(sm + L::kOffStats);  // [warp][row]: m, l
    int *refs = reinterpret_cast<int *>(sm + L::kOffRef);
    float *join = reinterpret_cast<float *>(sm + L::kOffJoin);      // [warp][row of 8][lane]
    if (g == 0)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) stats[warp * 8 * NT + 8 * nt + 2 * c + i] = make_float2(m[nt][i], l[nt][i]);
    if (lane == 0) refs[warp] = ref;
    __syncthreads();
    const bool whole = u.s0 == 0 && u.s1 == u.n;
    const int64_t piece = int64_t(2 * blockIdx.x + (u.first ? 0 : 1)) * 8 * NT;
    const int jrow = tid >> 5;  // row of a tile that this thread joins
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (8 * nt >= rows) break;
      const int row = 8 * nt + jrow;
      float top = neg_inf(), all = 0.f, f[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[w * 8 * NT + row].x);
      const float base = top == neg_inf() ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 x = stats[w * 8 * NT + row];
        f[w] = ex2(x.x - base);
        all += x.y * f[w];
      }
      const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) f[w] = stats[w * 8 * NT + row].y == 0.f ? 0.f : f[w] * inv * scale_value(uint32_t(refs[w]));
      const bool live = row < rows;
      const int64_t out = (int64_t(r.token0) + row / p.G) * p.Hq + u.kv * p.G + row % p.G;
      const int64_t dst = (whole ? out : piece + row) * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float4 *to = reinterpret_cast<float4 *>(join + warp * 256);
        to[(2 * c) * 8 + g] = make_float4(o[nt][2 * i][0], o[nt][2 * i][2], o[nt][2 * i + 1][0], o[nt][2 * i + 1][2]);
        to[(2 * c + 1) * 8 + g] = make_float4(o[nt][2 * i][1], o[nt][2 * i][3], o[nt][2 * i + 1][1], o[nt][2 * i + 1][3]);
        __syncthreads();
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          y = fmaf(join[w * 256 + tid], f[w], y);
        }
        if (live) {
          const int64_t to_at = dst + (lane >> 2) * (D / 8) + 4 * i + (lane & 3);
          if (!whole) p.part_o[to_at] = y;
          else if (p.out_f32) static_cast<float *>(p.o)[to_at] = y;
          else static_cast<__nv_bfloat16 *>(p.o)[to_at] = __float2bfloat16_rn(y);
        }
        __syncthreads();
      }
      if (live && lane == 0) {
        const float v = all == 0.f ? neg_inf() : top + log2f(all);
        if (!whole) p.part_lse[piece + row] = v;
        else if (p.lse) p.lse[out] = v;
      }
    }
    __syncthreads();  // stats and refs are free
  }
  copies_wait<0>();
  if (bad) raise_fault(p.fault, bad);
}

// A unit that stretches' bounds cut.
struct Cut {
  int64_t out;    // output row of its first token and head
  int16_t rows;
  int16_t n;      // its pieces, one a CTA
  int16_t first;  // the CTA of the first
  int16_t late;   // the first piece is the second of its CTA
};
struct Cuts {
  Cut c[kMaxCtas - 1];
};

// Joins the pieces of a unit, in key order: D / 4 threads a row.
template <int D>
__global__ void __launch_bounds__(256) rows_join_kernel(const RowsParams p, const __grid_constant__ Cuts cuts, int unit_rows) {
  constexpr int kRows = 256 / (D / 4);
  const Cut &u = cuts.c[blockIdx.x];
  const int row = blockIdx.y * kRows + threadIdx.x / (D / 4), col = threadIdx.x % (D / 4) * 4;
  wait_for_prior_grid();
  if (row >= u.rows) return;
  auto at = [&](int i) { return int64_t(2 * (u.first + i) + (i == 0 ? u.late : 0)) * unit_rows + row; };
  float m = neg_inf();
  for (int i = 0; i < u.n; ++i) m = fmaxf(m, p.part_lse[at(i)]);
  const float from = m == neg_inf() ? 0.f : m;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < u.n; ++i) {
    const float4 y = *reinterpret_cast<const float4 *>(p.part_o + at(i) * D + col);
    const float s = p.part_lse[at(i)], w = ex2(s - from);
    sum += w;
    if (s == neg_inf()) continue;
    x.x = fmaf(w, y.x, x.x), x.y = fmaf(w, y.y, x.y), x.z = fmaf(w, y.z, x.z), x.w = fmaf(w, y.w, x.w);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t out = u.out + int64_t(row / p.G) * p.Hq + row % p.G, o = out * D + col;
  const float4 y = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  if (p.out_f32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + o) = y;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(y.x, y.y), b = __floats2bfloat162_rn(y.z, y.w);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + o) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  }
  if (col == 0 && p.lse) p.lse[out] = sum == 0.f ? neg_inf() : m + log2f(sum);
}

template <int D, int NT, int TERMS>
psd_status run(const StepParams &S, const StepRequests &sreq, float *base, const DeviceInfo &dev, cudaStream_t s) {
  using L = Lay<D, NT>;
  RowsParams p;
  p.q = S.q;
  p.k_pool = static_cast<const uint8_t *>(S.k_pool);
  p.v_pool = static_cast<const uint8_t *>(S.v_pool);
  p.k_scales = S.scales.k;
  p.v_scales = S.scales.v;
  p.page_indices = S.page_indices;
  p.tree = S.tree;
  p.o = S.o;
  p.lse = S.lse;
  p.fault = S.fault;
  p.q_stride = S.q_stride;
  p.num_pages = S.num_pages;
  p.num_scales = S.num_pages * (S.page_size >> S.scales.shift) * S.Hkv;
  p.Hq = S.Hq;
  p.Hkv = S.Hkv;
  p.G = S.G;
  p.page_size = S.page_size;
  p.shift = S.scales.shift;
  p.out_f32 = S.out_f32;
  p.q_scale = S.q_scale;
  RowsRequests req;
  std::memcpy(req.r, sreq.r, sizeof(psd_token_request) * size_t(S.B));
  auto steps_of = [&](int b) { return (int64_t(req.r[b].kv_len) + kStep - 1) / kStep; };
  int64_t cost = 0, longest = 0;
  for (int b = 0; b < S.B; ++b) {
    cost += (steps_of(b) + kUnitCost) * S.Hkv;
    longest = std::max(longest, steps_of(b) + kUnitCost);
  }
  // Stretches of at least four steps a warp.
  const int64_t room = std::min(L::kCtasPerSm * dev.num_sms, kMaxCtas), units = int64_t(S.B) * S.Hkv;
  int ctas = int(std::max<int64_t>(1, std::min<int64_t>(room, cost / (4 * kWarps))));
  // Units left whole need no second kernel, which costs what some 30 steps a warp more would.
  const bool whole = units <= room && longest <= cost / ctas + 30;
  Cuts cuts;
  int n_cuts = 0;
  if (whole) {
    ctas = int(units);
    for (int u = 0; u < ctas; ++u) req.start[u] = Start{uint16_t(u / S.Hkv), uint16_t(u % S.Hkv), 0, int32_t(steps_of(u / S.Hkv))};
  } else {
    // Where the stretches begin: the unit and its step at c / ctas of the cost.
    int b = 0, last_cut_unit = -1;
    int64_t before = 0, line = 0, unit0 = 0;  // cost and steps before request b; its first unit
    int64_t began = 0;                        // the step on the line at which the stretch before begins
    for (int c = 0; c <= ctas; ++c) {
      int64_t here;
      if (c < ctas) {
        const int64_t want = c * cost / ctas;
        while (want >= before + (steps_of(b) + kUnitCost) * S.Hkv) {
          before += (steps_of(b) + kUnitCost) * S.Hkv;
          line += steps_of(b) * S.Hkv;
          unit0 += S.Hkv;
          ++b;
        }
        const int64_t n = steps_of(b);
        const int kv = int((want - before) / (n + kUnitCost));
        const int64_t j = std::max<int64_t>(0, want - before - kv * (n + kUnitCost) - kUnitCost);
        here = line + kv * n + j;
        req.start[c] = Start{uint16_t(b), uint16_t(kv), int32_t(j), 0};
        if (j > 0) {
          const int unit = int(unit0 + kv);
          if (unit != last_cut_unit) {
            last_cut_unit = unit;
            Cut &u = cuts.c[n_cuts++];
            u.out = int64_t(req.r[b].token0) * S.Hq + int64_t(kv) * S.G;
            u.rows = int16_t(req.r[b].num_new * S.G);
            u.n = 1;
            u.first = int16_t(c - 1);
            u.late = began < line + kv * n;
          }
          ++cuts.c[n_cuts - 1].n;
        }
      } else {
        while (b < S.B) line += steps_of(b++) * S.Hkv;
        here = line;
      }
      if (c > 0) req.start[c - 1].steps = int32_t(here - began);
      began = here;
    }
  }
  p.part_o = base;
  p.part_lse = base + int64_t(ctas) * 2 * 8 * NT * D;
  auto kern = rows_kernel<D, NT, TERMS>;
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = dev.device < 64 ? uint64_t(1) << dev.device : 0;
  cudaError_t e = cudaSuccess;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(L::kSmem));
    if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    ready.fetch_or(bit, std::memory_order_release);
  }
  kern<<<ctas, kThreads, L::kSmem, s>>>(p, req);
  e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "multi_token_decode_scaled launch: %s", cudaGetErrorString(e));
  if (n_cuts == 0) return PSD_OK;
  cudaLaunchConfig_t cfg = {};
  constexpr int kRows = 256 / (D / 4);
  cfg.gridDim = dim3(unsigned(n_cuts), unsigned((8 * NT + kRows - 1) / kRows));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, rows_join_kernel<D>, p, cuts, 8 * NT);
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "multi_token_decode_scaled join launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}

}  // namespace

bool step_rows_supports(const StepParams &p) {
  return p.scaled && (p.D == 64 || p.D == 128) && p.G <= kFewRows &&
         ((reinterpret_cast<uintptr_t>(p.scales.k) | reinterpret_cast<uintptr_t>(p.scales.v)) & 3) == 0;
}

size_t step_rows_floats(int sms, int D) {
  return size_t(std::min(2 * sms, kMaxCtas)) * 2 * kFewRows * (size_t(D) + 1);
}

psd_status launch_step_rows(const StepParams &p, const StepRequests &req, float *base, const DeviceInfo &dev, cudaStream_t s) {
  int rows = 0;
  for (int b = 0; b < p.B; ++b) rows = std::max(rows, req.r[b].num_new * p.G);
  auto go = [&](auto d) {
    constexpr int D = decltype(d)::value;
    auto by = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      return p.out_f32 ? run<D, NT, 2>(p, req, base, dev, s) : run<D, NT, 1>(p, req, base, dev, s);
    };
    if (rows <= 8) return by(std::integral_constant<int, 1>{});
    if (rows <= 16) return by(std::integral_constant<int, 2>{});
    if (rows <= 24) return by(std::integral_constant<int, 3>{});
    return by(std::integral_constant<int, 4>{});
  };
  return p.D == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace psd
