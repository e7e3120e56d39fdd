// append_tokens into a cache of 8-bit blocks with a scale each (the contract is in include/psd.h).
//
// Mathematics.  The scale of a block is the least power of two that brings its largest magnitude within e4m3's
// 448 = 1.75 2^8: with A = f 2^E, f in [1, 2), that is 2^(E - 8), or 2^(E - 7) where f > 1.75, read off A's bits.
// x 2^-k is exact in f32, so a code is rounded once.  A block that holds older tokens keeps its scale or takes a
// larger one; older codes then go down by a power of two, which rounds only what falls below 2^-6.
//
// Blocks are written by the CTA that has their first new token, the tokens of such a block behind its own included.  So
// every block has one writer, whatever the lengths, without a list of blocks and without atomics on scales.  A warp takes one
// block of one head's K or V, D / 16 lanes a token, and keeps the rotated values between finding the scale and writing the
// codes (blocks of 16 tokens up to 128 columns; larger ones are read and rotated twice).
//   8118 prompt tokens, 32 query heads and 8 of K and V, of 128: 36 us, 0.75 of the copy rate (183 MB): K and V 19, the queries
// 20, which is their bytes at the copy rate, a few of them beside each other.  32 single tokens: 5.2 us, all of it latency.
#include <algorithm>
#include <atomic>

#include "append.cuh"
#include "block_scales.cuh"

namespace psd {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kLeast = 95;  // 2^-32
constexpr int kMaxBlock = 64, kMany = 16, kManyQueries = 16;  // tokens a CTA at most
constexpr int kBlockCtas = 2, kQueryCtas = 4;  // CTAs an SM

struct ScaledParams {
  AppendParams a;
  uint8_t *k_scales, *v_scales;
  int block, shift;  // 2^shift tokens
};

// A token of the CTA.
struct Token {
  int pos;       // rotation position; negative: left as it is
  int count;     // tokens of the block from this one on, if it is the block's first new one, else 0
  int older;     // tokens of the block before this one
  int64_t slot;  // pool row, or -1
};

// The request of token t0 + lane, for the lanes below `own` (uniform): the warp finds the first one's, and one load of 32 bounds
// behind it tells the others'.
__device__ __forceinline__ int request_of_lane(const AppendParams &p, int t0, int own) {
  const int lane = threadIdx.x & 31, b0 = request_of(p.q_indptr, p.B, t0);
  if (own == 1) return b0;
  const int bound = b0 + 1 + lane < p.B ? __ldg(p.q_indptr + b0 + 1 + lane) : 0x7fffffff;
  int b = b0;
  for (int i = 0; i < own; ++i) {
    const int behind = __popc(__ballot_sync(0xffffffffu, bound <= t0 + i));
    if (lane == i) b = b0 + behind;
  }
  if (b == b0 + 32)  // (many requests without tokens)
    while (b + 1 < p.B && __ldg(p.q_indptr + b + 1) <= t0 + lane) ++b;
  return b;
}
// Token t0 + lane of a warp's, for the lanes below `own`.  (A search for each token, two a warp one after the other, took twice
// the time of these dependent loads.)
__device__ __forceinline__ Token locate(const ScaledParams &s, int t0, int own, uint32_t &faults) {
  const AppendParams &p = s.a;
  Token x{-1, 0, 0, -1};
  faults = 0;
  const int t = t0 + int(threadIdx.x & 31), all = __ldg(p.q_indptr + p.B);
  const int b = request_of_lane(p, t0, own);
  if (t >= t0 + own || t >= p.T || t >= all) return x;  // not the CTA's, or behind the last request
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
  x.older = at & (s.block - 1);
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
__device__ __forceinline__ float max_abs(float a, float b, float c) {  // of the magnitudes; NaN operands lose, as in fmaxf
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
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

// The angles of tokens from .. n - 1 into `cosine` and `sine`, all kThreads threads; `freq`: the turns per position, in shared
// memory (lanes that read different parameters of a launch wait for each other).
struct Deal {  // of (token, pair) to the threads: the first, and the way to the next
  int m, k, step, rest;
  __device__ __forceinline__ explicit Deal(int half) : m(0), k(0), step(1), rest(0) {
    if (half == 0) return;
    step = kThreads / half, rest = kThreads - step * half;
    m = int(threadIdx.x) / half, k = int(threadIdx.x) - m * half;
  }
};
__device__ __forceinline__ void make_angles(const Deal &deal, const int *pos, int from, int n, int half, const uint64_t *freq, float magnitude,
                                            float *cosine, float *sine) {
  if (half == 0) return;
  int k = deal.k;
  for (int m = deal.m + from; m < n; m += deal.step) {
    const float2 cs = pos[m] >= 0 ? short_turn(freq[k], pos[m], magnitude) : make_float2(0.f, 0.f);
    const int at = m * half + angle_at(k, half);
    cosine[at] = cs.x;
    sine[at] = cs.y;
    k += deal.rest;
    if (k >= half) k -= half, ++m;
  }
}
// A warp's lanes among the tokens of a block: D / 16 a token.
struct Lanes {
  int a_pass, mine, k;  // tokens a pass; the lane's token of a pass and its place in it
  __device__ __forceinline__ explicit Lanes(int width) {
    const int lane = threadIdx.x & 31, lanes = (width + 15) / 16;
    a_pass = 32 / lanes, mine = lane / lanes, k = lane - mine * lanes;
  }
};
// A thread's place in a token's query heads: a group of pairs, or a run that is not rotated.
struct Column {
  int at;       // of the first run of 8 (element in the token's row)
  int group;    // of pairs; negative: not rotated
  __device__ __forceinline__ Column(const AppendParams &p, int job, int groups, int per_head, bool neox) {
    const int h = job / per_head, g = job - h * per_head;
    group = g < groups ? g : -1;
    int col = g < groups ? p.rot_col + (neox ? 8 * g : 16 * g) : 8 * (g - groups);
    if (g >= groups && col >= p.rot_col) col += p.rot;
    at = h * p.D + col;
  }
};

// Queries of `per` tokens a CTA: a thread has the same column of all of them, two tokens on their way.  (With two tokens a CTA
// every other cycle went into waiting for their places: 26 us for 8118 tokens of 32 heads of 128.)
template <bool NEOX>
__global__ void __launch_bounds__(kThreads, kQueryCtas) append_queries_kernel(const ScaledParams s, const __grid_constant__ Turns turns, int per) {
  extern __shared__ __align__(16) float table[];  // cosines [tokens][half], then sines
  __shared__ int pos[kManyQueries];
  __shared__ uint64_t freq[kMaxPairs / 2];
  const AppendParams &p = s.a;
  const int tid = threadIdx.x, lane = tid & 31;
  for (int k = tid; k < p.rot / 2; k += kThreads) freq[k] = turns.f[k];
  const int half = p.rot / 2, groups = half / 8, far = NEOX ? half : 8;
  const int per_head = groups + (p.D - p.rot) / 8, jobs = p.Hq * per_head;
  const int t0 = blockIdx.x * per, n = min(per, p.T - t0);
  uint4 wa[2], wb[2];
  auto fetch = [&](const Column &c, int i, uint4 &a, uint4 &b) {
    if (i < n) {
      const __nv_bfloat16 *at = p.q + (t0 + i) * p.q_stride + c.at;
      a = load_raw(at);
      if (c.group >= 0) b = load_raw(at + far);
    }
  };
  Column c(p, min(tid, jobs - 1), groups, per_head, NEOX);
  if (tid < jobs) {  // on their way before their places are known
    fetch(c, 0, wa[0], wb[0]);
    fetch(c, 1, wa[1], wb[1]);
  }
  if (tid < 32) {
    const int t = t0 + lane, all = __ldg(p.q_indptr + p.B), b = request_of_lane(p, t0, n);
    int at = -1;
    if (lane < n && t < all) {
      const int begin = __ldg(p.q_indptr + b), end = __ldg(p.q_indptr + b + 1);
      at = p.positions ? __ldg(p.positions + t) : __ldg(p.kv_len + b) - (end - t);
      if (t < begin || t >= end) at = -1;  // (K's CTAs report it)
    }
    if (lane < n) pos[lane] = max(at, -1);
  }
  __syncthreads();
  float *cosine = table, *sine = table + n * half;
  make_angles(Deal(half), pos, 0, n, half, freq, p.magnitude, cosine, sine);
  __syncthreads();
  // (q_out may be q: both runs of a group are read before either is written)
  for (int job = tid; job < jobs; job += kThreads) {
    if (job != tid) {
      c = Column(p, job, groups, per_head, NEOX);
      fetch(c, 0, wa[0], wb[0]);
      fetch(c, 1, wa[1], wb[1]);
    }
    __nv_bfloat16 *to = p.q_out + int64_t(t0) * p.Hq * p.D + c.at;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 2) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = i0 + k;
        const bool there = i < n && pos[i] >= 0;
        if (c.group >= 0) {
          F8 x = unpack(wa[k]), y = unpack(wb[k]);
          fetch(c, i + 2, wa[k], wb[k]);
          if (there) {
            rotate<NEOX>(x, y, cosine + i * half, sine + i * half, c.group, half);
            store8(to, x);
            store8(to + far, y);
          }
        } else {
          const uint4 w = wa[k];
          fetch(c, i + 2, wa[k], wb[k]);
          if (there) *reinterpret_cast<uint4 *>(to) = w;
        }
        to += int64_t(p.Hq) * p.D;
      }
    }
  }
  wait_for_prior_grid();  // what waits for this launch waits for K and V too
}

// Tokens t0 .. t0 + own - 1 as K's and V's CTAs take them.
template <int NT>
struct Tile {
  Token tokens[NT];
  int pos[NT + kMaxBlock];
  int n_table, n_starts, starts[NT];  // tokens whose angles are needed; tokens that begin their block
};
// A warp fills it in; returns the faults.
template <int NT>
__device__ __forceinline__ uint32_t fill(const ScaledParams &s, int t0, int own, Tile<NT> &tile) {
  static_assert(NT <= 32, "a lane a token");
  const int lane = threadIdx.x & 31;
  uint32_t faults;
  const Token x = locate(s, t0, own, faults);
  if (lane < own) tile.tokens[lane] = x;
  faults = __reduce_or_sync(0xffffffffu, faults);
  __syncwarp();
  // the tokens whose angles are needed: its own, and those of its last block behind them
  const bool begins = x.slot >= 0 && x.count > 0;
  const uint32_t who = __ballot_sync(0xffffffffu, begins);
  const int most = __reduce_max_sync(0xffffffffu, begins ? max(own, lane + x.count) : own);
  for (int n = lane; n < most; n += 32) {
    if (n < own) {
      tile.pos[n] = tile.tokens[n].pos;
    } else {  // of the request of the last block that starts here
      int at = -1;
      if (s.a.positions) {
        at = __ldg(s.a.positions + t0 + n);
      } else {
        const int i = 31 - __clz(who);
        if (tile.tokens[i].count > n - i) at = tile.tokens[i].pos + (n - i);
      }
      tile.pos[n] = max(at, -1);
    }
  }
  if (begins) tile.starts[__popc(who & ((1u << lane) - 1u))] = lane;
  if (lane == 0) tile.n_table = most, tile.n_starts = __popc(who);
  return faults;
}
// The rows of K or V, as far as the CTA's own tokens go, to the second-level cache; all threads, 16 a row.
__device__ __forceinline__ void prefetch_rows(const AppendParams &p, bool is_v, int t0, int own) {
  const int bytes = (is_v ? p.Dv : p.D) * p.Hkv * 2, n = min(own, p.T - t0);
  const int64_t stride = 2 * (is_v ? p.v_stride : p.k_stride);
  for (int row = threadIdx.x / 16; row < n; row += kThreads / 16)
    for (int at = 128 * (threadIdx.x % 16); at < bytes; at += 128 * 16)
      prefetch_l2(reinterpret_cast<const uint8_t *>(is_v ? p.v : p.k) + (t0 + row) * stride + at);
}

// The blocks that begin in a tile: K of head h, or V of it, a warp each.  A lane has two runs of 8 columns of a token, up to
// kPasses tokens at once.  K's angles are made by all kWarps warps, a barrier behind them, while the first block's rows are on
// their way: `joined` is that barrier.
template <int NT, bool NEOX, typename Barrier>
__device__ __forceinline__ void write_blocks(const ScaledParams &s, const uint64_t *freq, const Deal &deal, const Lanes &lanes, const Tile<NT> &tile, int t0,
                                             bool is_v, float *table, Barrier joined) {
  constexpr int kPasses = 4;
  const AppendParams &p = s.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = p.rot / 2;
  const int groups = half / 8, far = NEOX ? half : 8;  // groups of 8 pairs; their second run of 8 columns is `far` behind
  const int nt = tile.n_table, n_starts = tile.n_starts, W = is_v ? p.Dv : p.D;
  const int *pos = tile.pos;
  float *cosine = table, *sine = table + nt * half;
  bool ready = is_v;
  auto angles = [&]() {
    if (ready) return;
    const int from = n_starts == 0 ? nt : tile.starts[0];  // (tokens before the first block's begin are another CTA's)
    make_angles(deal, pos, from, nt, half, freq, p.magnitude, cosine, sine);
    joined();
    ready = true;
  };
  const int a_pass = lanes.a_pass, mine = lanes.mine, k = lanes.k;
  for (int start = 0, h = warp;; h += kWarps) {
    while (h >= p.Hkv && start < n_starts) h -= p.Hkv, ++start;
    if (start >= n_starts) break;
    const int n = tile.starts[start];
    const Token x = tile.tokens[n];
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
    any = __any_sync(0xffffffffu, any);
    const int passes = x.count <= kPasses * a_pass ? kPasses : (x.count + a_pass - 1) / a_pass;
    F8 a[kPasses], b[kPasses];
    uint4 wa[kPasses], wb[kPasses];
    uint32_t valid = 0;  // passes of those at hand that have a token for this lane
    auto fetch = [&](int pass0) {
      valid = 0;
      const __nv_bfloat16 *at = src + (t0 + n + pass0 * a_pass + mine) * stride;
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
    };
    auto turn = [&](int pass0) {
#pragma unroll
      for (int q = 0; q < kPasses; ++q) {
        a[q] = unpack(wa[q]), b[q] = unpack(wb[q]);
        const int i = (n + (pass0 + q) * a_pass + mine) * half;
        if (turned && (valid >> q & 1)) rotate<NEOX>(a[q], b[q], cosine + i, sine + i, k, half);
      }
    };
    fetch(0);
    angles();
    if (!any) continue;
    turn(0);
    float top = 0.f;
    // (NaN loses; infinities are looked for again, and left out, where there are any)
    auto larger = [&](const F8 &f, bool finite) {
      if (!finite) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) top = max_abs(top, f.v[i], f.v[i + 1]);
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
        if (passes > kPasses && (finite || pass0 > 0)) fetch(pass0), turn(pass0);
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
    uint8_t *scale = (is_v ? s.v_scales : s.k_scales) + (first >> s.shift) * p.Hkv + h;
    uint8_t *pool = static_cast<uint8_t *>(is_v ? p.v_pool : p.k_pool) + (first * p.Hkv + h) * W;
    const int64_t pool_stride = int64_t(p.Hkv) * W;
    int e = scale_of(top);
    if (x.older > 0) {
      const int had = *scale;
      if (e > had) {
        const float down = power_of_two(had - e);        // (ties are kept; 0 below 2^-126)
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
    const float by = __uint_as_float(e >= 254 ? 0x00400000u : uint32_t(254 - e) << 23);  // (2^-127 is subnormal)
#pragma unroll 1
    for (int pass0 = 0; pass0 < passes; pass0 += kPasses) {
      if (passes > kPasses) fetch(pass0), turn(pass0);   // (otherwise they are there)
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
  angles();
}

// K and V of many tokens: a CTA takes tiles of kMany tokens, of K and of V in turn.  Its warps find the places of one tile each,
// all at once; a tile's rows are brought to the second-level cache while the tile before is worked on.  (With a CTA a tile,
// seven warps waited for the eighth's dependent loads: 26 us for 8118 tokens of 8 heads of 128 against 19.)  Bound by the chain
// of a tile (rows, angles, largest, scale, codes: 3 us), with 16 warps an SM at 47 % of the issue slots.
template <bool NEOX>
__global__ void __launch_bounds__(kThreads, kBlockCtas) append_blocks_kernel(const ScaledParams s, const __grid_constant__ Turns turns, int) {
  extern __shared__ __align__(16) float table[];  // cosines [tokens][half], then sines
  __shared__ Tile<kMany> tiles[kWarps];
  __shared__ uint64_t freq[kMaxPairs / 2];
  const AppendParams &p = s.a;
  for (int k = threadIdx.x; k < p.rot / 2; k += kThreads) freq[k] = turns.f[k];
  dependents_may_launch();  // the queries
  const int items = 2 * ((p.T - 1) / kMany + 1), lane = threadIdx.x & 31, warp = threadIdx.x >> 5, step = gridDim.x;
  if (int(blockIdx.x) < items) prefetch_rows(p, blockIdx.x & 1, int(blockIdx.x) / 2 * kMany, kMany);
  const Deal deal(p.rot / 2);
  const Lanes of_k(p.D), of_v(p.Dv);
  int turn = 0;
  for (int item = blockIdx.x; item < items; item += step, ++turn) {
    __syncthreads();  // the table and the tile before are free
    if (turn % kWarps == 0) {
      const int64_t mine = item + int64_t(warp) * step;
      if (mine < items) {
        const uint32_t faults = fill(s, int(mine / 2) * kMany, kMany, tiles[warp]);
        if (faults && lane == 0 && !((mine + warp) & 1)) atomicOr(p.fault, int32_t(faults));
      }
      __syncthreads();
    }
    const bool is_v = (item + turn) & 1;
    // (one tile ahead: with all tiles' rows asked for at the start, the first places took 6 us to be found)
    if (item + step < items) prefetch_rows(p, (item + step + turn + 1) & 1, (item + step) / 2 * kMany, kMany);
    write_blocks<kMany, NEOX>(s, freq, deal, is_v ? of_v : of_k, tiles[turn % kWarps], item / 2 * kMany, is_v, table, [] { __syncthreads(); });
  }
}

// Few tokens: a CTA a token's K, its V and its queries, all in one launch.
template <bool NEOX>
__global__ void __launch_bounds__(kThreads, 2) append_few_kernel(const ScaledParams s, const __grid_constant__ Turns turns, int) {
  extern __shared__ __align__(16) float table[];  // cosines [tokens][half], then sines
  __shared__ Tile<1> tile;
  __shared__ uint64_t freq[kMaxPairs / 2];
  const AppendParams &p = s.a;
  for (int k = threadIdx.x; k < p.rot / 2; k += kThreads) freq[k] = turns.f[k];
  const int tid = threadIdx.x, warp = tid >> 5;
  const int half = p.rot / 2, groups = half / 8, far = NEOX ? half : 8;
  // CTAs of K (0) and V (1) in turn, then those of the queries (2).
  const int kv_ctas = 2 * p.T, cta = blockIdx.x, part = cta >= kv_ctas ? 2 : cta & 1, t0 = part == 2 ? cta - kv_ctas : cta / 2;
  // The row is on its way before its place is known.
  const int per_head = groups + (p.D - p.rot) / 8, jobs = p.Hq * per_head;
  uint4 qa, qb;
  Column c(p, min(tid, max(jobs - 1, 0)), groups, per_head, NEOX);
  auto fetch_q = [&]() {
    const __nv_bfloat16 *at = p.q + t0 * p.q_stride + c.at;
    qa = load_raw(at);
    if (c.group >= 0) qb = load_raw(at + far);
  };
  if (part < 2) prefetch_rows(p, part == 1, t0, 1);
  else if (tid < jobs) fetch_q();
  if (warp == 0) {
    const uint32_t faults = fill(s, t0, 1, tile);
    if (faults && tid == 0 && part == 0) atomicOr(p.fault, int32_t(faults));
  }
  __syncthreads();
  if (part < 2) {
    write_blocks<1, NEOX>(s, freq, Deal(half), Lanes(part ? p.Dv : p.D), tile, t0, part == 1, table, [] { __syncthreads(); });
    return;
  }
  // (q_out may be q: both runs of a group are read before either is written)
  const int pos = tile.pos[0];
  if (pos < 0) return;
  float *cosine = table, *sine = table + half;
  for (int k = tid; k < half; k += kThreads) {
    const float2 cs = short_turn(freq[k], pos, p.magnitude);
    cosine[angle_at(k, half)] = cs.x;
    sine[angle_at(k, half)] = cs.y;
  }
  __syncthreads();
  for (int job = tid; job < jobs; job += kThreads) {
    if (job != tid) {
      c = Column(p, job, groups, per_head, NEOX);
      fetch_q();
    }
    __nv_bfloat16 *to = p.q_out + int64_t(t0) * p.Hq * p.D + c.at;
    if (c.group >= 0) {
      F8 x = unpack(qa), y = unpack(qb);
      rotate<NEOX>(x, y, cosine, sine, c.group, half);
      store8(to, x);
      store8(to + far, y);
    } else {
      *reinterpret_cast<uint4 *>(to) = qa;
    }
  }
}

template <typename Kernel>
psd_status start(Kernel kern, std::atomic<uint64_t> &ready, int64_t ctas, int threads, size_t shared, size_t most_shared, bool behind,
                 const ScaledParams &p, const Turns &turns, int per, const DeviceInfo &dev, cudaStream_t s) {
  if (ctas > 0x7fffffffLL) return fail(PSD_ERR_UNSUPPORTED, "append_tokens_scaled: %d tokens", p.a.T);
  const uint64_t bit = dev.device < 64 ? uint64_t(1) << dev.device : 0;
  cudaError_t e = cudaSuccess;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most_shared));
    if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = shared;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = behind ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, p, turns, per);
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "append_tokens_scaled launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}

// Tokens a CTA of the queries, so that they fill whole rounds of the CTAs that run at once.
int tokens_a_cta(int64_t tokens, int64_t at_once) {
  const int64_t rounds = (tokens + at_once * kManyQueries - 1) / (at_once * kManyQueries);
  return int((tokens + at_once * rounds - 1) / (at_once * rounds));
}

template <bool NEOX>
psd_status launch_all(const ScaledParams &p, const Turns &turns, const DeviceInfo &dev, cudaStream_t s) {
  const int64_t T = p.a.T;
  const size_t angles = size_t(p.a.rot) * 4;  // bytes a token
  static std::atomic<uint64_t> one{0}, queries{0}, blocks{0};
  // One launch while its CTAs fit on the SMs at once.
  if (T <= 2 * dev.num_sms)
    return start(append_few_kernel<NEOX>, one, (p.a.Hq ? 3 : 2) * T, kThreads, p.block * angles, kMaxBlock * kMaxPairs * 4, false, p, turns,
                 1, dev, s);
  // K and V first: the queries, which wait for memory, start where their CTAs end.  (39.3 us against 40.1 the other way round.)
  const int64_t items = 2 * ((T + kMany - 1) / kMany);
  const psd_status st =
      start(append_blocks_kernel<NEOX>, blocks, std::min<int64_t>(items, kBlockCtas * dev.num_sms), kThreads, (kMany + p.block - 1) * angles,
            (kMany + kMaxBlock - 1) * kMaxPairs * 4, false, p, turns, kMany, dev, s);
  if (st != PSD_OK || p.a.Hq == 0) return st;
  const int per = tokens_a_cta(T, kQueryCtas * dev.num_sms);
  return start(append_queries_kernel<NEOX>, queries, (T + per - 1) / per, kThreads, per * angles, kManyQueries * kMaxPairs * 4, true, p, turns,
               per, dev, s);
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
  p.shift = scales->block == 16 ? 4 : scales->block == 32 ? 5 : 6;
  const Turns turns = append_turns(a);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a->neox ? launch_all<true>(p, turns, ctx->dev, s) : launch_all<false>(p, turns, ctx->dev, s);
}
