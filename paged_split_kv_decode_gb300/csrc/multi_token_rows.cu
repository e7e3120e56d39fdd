// Attention of few rows (a request's new tokens times the G query heads of a KV head, at most 32) over a cache of
// 8-bit blocks with a scale each: single tokens and short drafts, where reading the cache is all the work.
//
// Mathematics.  S^T = K Q^T and O^T += V^T P^T, keys and columns as the 16 rows of an mma.sync, query rows as its 8
// columns: 8 rows fill an MMA, where S = Q K^T would take 16.  Which columns a lane takes is free as long as Q and K
// agree, so each lane's 16 bytes of a key are its operands as they lie: no shuffles, no transposition of K.
// Codes become f16 exactly; V's bytes of two keys are paired by one permute for four codes.  Q is f16 scaled row by
// row (exact but for elements 2^-31 below the row's top).  (mma.sync on e4m3 operands is made of conversions and the
// f16 MMA here: with Q as two e4m3 terms 16 keys took 90 instructions more.)
//   K's scale 2^a multiplies the scores of its block's 16 keys.  V's 2^b goes into P: P' = P 2^(b - r), r the largest b
// so far (O follows when r grows), so that P' <= P and f16 holds it to 2^-12 of itself down to b = r - 21 and
// beyond that to 2^-32 of the row's largest; the sum l is of P.  The row maximum follows lazily, as in the
// tensor-core kernel for many rows: P <= 2^15, and O and l are rescaled only when it grows by more than 2^8.
// f32 outputs take P' as two f16 terms (2^-22).
//
// Bytes: a key's row of a head is 64 or 128 bytes, and a step of a warp is 32 keys in two halves of 16, whose chains of
// dependent instructions are independent of each other.  A warp copies whole rows (cp.async) into a ring of its own, which
// needs no barrier, chunks of 16 bytes swizzled so that eight neighbouring lanes read eight different bank groups: K's
// chunk k of row r lies at k ^ 4 (r & 1), V's at k ^ 2 (r / 2 % 4) (64-byte rows: V's rows 0, 2, .. 14, 1, 3, .. and k ^ 2 for
// every other pair).  Two steps of 8 KB a warp, 12 warps an SM, are 192 KB; DRAM at its full rate wants about 50 on their
// way.  (Copies by the lanes that use the bytes fetched V twice from the second-level cache, 64 bytes at a time for 32.)
//
// Split: a worker is a warp with one KV head; the heads' workers of one slot are neighbours and read the same tokens'
// rows side by side.  The requests' steps lie on one line, the same for every head, and each slot takes a stretch of
// it that costs the same.  A request that a stretch's bound cuts leaves normalised pieces, which a second kernel
// joins in key order.  Nothing is added atomically.  (With a unit's steps dealt out to the eight warps of a CTA and
// their O joined in shared memory, that joining took more instructions than the steps.)
//
// Bound by DRAM in its steady state: 32 single tokens over 512 to 4096 keys (140 MB, 21 us at the copy rate) take 30 us without
// the join and 34 with it; three over 20000 to 65536 with f32 outputs (27 us) 36 and 42.  The rest is the launch, the ramp
// to the first step and the slots' ends.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

#include "device.cuh"
#include "multi_token.h"

namespace psd {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kHalf = 16, kStep = 2 * kHalf;  // keys
constexpr float kLazy = 8.f, kBias = 7.f;  // log2 units: P's top is 2^7, and grows to 2^15 at most
constexpr int kSegmentCost = 2;  // of a request beside its steps, in steps
constexpr int kLeastSteps = 1;   // of a slot (3: 4 tokens over 60 to 400 keys took 9.9 us against 7.8)
constexpr int kJoinSteps = 4;    // what joining takes, in steps
constexpr int kMostPieces = 2048; // slots at most
constexpr int kFewPieces = 16;   // that a warp joins by itself

template <int D, int NT>
struct Lay {
  static constexpr int kCtasPerSm = NT == 1 ? 3 : 2;
  static constexpr bool kQInRegs = NT <= 2 || D == 64;
  static constexpr int kStages = NT == 1 ? 2 : kQInRegs ? 3 : 2;
  static constexpr uint32_t kHalfBytes = 2 * kHalf * D;              // K, then V
  static constexpr uint32_t kStageBytes = 2 * kHalfBytes;
  static constexpr uint32_t kOffMeta = kWarps * kStages * kStageBytes;  // a half's scales: two words and a shift
  static constexpr uint32_t kOffQ = kOffMeta + kWarps * kStages * 32;
  static constexpr uint32_t kSmem = kOffQ + (kQInRegs ? 0 : kWarps * NT * (D / 16) * 32 * 8);
  static_assert(kCtasPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory");
};

struct RowsParams {
  const __nv_bfloat16 *q;
  const uint8_t *k_pool, *v_pool, *k_scales, *v_scales;
  const int32_t *page_indices;
  const uint64_t *tree;
  void *o;
  float *lse;
  float *part_o, *part_lse;  // [slots][2][KV heads][rows of a unit][D], and without D
  FaultRef fault;
  int64_t q_stride, num_pages;
  int num_scales;            // bytes
  int Hq, Hkv, G, page_size, shift, out_f32;
  float q_scale;
  int B, slots;
  bool narrow;  // the line's length times the slots fits 32 bits
  bool whole;   // slot x has request x
};
// A launch's requests, and what those before each cost: their steps, and kSegmentCost each.
struct RowsRequests {
  psd_token_request r[kStepRequests];
  int64_t before[kStepRequests + 1];
};

__host__ __device__ __forceinline__ int steps_of(const psd_token_request &r) { return (r.kv_len - 1) / kStep + 1; }
// (64-bit divisions take ten times as long.)
__host__ __device__ __forceinline__ int64_t divide(const RowsParams &p, int64_t a, int64_t b) {
  return p.narrow ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}
// The request and step at which slot `x` begins.
__device__ __forceinline__ int2 begin_of(const RowsParams &p, const RowsRequests &req, int x) {
  if (p.whole) return make_int2(x, 0);
  const int64_t want = divide(p, x * req.before[p.B], p.slots);
  int b = 0;
  for (int n = p.B; n > 1;) {  // the last request with before <= want
    const int mid = n / 2;
    if (req.before[b + mid] <= want) b += mid, n -= mid;
    else n = mid;
  }
  if (x >= p.slots) return make_int2(p.B, 0);
  return make_int2(b, int(max(int64_t(0), want - req.before[b] - kSegmentCost)));
}

// A stretch's part of one request.
struct Segment {
  int b, s0, s1, n;
  bool first;
};
struct Walk {
  const RowsRequests &req;
  int2 at, end;
  bool first = true;
  __device__ Walk(const RowsRequests &r, int2 begin, int2 end_) : req(r), at(begin), end(end_) {}
  __device__ bool next(Segment &g) {
    if (at.x > end.x || (at.x == end.x && at.y >= end.y)) return false;
    g.b = at.x, g.s0 = at.y, g.first = first;
    g.n = steps_of(req.r[at.x]);
    g.s1 = at.x == end.x ? end.y : g.n;
    first = false;
    at = make_int2(at.x + 1, 0);
    return true;
  }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
template <int SEL>
__device__ __forceinline__ uint32_t pair(uint32_t a, uint32_t b) {
  uint32_t r;
  asm volatile("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "n"(SEL));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN operands lose, as in fmaxf
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
  constexpr int NS = L::kStages, kCols = D / 64, kMmas = D / 16;  // 64-column parts of a row; MMAs of S for 16 keys, and of O
  extern __shared__ __align__(128) uint8_t sm[];
  dependents_may_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int worker = blockIdx.x * kWarps + warp, slot = worker / p.Hkv, kv = worker - slot * p.Hkv;
  if (slot >= p.slots) return;
  const uint32_t ring = smem_u32(sm) + warp * NS * L::kStageBytes;
  const uint8_t *ring_at = sm + warp * NS * L::kStageBytes;
  const uint32_t meta = smem_u32(sm) + L::kOffMeta + warp * NS * 32;
  const uint32_t row_bytes = uint32_t(p.Hkv) * D, half_bytes = kHalf * row_bytes;  // between a head's rows of neighbouring slots
  uint32_t bad = 0;
  const int2 begin = begin_of(p, req, slot), end = begin_of(p, req, slot + 1);

  // ------------------------------------------------------------------------------ copies
  // The steps to be copied run NS ahead of those worked on, across the requests' ends.
  Walk ahead(req, begin, end);
  Segment from;
  bool more = ahead.next(from);
  int at = more ? from.s0 : 0;
  int halves = -1, window = 32;  // pool halves (16 slots) of 32 of the worker's halves, one a lane; -1: not there
  // A lane copies 16 bytes of every kRowsACopy-th row.
  constexpr int kChunks = D / 16, kRowsACopy = 32 / kChunks, kCopies = kHalf / kRowsACopy;
  const int row0 = lane / kChunks, chunk = lane % kChunks;
  const uint64_t lane_bytes = uint64_t(row0) * row_bytes + uint32_t(16 * chunk + kv * D);
  const uint8_t *k_lane = p.k_pool + lane_bytes, *v_lane = p.v_pool + lane_bytes;
  const uint32_t copy_bytes = kRowsACopy * row_bytes;
  const uint32_t k_to = ring + (D == 128 ? row0 * 128 + ((chunk ^ (row0 & 1) * 4) << 4) : lane * 16);
  const uint32_t v_to = ring + kHalf * D + (D == 128 ? row0 * 128 + ((chunk ^ (row0 >> 1) * 2) << 4)
                                                     : ((row0 & 1) * 8 + (row0 >> 1)) * 64 + ((chunk ^ (row0 >> 2) * 2) << 4));
  // and reads K's rows g and g + 8, and columns D / 8 g .. of V's rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9
  const uint32_t k_from = D == 128 ? g * 128 + c * 16 + (g & 1) * 64 : g * 64 + c * 16;
  const uint32_t v_from = kHalf * D + (D == 128 ? 2 * c * 128 + ((g ^ 2 * c) << 4) : c * 64 + (((g >> 1) ^ (c >> 1) * 2) << 4) + (g & 1) * 8);
  const uint8_t *scale_lane = lane ? p.v_scales : p.k_scales;
  const int page_halves = p.page_size / kHalf;
  auto issue = [&](int stage) {
    if (more && at >= from.s1) {
      more = ahead.next(from);
      at = from.s0;
      window = 32;
    }
    if (more) {
      if (window == 32) {
        window = 0;
        const psd_token_request &r = req.r[from.b];
        const int mine = 2 * at + lane, page = mine / page_halves;
        const bool wanted = mine < 2 * from.s1 && mine <= (r.kv_len - 1) / kHalf;
        int id = -1;
        if (wanted) id = __ldg(p.page_indices + r.page_off + page);
        const bool there = id >= 0 && int64_t(id) < p.num_pages;
        if (wanted && !there) bad |= PSD_FAULT_PAGE_ID;
        halves = there ? (id - page) * page_halves + mine : -1;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int half = __shfl_sync(0xffffffffu, halves, window + x);
        const uint32_t dst = stage * L::kStageBytes + x * L::kHalfBytes;
        const uint32_t scales = meta + stage * 32 + x * 16;
        // a half that is not there (its page, or it lies behind the last token) is hidden: a shift of 32 says so
        uint32_t shift = 32;
        if (half >= 0) {
          const uint64_t off = uint64_t(uint32_t(half)) * half_bytes;
          const uint8_t *k = k_lane + off, *v = v_lane + off;
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            copy16(k_to + dst + i * 512, k);
            k += copy_bytes;
          }
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            copy16((D == 128 ? v_to ^ (i & 1) * 64 : v_to) + dst + i * (D == 128 ? 512 : 256), v);
            v += copy_bytes;
          }
          const int scale = (half >> (p.shift - 4)) * p.Hkv + kv, word = scale & ~3;
          shift = uint32_t(scale & 3) * 8;
          if (lane < 2) copy4(scales + 4 * lane, scale_lane + word, uint32_t(min(4, p.num_scales - word)));
        }
        if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(scales + 8), "r"(shift) : "memory");
      }
      window += 2;
      ++at;
    }
    copies_end();
  };
  for (int s = 0; s < NS; ++s) issue(s);

  // ----------------------------------------------------------------------------- requests
  Walk walk(req, begin, end);
  Segment u;
  int stage = 0;
  while (walk.next(u)) {
    const psd_token_request r = req.r[u.b];
    const int start = r.kv_len - r.num_new, rows = r.num_new * p.G;
    const bool has_tree = p.tree != nullptr;
    // Q of row g of each tile, times the power of two that puts its top in [2^14, 2^15): exact but for elements
    // 2^-31 below the top.
    [[maybe_unused]] uint2 qf[L::kQInRegs ? NT : 1][kMmas];
    float qs[NT][2];  // score factors of rows 2 c and 2 c + 1
    uint2 *q_at = reinterpret_cast<uint2 *>(sm + L::kOffQ) + warp * NT * kMmas * 32 + lane;  // [tile][MMA][lane]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 8 * nt + g;
      uint4 w[kCols][2];
      const bool live = row < rows;
      const __nv_bfloat16 *src = p.q + (int64_t(r.token0) + (live ? row / p.G : 0)) * p.q_stride +
                                 (int64_t(kv) * p.G + (live ? row % p.G : 0)) * D + 16 * c;
      float top = 0.f;
#pragma unroll
      for (int h = 0; h < kCols; ++h)
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
      for (int i = 0; i < kMmas; ++i) {  // columns 64 (i / 4) + 16 c + 4 (i % 4) .. + 3
        const uint4 &x = w[i >> 2][(i >> 1) & 1];
        const uint32_t lo = i & 1 ? x.z : x.x, hi = i & 1 ? x.w : x.y;
        const uint2 q = make_uint2(f16x2_bits(bf16_lo(lo) * f, bf16_hi(lo) * f), f16x2_bits(bf16_lo(hi) * f, bf16_hi(hi) * f));
        if constexpr (L::kQInRegs) qf[nt][i] = q;
        else q_at[(nt * kMmas + i) * 32] = q;  // (read by this lane alone)
      }
      qs[nt][0] = __shfl_sync(0xffffffffu, back, 8 * c);
      qs[nt][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
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
    for (int s = u.s0; s < u.s1; ++s) {
      copies_wait<NS - 1>();
      __syncwarp();  // rows and scales came through other lanes
      const uint8_t *src = ring_at + stage * L::kStageBytes;
      uint32_t ke[2], ve[2];
      bool there[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4 w = *reinterpret_cast<const uint4 *>(sm + L::kOffMeta + ((warp * NS + stage) * 2 + x) * 16);
        there[x] = w.z < 32;
        ke[x] = there[x] ? (w.x >> w.z) & 255u : 127u;
        ve[x] = there[x] ? (w.y >> w.z) & 255u : 0u;
      }
      float sc[2][NT][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[x][nt][0] = sc[x][nt][1] = sc[x][nt][2] = sc[x][nt][3] = 0.f;
#pragma unroll
      for (int h = 0; h < kCols; ++h) {
        uint32_t wa[2][4], wb[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint8_t *at_k = src + x * L::kHalfBytes + (k_from ^ h * 64);
          const uint4 a = *reinterpret_cast<const uint4 *>(at_k);
          const uint4 b = *reinterpret_cast<const uint4 *>(at_k + 8 * D);
          wa[x][0] = a.x, wa[x][1] = a.y, wa[x][2] = a.z, wa[x][3] = a.w;
          wb[x][0] = b.x, wb[x][1] = b.y, wb[x][2] = b.z, wb[x][3] = b.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t f[4];
            widen(wa[x][i], f[0], f[2]);
            widen(wb[x][i], f[1], f[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint2 q;
              if constexpr (L::kQInRegs) q = qf[nt][4 * h + i];
              else q = q_at[(nt * kMmas + 4 * h + i) * 32];
              mma(sc[x][nt], f, q.x, q.y);
            }
          }
      }
      // V: four keys a lane and half, D / 8 columns of each, its bytes paired key by key.  (Volatile, as the copies are: the
      // stage has been read when the next copies into it begin.)
      constexpr int kWords = D / 32;
      uint32_t v[2][kWords][4];
      const int j0 = s * kStep;
      const bool tail = j0 + kStep > r.kv_len || !there[0] || !there[1];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t w[4][kWords];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint8_t *at_v = src + x * L::kHalfBytes + v_from;
          if constexpr (D == 128) {
            const uint4 y = *reinterpret_cast<const uint4 *>(at_v + (t & 1) * 128 + (t >> 1) * 1024);
            w[t][0] = y.x, w[t][1] = y.y, w[t][2] = y.z, w[t][3] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2 *>(at_v + (t & 1) * 512 + (t >> 1) * 256);
            w[t][0] = y.x, w[t][1] = y.y;
          }
        }
        if (tail) {  // slots behind the last token, or not there, may hold anything, NaN included
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (!there[x] || j0 + kHalf * x + 2 * c + (t & 1) + 8 * (t >> 1) >= r.kv_len)
#pragma unroll
              for (int i = 0; i < kWords; ++i) w[t][i] = 0u;
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          v[x][i][0] = pair<0x5140>(w[0][i], w[1][i]);
          v[x][i][1] = pair<0x5140>(w[2][i], w[3][i]);
          v[x][i][2] = pair<0x7362>(w[0][i], w[1][i]);
          v[x][i][3] = pair<0x7362>(w[2][i], w[3][i]);
        }
      }
      __syncwarp();  // every lane has read the stage
      issue(stage);
      const uint32_t most = max(ve[0], ve[1]);
      if (most > uint32_t(ref)) {  // the same in all lanes
        const uint32_t finite = max(ve[0] == 255 ? 0u : ve[0], ve[1] == 255 ? 0u : ve[1]);
        if (finite > uint32_t(ref)) {
          const float down = power_of_two(ref - int(finite));
          ref = int(finite);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < kMmas; ++j)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[nt][j][x] *= down;
        }
      }
      const bool masked = tail || j0 + kStep > clear;
      float ks[2], vf[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        ks[x] = scale_value(ke[x]);
        vf[x] = ve[x] == 255 ? scale_value(255) : __uint_as_float(uint32_t(max(127 + int(ve[x]) - ref, 0)) << 23);
      }
      uint32_t pb[2][NT][TERMS][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // log2 of the weights, relative to the running maximum; +inf while there is none
        float y[2][4];
        uint32_t hidden = 0;  // bit 4 half + element
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int k = 0; k < 4; ++k) y[x][k] = fmaf(sc[x][nt][k], qs[nt][k & 1] * ks[x], -m[nt][k & 1]);
        if (masked) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = j0 + kHalf * x + g + 8 * (k >> 1), row = 8 * nt + 2 * c + (k & 1);
              bool sees = row < rows && j < r.kv_len && there[x];
              if (sees && j >= start) {
                const int tok = row / p.G;
                sees = has_tree ? j - start < 64 && (__ldg(reinterpret_cast<const unsigned long long *>(p.tree) + r.token0 + tok) >> (j - start) & 1)
                                : j <= start + tok;
              }
              if (!sees) {
                y[x][k] = neg_inf();
                hidden |= 1u << (4 * x + k);
              }
            }
        }
        const float top = max3(max3(y[0][0], y[0][1], y[0][2]), max3(y[0][3], y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3]));
        if (__any_sync(0xffffffffu, top > kBias + kLazy)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float t = neg_inf();
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int k = i; k < 4; k += 2)
                if (!(hidden >> (4 * x + k) & 1)) t = fmaxf(t, sc[x][nt][k] * (qs[nt][i] * ks[x]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
            if (t > m[nt][i] + (kBias + kLazy)) {
              const float to = t - kBias, alpha = ex2(m[nt][i] - to);
              m[nt][i] = to;
              l[nt][i] *= alpha;
#pragma unroll
              for (int j = 0; j < kMmas; ++j) o[nt][j][i] *= alpha, o[nt][j][2 + i] *= alpha;
            }
            const float n = m[nt][i] == neg_inf() ? 0.f : m[nt][i];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int k = i; k < 4; k += 2)
                y[x][k] = hidden >> (4 * x + k) & 1 ? neg_inf() : fmaf(sc[x][nt][k], qs[nt][i] * ks[x], -n);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float e[4] = {ex2(y[x][0]), ex2(y[x][1]), ex2(y[x][2]), ex2(y[x][3])};
          l[nt][0] += e[0] + e[2];
          l[nt][1] += e[1] + e[3];
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] *= vf[x];
          if (hidden && ve[x] == 255) {  // 0 beside a scale of NaN
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (hidden >> (4 * x + k) & 1) e[k] = 0.f;
          }
#pragma unroll
          for (int z = 0; z < TERMS; ++z) {
            const uint32_t w0 = f16x2_bits(e[0], e[1]), w1 = f16x2_bits(e[2], e[3]);
            pb[x][nt][z][0] = transpose8(w0);
            pb[x][nt][z][1] = transpose8(w1);
            if (z + 1 < TERMS) {
              const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w0)), b = __half22float2(*reinterpret_cast<const __half2 *>(&w1));
              e[0] -= a.x, e[1] -= a.y, e[2] -= b.x, e[3] -= b.y;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        // The tensor cores' sums cut low bits towards zero.  f32 outputs see that: a step's O starts anew, and is added in f32
        // (three tokens over 20000 to 65536 keys: 2.5e-7 of the norm and 41.9 us, against 3.2e-7, most of it bias, and 41.2).
        float now[TERMS > 1 ? NT : 1][2][4] = {};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t f[4], h[4];
          widen(v[x][i][0], f[0], f[1]);
          widen(v[x][i][1], f[2], f[3]);
          widen(v[x][i][2], h[0], h[1]);
          widen(v[x][i][3], h[2], h[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < TERMS; ++z) {
              mma(TERMS > 1 ? now[TERMS > 1 ? nt : 0][0] : o[nt][2 * i], f, pb[x][nt][z][0], pb[x][nt][z][1]);
              mma(TERMS > 1 ? now[TERMS > 1 ? nt : 0][1] : o[nt][2 * i + 1], h, pb[x][nt][z][0], pb[x][nt][z][1]);
            }
        }
        if constexpr (TERMS > 1) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 8; ++k) o[nt][2 * i + (k >> 2)][k & 3] += now[nt][k >> 2][k & 3];
        }
      }
      if (++stage == NS) stage = 0;
    }

    // ------------------------------------------------------------------------ the request's end
    // Lane (g, c) holds columns D / 8 g .. of rows 2 c and 2 c + 1.
    const bool whole = u.s0 == 0 && u.s1 == u.n;
    const float unit = scale_value(uint32_t(ref));  // (times 1 / l first, its product could be too small for f32)
    const int64_t piece = ((int64_t(slot) * 2 + (u.first ? 0 : 1)) * p.Hkv + kv) * 8 * NT;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float all = l[nt][i];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) all += __shfl_xor_sync(0xffffffffu, all, x);
        const int row = 8 * nt + 2 * c + i;
        if (row >= rows) continue;
        const int tok = row / p.G;
        const int64_t out = (int64_t(r.token0) + tok) * p.Hq + kv * p.G + (row - tok * p.G);
        const float f = all == 0.f ? 0.f : 1.f / all;
        const int64_t dst = (whole ? out : piece + row) * D + (D / 8) * g;
        if (whole && TERMS == 1) {
          __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.o) + dst;
#pragma unroll
          for (int j = 0; j < kMmas; j += 4) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 x = __floats2bfloat162_rn(o[nt][j + k][i] * f * unit, o[nt][j + k][2 + i] * f * unit);
              w[k] = *reinterpret_cast<const uint32_t *>(&x);
            }
            *reinterpret_cast<uint4 *>(to + 2 * j) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float *to = (whole ? static_cast<float *>(p.o) : p.part_o) + dst;
#pragma unroll
          for (int j = 0; j < kMmas; j += 2)
            *reinterpret_cast<float4 *>(to + 2 * j) = make_float4(o[nt][j][i] * f * unit, o[nt][j][2 + i] * f * unit,
                                                                  o[nt][j + 1][i] * f * unit, o[nt][j + 1][2 + i] * f * unit);
        }
        if (g == 0) {
          const float v = all == 0.f ? neg_inf() : m[nt][i] + log2f(all);
          if (!whole) p.part_lse[piece + row] = v;
          else if (p.lse) p.lse[out] = v;
        }
      }
    }
  }
  copies_wait<0>();
  if (bad) raise_fault(p.fault, bad);
}

// A request's pieces, and the first one's slot.  The slots that have its first step and its last: slot x begins at cost
// floor(x C / slots), and all costs up to kSegmentCost behind the request's begin at its first step.
__host__ __device__ __forceinline__ int pieces_of(const RowsParams &p, const RowsRequests &req, int b, int64_t &first) {
  const int64_t all = req.before[p.B], n = steps_of(req.r[b]);
  first = divide(p, (req.before[b] + kSegmentCost + 1) * p.slots - 1, all);
  const int64_t last = divide(p, (req.before[b] + kSegmentCost + n) * p.slots - 1, all);
  return int((last < p.slots - 1 ? last : int64_t(p.slots) - 1) - first) + 1;
}

// Joins the pieces of a row, kFewPieces at most, a warp a row (request blockIdx.x, KV head blockIdx.y, four rows a CTA): a lane
// has D / 32 columns of all pieces, and its own piece's LSE.  (With the kernel below 32 single tokens took 36 us, 34 so.)
template <int D>
__global__ void __launch_bounds__(128) rows_join_few_kernel(const RowsParams p, const __grid_constant__ RowsRequests req, int unit_rows) {
  constexpr int N = D / 32;
  using Vec = std::conditional_t<N == 4, float4, float2>;
  const int b = blockIdx.x, kv = blockIdx.y, lane = threadIdx.x & 31, row = blockIdx.z * 4 + (threadIdx.x >> 5);
  const psd_token_request &r = req.r[b];
  int64_t first;
  const int pieces = pieces_of(p, req, b, first), late = begin_of(p, req, int(first)).x < b;
  wait_for_prior_grid();
  if (pieces == 1 || row >= r.num_new * p.G) return;
  // (all pieces' numbers fit 31 bits: step_rows_floats)
  const int stride = 2 * p.Hkv * unit_rows, at0 = int(first) * stride + kv * unit_rows + row, late_by = late * p.Hkv * unit_rows;
  auto at = [&](int i) { return at0 + i * stride + (i == 0 ? late_by : 0); };
  const float lse = lane < pieces ? p.part_lse[at(lane)] : neg_inf();
  float y[kFewPieces][N];
#pragma unroll
  for (int i = 0; i < kFewPieces; ++i)
    if (i < pieces) *reinterpret_cast<Vec *>(y[i]) = *reinterpret_cast<const Vec *>(p.part_o + at(i) * D + N * lane);
  float m = lse;
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float w = ex2(lse - (m == neg_inf() ? 0.f : m));
  float sum = w, x[N] = {};
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
  for (int i = 0; i < kFewPieces; ++i) {
    const float f = __shfl_sync(0xffffffffu, w, i);
    if (i < pieces)
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = fmaf(f, y[i][k], x[k]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] *= inv;
  const int tok = row / p.G;
  const int64_t out = (int64_t(r.token0) + tok) * p.Hq + kv * p.G + (row - tok * p.G), o = out * D + N * lane;
  if (p.out_f32) {
    *reinterpret_cast<Vec *>(static_cast<float *>(p.o) + o) = *reinterpret_cast<const Vec *>(x);
  } else {
    __nv_bfloat162 z[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) z[k] = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.o) + o;
    if constexpr (N == 4) *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(z);
    else *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(z);
  }
  if (lane == 0 && p.lse) p.lse[out] = sum == 0.f ? neg_inf() : m + log2f(sum);
}

// Joins the pieces of a row (request blockIdx.x, KV head blockIdx.y, row blockIdx.z): D / 4 threads a piece take every
// NG-th of them, in an order that does not change.
template <int D>
__global__ void __launch_bounds__(256) rows_join_kernel(const RowsParams p, const __grid_constant__ RowsRequests req, int unit_rows) {
  constexpr int kLanes = D / 4, NG = 256 / kLanes;
  __shared__ float4 part[NG][kLanes];
  constexpr int kAhead = 8;
  __shared__ float tops[8], sums[8], weight[kMostPieces];
  const int b = blockIdx.x, kv = blockIdx.y, row = blockIdx.z, tid = threadIdx.x;
  const psd_token_request &r = req.r[b];
  int64_t first;
  const int pieces = pieces_of(p, req, b, first), late = begin_of(p, req, int(first)).x < b;  // the first piece is the second of its slot
  wait_for_prior_grid();
  if (pieces == 1 || row >= r.num_new * p.G) return;    // whole
  // (all pieces' numbers fit 31 bits: step_rows_floats)
  const int stride = 2 * p.Hkv * unit_rows, at0 = int(first) * stride + kv * unit_rows + row, late_by = late * p.Hkv * unit_rows;
  auto at = [&](int i) { return at0 + i * stride + (i == 0 ? late_by : 0); };
  const int group = tid / kLanes, col = tid % kLanes * 4;
  const float *piece = p.part_o + col;
  float4 y[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)  // on their way beside the LSEs
    if (group + k * NG < pieces) y[k] = *reinterpret_cast<const float4 *>(piece + at(group + k * NG) * D);
  float m = neg_inf();
  for (int i = tid; i < pieces; i += 256) {
    weight[i] = p.part_lse[at(i)];
    m = fmaxf(m, weight[i]);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (tid % 32 == 0) tops[tid / 32] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, tops[w]);
  const float from = m == neg_inf() ? 0.f : m;
  float sum = 0.f;
  for (int i = tid; i < pieces; i += 256) {
    const float w = ex2(weight[i] - from);
    weight[i] = w;
    sum += w;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (tid % 32 == 0) sums[tid / 32] = sum;
  __syncthreads();
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = group; i0 < pieces; i0 += kAhead * NG) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * NG;
      if (i >= pieces) break;
      const float w = weight[i];
      const float4 z = y[k];
      if (i + kAhead * NG < pieces) y[k] = *reinterpret_cast<const float4 *>(piece + at(i + kAhead * NG) * D);
      x.x = fmaf(w, z.x, x.x), x.y = fmaf(w, z.y, x.y), x.z = fmaf(w, z.z, x.z), x.w = fmaf(w, z.w, x.w);
    }
  }
  part[group][tid % kLanes] = x;
  __syncthreads();
  if (group) return;
#pragma unroll
  for (int k = 1; k < NG; ++k) {
    const float4 z = part[k][tid];
    x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
  }
  sum = sums[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) sum += sums[k];
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int tok = row / p.G;
  const int64_t out = (int64_t(r.token0) + tok) * p.Hq + kv * p.G + (row - tok * p.G), o = out * D + col;
  if (p.out_f32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + o) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x * inv, x.y * inv), hi = __floats2bfloat162_rn(x.z * inv, x.w * inv);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + o) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  }
  if (tid == 0 && p.lse) p.lse[out] = sum == 0.f ? neg_inf() : m + log2f(sum);
}

// Slots for the workers of so many CTAs.
int slots_of(int ctas, int Hkv) { return std::max(1, std::min(ctas * kWarps / Hkv, kMostPieces)); }

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
  p.num_scales = int(S.num_pages * (S.page_size >> S.scales.shift) * S.Hkv);
  p.Hq = S.Hq;
  p.Hkv = S.Hkv;
  p.G = S.G;
  p.page_size = S.page_size;
  p.shift = S.scales.shift;
  p.out_f32 = S.out_f32;
  p.q_scale = S.q_scale;
  p.B = S.B;
  RowsRequests req;
  std::memcpy(req.r, sreq.r, sizeof(psd_token_request) * size_t(S.B));
  req.before[0] = 0;
  for (int b = 0; b < S.B; ++b) req.before[b + 1] = req.before[b] + steps_of(req.r[b]) + kSegmentCost;
  const int most = slots_of(L::kCtasPerSm * dev.num_sms, S.Hkv);
  p.slots = int(std::max<int64_t>(1, std::min<int64_t>(most, req.before[S.B] / kLeastSteps)));
  // A slot for each request, and nothing to join, where that takes no longer: 4 requests of 64 keys 4.9 us against 6.4, 50 of
  // 128 8.4 against 11.7; of 256 keys (8 steps) 9.8 against 7.0, and 12.8 against 13.8.
  int longest = 0;
  for (int b = 0; b < S.B; ++b) longest = std::max(longest, steps_of(req.r[b]));
  p.whole = S.B <= most && longest <= req.before[S.B] / p.slots + kJoinSteps;
  if (p.whole) p.slots = S.B;
  p.narrow = (req.before[S.B] + 1) * (int64_t(p.slots) + 1) < int64_t(1) << 32;
  const int64_t ctas = (int64_t(p.slots) * S.Hkv + kWarps - 1) / kWarps;
  p.part_o = base;
  p.part_lse = base + int64_t(p.slots) * 2 * S.Hkv * 8 * NT * D;
  auto kern = rows_kernel<D, NT, TERMS>;
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = dev.device < 64 ? uint64_t(1) << dev.device : 0;
  cudaError_t e = cudaSuccess;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(L::kSmem));
    if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    ready.fetch_or(bit, std::memory_order_release);
  }
  kern<<<unsigned(ctas), kThreads, L::kSmem, s>>>(p, req);
  e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "multi_token_decode_scaled launch: %s", cudaGetErrorString(e));
  if (p.slots == 1 || p.whole) return PSD_OK;
  cudaLaunchConfig_t cfg = {};
  int rows = 0, pieces = 0;
  int64_t first;
  for (int b = 0; b < S.B; ++b) {
    rows = std::max(rows, req.r[b].num_new * S.G);
    pieces = std::max(pieces, pieces_of(p, req, b, first));
  }
  const bool few = pieces <= kFewPieces;
  cfg.gridDim = dim3(unsigned(S.B), unsigned(S.Hkv), unsigned(few ? (rows + 3) / 4 : rows));
  cfg.blockDim = dim3(few ? 128 : 256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, few ? rows_join_few_kernel<D> : rows_join_kernel<D>, p, req, 8 * NT);
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "multi_token_decode_scaled join launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}

}  // namespace

bool step_rows_supports(const StepParams &p) {
  return p.scaled && (p.D == 64 || p.D == 128) && p.G <= kFewRows && p.num_pages * (p.page_size / kHalf) * p.Hkv <= 0x7fffffffLL &&
         ((reinterpret_cast<uintptr_t>(p.scales.k) | reinterpret_cast<uintptr_t>(p.scales.v)) & 3) == 0;
}

size_t step_rows_floats(int sms, int D) {
  // slots * Hkv is at most the workers of the CTAs, 12 an SM with 8 rows and 8 with up to four times as many; or, with
  // more heads than that, one slot, which leaves no pieces
  return size_t(sms) * 2 * kWarps * 2 * kFewRows * (size_t(D) + 1);
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
