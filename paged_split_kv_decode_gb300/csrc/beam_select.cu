// Beam search's selection (the contract is in include/psd.h).
//
// Mathematics.  v(r, t) = score(r) + x(r, t) - log sum exp x(r, s): within a row the order is that of the
// logits, so a row's k largest logits hold all of it that can be chosen, and its sum enters only when rows
// meet.  One pass over the logits finds both.
//   Sum: in units of 2^R, R an integer near the running maximum of a thread's logits in log2 units, -2^23 at least: the term
// is 2^(x log2 e - R), log2 e in two f32 pieces so that what is rounded is the difference, not the product.  16 terms are added
// pairwise, the 16-sums with the error of each addition kept beside it; threads and splits meet as such pairs too, rows in 64
// bits.  What is left is the rounding of the single terms: 2^-20 of a term at most (exp2 2 ulp, 2^-22; its argument, up to 16,
// rounded twice, 2^-21 ln 2 each), so that of the sum where one term is most of it, and some 1e-8 where many are alike.  It does
// not depend on where a row lies in memory: equal rows tie (those of a request are split alike).  Beyond 2^23 either way R would
// not be an integer near the maximum any more.  Logits of -2^23 and less, masks mostly, add nothing to a sum with larger ones; a
// row whose largest lies so far off is summed once more by the second kernel, relative to that logit, and its values are the
// logits' differences from it.
//   Candidates: each warp takes the r-th largest of its lanes' largest logits, r = ceil(k / 8); the least of the
// 8 warps' is a lower bound of the k-th largest (8 r >= k logits are no smaller), found without a sort.  The pass keeps
// each thread's largest of every tile; some 2 k of these are not below the bound, and only their 16 logits are read again.
// Order numbers (a count of the larger ones) give the exact k.  All in all a
// logit of bf16 takes 13 instructions; with a bound and a search tile by tile 240 rows of 131072 bf16 took 34 us against 23.
// Where more is found than there is room for (many equal logits) the CTA goes over its logits again and thins them out on the
// way, which is slow: with half of the logits equal, at the top, 128 rows of 98305 f32 take 430 us against 20, and 421 with nine
// tenths of each row at a finite mask such as -1e10 (a CTA's share of a row may be masked whole; masks of -inf: 18).
//
// Rows are split so that all SMs have equal work: the rows that are read (not finished, not empty) share the CTAs that run
// at once, to within a split.  A second kernel, one CTA a request, joins the splits' sums and takes the k largest of the
// rows' candidates in 64 bits.
//
// 128 rows of 98305 f32, a fifth of them finished: 17 us (40 MB, 6 us at the copy rate), 11 of them the first kernel; bound by the
// chain of a CTA's steps around its 16000 logits (its row, the bound, the search, the order), then by the second kernel's
// chain.  240 rows of 131072 bf16: 23 us (8 us at the copy rate); f16 25 and bf16 26 with no beam finished.  59 % of the issue
// slots and 32 % of DRAM: its warps wait for the tile ahead (38 % of their time) and for results (18 %) more than for either.  A
// row that lies far from zero: 24 us more, for the second kernel's pass over 98305 logits.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "context.h"
#include "device.cuh"
#include "kernels.h"

namespace psd {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 2048;                 // a split's logits are a multiple of this
constexpr int kSlots = 16;                   // a thread's maxima that are kept: of a tile each, or of several
constexpr int kKeep = 1024;                  // candidates there is room for, and threads' tiles that hold some
constexpr int kFew = 256;                    // candidates that are put in order among themselves
constexpr int kMaxK = 64, kMaxBeams = 64, kMaxVocab = 1 << 30;  // (so that a place behind the last tile is an int)
constexpr int kMost = 8192;                  // candidates of a request in the second kernel
constexpr float kFar = 8388608.f;            // 2^23, in log2 units

struct SelectParams {
  const void *logits;
  int64_t stride;
  int type;                  // psd_logits_type
  const float *scores;
  const uint8_t *finished;
  int rows, beams, vocab, k, pad;
  int pieces, most_splits;   // CTAs of the first kernel; of a row at most (1: piece and row are the same number)
  float *out_scores;
  int32_t *out_rows, *out_tokens, *fault;
  float2 *sums;              // [pieces] in units of 2^ref, two pieces of a number
  int2 *refs;                // [pieces] R's bits, and the row's number in its request
  unsigned long long *keys;  // [pieces][k] descending, 0: none
  uint32_t *marks;           // the rows that are read, for calls that write the scores over those they had
  bool in_place;
};

// Rows whose logits are read share the pieces: of L such rows the j-th has those from first(j) to first(j + 1), `splits` of
// them or, the rows of the first requests, one more.  The rows of a request are split alike, so that equal ones have
// equal sums.  (A NaN score is reported by the second kernel.)
constexpr int kMostRanked = 1024;
static_assert(kMostRanked / 32 == 32, "a lane a word");
struct Shares {
  int rows, splits, more;  // L, and how many rows have one more
  __device__ __forceinline__ int pieces() const { return rows * splits + more; }
  __device__ __forceinline__ int first(int j) const { return j * splits + min(j, more); }
  __device__ __forceinline__ int row_of(int piece) const {
    const int those = more * (splits + 1);
    return piece < those ? int(uint32_t(piece) / uint32_t(splits + 1)) : more + int(uint32_t(piece - those) / uint32_t(splits));
  }
};
// All rows' bits, 32 a word; all kThreads threads.
__device__ __forceinline__ void mark_rows(const SelectParams &p, uint32_t *words) {
  constexpr int kEach = kMostRanked / kThreads;
  float score[kEach];
  uint8_t done[kEach];
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    if (n * kThreads >= p.rows) break;
    const int i = n * kThreads + int(threadIdx.x);
    score[n] = i < p.rows ? p.scores[i] : neg_inf();
    done[n] = i < p.rows && p.finished ? p.finished[i] : uint8_t(0);
  }
#pragma unroll
  for (int n = 0; n < kEach; ++n) {
    if (n * kThreads >= p.rows) {
      if (threadIdx.x < kWarps) words[n * kWarps + threadIdx.x] = 0;
      continue;
    }
    const uint32_t is = __ballot_sync(0xffffffffu, score[n] != neg_inf() && !done[n]);
    if ((threadIdx.x & 31) == 0) words[(n * kThreads + int(threadIdx.x)) / 32] = is;
  }
}
// A warp's view of the marks: rows of the lane's word, and before it.
struct Ranks {
  const uint32_t *words;
  int here, before, all;
  __device__ __forceinline__ explicit Ranks(const uint32_t *w) : words(w) {
    here = __popc(words[threadIdx.x & 31]);
    before = here;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, d);
      if ((threadIdx.x & 31) >= d) before += y;
    }
    all = __shfl_sync(0xffffffffu, before, 31);
    before -= here;
  }
  __device__ __forceinline__ int row_of(int rank) const {  // the same in all lanes, below `all`
    const int lane = threadIdx.x & 31;
    const int word = __ffs(__ballot_sync(0xffffffffu, rank >= before && rank < before + here)) - 1;
    const uint32_t is = words[word];
    const int in_word = rank - __shfl_sync(0xffffffffu, before, word);
    return 32 * word + __ffs(__ballot_sync(0xffffffffu, (is >> lane & 1) && __popc(is & ((1u << lane) - 1u)) == in_word)) - 1;
  }
  __device__ __forceinline__ int rank_of(int row) const {  // rows that are read before it; each lane its own, up to kMostRanked
    const int x = __shfl_sync(0xffffffffu, before, row / 32 & 31);
    return row >= kMostRanked ? all : x + __popc(words[row / 32] & ((1u << (row & 31)) - 1u));
  }
  __device__ __forceinline__ Shares shares(const SelectParams &p) const {
    Shares s{all, 1, 0};
    if (all == 0) return s;
    s.splits = min(int(uint32_t(p.pieces) / uint32_t(all)), p.most_splits);
    const int spare = s.splits < p.most_splits ? p.pieces - all * s.splits : 0;  // (fewer than the rows)
    if (spare > 0) {
      const int row = row_of(spare);
      s.more = rank_of(row - row % p.beams);
    }
    return s;
  }
};
// log2 of s + e to 1.4e-9, as its integer part and the rest: with r near 1 / m, 9 bits, m = s 2^-n in [1, 2),
// log2 m = -log2 r + log2(1 + t), t = m r - 1 below 2^-7 exact but for its last bit, and four terms of a series.  (In 64 bits
// a logarithm is some 40 slow operations that a whole CTA waits for: 0.7 us of 18.)
struct Logs {
  float r[128], high[128], low[128];  // r, and -log2 r in two pieces
  constexpr Logs() : r{}, high{}, low{} {
    for (int i = 0; i < 128; ++i) {
      const int k = int(512.0 * 128.0 / (128.0 + i + 0.5) + 0.5);  // r = k / 512
      const double x = k / 512.0, y = (x - 1) / (x + 1);           // ln x = 2 (y + y^3 / 3 + ..)
      double sum = 0, power = y;
      for (int n = 0; n < 40; ++n) sum += power / (2 * n + 1), power *= y * y;
      const double log2 = -2 * sum * 1.4426950408889634074;
      r[i] = float(x), high[i] = float(log2), low[i] = float(log2 - double(float(log2)));
    }
  }
};
__constant__ const Logs kLogs = Logs();
__device__ __forceinline__ double log2_of(float s, float e, float ref) {  // 2^ref (s + e), s normal
  const int u = __float_as_int(s), n = (u >> 23) - 127, i = u >> 16 & 127;
  const float m = __int_as_float((u & 0x7fffff) | 0x3f800000), tail = e * __int_as_float((127 - max(n, -126)) << 23);
  const float r = kLogs.r[i], t = fmaf(tail, r, fmaf(m, r, -1.f));
  const float p = t * fmaf(t, fmaf(t, fmaf(t, -0.360673760f, 0.480898347f), -0.721347520f), 1.442695041f);
  return double(ref) + double(n) + (double(kLogs.high[i]) + double(kLogs.low[i] + p));
}
// (s, e) += (t, f), s and e two pieces of a number: f32 with an error of some 2^-47.
__device__ __forceinline__ void add_pairs(float &s, float &e, float t, float f) {
  const float sum = s + t, part = sum - s;
  e = e + f + ((s - (sum - part)) + (t - part));
  s = sum;
}

// Unsigned numbers that are ordered as floats and doubles are (no NaN; -0 is made 0 before).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) { return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu)); }
__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long u = __double_as_longlong(x + 0.0);
  return u ^ (u >> 63 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double from_ordered(unsigned long long o) {
  return __longlong_as_double((long long)(o ^ (o >> 63 ? 1ull << 63 : ~0ull)));
}
// A candidate: larger logits first, then lower tokens.  0 is less than all.
__device__ __forceinline__ unsigned long long key_of(float x, uint32_t token) {
  return (unsigned long long)(ordered(x)) << 32 | (0xffffffffu - token);
}

__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN operands lose, as in fmaxf
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The r-th largest of the lanes' values (equal ones count singly).
__device__ __forceinline__ uint32_t nth_largest(uint32_t v, int r) {
  uint32_t top = 0;
  for (int i = 0; i < r; ++i) {
    top = __reduce_max_sync(0xffffffffu, v);
    const uint32_t who = __ballot_sync(0xffffffffu, v == top);
    if ((threadIdx.x & 31) == __ffs(who) - 1) v = 0;
  }
  return top;
}
template <typename T> __device__ __forceinline__ float logit(T x);
template <> __device__ __forceinline__ float logit<float>(float x) { return x; }
template <> __device__ __forceinline__ float logit<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float logit<__half>(__half x) { return __half2float(x); }
// A 32-bit word's logits.
template <typename T> __device__ __forceinline__ void unpack(uint32_t w, float *x) {
  if constexpr (sizeof(T) == 4) {
    x[0] = __uint_as_float(w);
  } else if constexpr (std::is_same_v<T, __half>) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    x[0] = f.x, x[1] = f.y;
  } else {
    x[0] = bf16_lo(w), x[1] = bf16_hi(w);
  }
}

// What a CTA takes at a time: 16 logits a thread, the next on their way while a tile is worked on.
constexpr int kPer = 16, kTile = kThreads * kPer;
constexpr int kStep = kThreads * 4;          // the same where candidates are thinned out on the way

// A CTA a piece.  VEC: rows are 16-byte aligned; otherwise a warp's loads are
// neighbours one by one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) select_rows_kernel(const SelectParams p) {
  constexpr int N = 16 / int(sizeof(T));  // logits of a 16-byte load
  __shared__ float tops[kSlots][kThreads];
  __shared__ unsigned long long kept[kKeep + kStep], few[kFew], chosen[kMaxK];
  __shared__ uint16_t found[kKeep];         // slot and thread
  __shared__ float bound[kWarps];
  __shared__ int n_found, n_kept, n_few;
  __shared__ float warp_ref[kWarps], warp_sum[kWarps], warp_rest[kWarps];
  dependents_may_launch();
  const int piece = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int row = piece, begin = 0, size = p.vocab;
  if (p.most_splits > 1) {
    __shared__ uint32_t words[kMostRanked / 32];
    mark_rows(p, words);
    __syncthreads();
    const Ranks ranks(words);
    const Shares shares = ranks.shares(p);
    if (p.in_place && piece == 0 && tid < kMostRanked / 32) p.marks[tid] = words[tid];
    if (piece >= shares.pieces()) return;
    const int j = shares.row_of(piece), first = shares.first(j), splits = shares.first(j + 1) - first;
    row = ranks.row_of(j);
    const int chunks = (p.vocab + kChunk - 1) / kChunk, at = piece - first;
    begin = int(uint32_t(at * chunks) / uint32_t(splits)) * kChunk;  // (at < 64, chunks < 2^20)
    size = min(int(uint32_t((at + 1) * chunks) / uint32_t(splits)) * kChunk, p.vocab) - begin;
  } else if (p.scores[row] == neg_inf() || (p.finished && p.finished[row])) {
    return;  // no continuations, or one: the second kernel sees to it
  }
  const T *x_split = static_cast<const T *>(p.logits) + int64_t(row) * p.stride + begin;
  const int r = (p.k + kWarps - 1) / kWarps;
  if (tid == 0) n_found = n_kept = 0;
  // Where a thread's c-th logit lies in a tile.
  auto place_of = [&](int t, int c) { return VEC ? (c / N) * (kThreads * N) + t * N + c % N : c * kThreads + t; };
  auto place = [&](int c) { return place_of(tid, c); };
  constexpr int kRaw = VEC ? kPer * int(sizeof(T)) / 4 : kPer;  // words on their way
  uint32_t raw[kRaw];
  const T *x_mine = x_split + place(0);
  auto load = [&](int tile) {
    const bool all = tile + kTile <= size;
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < kPer; c += N)
        if (all || tile + place(c) + N <= size) {
          const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(x_mine + tile + (place(c) - place(0))));
          raw[4 * (c / N)] = w.x, raw[4 * (c / N) + 1] = w.y, raw[4 * (c / N) + 2] = w.z, raw[4 * (c / N) + 3] = w.w;
        }
    } else {
      using Word = std::conditional_t<sizeof(T) == 4, uint32_t, unsigned short>;
      const Word *at = reinterpret_cast<const Word *>(x_mine + tile);
      if (all) {
#pragma unroll
        for (int c = 0; c < kPer; ++c) raw[c] = __ldcs(at + c * kThreads);
      } else {
#pragma unroll
        for (int c = 0; c < kPer; ++c)
          if (tile + place(c) < size) raw[c] = __ldcs(at + c * kThreads);
      }
    }
  };
  float x[kPer];
  auto values = [&](int tile) {
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < kPer; c += N)
#pragma unroll
        for (int w = 0; w < 4; ++w) unpack<T>(raw[4 * (c / N) + w], x + c + w * (N / 4));
      if (tile + kTile > size) {
#pragma unroll
        for (int c = 0; c < kPer; c += N)
          if (tile + place(c) + N > size)
#pragma unroll
            for (int i = 0; i < N; ++i) x[c + i] = tile + place(c + i) < size ? logit<T>(x_split[tile + place(c + i)]) : neg_inf();
      }
    } else {
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        float two[2];
        unpack<T>(raw[c], two);
        x[c] = two[0];
      }
      if (tile + kTile > size) {
#pragma unroll
        for (int c = 0; c < kPer; ++c)
          if (tile + place(c) >= size) x[c] = neg_inf();
      }
    }
  };
  constexpr float kL = 1.44269502f, kL2 = 1.92596303e-8f;  // log2 e, f32 and the rest
  float ref = -kFar, sum = 0.f, rest = 0.f, best = neg_inf();
  auto lowest = [&]() {
    float low = bound[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) low = fminf(low, bound[w]);
    return low;
  };
  // The k largest of those kept, in order, to the front; all threads, behind a barrier.
  auto thin = [&]() {
    const int n = n_kept;
    const float low = lowest();
    const unsigned long long least = low == neg_inf() ? 1ull : (unsigned long long)(ordered(low)) << 32;
    if (tid < p.k) chosen[tid] = 0;
    if (tid == 0) n_few = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
      if (kept[i] >= least) {
        const int at = atomicAdd(&n_few, 1);
        if (at < kFew) few[at] = kept[i];
      }
    __syncthreads();
    const int m = n_few <= kFew ? n_few : n;
    const unsigned long long *from = n_few <= kFew ? few : kept;
    for (int i = tid; i < m; i += kThreads) {
      const unsigned long long mine = from[i];
      int larger = 0;
#pragma unroll 8
      for (int j = 0; j < m; ++j) larger += from[j] > mine;
      if (mine >= least && larger < p.k) chosen[larger] = mine;
    }
    __syncthreads();
    if (tid < p.k) kept[tid] = chosen[tid];
    if (tid == 0) n_kept = min(n, p.k);
    __syncthreads();
  };
  auto sharpen = [&]() {
    const uint32_t mine = nth_largest(ordered(best), r);
    if (lane == 0) bound[warp] = from_ordered(mine);
  };

  // ---- one pass over the split's logits: the sum, and each thread's largest of every tile, or of `group` tiles
  const int tiles = (size + kTile - 1) / kTile, group = (tiles + kSlots - 1) / kSlots;
  int slot = 0, left = group;
  float slot_top = neg_inf();
  load(0);
  for (int tile = 0; tile < size; tile += kTile) {
    values(tile);
    if (size - tile > kTile) load(tile + kTile);
    float top = neg_inf();  // (NaN loses)
#pragma unroll
    for (int c = 0; c < kPer; c += 2) top = max3(top, x[c], x[c + 1]);
    slot_top = fmaxf(slot_top, top);
    if (--left == 0) {
      tops[slot++][tid] = slot_top;
      best = fmaxf(best, slot_top);
      slot_top = neg_inf();
      left = group;
    }
    if (__any_sync(0xffffffffu, top * kL > ref + 16.f)) {  // (the warp goes together: 240 rows of bf16 23.0 us against 23.7)
      const float to = fmaxf(ref, fminf(ceilf(top * kL), 3e38f));
      const float down = ex2(ref - to);
      sum *= down, rest *= down;
      ref = to;
    }
    const float from = -ref;
    const float2 from2 = make_float2(from, from), l2 = make_float2(kL, kL), l22 = make_float2(kL2, kL2);
    float2 e[kPer / 2];
#pragma unroll
    for (int c = 0; c < kPer / 2; ++c) {
      const float2 y = make_float2(x[2 * c], x[2 * c + 1]);
      const float2 z = __ffma2_rn(y, l22, __ffma2_rn(y, l2, from2));
      e[c] = make_float2(ex2(z.x), ex2(z.y));
    }
#pragma unroll
    for (int d = kPer / 4; d; d >>= 1)
#pragma unroll
      for (int c = 0; c < d; ++c) e[c] = __fadd2_rn(e[c], e[c + d]);
    float e0 = e[0].x + e[0].y;
    if (e0 != e0) {  // NaN counts as -inf (a sum that is NaN without one: +inf among the logits)
      e0 = 0.f;
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const float y = fmaxf(x[c], neg_inf());
        e0 += ex2(fmaf(y, kL2, fmaf(y, kL, from)));
      }
    }
    const float s = sum + e0, t = s - sum;
    rest += (sum - (s - t)) + (e0 - t);
    sum = s;
  }
  if (left != group) {
    tops[slot++][tid] = slot_top;
    best = fmaxf(best, slot_top);
  }
  sharpen();
  {  // the warp's sum, to its lanes' largest reference.  (A factor below 2^-126 is 0: so are its terms beside the largest.  In
     // 64 bits, which are slow here, this took a fifth of the kernel's time.)
    float most = ref;
#pragma unroll
    for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    const float f = ex2(ref - most);
    sum *= f, rest *= f;
#pragma unroll
    for (int d = 16; d; d >>= 1) add_pairs(sum, rest, __shfl_xor_sync(0xffffffffu, sum, d), __shfl_xor_sync(0xffffffffu, rest, d));
    if (lane == 0) warp_ref[warp] = most, warp_sum[warp] = sum, warp_rest[warp] = rest;
  }
  __syncthreads();

  // ---- the logits that are not below the bound (-inf is no candidate): which threads' tiles have any, then those read anew
  const float low = fmaxf(lowest(), -3.402823466e38f);
  if (best >= low)
    for (int i = 0; i < slot; ++i)
      if (tops[i][tid] >= low) {
        const int at = atomicAdd(&n_found, 1);
        if (at < kKeep) found[at] = uint16_t(i * kThreads + tid);
      }
  __syncthreads();
  bool careful = n_found > kKeep;
  if (!careful) {
    constexpr int kLanes = 16, kAtOnce = kThreads / kLanes, kBatch = 4;  // lanes a thread's tile
    static_assert(kLanes == kPer && kSlots * kThreads <= 65536, "a lane a logit");
    const int jobs = n_found * group, c = tid % kLanes;
    for (int job0 = tid / kLanes; job0 < jobs; job0 += kBatch * kAtOnce) {
      int at[kBatch];
      float v[kBatch];
#pragma unroll
      for (int n = 0; n < kBatch; ++n) {
        const int job = job0 + n * kAtOnce, f = group == 1 ? job : job / group;
        at[n] = -1, v[n] = neg_inf();
        if (job < jobs) {
          const int which = found[f], tile = (which / kThreads) * group + (job - f * group);
          at[n] = tile * kTile + place_of(which % kThreads, c);
          if (at[n] < size) v[n] = logit<T>(x_split[at[n]]);
        }
      }
#pragma unroll
      for (int n = 0; n < kBatch; ++n)
        if (v[n] >= low) {
          const int to = atomicAdd(&n_kept, 1);
          if (to < kKeep) kept[to] = key_of(v[n], uint32_t(begin + at[n]));
        }
    }
    __syncthreads();
    careful = n_kept > kKeep;
  }
  if (careful) {  // logits that rise along the row, many equal ones: tile by tile, the k largest so far
    __syncthreads();
    if (tid == 0) n_kept = 0;
    best = neg_inf();
    unsigned long long least = 0;  // the k-th largest, once there is one
    for (int at = 0; at < size; at += kStep) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kStep / kThreads; ++c) {
        const int i = at + c * kThreads + tid;
        const float y = i < size ? fmaxf(logit<T>(x_split[i]), neg_inf()) : neg_inf();
        const unsigned long long key = key_of(y, uint32_t(begin + i));
        best = fmaxf(best, y);
        if (y != neg_inf() && key > least) kept[atomicAdd(&n_kept, 1)] = key;
      }
      sharpen();
      __syncthreads();
      if (n_kept > kKeep) {
        thin();
        least = kept[p.k - 1];
      }
    }
  }
  unsigned long long *keys = p.keys + int64_t(piece) * p.k;
  if (careful) {
    thin();
    if (tid < p.k) keys[tid] = kept[tid];
  } else {  // (none is below the bound: all are put in order at once)
    const int n = n_kept;
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long mine = kept[i];
      int larger = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) larger += kept[j] > mine;
      if (larger < p.k) keys[larger] = mine;
    }
    for (int i = n + tid; i < p.k; i += kThreads) keys[i] = 0;
  }
  if (warp == kWarps - 1) {  // the warps' sums to the largest reference
    const float own = warp_ref[lane % kWarps];
    float most = own;
#pragma unroll
    for (int d = kWarps / 2; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    const float f = ex2(own - most);
    sum = warp_sum[lane % kWarps] * f, rest = warp_rest[lane % kWarps] * f;
#pragma unroll
    for (int d = kWarps / 2; d; d >>= 1) add_pairs(sum, rest, __shfl_xor_sync(0xffffffffu, sum, d), __shfl_xor_sync(0xffffffffu, rest, d));
    if (lane == 0) {
      p.sums[piece] = make_float2(sum, rest);
      p.refs[piece] = make_int2(__float_as_int(most), row % p.beams);
    }
  }
}

// (s, e): the sum of exp(x - top) over a row, of 2^23 or more in magnitude, where top is its largest logit; all threads.
template <typename T>
__device__ __noinline__ float2 sum_far(const T *x, int vocab, float top) {
  __shared__ float2 of_warp[kWarps];
  float s = 0.f, e = 0.f;
  constexpr int kAtOnce = 16;  // loads on their way
  for (int i0 = threadIdx.x; i0 < vocab; i0 += kAtOnce * kThreads) {
    float y[kAtOnce];
#pragma unroll
    for (int c = 0; c < kAtOnce; ++c) y[c] = i0 + c * kThreads < vocab ? logit<T>(x[i0 + c * kThreads]) : neg_inf();
#pragma unroll
    for (int c = 0; c < kAtOnce; ++c) {
      const float d = y[c] - top;  // (exact where it is not far below 0; NaN is no continuation)
      add_pairs(s, e, d <= 0.f ? ex2(d * 1.44269502f) : 0.f, 0.f);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) add_pairs(s, e, __shfl_xor_sync(0xffffffffu, s, d), __shfl_xor_sync(0xffffffffu, e, d));
  __syncthreads();  // (of the row before)
  if (threadIdx.x % 32 == 0) of_warp[threadIdx.x / 32] = make_float2(s, e);
  __syncthreads();
  s = e = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) add_pairs(s, e, of_warp[w].x, of_warp[w].y);
  return make_float2(s, e);
}

// Of the rows whose far_top is not 0: that becomes their largest logit (0: there is none; +inf stays), and the sums are relative to it.
__device__ __noinline__ void sum_far_rows(const SelectParams &p, int row0, const int *first_of, float *far_top, float *row_sum,
                                          float *row_rest, float *row_ref) {
  for (int w = 0; w < p.beams; ++w) {
    if (far_top[w] == 0.f) continue;
    unsigned long long first_key = 0;  // of the row's pieces
    for (int s = first_of[w]; s < first_of[w + 1]; ++s) first_key = max(first_key, p.keys[int64_t(s) * p.k]);
    const float top = first_key ? from_ordered(uint32_t(first_key >> 32)) : 0.f;
    float2 sum = make_float2(first_key ? 1.f : 0.f, 0.f);
    if (first_key && top < -neg_inf()) {
      const int64_t at = int64_t(row0 + w) * p.stride;
      sum = p.type == PSD_LOGITS_F32   ? sum_far(static_cast<const float *>(p.logits) + at, p.vocab, top)
            : p.type == PSD_LOGITS_F16 ? sum_far(static_cast<const __half *>(p.logits) + at, p.vocab, top)
                                       : sum_far(static_cast<const __nv_bfloat16 *>(p.logits) + at, p.vocab, top);
    }
    __syncthreads();  // (all have seen far_top)
    if (threadIdx.x == 0) far_top[w] = top, row_sum[w] = sum.x, row_rest[w] = sum.y, row_ref[w] = 0.f;
  }
}

// One CTA a request: its rows' logarithms, then the k largest of their candidates.  64 bits are slow here, so f32 sums
// rounded down give a bound, those rounded up say who may reach it, and only these are added and put in order in 64 bits.
__global__ void __launch_bounds__(kThreads) select_join_kernel(const SelectParams p) {
  extern __shared__ unsigned long long shared[];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int most = p.beams * (p.most_splits * p.k + 1);
  unsigned long long *value = shared, *key = shared + most;  // candidates: v in order, and the logit and token
  uint8_t *of = reinterpret_cast<uint8_t *>(key + most);     // and the row
  __shared__ double base[kMaxBeams];                         // what a row's logits, less `far_top`, are added to
  __shared__ float far_top[kMaxBeams];                       // 0, or the largest logit of a row that lies far off
  __shared__ float row_ref[kMaxBeams], row_sum[kMaxBeams], row_rest[kMaxBeams], base_down[kMaxBeams], base_up[kMaxBeams];
  __shared__ uint8_t kind[kMaxBeams];                        // 0: no continuation, 1: pad_token, 2: candidates
  __shared__ float bound[kWarps];
  __shared__ int n_shared, first_of[kMaxBeams + 1];          // a row's first piece
  __shared__ uint32_t words[kMostRanked / 32];
  const int row0 = b * p.beams;
  float score = 0.f;
  bool done = false;
  if (tid < p.beams) {
    score = p.scores[row0 + tid];
    done = p.finished && p.finished[row0 + tid];
  }
  if (tid == 0) n_shared = 0;
  if (p.most_splits > 1) {
    if (!p.in_place) {
      mark_rows(p, words);
    } else {  // (other requests' scores may have been written already)
      wait_for_prior_grid();
      if (tid < kMostRanked / 32) words[tid] = p.marks[tid];
    }
    __syncthreads();
    if (warp < 3) {
      const Ranks ranks(words);
      const Shares shares = ranks.shares(p);
      const int rank = ranks.rank_of(min(row0 + tid, kMostRanked));
      if (tid <= p.beams) first_of[tid] = shares.first(rank);
    }
  } else {
    if (tid <= p.beams) first_of[tid] = row0 + tid;
  }
  __syncthreads();
  const int piece0 = first_of[0], n_keys = (first_of[p.beams] - piece0) * p.k, n_all = n_keys + p.beams;
  wait_for_prior_grid();
  // The i-th candidate's logit and token, 0: none, and its row: the pieces' first, then one for each row that may be finished.
  const uint32_t by_k = (1u << 20) / uint32_t(p.k) + 1u;      // i / k = i by_k >> 20, i < 2^14 and k <= 64
  auto fetch = [&](int i, int &w) {
    w = i - n_keys;
    if (i >= n_keys) return 0ull;
    const int piece = int(uint64_t(uint32_t(i)) * by_k >> 20);
    w = p.most_splits > 1 ? p.refs[piece0 + piece].y : piece;  // (of rows that are not read nothing was written)
    return p.keys[int64_t(piece0) * p.k + i];
  };
  auto candidate = [&](int i, int w, unsigned long long x) {
    if (i >= n_keys) return kind[w] == 1 ? key_of(0.f, uint32_t(p.pad)) : 0ull;
    return kind[w] == 2 ? x : 0ull;  // (rows that are not read have left nothing)
  };
  // A warp takes every eighth candidate, so that all have some of every row: one without any leaves no bound.  A thread's
  // first are on their way beside the sums.
  constexpr int kHeld = 4;
  const int first = lane * kWarps + warp;
  unsigned long long held[kHeld];
  int held_of[kHeld];
#pragma unroll
  for (int n = 0; n < kHeld; ++n)
    if (first + n * kThreads < n_all) held[n] = fetch(first + n * kThreads, held_of[n]);
  bool far_off = false;
  if (tid < p.beams) far_top[tid] = 0.f;
  for (int w = warp; w < p.beams; w += kWarps) {
    const int at = first_of[w], splits = first_of[w + 1] - at;
    float refs[2];
    float2 sums[2];  // at most 64 splits: two a lane
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = lane + 32 * i;
      refs[i] = s < splits ? __int_as_float(p.refs[at + s].x) : neg_inf();
      sums[i] = s < splits ? p.sums[at + s] : make_float2(0.f, 0.f);
    }
    float ref = fmaxf(refs[0], refs[1]);
#pragma unroll
    for (int d = 16; d; d >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, d));
    float total = 0.f, rest = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f = refs[i] == neg_inf() ? 0.f : ex2(refs[i] - ref);
      add_pairs(total, rest, sums[i].x * f, sums[i].y * f);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
      if (d < splits) add_pairs(total, rest, __shfl_xor_sync(0xffffffffu, total, d), __shfl_xor_sync(0xffffffffu, rest, d));
    if (lane == 0) row_sum[w] = total, row_rest[w] = rest, row_ref[w] = ref;  // (lanes behind the splits hold 0)
    far_off |= splits > 0 && !(fabsf(ref) < kFar);
  }
  // (finished rows and those that were never filled have left no sums)
  const bool read = tid < p.beams && !done && fabsf(score) < -neg_inf();
  if (__syncthreads_or(far_off)) {
    if (read) far_top[tid] = fabsf(row_ref[tid]) < kFar ? 0.f : -neg_inf();
    __syncthreads();
    sum_far_rows(p, row0, first_of, far_top, row_sum, row_rest, row_ref);
    __syncthreads();
  }
  if (tid < p.beams) {  // a lane a row: the logarithms at once
    int what = score == neg_inf() ? 0 : done ? 1 : 2;
    bool bad = isnan(score) || score == -neg_inf();
    const float top = far_top[tid];
    double add = double(score);
    if (read) {
      const float sum = row_sum[tid];
      if (sum == 0.f) what = 0;  // nothing but -inf
      else if (top == -neg_inf()) bad = true;
      else add -= log2_of(sum, row_rest[tid], row_ref[tid]) * 0.69314718055994530942;
    }
    if (bad) {
      what = 0;
      atomicOr(p.fault, PSD_FAULT_RANGE);
    }
    base[tid] = add;
    base_down[tid] = top == 0.f ? __double2float_rd(add) : neg_inf();  // (of rows far off all candidates are put in order)
    base_up[tid] = top == 0.f ? __double2float_ru(add) : -neg_inf();
    kind[tid] = uint8_t(what);
  }
  __syncthreads();
  float best = neg_inf();
  auto see = [&](int i, int w, unsigned long long x) {
    x = candidate(i, w, x);
    if (x) best = fmaxf(best, __fadd_rd(from_ordered(uint32_t(x >> 32)), base_down[w]));
  };
#pragma unroll
  for (int n = 0; n < kHeld; ++n)
    if (first + n * kThreads < n_all) see(first + n * kThreads, held_of[n], held[n]);
  for (int i = first + kHeld * kThreads; i < n_all; i += kThreads) {
    int w;
    const unsigned long long x = fetch(i, w);
    see(i, w, x);
  }
  const uint32_t mine = nth_largest(ordered(best), (p.k + kWarps - 1) / kWarps);
  if (lane == 0) bound[warp] = from_ordered(mine);
  __syncthreads();
  float low = bound[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) low = fminf(low, bound[w]);
  auto take = [&](int i, int w, unsigned long long k) {
    k = candidate(i, w, k);
    if (k == 0) return;
    const float x = from_ordered(uint32_t(k >> 32));
    if (__fadd_ru(x, base_up[w]) < low) return;
    const int at = atomicAdd(&n_shared, 1);
    value[at] = ordered((double(x) - double(far_top[w])) + base[w]);
    key[at] = k;
    of[at] = uint8_t(w);
  };
#pragma unroll
  for (int n = 0; n < kHeld; ++n)
    if (first + n * kThreads < n_all) take(first + n * kThreads, held_of[n], held[n]);
  for (int i = first + kHeld * kThreads; i < n_all; i += kThreads) {
    int w;
    const unsigned long long x = fetch(i, w);
    take(i, w, x);
  }
  __syncthreads();
  const int n = n_shared;
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long v = value[i], x = key[i];
    const uint8_t w = of[i];
    int larger = 0, equal = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      larger += value[j] > v;
      equal += value[j] == v;
    }
    if (equal > 1)
      for (int j = 0; j < n; ++j) larger += value[j] == v && (of[j] < w || (of[j] == w && key[j] > x));
    if (larger < p.k) {
      const int64_t to = int64_t(b) * p.k + larger;
      p.out_scores[to] = float(from_ordered(v));
      p.out_rows[to] = b * p.beams + w;
      p.out_tokens[to] = int32_t(0xffffffffu - uint32_t(x));
    }
  }
  for (int i = n + tid; i < p.k; i += kThreads) {
    const int64_t to = int64_t(b) * p.k + i;
    p.out_scores[to] = neg_inf();
    p.out_rows[to] = -1;
    p.out_tokens[to] = -1;
  }
}

// CTAs of the first kernel: those that run at once, four an SM, or the rows if they are more.  (A second wave of few CTAs
// takes as long as the first.)
int pieces_of(int sms, int rows) { return std::max(std::min(4 * sms, kMostRanked), rows); }
// CTAs a row may be split over: what the second kernel's CTA can hold, and twice what all rows would have.
int most_splits(int pieces, int rows, int chunks, int beams, int k) {
  return std::max(1, std::min({2 * ((pieces + rows - 1) / rows), chunks, kMost / (beams * k), 64}));
}

size_t join_bytes(const SelectParams &p) { return size_t(p.beams) * (p.most_splits * p.k + 1) * 17; }

}  // namespace

static psd_status launch_select(const psd_beam_args *a, void *workspace, const DeviceInfo &dev, cudaStream_t s) {
  SelectParams p;
  p.logits = a->logits;
  p.stride = a->logits_stride;
  p.type = a->logits_type;
  p.scores = a->scores;
  p.finished = a->finished;
  p.rows = a->rows;
  p.beams = a->beams;
  p.vocab = a->vocab;
  p.k = a->k;
  p.pad = a->pad_token;
  p.out_scores = a->out_scores;
  p.out_rows = a->out_rows;
  p.out_tokens = a->out_tokens;
  p.fault = a->fault_dev;
  const int chunks = int((int64_t(a->vocab) + kChunk - 1) / kChunk);
  p.pieces = pieces_of(dev.num_sms, a->rows);
  p.most_splits = p.pieces == a->rows ? 1 : most_splits(p.pieces, a->rows, chunks, a->beams, a->k);
  if (p.most_splits == 1) p.pieces = a->rows;
  p.pieces = int(std::min(int64_t(p.pieces), int64_t(p.most_splits) * a->rows));
  uint8_t *at = static_cast<uint8_t *>(workspace);
  const size_t pieces = size_t(p.pieces);
  p.sums = reinterpret_cast<float2 *>(at);
  p.keys = reinterpret_cast<unsigned long long *>(at + pieces * 8);
  p.refs = reinterpret_cast<int2 *>(at + pieces * 8 * (1 + size_t(a->k)));
  p.marks = reinterpret_cast<uint32_t *>(p.refs + pieces);
  p.in_place = a->out_scores == a->scores;
  const size_t size = a->logits_type == PSD_LOGITS_F32 ? 4 : 2;
  const bool vec = aligned16(a->logits) && (a->logits_stride * int64_t(size)) % 16 == 0;
  auto go = [&](auto type) {
    using T = decltype(type);
    auto kern = vec ? select_rows_kernel<T, true> : select_rows_kernel<T, false>;
    kern<<<unsigned(p.pieces), kThreads, 0, s>>>(p);
  };
  if (a->logits_type == PSD_LOGITS_F32) go(float{});
  else if (a->logits_type == PSD_LOGITS_BF16) go(__nv_bfloat16{});
  else go(__half{});
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "beam_select launch: %s", cudaGetErrorString(e));
  const size_t shared = join_bytes(p);
  if (shared > 40 * 1024) {
    e = cudaFuncSetAttribute(select_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 17 * (kMost + kMaxBeams));
    if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a->rows / a->beams));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, select_join_kernel, p);
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "beam_select join launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}

}  // namespace psd

using namespace psd;

extern "C" size_t psd_beam_workspace_bytes(const psd_ctx *ctx, int32_t rows, int32_t beams, int32_t k) {
  if (!ctx || rows < 0 || beams < 1 || beams > kMaxBeams || k < 1 || k > kMaxK || beams * k > 4096) return 0;
  return 256 + size_t(pieces_of(ctx->dev.num_sms, rows)) * (16 + 8 * size_t(k));
}

extern "C" psd_status beam_select(psd_ctx *ctx, const psd_beam_args *a, void *workspace, size_t workspace_bytes,
                                  psd_stream_t stream) {
  clear_error();
  if (!ctx || !a) return fail(PSD_ERR_INVALID_ARG, "beam_select: NULL");
  if (a->beams < 1 || a->k < 1 || a->vocab < 1 || a->rows < 0 || a->rows % a->beams)
    return fail(PSD_ERR_INVALID_ARG, "beam_select: %d rows, %d beams, vocab %d, k %d", a->rows, a->beams, a->vocab, a->k);
  if (a->beams > kMaxBeams || a->k > kMaxK || a->beams * a->k > 4096 || a->vocab > kMaxVocab)
    return fail(PSD_ERR_UNSUPPORTED, "beam_select: at most %d beams, k %d, beams * k 4096, vocab %d (beams %d, k %d, vocab %d)",
                kMaxBeams, kMaxK, kMaxVocab, a->beams, a->k, a->vocab);
  if (a->logits_type < PSD_LOGITS_F32 || a->logits_type > PSD_LOGITS_F16)
    return fail(PSD_ERR_INVALID_ARG, "beam_select: logits_type %d", a->logits_type);
  if (a->logits_stride < a->vocab) return fail(PSD_ERR_INVALID_ARG, "beam_select: logits_stride shorter than a row");
  if (a->rows == 0) return PSD_OK;
  if (!a->logits || !a->scores || !a->out_scores || !a->out_rows || !a->out_tokens || !a->fault_dev)
    return fail(PSD_ERR_INVALID_ARG, "beam_select: NULL pointer");
  if (reinterpret_cast<uintptr_t>(a->logits) % (a->logits_type == PSD_LOGITS_F32 ? 4 : 2))
    return fail(PSD_ERR_INVALID_ARG, "beam_select: logits alignment");
  const int64_t outputs = int64_t(a->rows / a->beams) * a->k;
  auto over = [&](const void *out, const void *in, int size) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(out), y = reinterpret_cast<uintptr_t>(in);
    return in && x < y + uintptr_t(a->rows) * size && y < x + uintptr_t(outputs) * 4;
  };
  if (over(a->out_rows, a->finished, 1) || over(a->out_tokens, a->finished, 1) || over(a->out_scores, a->finished, 1))
    return fail(PSD_ERR_INVALID_ARG, "beam_select: outputs overlap finished");
  if (over(a->out_rows, a->scores, 4) || over(a->out_tokens, a->scores, 4) ||
      (over(a->out_scores, a->scores, 4) && !(a->out_scores == a->scores && a->k == a->beams)))
    return fail(PSD_ERR_INVALID_ARG, "beam_select: outputs overlap scores (out_scores may be scores where k is beams)");
  if (!workspace || !aligned16(workspace)) return fail(PSD_ERR_INVALID_ARG, "beam_select: workspace must be 16-byte aligned");
  const size_t need = psd_beam_workspace_bytes(ctx, a->rows, a->beams, a->k);
  if (workspace_bytes < need) return fail(PSD_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", workspace_bytes, need);
  DeviceGuard g(ctx->dev.device);
  return launch_select(a, workspace, ctx->dev, reinterpret_cast<cudaStream_t>(stream));
}
