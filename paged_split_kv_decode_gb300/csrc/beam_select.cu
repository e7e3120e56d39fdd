// Beam search's selection (the contract is in include/psd.h).
//
// Mathematics.  v(r, t) = score(r) + x(r, t) - log sum exp x(r, s): within a row the order is that of the
// logits, so a row's k largest logits hold all of it that can be chosen, and its sum enters only when rows
// meet.  One pass over the logits finds both.
//   Sum: in units of 2^R, R an integer near the running maximum of a thread's logits in log2 units: the term is
// 2^(x log2 e - R), log2 e in two f32 pieces so that what is rounded is the difference, not the product.  16
// terms are added pairwise, the 16-sums with the error of each addition kept beside it, and threads, splits and
// rows meet in 64 bits.  What is left is the rounding of the single terms, some 1e-8 of the sum, and does not
// depend on where a row lies in memory: equal rows tie.
//   Candidates: each warp keeps the r-th largest of its lanes' largest logits, r = ceil(k / 8); the least of the
// 8 warps' is a lower bound of the k-th largest so far (8 r >= k logits are no smaller), found without a sort, and
// rises tile by tile.  What is not below it is kept: some k ln(tiles) + k of a CTA's logits.  Order numbers
// among those that are not below the last bound (a count of the larger ones) give the exact k.  Warps wait for each
// other only after the first tile, which makes the bound: with two barriers a tile 240 rows of 131072 took 38 us.
// Where more is kept than there is room for (logits that rise, many equal ones) the CTA begins again and thins them
// out tile by tile.
//
// A row is split over CTAs so that all SMs have work; a second kernel, one CTA a request, joins the
// splits' sums and takes the k largest of the rows' candidates in 64 bits.
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
constexpr int kKeep = 1024;                  // candidates before they are thinned out
constexpr int kFew = 256;                    // candidates at the end that are put in order among themselves
constexpr int kMaxK = 64, kMaxBeams = 64, kMaxVocab = 1 << 30;  // (so that a place behind the last tile is an int)
constexpr int kMost = 8192;                  // candidates of a request in the second kernel

struct SelectParams {
  const void *logits;
  int64_t stride;
  const float *scores;
  const uint8_t *finished;
  int rows, beams, vocab, k, pad, splits, chunk;
  float *out_scores;
  int32_t *out_rows, *out_tokens, *fault;
  double *sums;              // [rows][splits] in units of 2^ref
  float *refs;               // [rows][splits]
  unsigned long long *keys;  // [rows][splits][k] descending, 0: none
};

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

// blockIdx.x: split, blockIdx.y (and z): row.  VEC: rows are 16-byte aligned; otherwise a warp's loads are
// neighbours one by one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) select_rows_kernel(const SelectParams p) {
  constexpr int N = 16 / int(sizeof(T));  // logits of a 16-byte load
  __shared__ unsigned long long kept[kKeep + kTile], few[kFew], chosen[kMaxK];
  __shared__ volatile float bound[kWarps];
  __shared__ int n_kept, n_few;
  __shared__ double warp_sum[kWarps];
  __shared__ float warp_ref[kWarps];
  dependents_may_launch();
  const int row = int(blockIdx.y + gridDim.y * blockIdx.z), split = blockIdx.x;
  if (row >= p.rows) return;
  const float score = p.scores[row];
  // no continuations, or one: the second kernel sees to it (a NaN goes on, to be reported there)
  if (score == neg_inf() || (p.finished && p.finished[row])) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int begin = split * p.chunk, size = min(p.vocab - begin, p.chunk);  // (below 2^31: the splits cover the row just)
  const T *x_split = static_cast<const T *>(p.logits) + int64_t(row) * p.stride + begin;
  const int r = (p.k + kWarps - 1) / kWarps;
  if (tid == 0) n_kept = 0;
  // Where a thread's c-th logit lies in a tile.
  auto place = [&](int c) { return VEC ? (c / N) * (kThreads * N) + tid * N + c % N : c * kThreads + tid; };
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
  float ref = neg_inf(), sum = 0.f, rest = 0.f, best = neg_inf();
  auto lowest = [&]() {
    float low = bound[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) low = fminf(low, bound[w]);
    return low;
  };
  // The k largest of those kept, in order, to the front; all threads.
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
  // One pass over the split's logits.  Careful: what is kept is thinned out wherever there could be too much of it.
  // Otherwise false where there was.
  auto pass = [&](bool careful) {
    const int room = careful ? kKeep : kKeep + kTile;
    bool full = false;  // this thread has found no room, or, careful, put one behind the kKeep-th
    load(0);
    for (int tile = 0; tile < size; tile += kTile) {
      values(tile);
      if (size - tile > kTile) load(tile + kTile);
      float top = neg_inf();  // (NaN loses)
#pragma unroll
      for (int c = 0; c < kPer; c += 2) top = max3(top, x[c], x[c + 1]);
      if (top * kL > ref + 16.f) {  // (false while all are -inf)
        const float to = fminf(ceilf(top * kL), 3e38f);
        const float down = ref == neg_inf() ? 0.f : ex2(ref - to);
        sum *= down, rest *= down;
        ref = to;
      }
      const float from = ref == neg_inf() ? 0.f : -ref;
      const float2 from2 = make_float2(from, from), l2 = make_float2(kL, kL), l22 = make_float2(kL2, kL2);
      float e0;
      for (;;) {
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
        e0 = e[0].x + e[0].y;
        if (e0 == e0) break;
        bool nan = false;  // NaN counts as -inf (a sum that is NaN without one: +inf among the logits)
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          nan |= x[c] != x[c];
          x[c] = fmaxf(x[c], neg_inf());
        }
        if (!nan) break;
      }
      const float s = sum + e0, t = s - sum;
      rest += (sum - (s - t)) + (e0 - t);
      sum = s;
      const bool first = tile == 0;
      if (__any_sync(0xffffffffu, first || top > best)) {
        best = fmaxf(best, top);
        const uint32_t mine = nth_largest(ordered(best), r);
        if (lane == 0) bound[warp] = from_ordered(mine);
      }
      if (careful) {
        if (__syncthreads_or(full)) {
          thin();
          full = false;
        }
      } else if (first) {
        __syncthreads();
      }
      const float low = lowest();  // (what others have put since only makes it sharper)
      if (top >= low) {
#pragma unroll
        for (int c = 0; c < kPer; ++c)
          if (x[c] >= low && x[c] != neg_inf()) {
            const int at = atomicAdd(&n_kept, 1);
            if (at < kKeep + kTile) kept[at] = key_of(x[c], uint32_t(begin + tile + place(c)));
            full |= at >= room;
          }
      }
    }
    return !__syncthreads_or(full);
  };
  for (bool careful = false; !pass(careful) && !careful; careful = true) {
    if (tid == 0) n_kept = 0;
    ref = best = neg_inf(), sum = rest = 0.f;
    __syncthreads();
  }
  thin();
  const int64_t at = int64_t(row) * p.splits + split;
  if (tid < p.k) p.keys[at * p.k + tid] = kept[tid];
  // The threads' sums to the largest reference.
  float most = ref;
#pragma unroll
  for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
  if (lane == 0) warp_ref[warp] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) most = fmaxf(most, warp_ref[w]);
  // (a factor below 2^-126 is 0: so are its terms beside the largest)
  double all = ref == neg_inf() ? 0.0 : (double(sum) + double(rest)) * double(ex2(ref - most));
#pragma unroll
  for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
  if (lane == 0) warp_sum[warp] = all;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) all += warp_sum[w];
    p.sums[at] = all;
    p.refs[at] = most;
  }
}

// One CTA a request: its rows' logarithms, then the k largest of their candidates.  64 bits are slow here, so f32 sums
// rounded down give a bound, those rounded up say who may reach it, and only these are added and put in order in 64 bits.
__global__ void __launch_bounds__(kThreads) select_join_kernel(const SelectParams p) {
  extern __shared__ unsigned long long shared[];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_row = p.splits * p.k, most = p.beams * per_row;
  unsigned long long *value = shared, *key = shared + most;  // candidates: v in order, and the logit and token
  uint8_t *of = reinterpret_cast<uint8_t *>(key + most);     // and the row
  __shared__ double base[kMaxBeams];                         // what a row's logits are added to
  __shared__ float row_ref[kMaxBeams], base_down[kMaxBeams], base_up[kMaxBeams];
  __shared__ uint8_t kind[kMaxBeams];                        // 0: no continuation, 1: pad_token, 2: candidates
  __shared__ float bound[kWarps];
  __shared__ int n_shared;
  // A warp takes every eighth candidate, so that all have some of every row: one without any leaves no bound.
  wait_for_prior_grid();
  const int64_t from = int64_t(b) * most;
  const int first = lane * kWarps + warp;
  const unsigned long long early = first < most ? p.keys[from + first] : 0;  // on its way beside the sums
  float score = 0.f;
  bool done = false;
  if (tid < p.beams) {
    score = p.scores[b * p.beams + tid];
    done = p.finished && p.finished[b * p.beams + tid];
  }
  if (tid == 0) n_shared = 0;
  for (int w = warp; w < p.beams; w += kWarps) {
    const int64_t at = int64_t(b * p.beams + w) * p.splits;
    float refs[2];
    double sums[2];  // at most 64 splits: two a lane
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = lane + 32 * i;
      refs[i] = s < p.splits ? p.refs[at + s] : neg_inf();
      sums[i] = s < p.splits ? p.sums[at + s] : 0.0;
    }
    float ref = fmaxf(refs[0], refs[1]);
#pragma unroll
    for (int d = 16; d; d >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, d));
    double sum = 0.0;
    if (ref != neg_inf()) sum = sums[0] * double(ex2(refs[0] - ref)) + sums[1] * double(ex2(refs[1] - ref));
#pragma unroll
    for (int d = 16; d; d >>= 1)
      if (d < p.splits) sum += __shfl_xor_sync(0xffffffffu, sum, d);  // (lanes behind the splits hold 0)
    if (lane == 0) base[w] = sum, row_ref[w] = ref;
  }
  __syncthreads();
  if (tid < p.beams) {  // a lane a row: the logarithms at once
    int what = score == neg_inf() ? 0 : done ? 1 : 2;
    bool bad = isnan(score) || score == -neg_inf();
    double add = double(score);
    if (what == 2 && !bad) {  // (rows that are finished or were never filled have left no sums)
      const double sum = base[tid];
      const float ref = row_ref[tid];
      if (sum == 0.0) what = 0;  // nothing but -inf
      else if (!(sum < 1e300) || ref > 3e38f) bad = true;
      else add -= (double(ref) + log2(sum)) * 0.69314718055994530942;
    }
    if (bad) {
      what = 0;
      atomicOr(p.fault, PSD_FAULT_RANGE);
    }
    base[tid] = add;
    base_down[tid] = __double2float_rd(add);
    base_up[tid] = __double2float_ru(add);
    kind[tid] = uint8_t(what);
  }
  __syncthreads();
  // A candidate's logit and token; 0: none.
  auto candidate = [&](int i, int w) {
    if (kind[w] == 2) return i == first ? early : p.keys[from + i];
    return kind[w] == 1 && i == w * per_row ? key_of(0.f, uint32_t(p.pad)) : 0ull;
  };
  float best = neg_inf();
  for (int i = first; i < most; i += kThreads) {
    const int w = i / per_row;
    const unsigned long long k = candidate(i, w);
    if (k) best = fmaxf(best, __fadd_rd(from_ordered(uint32_t(k >> 32)), base_down[w]));
  }
  const uint32_t mine = nth_largest(ordered(best), (p.k + kWarps - 1) / kWarps);
  if (lane == 0) bound[warp] = from_ordered(mine);
  __syncthreads();
  float low = bound[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) low = fminf(low, bound[w]);
  for (int i = first; i < most; i += kThreads) {
    const int w = i / per_row;
    const unsigned long long k = candidate(i, w);
    if (k == 0) continue;
    const float x = from_ordered(uint32_t(k >> 32));
    if (__fadd_ru(x, base_up[w]) < low) continue;
    const int at = atomicAdd(&n_shared, 1);
    value[at] = ordered(double(x) + base[w]);
    key[at] = k;
    of[at] = uint8_t(w);
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

// CTAs a row may be split over: those that run at once, four an SM, and what the second kernel's CTA can hold.  (A second
// wave of few CTAs takes as long as the first.)
int most_splits(int sms, int rows, int beams, int k) {
  return int(std::max<int64_t>(1, std::min<int64_t>({4 * int64_t(sms) / rows, kMost / (beams * k), 64})));
}

size_t join_bytes(const SelectParams &p) { return size_t(p.beams) * p.splits * p.k * 17; }

}  // namespace

static psd_status launch_select(const psd_beam_args *a, void *workspace, const DeviceInfo &dev, cudaStream_t s) {
  SelectParams p;
  p.logits = a->logits;
  p.stride = a->logits_stride;
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
  const int splits = std::min(chunks, most_splits(dev.num_sms, a->rows, a->beams, a->k));
  const int each = (chunks + splits - 1) / splits;
  p.splits = (chunks + each - 1) / each;
  p.chunk = each * kChunk;
  uint8_t *at = static_cast<uint8_t *>(workspace);
  const size_t pieces = size_t(a->rows) * p.splits;
  p.sums = reinterpret_cast<double *>(at);
  p.keys = reinterpret_cast<unsigned long long *>(at + pieces * 8);
  p.refs = reinterpret_cast<float *>(at + pieces * 8 * (1 + size_t(a->k)));
  const size_t size = a->logits_type == PSD_LOGITS_F32 ? 4 : 2;
  const bool vec = aligned16(a->logits) && (a->logits_stride * int64_t(size)) % 16 == 0;
  const int high = std::min(a->rows, 32768);
  const dim3 grid(unsigned(p.splits), unsigned(high), unsigned((a->rows + high - 1) / high));
  auto go = [&](auto type) {
    using T = decltype(type);
    auto kern = vec ? select_rows_kernel<T, true> : select_rows_kernel<T, false>;
    kern<<<grid, kThreads, 0, s>>>(p);
  };
  if (a->logits_type == PSD_LOGITS_F32) go(float{});
  else if (a->logits_type == PSD_LOGITS_BF16) go(__nv_bfloat16{});
  else go(__half{});
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "beam_select launch: %s", cudaGetErrorString(e));
  const size_t shared = join_bytes(p);
  if (shared > 40 * 1024) {
    e = cudaFuncSetAttribute(select_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 17 * kMost);
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
  // rows * splits is at most 4 an SM, or the rows: more rows never need less
  return 256 + size_t(std::max(4 * ctx->dev.num_sms, rows)) * (12 + 8 * size_t(k));
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
  if (!workspace || !aligned16(workspace)) return fail(PSD_ERR_INVALID_ARG, "beam_select: workspace must be 16-byte aligned");
  const size_t need = psd_beam_workspace_bytes(ctx, a->rows, a->beams, a->k);
  if (workspace_bytes < need) return fail(PSD_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", workspace_bytes, need);
  DeviceGuard g(ctx->dev.device);
  return launch_select(a, workspace, ctx->dev, reinterpret_cast<cudaStream_t>(stream));
}
