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
// among those (a count of the larger ones) give the exact k.
//
// A row is split over CTAs so that all SMs have work; a second kernel, one CTA a request, joins the
// splits' sums and takes the k largest of the rows' candidates in 64 bits.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "context.h"
#include "device.cuh"
#include "kernels.h"

namespace psd {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kPer = 16;
constexpr int kTile = kThreads * kPer;       // logits a CTA takes at a time
constexpr int kKeep = 1024;                  // candidates before they are thinned out
constexpr int kMaxK = 64, kMaxBeams = 64;
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
__device__ __forceinline__ unsigned long long nth_largest(unsigned long long v, int r) {
  unsigned long long top = 0;
  for (int i = 0; i < r; ++i) {
    top = v;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    const uint32_t who = __ballot_sync(0xffffffffu, v == top);
    if ((threadIdx.x & 31) == __ffs(who) - 1) v = 0;
  }
  return top;
}

template <typename T> struct Raw;  // 16 logits of a thread as they come
template <> struct Raw<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ void unpack(const uint4 &w, float *x) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ float one(const float *p) { return __ldcs(p); }
};
template <> struct Raw<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void unpack(const uint4 &w, float *x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(u[i]), x[2 * i + 1] = bf16_hi(u[i]);
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
};
template <> struct Raw<__half> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void unpack(const uint4 &w, float *x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(u + i));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float one(const __half *p) { return __half2float(*p); }
};

// blockIdx.x: split, blockIdx.y (and z): row.  VEC: rows are 16-byte aligned; otherwise a warp's loads are
// neighbours one by one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) select_rows_kernel(const SelectParams p) {
  constexpr int N = Raw<T>::kVec, kLoads = kPer / N;
  __shared__ unsigned long long kept[kKeep + kTile];
  __shared__ float bound[kWarps];
  __shared__ int n_kept;
  __shared__ double warp_sum[kWarps];
  __shared__ float warp_ref[kWarps];
  dependents_may_launch();
  const int row = int(blockIdx.y + gridDim.y * blockIdx.z), split = blockIdx.x;
  if (row >= p.rows) return;
  const float score = p.scores[row];
  // no continuations, or one: the second kernel sees to it (a NaN goes on, to be reported there)
  if (score == neg_inf() || (p.finished && p.finished[row])) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t begin = int64_t(split) * p.chunk, end = min(int64_t(p.vocab), begin + p.chunk);
  const T *x_row = static_cast<const T *>(p.logits) + int64_t(row) * p.stride;
  const int r = (p.k + kWarps - 1) / kWarps;
  if (tid == 0) n_kept = 0;

  uint4 raw[kLoads];
  float x[kPer];
  // where element c of a thread's 16 lies in a tile
  auto place = [&](int c) { return VEC ? (c / N) * (kThreads * N) + tid * N + c % N : c * kThreads + tid; };
  auto load = [&](int64_t tile) {
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < kLoads; ++c)
        if (tile + place(c * N) + N <= end) raw[c] = __ldcs(reinterpret_cast<const uint4 *>(x_row + tile + place(c * N)));
    }
  };
  auto values = [&](int64_t tile) {
    if constexpr (VEC) {
#pragma unroll
      for (int c = 0; c < kLoads; ++c) {
        if (tile + place(c * N) + N <= end) {
          Raw<T>::unpack(raw[c], x + c * N);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) x[c * N + i] = tile + place(c * N + i) < end ? Raw<T>::one(x_row + tile + place(c * N + i)) : neg_inf();
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < kPer; ++c) x[c] = tile + place(c) < end ? Raw<T>::one(x_row + tile + place(c)) : neg_inf();
    }
  };
  constexpr float kL = 1.44269502f, kL2 = 1.92596303e-8f;  // log2 e, f32 and the rest
  float ref = neg_inf(), sum = 0.f, rest = 0.f, best = neg_inf();
  auto thin = [&]() {  // the k largest of those kept, in order, to the front; all threads
    const int n = n_kept;
    float low = bound[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) low = fminf(low, bound[w]);
    const unsigned long long least = low == neg_inf() ? 1ull : (unsigned long long)(ordered(low)) << 32;
    __shared__ unsigned long long chosen[kMaxK];
    if (tid < p.k) chosen[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long mine = kept[i];
      if (mine < least) continue;
      int larger = 0;
      for (int j = 0; j < n; ++j) larger += kept[j] > mine;
      if (larger < p.k) chosen[larger] = mine;
    }
    __syncthreads();
    if (tid < p.k) kept[tid] = chosen[tid];
    if (tid == 0) n_kept = min(n, p.k);
    __syncthreads();
  };
  load(begin);
  for (int64_t tile = begin; tile < end; tile += kTile) {
    values(tile);
    if (tile + kTile < end) load(tile + kTile);
    float top = neg_inf();
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      x[c] = fmaxf(x[c], neg_inf());  // NaN counts as -inf
      top = fmaxf(top, x[c]);
    }
    if (top * kL > ref + 16.f) {  // (false while all are -inf)
      const float to = fminf(ceilf(top * kL), 3e38f);
      const float down = ref == neg_inf() ? 0.f : ex2(ref - to);
      sum *= down, rest *= down;
      ref = to;
    }
    const float from = ref == neg_inf() ? 0.f : -ref;
    float e[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) e[c] = ex2(fmaf(x[c], kL, from) + x[c] * kL2);
#pragma unroll
    for (int d = kPer / 2; d; d >>= 1)
#pragma unroll
      for (int c = 0; c < d; ++c) e[c] += e[c + d];
    const float s = sum + e[0], t = s - sum;
    rest += (sum - (s - t)) + (e[0] - t);
    sum = s;
    best = fmaxf(best, top);
    const uint32_t mine = nth_largest(ordered(best), r);
    if (lane == 0) reinterpret_cast<volatile float *>(bound)[warp] = from_ordered(mine);
    __syncthreads();  // (the first tile's bounds are needed; later ones only become sharper)
    float low = bound[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) low = fminf(low, bound[w]);
    if (top >= low) {
#pragma unroll
      for (int c = 0; c < kPer; ++c)
        if (x[c] >= low && x[c] != neg_inf()) kept[atomicAdd(&n_kept, 1)] = key_of(x[c], uint32_t(tile + place(c)));
    }
    __syncthreads();
    if (n_kept > kKeep) thin();  // the same for all
  }
  __syncthreads();
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

// One CTA a request: its rows' logarithms, then the k largest of their candidates.  As in the first kernel a bound
// leaves few of them to be put in order: all ranks of 640 candidates took 80 us.
__global__ void __launch_bounds__(kThreads) select_join_kernel(const SelectParams p) {
  extern __shared__ unsigned long long shared[];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_row = p.splits * p.k, most = p.beams * per_row;
  unsigned long long *value = shared, *key = shared + most;  // candidates: v in order, and the logit and token
  uint8_t *of = reinterpret_cast<uint8_t *>(key + most);     // and the row
  __shared__ double base[kMaxBeams];                         // what a row's logits are added to
  __shared__ uint8_t kind[kMaxBeams];                        // 0: no continuation, 1: pad_token, 2: candidates
  __shared__ unsigned long long bound[kWarps];
  __shared__ int n_shared;
  wait_for_prior_grid();
  const int64_t from = int64_t(b) * most;
  const unsigned long long early = tid < most ? p.keys[from + tid] : 0;  // on its way beside the sums
  if (tid == 0) n_shared = 0;
  for (int w = warp; w < p.beams; w += kWarps) {
    const int row = b * p.beams + w;
    const float score = p.scores[row];
    const bool done = p.finished && p.finished[row];
    float ref = neg_inf(), refs[2];
    double sums[2];  // at most 64 splits: two a lane
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = lane + 32 * i;
      refs[i] = s < p.splits ? p.refs[int64_t(row) * p.splits + s] : neg_inf();
      sums[i] = s < p.splits ? p.sums[int64_t(row) * p.splits + s] : 0.0;
    }
    double add = double(score);
    int what = score == neg_inf() ? 0 : done ? 1 : 2;
    bool bad = isnan(score) || score == -neg_inf();
    if (what == 2 && !bad) {
      ref = fmaxf(refs[0], refs[1]);
#pragma unroll
      for (int d = 16; d; d >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, d));
      double sum = 0.0;
      if (ref != neg_inf()) sum = sums[0] * double(ex2(refs[0] - ref)) + sums[1] * double(ex2(refs[1] - ref));
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (sum == 0.0) what = 0;  // nothing but -inf
      else if (!(sum < 1e300) || ref > 3e38f) bad = true;
      else add -= (double(ref) + log2(sum)) * 0.69314718055994530942;
    }
    if (bad) what = 0;
    if (lane == 0) {
      base[w] = add;
      kind[w] = uint8_t(what);
      if (bad) atomicOr(p.fault, PSD_FAULT_RANGE);
    }
  }
  __syncthreads();
  auto candidate = [&](int i, unsigned long long &k) {  // v in order; 0: none
    const int w = i / per_row;
    if (kind[w] == 2) {
      k = i == tid ? early : p.keys[from + i];
      return k ? ordered(double(from_ordered(uint32_t(k >> 32))) + base[w]) : 0ull;
    }
    k = key_of(0.f, uint32_t(p.pad));
    return kind[w] == 1 && i == w * per_row ? ordered(base[w]) : 0ull;
  };
  unsigned long long best = 0, k;
  for (int i = tid; i < most; i += kThreads) best = max(best, candidate(i, k));
  const unsigned long long mine = nth_largest(best, (p.k + kWarps - 1) / kWarps);
  if (lane == 0) bound[warp] = mine;
  __syncthreads();
  unsigned long long low = bound[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) low = min(low, bound[w]);
  for (int i = tid; i < most; i += kThreads) {
    const unsigned long long v = candidate(i, k);
    if (v == 0 || v < low) continue;
    const int at = atomicAdd(&n_shared, 1);
    value[at] = v;
    key[at] = k;
    of[at] = uint8_t(i / per_row);
  }
  __syncthreads();
  const int n = n_shared;
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long v = value[i], x = key[i];
    const uint8_t w = of[i];
    int larger = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const unsigned long long y = value[j];
      larger += y > v;
      if (y == v) larger += of[j] < w || (of[j] == w && key[j] > x);
    }
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

// CTAs a row may be split over: two an SM in all, and what the second kernel's CTA can hold.
int most_splits(int sms, int rows, int beams, int k) {
  return int(std::max<int64_t>(1, std::min<int64_t>({(4 * int64_t(sms) + rows - 1) / rows, kMost / (beams * k), 64})));
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
  const int tiles = int((int64_t(a->vocab) + kTile - 1) / kTile);
  const int splits = std::min(tiles, most_splits(dev.num_sms, a->rows, a->beams, a->k));
  const int each = (tiles + splits - 1) / splits;
  p.splits = (tiles + each - 1) / each;
  p.chunk = int(std::min<int64_t>(int64_t(each) * kTile, 0x7fffffff));
  uint8_t *at = static_cast<uint8_t *>(workspace);
  const size_t pieces = size_t(a->rows) * p.splits;
  p.sums = reinterpret_cast<double *>(at);
  p.keys = reinterpret_cast<unsigned long long *>(at + pieces * 8);
  p.refs = reinterpret_cast<float *>(at + pieces * 8 * (1 + size_t(a->k)));
  const size_t size = a->logits_type == PSD_LOGITS_F32 ? 4 : 2;
  const bool vec = aligned16(a->logits) && (a->logits_stride * int64_t(size)) % 16 == 0;
  const int high = std::min(a->rows, 32768);
  const dim3 grid(unsigned(p.splits), unsigned(high), unsigned((a->rows + high - 1) / high));
  auto go = [&](auto kern) { kern<<<grid, kThreads, 0, s>>>(p); };
  if (a->logits_type == PSD_LOGITS_F32) go(vec ? select_rows_kernel<float, true> : select_rows_kernel<float, false>);
  else if (a->logits_type == PSD_LOGITS_BF16) go(vec ? select_rows_kernel<__nv_bfloat16, true> : select_rows_kernel<__nv_bfloat16, false>);
  else go(vec ? select_rows_kernel<__half, true> : select_rows_kernel<__half, false>);
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
  return 256 + size_t(rows) * size_t(most_splits(ctx->dev.num_sms, std::max(rows, 1), beams, k)) * (12 + 8 * size_t(k));
}

extern "C" psd_status beam_select(psd_ctx *ctx, const psd_beam_args *a, void *workspace, size_t workspace_bytes,
                                  psd_stream_t stream) {
  clear_error();
  if (!ctx || !a) return fail(PSD_ERR_INVALID_ARG, "beam_select: NULL");
  if (a->beams < 1 || a->k < 1 || a->vocab < 1 || a->rows < 0 || a->rows % a->beams)
    return fail(PSD_ERR_INVALID_ARG, "beam_select: %d rows, %d beams, vocab %d, k %d", a->rows, a->beams, a->vocab, a->k);
  if (a->beams > kMaxBeams || a->k > kMaxK || a->beams * a->k > 4096)
    return fail(PSD_ERR_UNSUPPORTED, "beam_select: at most %d beams, k %d, beams * k 4096 (beams %d, k %d)", kMaxBeams, kMaxK,
                a->beams, a->k);
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
