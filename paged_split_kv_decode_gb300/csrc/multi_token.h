// A step's attention over several new tokens a request: what the entry point hands to the
// kernels.
#pragma once

#include <cuda_bf16.h>

#include "block_scales.cuh"
#include "kernels.h"

namespace psd {

// Requests of one launch, carried in its parameters: no list in memory that a captured call
// would read again.  A batch with more takes several launches; parameters cost about 0.1 us a
// KB, here 20 bytes a request, in every launch.
constexpr int kStepRequests = 256;
struct StepRequests {
  psd_token_request r[kStepRequests];
};

struct StepParams {
  const __nv_bfloat16 *q;
  const void *k_pool, *v_pool;
  const int32_t *page_indices;
  const uint64_t *tree;
  void *o;
  float *lse;
  FaultRef fault;
  int64_t q_stride, num_pages;
  int B;           // requests of this launch
  int num_tokens;  // rows of q
  int Hq, Hkv, G, D, page_size, fp8, out_f32;
  float q_scale;  // sm_scale * log2(e) * k_scale
  float v_scale;
  bool scaled;         // each block of the pools has its own scale
  BlockScales scales;
};

// The tensor-core kernel's CTAs, and where they keep the partial rows of units they share and
// the sums of f32 outputs: `floats` from a 16-byte aligned base on.
struct StepPlace {
  int ctas;
  float *part_o, *sum_o, *part_lse;
  size_t floats;
};
StepPlace step_tc_place(int ctas, int D, float *base);
bool step_tc_supports(const StepParams &p);
psd_status launch_step_tc(const StepParams &p, const StepRequests &req, const StepPlace &place, const DeviceInfo &dev,
                          cudaStream_t s);
// Few rows a KV head (new tokens times query heads) over a cache of 8-bit blocks.  32 requests over 512 to 4096 keys, 8 KV heads
// of 128, on mma.sync and on tcgen05: 4 rows 31 and 58 us, 8 rows 32 and 58, 16 rows 41 and 60, 24 rows 52 and 60, 28 rows 87 and
// 60, 32 rows 85 and 60; f32 outputs: 4 rows 32 and 83, 16 rows 43 and 86, 32 rows 91 and 88.  4 requests over 60 to 400: 16 rows 13
// and 14, 32 rows 20 and 15.  (So the two meet between 24 and 28 rows, not at 32.)
constexpr int kFewRows = 32;
bool step_rows_supports(const StepParams &p);
size_t step_rows_floats(int sms, int D);  // what it keeps from its base on
psd_status launch_step_rows(const StepParams &p, const StepRequests &req, float *base, const DeviceInfo &dev, cudaStream_t s);
psd_status launch_step_general(const StepParams &p, const StepRequests &req, float *base, const DeviceInfo &dev, cudaStream_t s);

}  // namespace psd
