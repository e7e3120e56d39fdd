// A step's attention over several new tokens a request: what the entry point hands to the
// kernels.
#pragma once

#include <cuda_bf16.h>

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
psd_status launch_step_general(const StepParams &p, const StepRequests &req, float *base, const DeviceInfo &dev, cudaStream_t s);

}  // namespace psd
