// q4.cuh -- what the kernels of the 4-bit base projection share.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "internal.h"

namespace lora {

struct Q4Work {
  int blk_begin[LORA_MAX_SLICES + 1];  // first block of outputs of each slice
  int nsplit;                          // partial planes of u
  long long plane_stride;              // floats between planes
  int wait_first;                      // 1: no shrink precedes
};

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// The bf16 of a whole number up to 256.
__device__ __forceinline__ uint32_t small_bf16(int n) { return __float_as_uint((float)n) >> 16; }
#endif

// q4_tc.cu.  Shapes are those of q4_fast_ok, and q4_tc_ok.
bool q4_tc_ok(const ProblemDesc& p, const Q4Weights& w);
cudaError_t launch_q4_tc(const ProblemDesc& p, const Q4Weights& wts, Q4Work w, const float* u, cudaStream_t s);

}  // namespace lora
