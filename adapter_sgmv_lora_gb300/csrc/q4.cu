// q4.cu -- the base projection on 4-bit weights with the LoRA delta joined
// (lora_base_q4_apply):
//
//   y_j[t, o] = rn( sum_i s_j[o, i/g] (c_j[o, i] - z_j[o, i/g]) x[t, i]
//                   + [t < end] (bias_j[slot, o] + sum_k B_j[slot, o, k] u[t, j*R + k]) )
//
// u comes from the library's shrink kernels, launched first on the same stream.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "tiles.cuh"

namespace lora {
namespace {

__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* dst, float v) { *dst = v; }
__device__ __forceinline__ void put(__nv_bfloat16* dst, float v) { *dst = __float2bfloat16_rn(v); }

// Any shape and type: a warp has one output of up to kRows rows, its lanes
// share the inputs out byte by byte.  u is the generic shrink's single plane.
constexpr int kRows = 8, kWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) q4_simple_kernel(const __grid_constant__ ProblemDesc p,
                                                                const __grid_constant__ Q4Weights w, int O,
                                                                const float* __restrict__ u) {
  __shared__ int s_ok;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    const bool ok = p.G == 0 || warp_check_routing(p);
    if (lane == 0) s_ok = ok;
  }
  __syncthreads();
  if (!s_ok) return;
  int col = blockIdx.x * kWarps + warp;
  if (col >= O) return;
  int j = 0;
  while (col >= p.sl[j].out_dim) col -= p.sl[j++].out_dim;
  const SliceDesc& sl = p.sl[j];
  const Q4Desc& d = w.w[j];
  const uint8_t* q = d.q + col * d.q_stride;
  const T* scales = static_cast<const T*>(d.scales) + col * d.s_stride;
  const uint8_t* zeros = d.zeros ? d.zeros + col * d.z_stride : nullptr;
  for (int t0 = blockIdx.y * kRows; t0 < p.num_tokens; t0 += gridDim.y * kRows) {
    const int rows = min(kRows, p.num_tokens - t0);
    const T* x = static_cast<const T*>(p.x) + t0 * p.x_row_stride;
    float acc[kRows] = {};
    for (int i = 2 * lane; i < p.in_dim; i += 64) {
      const int code = q[i >> 1], g = i / d.group, g1 = (i + 1) / d.group;
      const bool two = i + 1 < p.in_dim;
      const float w0 = value(scales[g]) * (float)((code & 15) - (zeros ? zeros[g] : 8));
      const float w1 = two ? value(scales[g1]) * (float)((code >> 4) - (zeros ? zeros[g1] : 8)) : 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= rows) break;
        const T* xr = x + r * p.x_row_stride + i;
        acc[r] = fmaf(w0, value(xr[0]), acc[r]);
        if (two) acc[r] = fmaf(w1, value(xr[1]), acc[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r >= rows) break;
      const int t = t0 + r;
      if (t < p.end) {
        const int slot = p.lora_ids[group_of_row(p, t)];
        const int kmax = slot_kmax(p, slot);
        const T* b = static_cast<const T*>(sl.B) + slot * sl.B_slot_stride + (long long)col * p.R;
        const float* ur = u + ((long long)t * p.n_slices + j) * p.R;
        for (int k = lane; k < kmax; k += 32) acc[r] = fmaf(value(b[k]), ur[k], acc[r]);
        if (sl.bias && lane == 0)
          acc[r] += value(static_cast<const T*>(sl.bias)[slot * sl.bias_slot_stride + col]);
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], m);
      if (lane == 0) put(static_cast<T*>(sl.y) + t * sl.y_row_stride + col, acc[r]);
    }
  }
}

}  // namespace

cudaError_t launch_q4_simple(const ProblemDesc& p, const Q4Weights& w, const float* u, cudaStream_t s) {
  long long O = 0;
  for (int j = 0; j < p.n_slices; ++j) O += p.sl[j].out_dim;
  if (O > INT32_MAX - kWarps) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((O + kWarps - 1) / kWarps), (unsigned)std::min((p.num_tokens + kRows - 1) / kRows, 65535));
  if (p.dtype == LORA_DTYPE_BF16) q4_simple_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(p, w, (int)O, u);
  else q4_simple_kernel<float><<<grid, kWarps * 32, 0, s>>>(p, w, (int)O, u);
  return noted(cudaGetLastError(), LORA_PATH_GENERIC_Q4);
}

bool q4_fast_ok(const ProblemDesc&, const Q4Weights&) { return false; }
cudaError_t launch_q4(const ProblemDesc& p, const Q4Weights& w, const float* u, int, bool, cudaStream_t s) {
  return launch_q4_simple(p, w, u, s);
}

}  // namespace lora
