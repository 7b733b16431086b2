// rope.cu -- norm, position rotation and cache append of a batch's q/k/v rows
// (lora_rope_append).
//
// For each token t and head, with x the head's row:
//   n = x * rsqrt(mean(x^2) + eps) * w                (norm given, else n = x)
//   (a, b) -> s (a cos - b sin, a sin + b cos)         for the rotated pairs
// in fp32, rounded once to the storage type.
//
// The angle.  turns[i] is the pair's frequency as a 64-bit fixed-point
// fraction of a turn, so the wrapped product position * turns[i] IS the
// fractional turn: its top 32 bits, read as a signed number of 2^-31 half
// turns, go to sincospi.  No range reduction is needed and the error stays
// near 2^-32 of a turn at any position, where an fp32 product position * f
// loses whole hundredths of a radian at 100k tokens.  The table is one
// 64-bit word per pair instead of a cos/sin row per position.
#include <cuda_bf16.h>

#include "internal.h"

namespace lora {
namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// cos and sin, times the attention scale, of pair i at a position.
__device__ __forceinline__ float2 rope_cos_sin(const RopeDesc& p, int position, int i) {
  const unsigned long long phase = (unsigned long long)(long long)position * p.turns[i];
  float s, c;
  sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c * p.attention_scale, s * p.attention_scale);
}

// Element offset of the cache row of token t (head 0), or -1 when the token
// is not stored.
__device__ __forceinline__ long long cache_offset(const RopeDesc& p, int t) {
  if (!p.cache_rows) return -1;
  const int row = p.cache_rows[t];
  if (row == -1) return -1;
  const int page = row / p.cache.page_size;
  if (row < 0 || page >= p.cache.num_pages) {
    atomicOr(p.status, LORA_DEV_BAD_PAGE);
    return -1;
  }
  return page * p.cache.page_stride + (row - page * p.cache.page_size) * p.cache.token_stride;
}

// Any type, size and alignment: one warp per head, element by element.  Block
// = one token and a share of its heads (query, key, then value heads).
constexpr int kGenericWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kGenericWarps * 32) rope_generic_kernel(const __grid_constant__ RopeDesc p) {
  __shared__ float2 cs[LORA_MAX_HEAD_DIM / 2];
  __shared__ long long s_row;
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < half; i += blockDim.x) cs[i] = rope_cos_sin(p, p.positions[t], i);
  if (threadIdx.x == 0) s_row = cache_offset(p, t);
  __syncthreads();
  const long long row = s_row;
  const int heads = p.H + p.Hk + (p.cache_rows ? p.Hk : 0);
  for (int h = blockIdx.y * kGenericWarps + warp; h < heads; h += gridDim.y * kGenericWarps) {
    if (h >= p.H + p.Hk) {  // value heads: copied
      if (row < 0) continue;
      const int hv = h - p.H - p.Hk;
      const T* src = static_cast<const T*>(p.v.data) + t * p.v.row_stride + hv * p.v.head_stride;
      T* dst = static_cast<T*>(p.cache.v) + row + hv * p.cache.head_stride;
      for (int d = lane; d < p.hd; d += 32) dst[d] = src[d];
      continue;
    }
    const bool is_q = h < p.H;
    const int hh = is_q ? h : h - p.H;
    const HeadsDesc& in = is_q ? p.q : p.k;
    const HeadsDesc& out = is_q ? p.q_out : p.k_out;
    const T* w = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
    const T* x = static_cast<const T*>(in.data) + t * in.row_stride + hh * in.head_stride;
    T* o = out.data ? static_cast<T*>(out.data) + t * out.row_stride + hh * out.head_stride : nullptr;
    T* c = !is_q && row >= 0 ? static_cast<T*>(p.cache.k) + row + hh * p.cache.head_stride : nullptr;
    float r = 1.f;
    if (w) {
      float sum = 0.f;
      for (int d = lane; d < p.hd; d += 32) sum = fmaf(to_f(x[d]), to_f(x[d]), sum);
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      r = rsqrtf(sum / p.hd + p.eps);
    }
    auto put = [&](int d, float v) {
      if (o) o[d] = from_f<T>(v);
      if (c) c[d] = from_f<T>(v);
    };
    // Each pair is read and written by one lane, so out may be the input.
    for (int i = lane; i < half; i += 32) {
      const int da = p.layout == LORA_ROPE_HALVES ? i : 2 * i;
      const int db = p.layout == LORA_ROPE_HALVES ? i + half : 2 * i + 1;
      float a = to_f(x[da]), b = to_f(x[db]);
      if (w) {
        a *= r * to_f(w[da]);
        b *= r * to_f(w[db]);
      }
      put(da, a * cs[i].x - b * cs[i].y);
      put(db, a * cs[i].y + b * cs[i].x);
    }
    for (int d = p.rot + lane; d < p.hd; d += 32) {
      float v = to_f(x[d]);
      if (w) v *= r * to_f(w[d]);
      put(d, v);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeDesc& p, cudaStream_t s) {
  const int heads = p.H + p.Hk + (p.cache_rows ? p.Hk : 0);
  // A block takes one token; its heads are shared by several blocks while the
  // batch is too small to give every SM some.
  const int sms = device_sm_count();
  int split = (heads + kGenericWarps - 1) / kGenericWarps;
  while (split > 1 && (long long)p.T * split > 8LL * sms) split = (split + 1) / 2;
  const dim3 grid(p.T, split);
  if (p.dtype == LORA_DTYPE_BF16)
    rope_generic_kernel<__nv_bfloat16><<<grid, kGenericWarps * 32, 0, s>>>(p);
  else
    rope_generic_kernel<float><<<grid, kGenericWarps * 32, 0, s>>>(p);
  return noted(cudaGetLastError(), LORA_PATH_GENERIC_ROPE);
}

}  // namespace lora
