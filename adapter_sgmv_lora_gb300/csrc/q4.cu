// q4.cu -- the base projection on 4-bit weights with the LoRA delta joined
// (lora_base_q4_apply):
//
//   y_j[t, o] = rn( sum_i s_j[o, i/g] (c_j[o, i] - z_j[o, i/g]) x[t, i]
//                   + [t < end] (bias_j[slot, o] + sum_k B_j[slot, o, k] u[t, j*R + k]) )
//
// u comes from the library's shrink kernels, launched first on the same stream.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

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

namespace {

// Tensor cores (mma.sync m16n8k16): outputs are the rows of the product, the
// batch's rows its columns, so one row fills an eighth of an instruction and
// the weights are still unpacked once.  A CTA has 32 outputs; its 8 warps share
// the inputs out in blocks of 128 and their sums meet in shared memory.  Each
// warp has a ring of asynchronous copies of its own, four blocks of 2 KB deep.
//
// Any order of the inputs will do as long as weights and x agree.  A 32-bit
// word holds 8 inputs; its nibbles 0 and 4, 1 and 5, ... masked into the low
// bits of two bf16 of 128 are 128 + code, less 128 + zero the exact operand,
// and x is paired alike.  A quad's words are 32 inputs, so two instructions
// stay within a group of 32.  The products are exact, a group's sum is fp32,
// and its scale multiplies the sum.
constexpr int kMmaWarps = 8, kMmaOuts = 32, kMmaAhead = 4;
constexpr int kMmaPitch = 80;  // bytes of a row of a block: 8 rows' words fall on 32 banks
constexpr int kMmaStage = kMmaOuts * kMmaPitch;
constexpr int kMmaRing = kMmaWarps * kMmaAhead * kMmaStage;
constexpr int kMmaSmemMost = 200 * 1024;

struct Q4Work {
  int blk_begin[LORA_MAX_SLICES + 1];  // first block of 32 outputs of each slice
  int nsplit;                          // partial planes of u
  long long plane_stride;              // floats between planes
  int wait_first;                      // 1: no shrink precedes
};

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// The bf16 of a whole number up to 256.
__device__ __forceinline__ uint32_t small_bf16(int n) { return __float_as_uint((float)n) >> 16; }

// Word of 8 codes -> the pairs (0,4) (1,5) (2,6) (3,7) of code - zero; low:
// 128 + zero, twice.
__device__ __forceinline__ void unpack(uint32_t w, uint32_t low, uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = sub_bf16x2(((w >> (4 * i)) & 0x000f000fu) | 0x43004300u, low);
}

// WPG: words of a thread that surely share a group: 4 where groups are whole
// blocks, else 2 (64) or 1 (32).
template <int NT, int WPG>
__global__ void __launch_bounds__(kMmaWarps * 32, 2)
    q4_mma_kernel(const __grid_constant__ ProblemDesc p, const __grid_constant__ Q4Weights wts,
                  const __grid_constant__ Q4Work w, const float* __restrict__ u) {
  constexpr int MW = kMmaOuts / 16, TN = 8 * NT, SUM_PITCH = TN + 1;
  using T = __nv_bfloat16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_ok, s_far, s_slot[TN];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (w.wait_first) pdl_wait();
  int j = 0;
  while (j + 1 < p.n_slices && (int)blockIdx.x >= w.blk_begin[j + 1]) ++j;
  const SliceDesc& sl = p.sl[j];
  const Q4Desc& d = wts.w[j];
  const int o0 = (blockIdx.x - w.blk_begin[j]) * kMmaOuts, t0 = blockIdx.y * TN;
  const int nb = (p.in_dim + 127) / 128;
  const int b_lo = nb * warp / kMmaWarps, b_hi = nb * (warp + 1) / kMmaWarps;
  uint8_t* ring = smem + warp * kMmaAhead * kMmaStage;
  // A copy covers 8 rows of 64 bytes; outputs past the slice's last read its
  // last row and are not stored.
  const uint8_t* qrow[kMmaOuts / 8];
#pragma unroll
  for (int i = 0; i < kMmaOuts / 8; ++i)
    qrow[i] = d.q + (long long)min(o0 + i * 8 + g, sl.out_dim - 1) * d.q_stride + t * 16;
  auto load = [&](int blk) {
    if (blk < b_hi) {
      uint8_t* dst = ring + (blk - b_lo) % kMmaAhead * kMmaStage + g * kMmaPitch + t * 16;
      const uint32_t bytes = blk * 128 + t * 32 < p.in_dim ? 16 : 0;
      const long long at = bytes ? blk * 64 : 0;
#pragma unroll
      for (int i = 0; i < kMmaOuts / 8; ++i)
        cp_async16_zfill(dst + i * 8 * kMmaPitch, qrow[i] - (bytes ? 0 : t * 16) + at, bytes);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kMmaAhead; ++i) load(b_lo + i);
  // Scales and zeros of the CTA's outputs: the scale's bits above those of 128 + zero.
  const int groups = (p.in_dim + d.group - 1) / d.group, sz_pitch = groups + 1 + (groups & 1);
  uint32_t* s_sz = reinterpret_cast<uint32_t*>(smem + kMmaRing);
  if (threadIdx.x == 0) s_far = 0;
  __syncthreads();
  for (int r = warp; r < kMmaOuts; r += kMmaWarps) {
    const long long o = min(o0 + r, sl.out_dim - 1);
    const uint16_t* scales = static_cast<const uint16_t*>(d.scales) + o * d.s_stride;
    const uint8_t* zeros = d.zeros ? d.zeros + o * d.z_stride : nullptr;
    for (int e = lane; e < groups; e += 32) {
      const int z = zeros ? zeros[e] : 8;
      if (z > 127) s_far = 1;
      s_sz[r * sz_pitch + e] = (uint32_t)scales[e] << 16 | small_bf16(128 + min(z, 127));
    }
  }
  if (warp == 0) {
    const bool ok = p.G == 0 || warp_check_routing(p);
    if (lane == 0) s_ok = ok;
    for (int r = lane; r < TN; r += 32) s_slot[r] = ok && t0 + r < p.end ? p.lora_ids[group_of_row(p, t0 + r)] : -1;
  }
  __syncthreads();
  const bool far = s_far != 0;
  float y[MW][NT][4] = {};
  // Rows of x past the batch's last count as zero.
  const T* xrow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = t0 + n * 8 + g;
    xrow[n] = row < p.num_tokens ? static_cast<const T*>(p.x) + row * p.x_row_stride + 8 * t : nullptr;
  }
  for (int blk = b_lo; blk < b_hi; ++blk) {
    cp_async_wait<kMmaAhead - 1>();
    __syncwarp();
    const uint8_t* stage = ring + (blk - b_lo) % kMmaAhead * kMmaStage;
#pragma unroll
    for (int c = 0; c < 4 / WPG; ++c) {
      const int k0 = blk * 128 + c * 32 * WPG;
      if (k0 >= p.in_dim) break;
      const int grp = k0 / d.group;
      uint32_t sz[MW][2];
#pragma unroll
      for (int m = 0; m < MW; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) sz[m][h] = s_sz[(m * 16 + h * 8 + g) * sz_pitch + grp];
      float acc[MW][NT][4] = {};
#pragma unroll
      for (int i = 0; i < WPG; ++i) {
        uint32_t a[MW][2][4];
#pragma unroll
        for (int m = 0; m < MW; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t word = *reinterpret_cast<const uint32_t*>(
                stage + (m * 16 + h * 8 + g) * kMmaPitch + (c * WPG + i) * 16 + t * 4);
            unpack(word, __byte_perm(sz[m][h], 0, 0x1010), a[m][h]);
          }
        if (far) {  // a zero past 127 has a rest
#pragma unroll
          for (int m = 0; m < MW; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const long long o = min(o0 + m * 16 + h * 8 + g, sl.out_dim - 1);
              const uint32_t rest = small_bf16(max((int)d.zeros[o * d.z_stride + grp], 127) - 127);
#pragma unroll
              for (int e = 0; e < 4; ++e) a[m][h][e] = sub_bf16x2(a[m][h][e], rest | rest << 16);
            }
        }
        const int k = k0 + 32 * i;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (xrow[n] && k < p.in_dim) x = __ldg(reinterpret_cast<const uint4*>(xrow[n] + k));
          const uint32_t b0 = __byte_perm(x.x, x.z, 0x5410), b1 = __byte_perm(x.x, x.z, 0x7632);
          const uint32_t b2 = __byte_perm(x.y, x.w, 0x5410), b3 = __byte_perm(x.y, x.w, 0x7632);
#pragma unroll
          for (int m = 0; m < MW; ++m) {
            const uint32_t a0[4] = {a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1]};
            const uint32_t a1[4] = {a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3]};
            mma_bf16_16816(acc[m][n], a0, b0, b1);
            mma_bf16_16816(acc[m][n], a1, b2, b3);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MW; ++m) {
        const float s0 = __uint_as_float(sz[m][0] & 0xffff0000u), s1 = __uint_as_float(sz[m][1] & 0xffff0000u);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          y[m][n][0] = fmaf(s0, acc[m][n][0], y[m][n][0]);
          y[m][n][1] = fmaf(s0, acc[m][n][1], y[m][n][1]);
          y[m][n][2] = fmaf(s1, acc[m][n][2], y[m][n][2]);
          y[m][n][3] = fmaf(s1, acc[m][n][3], y[m][n][3]);
        }
      }
    }
    __syncwarp();
    load(blk + kMmaAhead);
  }
  cp_async_wait<0>();
  __syncthreads();  // the rings are free
  float* s_sum = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < MW; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s_sum[(warp * kMmaOuts + m * 16 + g + (e >> 1) * 8) * SUM_PITCH + n * 8 + 2 * t + (e & 1)] = y[m][n][e];
  __syncthreads();
  if (!w.wait_first) pdl_wait();  // u comes from the shrink
  if (!s_ok) return;
  for (int e = threadIdx.x; e < kMmaOuts * TN; e += kMmaWarps * 32) {
    const int o = e % kMmaOuts, r = e / kMmaOuts, row = t0 + r;
    if (row >= p.num_tokens || o0 + o >= sl.out_dim) continue;
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kMmaWarps; ++v) sum += s_sum[(v * kMmaOuts + o) * SUM_PITCH + r];
    const int slot = s_slot[r];
    if (slot >= 0) {
      const int kmax = slot_kmax(p, slot);
      const T* b = static_cast<const T*>(sl.B) + slot * sl.B_slot_stride + (long long)(o0 + o) * p.R;
      const float* ur = u + ((long long)row * p.n_slices + j) * p.R;
      for (int k = 0; k < kmax; ++k) {
        float v = 0.f;
        for (int c = 0; c < w.nsplit; ++c) v += ur[c * w.plane_stride + k];
        sum = fmaf(value(b[k]), v, sum);
      }
      if (sl.bias) sum += value(static_cast<const T*>(sl.bias)[slot * sl.bias_slot_stride + o0 + o]);
    }
    put(static_cast<T*>(sl.y) + row * sl.y_row_stride + o0 + o, sum);
  }
}

// Words of a thread that surely share a group in every slice; 0: not one.
int q4_words_per_group(const ProblemDesc& p, const Q4Weights& w) {
  int words = 4;
  for (int j = 0; j < p.n_slices; ++j) {
    const int g = w.w[j].group;
    if (g >= p.in_dim || g % 128 == 0) continue;
    if (g % 32 != 0) return 0;
    words = std::min(words, g % 64 == 0 ? 2 : 1);
  }
  return words;
}

// Scales and zeros of 32 outputs in shared memory, bytes.
int q4_scale_bytes(const ProblemDesc& p, const Q4Weights& w) {
  int most = 0;
  for (int j = 0; j < p.n_slices; ++j) most = std::max(most, (p.in_dim + w.w[j].group - 1) / w.w[j].group);
  return kMmaOuts * (most + 1 + (most & 1)) * 4;
}

template <int NT, int WPG>
cudaError_t launch_q4_mma(const ProblemDesc& p, const Q4Weights& wts, Q4Work w, const float* u, cudaStream_t s) {
  int blocks = 0;
  for (int j = 0; j < p.n_slices; ++j) {
    w.blk_begin[j] = blocks;
    blocks += (p.sl[j].out_dim + kMmaOuts - 1) / kMmaOuts;
  }
  w.blk_begin[p.n_slices] = blocks;
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(q4_mma_kernel<NT, WPG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmaSmemMost);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, (p.num_tokens + 8 * NT - 1) / (8 * NT));
  cfg.blockDim = dim3(kMmaWarps * 32);
  cfg.dynamicSmemBytes = kMmaRing + q4_scale_bytes(p, wts);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return noted(cudaLaunchKernelEx(&cfg, q4_mma_kernel<NT, WPG>, p, wts, w, u), LORA_PATH_MMA_Q4);
}

template <int NT>
cudaError_t launch_q4_words(const ProblemDesc& p, const Q4Weights& wts, const Q4Work& w, const float* u, cudaStream_t s) {
  switch (q4_words_per_group(p, wts)) {
    case 4: return launch_q4_mma<NT, 4>(p, wts, w, u, s);
    case 2: return launch_q4_mma<NT, 2>(p, wts, w, u, s);
    default: return launch_q4_mma<NT, 1>(p, wts, w, u, s);
  }
}

}  // namespace

bool q4_fast_ok(const ProblemDesc& p, const Q4Weights& w) {
  if (p.dtype != LORA_DTYPE_BF16 || p.in_dim % 32 != 0 || p.token_rows) return false;
  if ((reinterpret_cast<uintptr_t>(p.x) & 15) != 0 || p.x_row_stride % 8 != 0) return false;
  if ((p.num_tokens + 31) / 32 > 65535 || kMmaRing + q4_scale_bytes(p, w) > kMmaSmemMost) return false;
  for (int j = 0; j < p.n_slices; ++j)
    if ((reinterpret_cast<uintptr_t>(w.w[j].q) & 15) != 0 || w.w[j].q_stride % 16 != 0) return false;
  return q4_words_per_group(p, w) > 0;
}

cudaError_t launch_q4(const ProblemDesc& p, const Q4Weights& wts, const float* u, int nsplit, bool after_shrink,
                      cudaStream_t s) {
  Q4Work w{};
  w.nsplit = nsplit;
  w.plane_stride = (long long)p.end * p.n_slices * p.R;
  w.wait_first = after_shrink ? 0 : 1;
  if (p.num_tokens <= 8) return launch_q4_words<1>(p, wts, w, u, s);
  if (p.num_tokens <= 16) return launch_q4_words<2>(p, wts, w, u, s);
  return launch_q4_words<4>(p, wts, w, u, s);
}

}  // namespace lora
