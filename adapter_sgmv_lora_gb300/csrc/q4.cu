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
#include <climits>

#include "internal.h"
#include "ptx.cuh"
#include "q4.cuh"
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
    int slot_of = -1, kmax_of = 0;  // of row t0 + lane
    if (lane < rows && t0 + lane < p.end) {
      slot_of = p.lora_ids[group_of_row(p, t0 + lane)];
      kmax_of = slot_kmax(p, slot_of);
    }
    for (int i = 2 * lane; i < p.in_dim; i += 64) {
      const int code = q[i >> 1], g = i / d.group, g1 = (i + 1) / d.group;
      const bool two = i + 1 < p.in_dim;
      const float w0 = value(scales[g]) * (float)((code & 15) - (zeros ? zeros[g] : 8));
      const float w1 = two ? value(scales[g1]) * (float)((code >> 4) - (zeros ? zeros[g1] : 8)) : 0.f;
      // Rows past the last read it again, so that all loads are under way at once.
      float x0[kRows], x1[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const T* xr = x + min(r, rows - 1) * p.x_row_stride + i;
        x0[r] = value(xr[0]);
        x1[r] = value(xr[two]);
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        acc[r] = fmaf(w0, x0[r], acc[r]);
        if (two) acc[r] = fmaf(w1, x1[r], acc[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r >= rows) break;
      const int t = t0 + r;
      if (t < p.end) {
        const int slot = __shfl_sync(0xffffffffu, slot_of, r), kmax = __shfl_sync(0xffffffffu, kmax_of, r);
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
//
// Unpacks for every 32 rows anew; warps wait most for x and their copies (issue
// slots a third taken, cold, 29 rows through 4096 outputs).  Gate and up of
// the 8B model 51 us for 16 rows, 68 for 32, 122 for 64 (which q4_tc.cu takes
// over).  Slower were 64 rows a CTA, one CTA an SM (150 for 64 rows: nothing runs
// under a CTA's start and end), x in the ring beside the weights (170), the delta
// on the tensor cores (144: registers), and fp8 or int8 operands (this GPU's
// mma.sync has neither at the rate of 16 bits).
constexpr int kMmaWarps = 8, kMmaOuts = 32, kMmaAhead = 4;
constexpr int kMmaPitch = 80;  // bytes of a row of a block: 8 rows' words fall on 32 banks
constexpr int kMmaStage = kMmaOuts * kMmaPitch;
constexpr int kMmaRing = kMmaWarps * kMmaAhead * kMmaStage;
constexpr int kMmaSmemMost = 200 * 1024;

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
  // The slots' B rows of these outputs are wanted at the end: into L2 now.
  const bool wide_b = p.R % 8 == 0 && ((reinterpret_cast<uintptr_t>(sl.B) | (uintptr_t)(sl.B_slot_stride * 2)) & 15) == 0;
  for (int r = warp; r < TN; r += kMmaWarps)
    if (s_slot[r] >= 0 && (r == 0 || s_slot[r] != s_slot[r - 1])) {
      const char* b = static_cast<const char*>(sl.B) + (s_slot[r] * sl.B_slot_stride + (long long)o0 * p.R) * 2;
      const int bytes = min(kMmaOuts, sl.out_dim - o0) * p.R * 2;
      for (int e = lane * 128; e < bytes; e += 32 * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(b + e));
    }
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
  // The delta, on the CUDA cores: a lane is an output, a warp takes every
  // eighth row; u's planes are summed into shared memory first.
  float* s_u = s_sum + kMmaWarps * kMmaOuts * SUM_PITCH;  // [TN][R]
  const int routed = min(max(p.end - t0, 0), TN);
  if (routed > 0) {
    const float* ur = u + ((long long)t0 * p.n_slices + j) * p.R;
    for (int e = threadIdx.x; e < routed * p.R; e += kMmaWarps * 32) {
      const int r = e / p.R, k = e - r * p.R;
      const float* at = ur + (long long)r * p.n_slices * p.R + k;
      float v = 0.f;
#pragma unroll 4
      for (int c = 0; c < w.nsplit; ++c) v += __ldcg(at + c * w.plane_stride);
      s_u[e] = v;
    }
    __syncthreads();
  }
  const int o = lane;
  if (o0 + o >= sl.out_dim) return;
  for (int r = warp; r < TN && t0 + r < p.num_tokens; r += kMmaWarps) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kMmaWarps; ++v) sum += s_sum[(v * kMmaOuts + o) * SUM_PITCH + r];
    const int slot = s_slot[r];
    if (slot >= 0) {
      const int kmax = slot_kmax(p, slot);
      const T* b = static_cast<const T*>(sl.B) + slot * sl.B_slot_stride + (long long)(o0 + o) * p.R;
      const float* ur = s_u + r * p.R;
      int k = 0;
      if (wide_b) {
#pragma unroll 2
        for (; k + 8 <= kmax; k += 8) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(b + k));
          const uint32_t bits[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum = fmaf(__uint_as_float(bits[e] << 16), ur[k + 2 * e], sum);
            sum = fmaf(__uint_as_float(bits[e] & 0xffff0000u), ur[k + 2 * e + 1], sum);
          }
        }
      }
      for (; k < kmax; ++k) sum = fmaf(value(b[k]), ur[k], sum);
      if (sl.bias) sum += value(static_cast<const T*>(sl.bias)[slot * sl.bias_slot_stride + o0 + o]);
    }
    put(static_cast<T*>(sl.y) + (t0 + r) * sl.y_row_stride + o0 + o, sum);
  }
}

// Few rows, many tiles.  x stays in shared memory and a CTA per SM goes through tile after
// tile of 32 outputs: 16 warps in teams, which share a tile's inputs out and
// only meet to sum.  Each warp's ring of copies runs on across its tiles, so
// memory never waits for a start or an end.
//
// Unpacking is most of the work (the shifts and masks run at half rate), and
// fp16 takes fewer instructions than bf16: its ten mantissa bits hold a nibble where
// it lies, 1024 + code from bits 0-3 and 1024 + 16 code from bits 4-7, less the
// zero (any byte) by one exact fused multiply-add.  So x is taken to fp16 by a
// power of two for each row that brings its largest value to 2^14; the sums are
// divided by that power.  That is exact for all values down to 2^-31 of the
// row's largest.  Where a row has smaller ones (its largest may meet a weight of
// zero), an infinity or a NaN, all rows stay bf16 and so do the weights: the same
// sums, five rows through the 8B gate and up with zeros 37.7 us, so 32.6 (one row
// 34.1 and 28.9, eight 40.0 and 35.1).
//
// A block is 256 inputs of 32 outputs, so a row's copies are whole lines.  One
// row through the 8B gate and up (61 MB): 22.2 us, 2.7 TB/s, the unpacking pipe
// 44% busy and 47% of issue slots taken, so nothing is full: warps wait for their
// copies and for one another at a tile's end.  The kernel above takes 30.3.
constexpr int kFewWarps = 16, kFewAhead = 2, kFewBlock = 256;
constexpr int kFewPitch = kFewBlock / 2 + 16;  // bytes of a row of a block: 8 rows' words fall on 32 banks
constexpr int kFewStage = kMmaOuts * kFewPitch;
constexpr int kFewSmemMost = 226 * 1024;
constexpr int kFewRing = kFewWarps * kFewAhead * kFewStage;

struct FewWork {
  int tile_begin[LORA_MAX_SLICES + 1];   // first tile of 32 outputs of each slice
  unsigned per_group[LORA_MAX_SLICES];   // ceil(2^32 / units of a group), 0 for one: unit -> group
  int team;                              // warps that share a tile: 1, 2, 4, 8 or 16
  int x_pitch;                           // bytes of a row of x in shared memory
  int nsplit;
  long long plane_stride;
  int wait_first;
};

template <int NT>
constexpr int few_sum_bytes() {
  return kFewWarps * 32 * 8 * NT * 4;
}

// D = A B (FIRST) or D += A B, fp16 operands.
template <bool FIRST>
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  if constexpr (FIRST)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// (w & mask) | magic in one instruction; magic stays in its register.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "n"(MASK), "r"(magic));
  return d;
}

// Word of 8 codes -> the fp16 pairs (0,4) (1,5) (2,6) (3,7) of code - zero;
// even: 1024 + zero, odd: -(64 + zero), magic: 1024, sixteenth: 1/16, twice each.
__device__ __forceinline__ void unpack_f16(uint32_t w, uint32_t even, uint32_t odd, uint32_t magic, uint32_t sixteenth,
                                           uint32_t (&v)[4]) {
  const uint32_t w8 = w >> 8;
  v[0] = sub_f16x2(pick<0x000f000fu>(w, magic), even);
  v[1] = fma_f16x2(pick<0x00f000f0u>(w, magic), sixteenth, odd);
  v[2] = sub_f16x2(pick<0x000f000fu>(w8, magic), even);
  v[3] = fma_f16x2(pick<0x00f000f0u>(w8, magic), sixteenth, odd);
}

// Word `word` of a block's row, all outputs and rows of x.  BF: both as bf16,
// even: 128 + zero as far as 127, odd: what is left of a zero past that.
template <int NT, bool FIRST, bool BF>
__device__ __forceinline__ void few_word(const uint8_t* at, const uint8_t* const (&xrow)[NT], int k_bytes, int word,
                                         const uint32_t (&even)[2][2], const uint32_t (&odd)[2][2], uint32_t magic,
                                         uint32_t sixteenth, float (&acc)[2][NT][4]) {
  uint32_t a[2][2][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t codes = *reinterpret_cast<const uint32_t*>(at + (m * 16 + h * 8) * kFewPitch + word * 16);
      if constexpr (BF) {
        unpack(codes, even[m][h], a[m][h]);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[m][h][e] = sub_bf16x2(a[m][h][e], odd[m][h]);
      } else {
        unpack_f16(codes, even[m][h], odd[m][h], magic, sixteenth, a[m][h]);
      }
    }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint4 x = *reinterpret_cast<const uint4*>(xrow[n] + k_bytes + word * 64);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if constexpr (BF) {
        if (FIRST) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
        const uint32_t a0[4] = {a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1]};
        const uint32_t a1[4] = {a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3]};
        mma_bf16_16816(acc[m][n], a0, x.x, x.y);
        mma_bf16_16816(acc[m][n], a1, x.z, x.w);
        continue;
      }
      mma_f16_16816<FIRST>(acc[m][n], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], x.x, x.y);
      mma_f16_16816<false>(acc[m][n], a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], x.z, x.w);
    }
  }
}

// One block from the ring: at, this thread's first word; xrow, its columns of x;
// raw, this lane's output's scales and zeros; left, the block's inputs.
template <int NT, int WPG, bool FULL, bool BF>
__device__ __forceinline__ void few_block(const uint8_t* at, const uint8_t* const (&xrow)[NT], int k_bytes,
                                          const uint32_t (&raw)[8 / WPG], int left, float (&y)[2][NT][4]) {
  static_assert(kMmaOuts == 32, "");
  const int g = (threadIdx.x & 31) >> 2;
  uint32_t magic, sixteenth;  // opaque, so that they stay in registers
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
  asm volatile("mov.b32 %0, 0x2c002c00;" : "=r"(sixteenth));
#pragma unroll
  for (int c = 0; c < 8 / WPG; ++c) {
    if (!FULL && c * 32 * WPG >= left) break;
    uint32_t even[2][2], odd[2][2];
    float scale[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t v = __shfl_sync(0xffffffffu, raw[c], m * 16 + h * 8 + g);
        scale[m][h] = __uint_as_float(v & 0xffff0000u);
        if constexpr (BF) {
          const int zero = v & 0xff, near = min(zero, 127);
          even[m][h] = small_bf16(128 + near) * 0x10001u;
          odd[m][h] = small_bf16(zero - near) * 0x10001u;
        } else {
          even[m][h] = (v & 0xffu) * 0x10001u + magic;     // 1024 + zero
          odd[m][h] = sub_f16x2(0x63806380u, even[m][h]);  // 960 - (1024 + zero) = -(64 + zero)
        }
      }
    float acc[2][NT][4];
    few_word<NT, true, BF>(at, xrow, k_bytes, c * WPG, even, odd, magic, sixteenth, acc);
#pragma unroll
    for (int i = 1; i < WPG; ++i) {
      if (!FULL && (c * WPG + i) * 32 >= left) break;
      few_word<NT, false, BF>(at, xrow, k_bytes, c * WPG + i, even, odd, magic, sixteenth, acc);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[m][n][e] = fmaf(scale[m][e >> 1], acc[m][n][e], y[m][n][e]);
  }
}

template <int NT, int WPG>
__global__ void __launch_bounds__(kFewWarps * 32, 1)
    q4_few_kernel(const __grid_constant__ ProblemDesc p, const __grid_constant__ Q4Weights wts,
                  const __grid_constant__ FewWork w, const float* __restrict__ u) {
  constexpr int MW = kMmaOuts / 16, GROUPS = 8 / WPG, ELEMS = MW * NT * 4;
  using T = __nv_bfloat16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_ok, s_slot[8 * NT];
  __shared__ unsigned s_top[8 * NT], s_low[8 * NT];  // bits of a row's largest |x|, of its smallest but 0 less 1
  float* s_part = reinterpret_cast<float*>(smem + kFewRing);             // [warps][ELEMS][32]
  uint8_t* s_x = smem + kFewRing + few_sum_bytes<NT>();                  // [rows][x_pitch]
  float* s_u = reinterpret_cast<float*>(s_x + p.num_tokens * w.x_pitch);  // [routed rows][slices * R]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = warp & (w.team - 1), per_cta = kFewWarps / w.team, team = blockIdx.x * per_cta + warp / w.team;
  const int teams = gridDim.x * per_cta, tiles = w.tile_begin[p.n_slices];
  if (w.wait_first) pdl_wait();
  const int nb = (p.in_dim + kFewBlock - 1) / kFewBlock;
  const int b_lo = nb * rank / w.team, b_hi = nb * (rank + 1) / w.team;
  uint8_t* ring = smem + warp * kFewAhead * kFewStage;
  auto slice_of = [&](int tile) {
    int j = 0;
    while (j + 1 < p.n_slices && tile >= w.tile_begin[j + 1]) ++j;
    return j;
  };

  // What is loaded next: block lb of tile lt, whose rows' addresses are kept.
  // Outputs past the slice's last read its last row and are not stored.
  int lt = team, lb = b_lo, stage_in = 0;
  const uint8_t* qrow[kMmaOuts / 8];
  const uint16_t* srow = nullptr;  // this lane's output
  const uint8_t* zrow = nullptr;
  unsigned per_group = 0;
  auto aim = [&] {
    if (lt >= tiles) return;
    const int j = slice_of(lt);
    const Q4Desc& d = wts.w[j];
    const int o0 = (lt - w.tile_begin[j]) * kMmaOuts, last = p.sl[j].out_dim - 1;
#pragma unroll
    for (int i = 0; i < kMmaOuts / 8; ++i) qrow[i] = d.q + (long long)min(o0 + i * 8 + g, last) * d.q_stride + t * 16;
    const long long o = min(o0 + lane, last);
    srow = static_cast<const uint16_t*>(d.scales) + o * d.s_stride;
    zrow = d.zeros ? d.zeros + o * d.z_stride : nullptr;
    per_group = w.per_group[j];
  };
  aim();
  auto load = [&](uint32_t (&sz)[GROUPS]) {
    if (lt < tiles && lb < b_hi) {
      uint8_t* dst = ring + stage_in * kFewStage + g * kFewPitch + t * 16;
      const int k = lb * kFewBlock + t * 32;
      if ((lb + 1) * kFewBlock <= p.in_dim) {
#pragma unroll
        for (int i = 0; i < kMmaOuts / 8; ++i) {
          const uint8_t* src = qrow[i] + lb * (kFewBlock / 2);
          cp_async16(dst + i * 8 * kFewPitch, src);
          cp_async16(dst + i * 8 * kFewPitch + 64, src + 64);
        }
      } else {  // what is not loaded is not used
#pragma unroll
        for (int i = 0; i < kMmaOuts / 8; ++i) {
          const uint8_t* src = qrow[i] + lb * (kFewBlock / 2);
          if (k < p.in_dim) cp_async16(dst + i * 8 * kFewPitch, src);
          if (k + 128 < p.in_dim) cp_async16(dst + i * 8 * kFewPitch + 64, src + 64);
        }
      }
#pragma unroll
      for (int c = 0; c < GROUPS; ++c) {
        const int unit = lb * GROUPS + c;
        if (unit * 32 * WPG < p.in_dim) {
          const unsigned grp = per_group == 0 ? unit : __umulhi(unit, per_group);
          sz[c] = (uint32_t)__ldg(srow + grp) << 16 | (zrow ? __ldg(zrow + grp) : 8u);
        }
      }
      stage_in = stage_in + 1 == kFewAhead ? 0 : stage_in + 1;
      if (++lb == b_hi) {
        lb = b_lo;
        lt += teams;
        aim();
      }
    }
    cp_async_commit();
  };
  uint32_t raw[kFewAhead][GROUPS] = {};  // the present block's first
#pragma unroll
  for (int i = 0; i < kFewAhead; ++i) load(raw[i]);

  if (warp == 0) {
    const bool ok = p.G == 0 || warp_check_routing(p);
    if (lane == 0) s_ok = ok;
    for (int r = lane; r < 8 * NT; r += 32) s_slot[r] = ok && r < p.end ? p.lora_ids[group_of_row(p, r)] : -1;
  }
  if (threadIdx.x < 8 * NT) {
    s_top[threadIdx.x] = 0;
    s_low[threadIdx.x] = 0xffffffffu;
  }
  __syncthreads();
  const int chunks = p.in_dim / 8, all = p.num_tokens * chunks;
  auto x_at = [&](int r, int c) {
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + r * p.x_row_stride) + c);
  };
  for (int e = threadIdx.x; e < all; e += kFewWarps * 32) {
    const int r = e / chunks;
    const uint4 x = x_at(r, e - r * chunks);
    unsigned top = 0, low = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
      const unsigned lo = v & 0x7fffu, hi = v >> 16 & 0x7fffu;
      top = max(top, max(lo, hi));
      low = min(low, min(lo - 1, hi - 1));
    }
    const unsigned mask = __activemask();
    if (__match_any_sync(mask, r) == mask) {
      top = __reduce_max_sync(mask, top);
      low = __reduce_min_sync(mask, low);
      if (lane == __ffs(mask) - 1) {
        atomicMax(&s_top[r], top);
        atomicMin(&s_low[r], low);
      }
    } else {
      atomicMax(&s_top[r], top);
      atomicMin(&s_low[r], low);
    }
  }
  __syncthreads();
  // The exponent that brings a row's largest value to 2^14.
  auto raise = [&](int r) { return min(14 + 127 - (int)(s_top[r] >> 7), 120); };
  // Whether fp16 has not all of a row: its smallest value's last bit, 2^-134
  // times 2 to the biased exponent, ends up below 2^-24.
  bool wide = false;
  if (lane < p.num_tokens && s_top[lane] > 0)
    wide = s_top[lane] >= 0x7f80u || (int)max((s_low[lane] + 1) >> 7, 1u) + raise(lane) < 134 - 24;
  wide = __any_sync(0xffffffffu, wide);
  auto lift = [&](int r) { return wide ? 0 : raise(r); };
  for (int e = threadIdx.x; e < all; e += kFewWarps * 32) {
    const int r = e / chunks, c = e - r * chunks;
    const uint4 x = x_at(r, c);
    if (wide) {
      *reinterpret_cast<uint4*>(s_x + r * w.x_pitch + c * 16) =
          make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                     __byte_perm(x.y, x.w, 0x7632));
      continue;
    }
    const float f = __uint_as_float((unsigned)(127 + lift(r)) << 23);
    auto pair = [&](uint32_t lo, uint32_t hi) {
      uint32_t v;
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(__uint_as_float(hi) * f), "f"(__uint_as_float(lo) * f));
      return v;
    };
    constexpr uint32_t kTop = 0xffff0000u;
    *reinterpret_cast<uint4*>(s_x + r * w.x_pitch + c * 16) =
        make_uint4(pair(x.x << 16, x.z << 16), pair(x.x & kTop, x.z & kTop), pair(x.y << 16, x.w << 16),
                   pair(x.y & kTop, x.w & kTop));
  }
  __syncthreads();
  const uint8_t* xrow[NT];  // columns past the batch's rows are the last row's and are not stored
#pragma unroll
  for (int n = 0; n < NT; ++n) xrow[n] = s_x + min(n * 8 + g, p.num_tokens - 1) * w.x_pitch + t * 16;

  const bool with_u = p.end > 0;
  bool have_u = false;
  auto take_u = [&] {  // the whole CTA, once
    if (!w.wait_first) pdl_wait();
    if (s_ok)
      for (int e = threadIdx.x; e < p.end * p.n_slices * p.R; e += kFewWarps * 32) {
        float v = 0.f;
#pragma unroll 4
        for (int c = 0; c < w.nsplit; ++c) v += __ldcg(u + c * w.plane_stride + e);
        s_u[e] = v;
      }
    __syncthreads();
    have_u = true;
  };
  int stage = 0;
  float y[MW][NT][4] = {};
  auto team_sync = [&] {
    __syncwarp();
    if (w.team > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / w.team), "r"(w.team * 32) : "memory");
  };
  // The end of a tile: the team's sums, the delta, the outputs.
  auto finish = [&](int tile) {
    float* mine = s_part + warp * ELEMS * 32 + lane;
#pragma unroll
    for (int m = 0; m < MW; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mine[((m * NT + n) * 4 + e) * 32] = y[m][n][e];
          y[m][n][e] = 0.f;
        }
    if (with_u && !have_u) take_u();
    team_sync();
    const int j = slice_of(tile);
    const SliceDesc& sl = p.sl[j];
    const int o = (tile - w.tile_begin[j]) * kMmaOuts + lane;
    if (o < sl.out_dim && s_ok) {
      const bool wide_b = p.R % 8 == 0 && ((reinterpret_cast<uintptr_t>(sl.B) | (uintptr_t)(sl.B_slot_stride * 2)) & 15) == 0;
      for (int r = rank; r < p.num_tokens; r += w.team) {
        // Output lane, row r lie in element e of lane 4 (o % 8) + (r % 8) / 2.
        const int e = ((lane >> 4) * NT + (r >> 3)) * 4 + ((lane >> 3) & 1) * 2 + (r & 1);
        const float* part = s_part + ((warp - rank) * ELEMS + e) * 32 + (lane & 7) * 4 + ((r & 7) >> 1);
        float sum = 0.f;
        for (int v = 0; v < w.team; ++v) sum += part[v * ELEMS * 32];
        sum *= __uint_as_float((unsigned)(127 - lift(r)) << 23);
        const int slot = s_slot[r];
        if (slot >= 0) {
          const int kmax = slot_kmax(p, slot);
          const T* b = static_cast<const T*>(sl.B) + slot * sl.B_slot_stride + (long long)o * p.R;
          const float* ur = s_u + (r * p.n_slices + j) * p.R;
          int k = 0;
          if (wide_b) {
#pragma unroll 2
            for (; k + 8 <= kmax; k += 8) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(b + k));
              const uint32_t bits[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                sum = fmaf(__uint_as_float(bits[q] << 16), ur[k + 2 * q], sum);
                sum = fmaf(__uint_as_float(bits[q] & 0xffff0000u), ur[k + 2 * q + 1], sum);
              }
            }
          }
          for (; k < kmax; ++k) sum = fmaf(value(b[k]), ur[k], sum);
          if (sl.bias) sum += value(static_cast<const T*>(sl.bias)[slot * sl.bias_slot_stride + o]);
        }
        put(static_cast<T*>(sl.y) + r * sl.y_row_stride + o, sum);
      }
    }
    team_sync();  // the sums are read
  };
  int tile = team, blk = b_lo;
  if (b_lo == b_hi) {  // more warps than blocks: this one only helps to finish
    for (; tile < tiles; tile += teams) finish(tile);
  }
#pragma unroll 1
  while (tile < tiles) {
    cp_async_wait<kFewAhead - 1>();
    __syncwarp();
    const uint8_t* at = ring + stage * kFewStage + g * kFewPitch + t * 4;
    const int left = p.in_dim - blk * kFewBlock;
    if (wide) few_block<NT, WPG, false, true>(at, xrow, blk * kFewBlock * 2, raw[0], left, y);
    else if (left >= kFewBlock) few_block<NT, WPG, true, false>(at, xrow, blk * kFewBlock * 2, raw[0], left, y);
    else few_block<NT, WPG, false, false>(at, xrow, blk * kFewBlock * 2, raw[0], left, y);
    stage = stage + 1 == kFewAhead ? 0 : stage + 1;
    __syncwarp();
#pragma unroll
    for (int i = 1; i < kFewAhead; ++i)
#pragma unroll
      for (int c = 0; c < GROUPS; ++c) raw[i - 1][c] = raw[i][c];
    load(raw[kFewAhead - 1]);
    if (++blk == b_hi) {
      finish(tile);
      blk = b_lo;
      tile += teams;
    }
  }
  cp_async_wait<0>();
  if (with_u && !have_u) take_u();  // the others wait for the whole CTA
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

// Warps to a team: what gives the fewest steps of a block, counting a tile's
// end as three quarters of one.
int few_team(int tiles, int nb, int sms) {
  int best = 16;
  long long least = LLONG_MAX;
  for (int team = 16; team >= 1; team /= 2) {
    const long long at_once = (long long)std::min<long long>(sms, ((long long)tiles * team + kFewWarps - 1) / kFewWarps) *
                              (kFewWarps / team);
    const long long steps = (tiles + at_once - 1) / at_once * (4 * ((nb + team - 1) / team) + 3);
    if (steps < least) {
      least = steps;
      best = team;
    }
  }
  return best;
}

int few_x_pitch(const ProblemDesc& p) { return p.in_dim * 2 + (p.in_dim % 64 == 0 ? 64 : 0); }

// Shared memory of the kernel for few rows; it is taken while that fits.
template <int NT>
long long few_smem(const ProblemDesc& p) {
  return kFewRing + few_sum_bytes<NT>() + (long long)p.num_tokens * few_x_pitch(p) + 4LL * p.end * p.n_slices * p.R;
}

template <int NT, int WPG>
cudaError_t launch_q4_few(const ProblemDesc& p, const Q4Weights& wts, const Q4Work& q, const float* u, cudaStream_t s) {
  FewWork w{};
  int tiles = 0;
  for (int j = 0; j < p.n_slices; ++j) {
    w.tile_begin[j] = tiles;
    tiles += (p.sl[j].out_dim + kMmaOuts - 1) / kMmaOuts;
  }
  w.tile_begin[p.n_slices] = tiles;
  const int sms = std::max(device_sm_count(), 1);
  w.team = few_team(tiles, (p.in_dim + kFewBlock - 1) / kFewBlock, sms);
  for (int j = 0; j < p.n_slices; ++j) {
    const int g = wts.w[j].group, units = g >= p.in_dim ? INT_MAX : g / (32 * WPG);
    w.per_group[j] = units == 1 ? 0u : (unsigned)((1ULL << 32) / units + ((1ULL << 32) % units != 0));
  }
  w.x_pitch = few_x_pitch(p);
  w.nsplit = q.nsplit;
  w.plane_stride = q.plane_stride;
  w.wait_first = q.wait_first;
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(q4_few_kernel<NT, WPG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmemMost);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(sms, ((long long)tiles * w.team + kFewWarps - 1) / kFewWarps));
  cfg.blockDim = dim3(kFewWarps * 32);
  cfg.dynamicSmemBytes = (size_t)few_smem<NT>(p);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return noted(cudaLaunchKernelEx(&cfg, q4_few_kernel<NT, WPG>, p, wts, w, u), LORA_PATH_MMA_Q4);
}

template <int NT>
cudaError_t launch_q4_few_words(const ProblemDesc& p, const Q4Weights& wts, const Q4Work& w, const float* u,
                                cudaStream_t s) {
  switch (q4_words_per_group(p, wts)) {
    case 4: return launch_q4_few<NT, 4>(p, wts, w, u, s);
    case 2: return launch_q4_few<NT, 2>(p, wts, w, u, s);
    default: return launch_q4_few<NT, 1>(p, wts, w, u, s);
  }
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
  if ((p.num_tokens + 31) / 32 > 65535 || p.R > 256 || kMmaRing + q4_scale_bytes(p, w) > kMmaSmemMost) return false;
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
  if (q4_tc_ok(p, wts)) {
    const cudaError_t e = launch_q4_tc(p, wts, w, u, s);
    if (e != cudaErrorNotSupported) return e;
  }
  // x in shared memory pays for the two smallest batches, and where the tiles of
  // 32 outputs are more than the other kernel's CTAs that fit at once and many
  // enough for the time that taking x in costs, which goes with rows and inputs.
  // us so and the other way:
  //   4096 inputs   28672 outputs 27.7 and 36.2 (1 row), 37.1 and 39.4 (8);
  //                 20480 29.2 and 32.9 (3), 31.3 and 33.3 (5), 34.1 and 34.0 (8);
  //                 12288 20.7 and 23.3 (3), 21.4 and 23.1 (4), 24.7 and 23.6 (5);
  //                 8192 15.0 and 15.3 (2), 17.0 and 15.6 (3), 21.8 and 16.4 (8)
  //   8192 inputs   28672 50.6 and 58.4 (4); 14336 35.5 and 33.9 (3)
  //   2048 inputs   28672 24.3 and 30.0 (8), 28.0 and 35.7 (9); 12288 18.9 and 18.8 (8)
  //   1024 inputs   28672 26.3 and 31.2 (16); 12288 14.8 and 16.6 (8), 19.8 and 20.6 (16)
  int tiles = 0;
  for (int j = 0; j < p.n_slices; ++j) tiles += (p.sl[j].out_dim + kMmaOuts - 1) / kMmaOuts;
  if (p.num_tokens <= 2 || (tiles > 2 * device_sm_count() && (long long)p.num_tokens * p.in_dim <= 44LL * tiles)) {
    if (p.num_tokens <= 8 && few_smem<1>(p) <= kFewSmemMost) return launch_q4_few_words<1>(p, wts, w, u, s);
    if (p.num_tokens <= 16 && few_smem<2>(p) <= kFewSmemMost) return launch_q4_few_words<2>(p, wts, w, u, s);
  }
  if (p.num_tokens <= 8) return launch_q4_words<1>(p, wts, w, u, s);
  if (p.num_tokens <= 16) return launch_q4_words<2>(p, wts, w, u, s);
  return launch_q4_words<4>(p, wts, w, u, s);
}

}  // namespace lora
