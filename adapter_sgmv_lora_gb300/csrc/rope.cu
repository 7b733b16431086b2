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

// 16-byte accesses.  A head is LPH lanes (a power of two) of two 16-byte
// chunks each.  In the halves layout the two chunks of a rotating lane are
// partners, chunk j of the first half and chunk j of the second, so a pair
// meets in one lane; interleaved pairs lie within a chunk.  A lane keeps its
// chunk position for every head it works on, so the cosines and sines of its
// pairs stay in registers.  Block = one token (times gridDim.y shares of its
// heads); the rows of the next heads are loaded before the present ones are
// rotated, and the first before the angles are worked out.
constexpr int kRopeThreads = 256;

template <typename T>
struct Chunk {
  static constexpr int V = 16 / sizeof(T);
  uint4 bits;
  __device__ __forceinline__ float get(int e) const { return to_f(reinterpret_cast<const T*>(&bits)[e]); }
};

__device__ __forceinline__ uint4 pack_chunk(const float* v, __nv_bfloat16) {
  __nv_bfloat162 r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  return *reinterpret_cast<const uint4*>(r);
}
__device__ __forceinline__ uint4 pack_chunk(const float* v, float) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeDesc p, int lph_log2) {
  constexpr int V = Chunk<T>::V;
  __shared__ float2 cs[LORA_MAX_HEAD_DIM / 2];
  const int t = blockIdx.x;
  const int lph = 1 << lph_log2, j = threadIdx.x & (lph - 1);
  const int half = p.rot / 2, chunks = p.hd / V, turning = half / V;  // turning: partner pairs (halves layout)
  int c0 = 2 * j, c1 = 2 * j + 1;
  if (!INTERLEAVED && j < turning) {
    c0 = j;
    c1 = j + turning;
  }
  const bool has0 = c0 < chunks, has1 = c1 < chunks;
  const int heads = p.H + p.Hk + (p.cache_rows ? p.Hk : 0);
  const int step = gridDim.y * (kRopeThreads >> lph_log2);

  auto load = [&](int h, Chunk<T>& x0, Chunk<T>& x1) {
    if (h >= heads) return;
    const HeadsDesc& in = h < p.H ? p.q : (h < p.H + p.Hk ? p.k : p.v);
    const int hh = h < p.H ? h : (h < p.H + p.Hk ? h - p.H : h - p.H - p.Hk);
    const uint4* row =
        reinterpret_cast<const uint4*>(static_cast<const T*>(in.data) + t * in.row_stride + hh * in.head_stride);
    if (has0) x0.bits = row[c0];
    if (has1) x1.bits = row[c1];
  };
  int h = blockIdx.y * (kRopeThreads >> lph_log2) + (threadIdx.x >> lph_log2);
  Chunk<T> x0{}, x1{}, n0{}, n1{};
  load(h, x0, x1);
  long long row = cache_offset(p, t);
  for (int i = threadIdx.x; i < half; i += kRopeThreads) cs[i] = rope_cos_sin(p, p.positions[t], i);
  __syncthreads();
  // Halves: V pairs; interleaved: V / 2 of each chunk.
  float2 w[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int i = INTERLEAVED ? (e < V / 2 ? c0 : c1) * (V / 2) + e % (V / 2) : c0 * V + e;
    w[e] = i < half ? cs[i] : make_float2(1.f, 0.f);
  }
  const bool turn = INTERLEAVED || j < turning;

  for (; h - (int)(threadIdx.x >> lph_log2) < heads; h += step) {
    load(h + step, n0, n1);
    const bool mine = h < heads;
    const bool is_v = h >= p.H + p.Hk, is_q = h < p.H;
    const T* weight = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
    float a[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      a[e] = x0.get(e);
      b[e] = x1.get(e);
    }
    if (p.q_weight || p.k_weight) {  // uniform, and so is the loop: the whole warp is here
      float sum = 0.f;               // chunks past the head are zero
#pragma unroll
      for (int e = 0; e < V; ++e) sum = fmaf(a[e], a[e], fmaf(b[e], b[e], sum));
      for (int m = lph / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      if (weight && !is_v) {
        const float r = rsqrtf(sum / p.hd + p.eps);
        Chunk<T> g0{}, g1{};
        if (has0) g0.bits = reinterpret_cast<const uint4*>(weight)[c0];
        if (has1) g1.bits = reinterpret_cast<const uint4*>(weight)[c1];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          a[e] *= r * g0.get(e);
          b[e] *= r * g1.get(e);
        }
      }
    }
    if (turn && !is_v) {
      if constexpr (INTERLEAVED) {
        // Chunks past the rotated part are skipped, not turned by 0: an
        // infinite neighbour would come out as NaN.
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 wa = w[e / 2], wb = w[V / 2 + e / 2];
          const float a0 = a[e], a1 = a[e + 1], b0 = b[e], b1 = b[e + 1];
          if (c0 * V < p.rot) {
            a[e] = a0 * wa.x - a1 * wa.y;
            a[e + 1] = a0 * wa.y + a1 * wa.x;
          }
          if (c1 * V < p.rot) {
            b[e] = b0 * wb.x - b1 * wb.y;
            b[e + 1] = b0 * wb.y + b1 * wb.x;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float a0 = a[e], b0 = b[e];
          a[e] = a0 * w[e].x - b0 * w[e].y;
          b[e] = a0 * w[e].y + b0 * w[e].x;
        }
      }
    }
    uint4 r0 = x0.bits, r1 = x1.bits;
    if ((turn || weight) && !is_v) {  // else the bits go through as they are
      r0 = pack_chunk(a, T());
      r1 = pack_chunk(b, T());
    }
    if (mine) {
      const int hh = is_q ? h : (is_v ? h - p.H - p.Hk : h - p.H);
      auto store = [&](void* base, long long off) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(base) + off);
        if (has0) dst[c0] = r0;
        if (has1) dst[c1] = r1;
      };
      if (is_q) {
        store(p.q_out.data, t * p.q_out.row_stride + hh * p.q_out.head_stride);
      } else {
        if (!is_v && p.k_out.data) store(p.k_out.data, t * p.k_out.row_stride + hh * p.k_out.head_stride);
        if (row >= 0) store(is_v ? p.cache.v : p.cache.k, row + hh * p.cache.head_stride);
      }
    }
    x0 = n0;
    x1 = n1;
  }
}

// Whether every row the call touches is whole 16-byte chunks on 16-byte
// boundaries and every rotating chunk's partner is a whole chunk too.
bool fast_ok(const RopeDesc& p) {
  const int V = p.dtype == LORA_DTYPE_BF16 ? 8 : 4;
  if (p.hd % V != 0) return false;
  if (p.rot % (p.layout == LORA_ROPE_HALVES ? 2 * V : V) != 0) return false;
  auto ok = [&](const HeadsDesc& h) {
    return (reinterpret_cast<uintptr_t>(h.data) & 15) == 0 && h.row_stride % V == 0 && h.head_stride % V == 0;
  };
  auto ptr = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  if (p.H > 0 && !(ok(p.q) && ok(p.q_out))) return false;
  if (p.Hk > 0 && !(ok(p.k) && (!p.k_out.data || ok(p.k_out)))) return false;
  if (p.cache_rows) {
    const CacheDesc& c = p.cache;
    if (!ok(p.v) || !ptr(c.k) || !ptr(c.v) || c.page_stride % V != 0 || c.token_stride % V != 0 ||
        c.head_stride % V != 0)
      return false;
  }
  return ptr(p.q_weight) && ptr(p.k_weight);
}

}  // namespace

cudaError_t launch_rope(const RopeDesc& p, cudaStream_t s) {
  const int heads = p.H + p.Hk + (p.cache_rows ? p.Hk : 0);
  const bool fast = fast_ok(p);
  const int V = p.dtype == LORA_DTYPE_BF16 ? 8 : 4;
  int lph_log2 = 0;
  while ((2 << lph_log2) < p.hd / V) ++lph_log2;
  const int at_once = fast ? kRopeThreads >> lph_log2 : kGenericWarps;  // heads a block works on at a time
  // A block takes one token; its heads are shared by several blocks while the
  // batch is too small to give every SM some.
  const int sms = device_sm_count();
  int split = (heads + at_once - 1) / at_once;
  while (split > 1 && (long long)p.T * split > 8LL * sms) split = (split + 1) / 2;
  const dim3 grid(p.T, split);
  const bool bf = p.dtype == LORA_DTYPE_BF16, inter = p.layout == LORA_ROPE_INTERLEAVED;
  if (!fast) {
    if (bf) rope_generic_kernel<__nv_bfloat16><<<grid, kGenericWarps * 32, 0, s>>>(p);
    else rope_generic_kernel<float><<<grid, kGenericWarps * 32, 0, s>>>(p);
    return noted(cudaGetLastError(), LORA_PATH_GENERIC_ROPE);
  }
  if (bf && inter) rope_kernel<__nv_bfloat16, true><<<grid, kRopeThreads, 0, s>>>(p, lph_log2);
  else if (bf) rope_kernel<__nv_bfloat16, false><<<grid, kRopeThreads, 0, s>>>(p, lph_log2);
  else if (inter) rope_kernel<float, true><<<grid, kRopeThreads, 0, s>>>(p, lph_log2);
  else rope_kernel<float, false><<<grid, kRopeThreads, 0, s>>>(p, lph_log2);
  return noted(cudaGetLastError(), LORA_PATH_ROPE);
}

}  // namespace lora
