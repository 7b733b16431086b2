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
// turns, go to sincospi.  No range reduction is needed.  What is lost is fp32's
// rounding of that number, 2^-26 of a turn at most, and the table's own (an
// entry comes from a double and is off by up to 2^-55 of a turn: 2^-24 at
// position 2^31), where an fp32 product position * f loses whole hundredths of
// a radian at 100k tokens.  The table is one 64-bit word per pair instead of a
// cos/sin row per position.
#include <cuda_bf16.h>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

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
// = one token and a share of its heads (query, key, then value heads).  Bound by
// its instructions, an access of 2 or 4 bytes per element: 8192 bf16 tokens of
// 32 + 2 x 8 heads, 80 wide, that rotate 20 take 106 us, rotating 64 by the
// kernel below 34; 96 wide and 24 123, all 96 36.
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
// chunks each, so a warp holds a group of 32 / LPH heads.  In the halves
// layout the two chunks of a rotating lane are partners, chunk j of the first
// half and chunk j of the second, so a pair meets in one lane; interleaved
// pairs lie within a chunk.  A lane keeps its chunk position for every head it
// works on, so the cosines and sines of its pairs stay in registers.
//
// A warp takes one token, or a share of its groups, and works the angles out
// for itself: no block barrier.  Query, key and value heads are grouped apart,
// so what a group needs is the same for the whole warp.  Four or five groups
// are loaded at a time (the first before the angles): 4 to 5 KB a warp in
// flight.  Products go two to an instruction (f32x2).  What is larger than L2
// anyway is read and written as streams (either alone gains nothing).
//
// Bounded by memory: 8192 bf16 tokens of 64 + 2 x 8 heads, 336 MB, take 55.6 us
// (6.0 TB/s; a plain copy of as many bytes takes 57.9), and took 66.6 where
// they take 57.3 with the streams.  With norms (40 + 2 x 8 heads, 235 MB) 57.3
// us: there the reductions' latency shows.
constexpr int kRopeWarps = 4;  // per block
// Groups a batch; measured 5 / 4: 80 heads 57.3 / 60.9 us, 48 heads 39.4 / 39.4,
// 56 heads with norms 60.9 / 57.9.
constexpr int kRopeBatch = 5, kRopeNormBatch = 4;

// A chunk's elements, eight (four of fp32), as fp32, and back.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void open(const uint4& b, float* v) {
    const unsigned w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 close(const float* v) {
    return make_uint4(round_pack_bf16x2(v[0], v[1]), round_pack_bf16x2(v[2], v[3]), round_pack_bf16x2(v[4], v[5]),
                      round_pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct Chunk<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void open(const uint4& b, float* v) {
    v[0] = __uint_as_float(b.x);
    v[1] = __uint_as_float(b.y);
    v[2] = __uint_as_float(b.z);
    v[3] = __uint_as_float(b.w);
  }
  static __device__ __forceinline__ uint4 close(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

template <typename T, bool INTERLEAVED, bool NORM, int BATCH>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const __grid_constant__ RopeDesc p, int lph_log2,
                                                               int shares) {
  constexpr int V = Chunk<T>::V;
  __shared__ float2 s_cs[kRopeWarps][LORA_MAX_HEAD_DIM / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long task = (long long)blockIdx.x * kRopeWarps + warp;
  const int t = (int)(task / shares), share = (int)(task - (long long)t * shares);
  if (t >= p.T) return;  // the whole warp
  const int lph = 1 << lph_log2, j = lane & (lph - 1), sub = lane >> lph_log2, at_once = 32 >> lph_log2;
  const int half = p.rot / 2, chunks = p.hd / V, turning = half / V;  // turning: partner pairs (halves layout)
  int c0 = 2 * j, c1 = 2 * j + 1;
  if (!INTERLEAVED && j < turning) {
    c0 = j;
    c1 = j + turning;
  }
  const bool has0 = c0 < chunks, has1 = c1 < chunks;
  const int q_groups = (p.H + at_once - 1) >> (5 - lph_log2), k_groups = (p.Hk + at_once - 1) >> (5 - lph_log2);
  const int groups = q_groups + (p.cache_rows ? 2 : 1) * k_groups;

  // This lane's head of group g, among those of its kind.
  auto head_of = [&](int g) {
    return (g < q_groups ? g : g - q_groups - (g < q_groups + k_groups ? 0 : k_groups)) * at_once + sub;
  };
  auto load = [&](int g, uint4 (&x)[2]) {
    if (g >= groups) return;
    const bool is_q = g < q_groups;
    const HeadsDesc& in = is_q ? p.q : (g < q_groups + k_groups ? p.k : p.v);
    const int h = head_of(g);
    if (h >= (is_q ? p.H : p.Hk)) return;
    const uint4* row =
        reinterpret_cast<const uint4*>(static_cast<const T*>(in.data) + t * in.row_stride + h * in.head_stride);
    if (has0) x[0] = BATCH > 1 ? __ldcs(row + c0) : row[c0];
    if (has1) x[1] = BATCH > 1 ? __ldcs(row + c1) : row[c1];
  };
  uint4 x[BATCH][2] = {};
#pragma unroll
  for (int i = 0; i < BATCH; ++i) load(share + i * shares, x[i]);
  const long long row = cache_offset(p, t);
  float2* cs = s_cs[warp];
  if (half > 0) {
    const int position = p.positions[t];
    for (int i = lane; i < half; i += 32) cs[i] = rope_cos_sin(p, position, i);
    __syncwarp();
  }
  // Halves: V pairs; interleaved: V / 2 of each chunk.
  float c[V], s[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int i = INTERLEAVED ? (e < V / 2 ? c0 : c1) * (V / 2) + e % (V / 2) : c0 * V + e;
    const float2 w = i < half ? cs[i] : make_float2(1.f, 0.f);
    c[e] = w.x;
    s[e] = w.y;
  }

  auto work = [&](int g, const uint4 (&x)[2]) {
    const bool is_q = g < q_groups, is_v = g >= q_groups + k_groups;
    const int h = head_of(g);
    uint4 r[2] = {x[0], x[1]};
    const T* weight = NORM ? static_cast<const T*>(is_q ? p.q_weight : p.k_weight) : nullptr;
    if (!is_v && (half > 0 || weight)) {  // else the bits go through as they are
      float a[V], b[V];
      Chunk<T>::open(x[0], a);
      Chunk<T>::open(x[1], b);
      if (NORM && weight) {
        float2 sum2 = make_float2(0.f, 0.f);  // chunks past the head are zero
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          sum2 = fma_f32x2(make_float2(a[e], a[e + 1]), make_float2(a[e], a[e + 1]), sum2);
          sum2 = fma_f32x2(make_float2(b[e], b[e + 1]), make_float2(b[e], b[e + 1]), sum2);
        }
        float sum = sum2.x + sum2.y;
        for (int m = lph / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const float n = rsqrtf(sum / p.hd + p.eps);
        uint4 g0 = {}, g1 = {};
        if (has0) g0 = reinterpret_cast<const uint4*>(weight)[c0];
        if (has1) g1 = reinterpret_cast<const uint4*>(weight)[c1];
        float wa[V], wb[V];
        Chunk<T>::open(g0, wa);
        Chunk<T>::open(g1, wb);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          a[e] *= n * wa[e];
          b[e] *= n * wb[e];
        }
      }
      // Chunks past the rotated part are skipped, not turned by 0: an
      // infinite neighbour would come out as NaN.
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float a0 = a[e], a1 = a[e + 1], b0 = b[e], b1 = b[e + 1];
          const float ca = c[e / 2], sa = s[e / 2], cb = c[V / 2 + e / 2], sb = s[V / 2 + e / 2];
          if (c0 * V < p.rot) {
            a[e] = a0 * ca - a1 * sa;
            a[e + 1] = a0 * sa + a1 * ca;
          }
          if (c1 * V < p.rot) {
            b[e] = b0 * cb - b1 * sb;
            b[e + 1] = b0 * sb + b1 * cb;
          }
        }
      } else if (j < turning) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 a2 = make_float2(a[e], a[e + 1]), b2 = make_float2(b[e], b[e + 1]);
          const float2 c2 = make_float2(c[e], c[e + 1]), s2 = make_float2(s[e], s[e + 1]);
          const float2 ra = fma_f32x2(make_float2(-b2.x, -b2.y), s2, mul_f32x2(a2, c2));
          const float2 rb = fma_f32x2(b2, c2, mul_f32x2(a2, s2));
          a[e] = ra.x;
          a[e + 1] = ra.y;
          b[e] = rb.x;
          b[e + 1] = rb.y;
        }
      }
      r[0] = Chunk<T>::close(a);
      r[1] = Chunk<T>::close(b);
    }
    if (h >= (is_q ? p.H : p.Hk)) return;
    auto store = [&](void* base, long long off) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(base) + off);
      if (has0) {
        if (BATCH > 1) __stcs(dst + c0, r[0]);
        else dst[c0] = r[0];
      }
      if (has1) {
        if (BATCH > 1) __stcs(dst + c1, r[1]);
        else dst[c1] = r[1];
      }
    };
    if (is_q) {
      store(p.q_out.data, t * p.q_out.row_stride + h * p.q_out.head_stride);
    } else {
      if (!is_v && p.k_out.data) store(p.k_out.data, t * p.k_out.row_stride + h * p.k_out.head_stride);
      if (row >= 0) store(is_v ? p.cache.v : p.cache.k, row + h * p.cache.head_stride);
    }
  };
#pragma unroll 1
  for (int g = share; g < groups; g += BATCH * shares) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (g + i * shares < groups) work(g + i * shares, x[i]);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) load(g + (BATCH + i) * shares, x[i]);
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
  const int at_once = fast ? 32 >> lph_log2 : kGenericWarps;  // heads a warp (or block) works on at a time
  const int sms = device_sm_count();
  const bool bf = p.dtype == LORA_DTYPE_BF16, inter = p.layout == LORA_ROPE_INTERLEAVED;
  if (!fast) {
    // Few tokens: their heads are shared out until every SM has work.
    int split = (heads + at_once - 1) / at_once;
    while (split > 1 && (long long)p.T * split > 8LL * sms) split = (split + 1) / 2;
    const dim3 grid(p.T, split);
    if (bf) rope_generic_kernel<__nv_bfloat16><<<grid, kGenericWarps * 32, 0, s>>>(p);
    else rope_generic_kernel<float><<<grid, kGenericWarps * 32, 0, s>>>(p);
    return noted(cudaGetLastError(), LORA_PATH_GENERIC_ROPE);
  }
  const int groups = (p.H + at_once - 1) / at_once + (p.cache_rows ? 2 : 1) * ((p.Hk + at_once - 1) / at_once);
  // Few tokens: a group to a warp, by the kernel whose code is short (256
  // tokens of 48 heads: 6.1 us against 8.2 by the long one, which is mostly
  // instructions not yet in any cache).
  const bool few = (long long)p.T * groups <= 32LL * sms;
  const bool norm = p.q_weight || p.k_weight;
  const int batch = norm ? kRopeNormBatch : kRopeBatch;
  const int shares = few ? groups : (groups + batch - 1) / batch;
  const unsigned grid = (unsigned)(((long long)p.T * shares + kRopeWarps - 1) / kRopeWarps);
  auto run = [&](auto kernel) { kernel<<<grid, kRopeWarps * 32, 0, s>>>(p, lph_log2, shares); };
  auto by_kind = [&](auto norm_c, auto batch_c) {
    constexpr bool N = decltype(norm_c)::value;
    constexpr int B = decltype(batch_c)::value;
    if (bf && inter) run(rope_kernel<__nv_bfloat16, true, N, B>);
    else if (bf) run(rope_kernel<__nv_bfloat16, false, N, B>);
    else if (inter) run(rope_kernel<float, true, N, B>);
    else run(rope_kernel<float, false, N, B>);
  };
  if (few && norm) by_kind(std::true_type(), std::integral_constant<int, 1>());
  else if (few) by_kind(std::false_type(), std::integral_constant<int, 1>());
  else if (norm) by_kind(std::true_type(), std::integral_constant<int, kRopeNormBatch>());
  else by_kind(std::false_type(), std::integral_constant<int, kRopeBatch>());
  return noted(cudaGetLastError(), LORA_PATH_ROPE);
}

}  // namespace lora
