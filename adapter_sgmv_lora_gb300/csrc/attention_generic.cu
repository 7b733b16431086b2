// attention_generic.cu -- paged decode attention in fp32 arithmetic on the
// CUDA cores: fp32 caches, and bf16 caches whose shapes or alignments the
// tensor-core core does not take.  The frame is attention.cuh.
//
// One warp works on a tile of TT = 8 or 16 tokens held as fp32 rows in shared
// memory.  Scores: lane (r, g) takes token r and every (32 / TT)-th 16-byte
// chunk of its key, so the queries come as broadcasts; the chunks are swizzled
// by the token so that 8 tokens' reads fall on different banks.  Output: each
// lane owns HD / 32 neighbouring columns and walks the tokens.
#include "attention.cuh"

namespace lora {
namespace {

// ASYNC: fp32 rows on 16-byte boundaries come in by asynchronous copies; else
// element by element, converted on the way.
template <typename T_, int HD_, int CH_, bool ASYNC>
struct GenericCore {
  using T = T_;
  // 16 tokens where a tile of them is small: the fixed steps of a tile weigh less.
  static constexpr int TT = HD_ == 64 ? 16 : 8, GRAIN = TT, GROUPS = 32 / TT, W = 4, HD = HD_, CH = CH_, COMB = CH_ < 4 ? CH_ : 4;
  static constexpr int STAGE_BYTES = 2 * TT * HD * 4;
  static constexpr int STAGES = CH == 8 && HD > 64 ? 2 : 3;
  static constexpr int CTAS = HD <= 128 ? 2 : 1;
  static constexpr int VPL = HD / 32;  // output columns per lane
  static constexpr int STREAM_COST = 6;
  static constexpr int EXTRA_BYTES = W * (CH * HD + TT * CH) * 4;
  static_assert(CH <= 8, "");

  float* shared;
  float* q;  // [CH][HD]: the CTA's queries, or this warp's where it is on its own
  float* prob;  // [TT][CH], this warp's
  float scale;
  uint64_t policy;
  int heads;
  float m[CH], l[CH], o[CH][VPL];
  float next_q[(CH * HD + W * 32 - 1) / (W * 32)];

  __device__ __forceinline__ GenericCore(const AttnDesc& p, uint8_t* extra)
      : shared(reinterpret_cast<float*>(extra)),
        q(shared),
        prob(q + W * CH * HD + (threadIdx.x >> 5) * TT * CH),
        scale(p.scale * kLog2e),
        policy(cache_policy(p)) {}

  static __device__ __forceinline__ int at(int r, int chunk) { return r * HD + ((chunk ^ (r & 7)) << 2); }

  __device__ __forceinline__ void load(const AttnDesc& p, uint8_t* stage, long long off, int n) const {
    float* k = reinterpret_cast<float*>(stage);
    float* v = k + TT * HD;
    const int lane = threadIdx.x & 31;
    const T* kg = static_cast<const T*>(p.cache.k);
    const T* vg = static_cast<const T*>(p.cache.v);
    // Offset of each row (lane r knows row r's), -1: none.
    if (p.whole_grains) off = off < 0 || (lane & (TT - 1)) >= n ? -1 : off + (lane & (TT - 1)) * p.cache.token_stride;
    if constexpr (ASYNC) {
#pragma unroll
      for (int i = 0; i < TT * HD / 4 / 32; ++i) {
        const int e = i * 32 + lane, r = e / (HD / 4), c = e % (HD / 4);
        const long long row = __shfl_sync(0xffffffffu, off, r);
        if (c * 4 < p.cache.head_dim) {
          const long long src = row < 0 ? 0 : row + c * 4;
          cp_async16_zfill(k + at(r, c), kg + src, row < 0 ? 0 : 16, policy);
          cp_async16_zfill(v + at(r, c), vg + src, row < 0 ? 0 : 16, policy);
        }
      }
    } else {
#pragma unroll 1
      for (int r = 0; r < TT; ++r) {
        const long long row = __shfl_sync(0xffffffffu, off, r);
        for (int d = lane; d < p.cache.head_dim; d += 32) {
          const int dst = at(r, d >> 2) + (d & 3);
          k[dst] = row < 0 ? 0.f : to_f(kg[row + d]);
          v[dst] = row < 0 ? 0.f : to_f(vg[row + d]);
        }
      }
    }
  }

  static constexpr int Q_PER_THREAD = (CH * HD + W * 32 - 1) / (W * 32);
  __device__ __forceinline__ void fetch(const AttnDesc& p, int seq, int head0, int heads_) {
    const T* src = static_cast<const T*>(p.q.data) + seq * p.q.row_stride + head0 * p.q.head_stride;
#pragma unroll
    for (int i = 0; i < Q_PER_THREAD; ++i) {
      const int e = i * W * 32 + threadIdx.x, h = e / HD, d = e % HD;
      next_q[i] = h < heads_ && d < p.cache.head_dim ? to_f(src[h * p.q.head_stride + d]) : 0.f;
    }
  }

  __device__ __forceinline__ void pass_on() const {
#pragma unroll
    for (int i = 0; i < Q_PER_THREAD; ++i)
      if (i * W * 32 + threadIdx.x < CH * HD) q[i * W * 32 + threadIdx.x] = next_q[i];
  }

  __device__ __forceinline__ void begin_solo(const AttnDesc& p, int seq, int head0, int heads_) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    q = shared + warp * CH * HD;
    const T* src = static_cast<const T*>(p.q.data) + seq * p.q.row_stride + head0 * p.q.head_stride;
    for (int h = 0; h < heads_; ++h) {  // rows of heads that are not there are not read
      float v[HD / 32];
#pragma unroll
      for (int i = 0; i < HD / 32; ++i)
        v[i] = i * 32 + lane < p.cache.head_dim ? to_f(src[h * p.q.head_stride + i * 32 + lane]) : 0.f;
#pragma unroll
      for (int i = 0; i < HD / 32; ++i) q[h * HD + i * 32 + lane] = v[i];
    }
    __syncwarp();
    begin(p, heads_);
  }

  __device__ __forceinline__ void begin(const AttnDesc&, int heads_) {
    heads = heads_;
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      m[h] = kNegInf;
      l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < VPL; ++e) o[h][e] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const AttnDesc& p, const uint8_t* stage, int n) {
    const float* k = reinterpret_cast<const float*>(stage);
    const float* v = k + TT * HD;
    const int lane = threadIdx.x & 31, r = lane % TT, g = lane / TT;
    float s[CH] = {};
#pragma unroll 4
    for (int i = 0; i < HD / 4 / GROUPS; ++i) {
      const int c = i * GROUPS + g;
      const float4 kv = *reinterpret_cast<const float4*>(k + at(r, c));
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        if (h < heads) {
          const float4 qv = *reinterpret_cast<const float4*>(q + h * HD + c * 4);
          s[h] = fmaf(kv.x, qv.x, s[h]);
          s[h] = fmaf(kv.y, qv.y, s[h]);
          s[h] = fmaf(kv.z, qv.z, s[h]);
          s[h] = fmaf(kv.w, qv.w, s[h]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      if (h >= heads) continue;
#pragma unroll
      for (int d = TT; d < 32; d <<= 1) s[h] += __shfl_xor_sync(0xffffffffu, s[h], d);
      s[h] = r < n ? s[h] * scale : kNegInf;
      float top = s[h];
#pragma unroll
      for (int d = TT / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float now = fmaxf(m[h], top);
      const float base = now == kNegInf ? 0.f : now;  // nothing but -inf so far: every weight is 0
      const float pr = pow2(s[h] - base);
      const float keep = pow2(m[h] - base);
      m[h] = now;
      l[h] = fmaf(l[h], keep, pr);  // this lane's token; the tokens are summed in put
#pragma unroll
      for (int e = 0; e < VPL; ++e) o[h][e] *= keep;
      if (g == 0) prob[r * CH + h] = pr;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      float vv[VPL];
#pragma unroll
      for (int e = 0; e < VPL; ++e) {
        const int d = lane * VPL + e;
        vv[e] = v[at(j, d >> 2) + (d & 3)];
      }
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        if (h >= heads) continue;
        const float pr = prob[j * CH + h];
#pragma unroll
        for (int e = 0; e < VPL; ++e) o[h][e] = fmaf(pr, vv[e], o[h][e]);
      }
    }
    __syncwarp();
  }

  __device__ __forceinline__ void put(int part, float* comb, float2* stat) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      if (h / COMB != part) continue;
      float sum = l[h];
#pragma unroll
      for (int d = TT / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) stat[h % COMB] = make_float2(m[h], sum);
#pragma unroll
      for (int e = 0; e < VPL; ++e) comb[(h % COMB) * (HD + 4) + lane * VPL + e] = o[h][e];
    }
  }
};

// fp32 rows on 16-byte boundaries.
bool async_ok(const AttnDesc& p) {
  const CacheDesc& c = p.cache;
  const auto low = reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v);
  return p.dtype == LORA_DTYPE_F32 && (low & 15) == 0 && c.head_dim % 4 == 0 && c.page_stride % 4 == 0 &&
         c.token_stride % 4 == 0 && c.head_stride % 4 == 0;
}

template <typename T, int HD, bool ASYNC>
cudaError_t by_group(const AttnDesc& p, void* ws, cudaStream_t s) {
  if (p.group == 1) return launch_core<GenericCore<T, HD, 1, ASYNC>>(p, ws, s, LORA_PATH_GENERIC_ATTENTION);
  return launch_core<GenericCore<T, HD, 8, ASYNC>>(p, ws, s, LORA_PATH_GENERIC_ATTENTION);
}

template <typename T, bool ASYNC>
cudaError_t by_width(const AttnDesc& p, void* ws, cudaStream_t s) {
  if (p.cache.head_dim <= 64) return by_group<T, 64, ASYNC>(p, ws, s);
  if (p.cache.head_dim <= 128) return by_group<T, 128, ASYNC>(p, ws, s);
  return by_group<T, 256, ASYNC>(p, ws, s);
}

}  // namespace

CoreShape generic_attention_shape(const AttnDesc& p) {
  const int hd = p.cache.head_dim <= 64 ? 64 : (p.cache.head_dim <= 128 ? 128 : 256);
  CoreShape c = shape_of<GenericCore<float, 64, 8, true>>();
  c.TT = hd <= 64 ? 16 : 8;
  c.HD = hd;
  c.CH = p.group == 1 ? 1 : 8;
  c.CTAS = hd <= 128 ? 2 : 1;
  return c;
}

cudaError_t launch_attention_generic(const AttnDesc& p, void* workspace, cudaStream_t s) {
  if (p.dtype == LORA_DTYPE_BF16) return by_width<__nv_bfloat16, false>(p, workspace, s);
  return async_ok(p) ? by_width<float, true>(p, workspace, s) : by_width<float, false>(p, workspace, s);
}

}  // namespace lora
