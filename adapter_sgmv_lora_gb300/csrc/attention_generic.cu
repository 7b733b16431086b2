// attention_generic.cu -- paged decode attention in fp32 arithmetic on the
// CUDA cores: fp32 caches, and bf16 caches whose page sizes, shapes or
// alignments the tensor-core core does not take (pages that are not whole
// grains of 8 tokens above all).  The frame is attention.cuh.
//
// One warp works on a tile of TT = 8 or 16 tokens held in shared memory in the
// cache's type (fp32 where rows are not on 16-byte boundaries).  Scores: lane
// (r, g) takes token r and every (32 / TT)-th 16-byte chunk of its key, so the
// queries come as broadcasts; the chunks are swizzled by the token so that 8
// tokens' reads fall on different banks.  Output: each lane owns HD / 32
// neighbouring columns and walks the tokens.
#include <type_traits>

#include "attention.cuh"

namespace lora {
namespace {

// N neighbouring values, 4 N or 2 N bytes on a boundary of as many.
template <int N>
__device__ __forceinline__ void read_row(const float* p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 w = *reinterpret_cast<const float4*>(p + i);
      v[i] = w.x;
      v[i + 1] = w.y;
      v[i + 2] = w.z;
      v[i + 3] = w.w;
    }
  } else {
    const float2 w = *reinterpret_cast<const float2*>(p);
    v[0] = w.x;
    v[1] = w.y;
  }
}
template <int N>
__device__ __forceinline__ void read_row(const __nv_bfloat16* p, float (&v)[N]) {
  uint32_t w[N / 2];
  if constexpr (N == 8) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
  else if constexpr (N == 4) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
  else w[0] = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// ASYNC: rows on 16-byte boundaries come in by asynchronous copies, as they
// are; else element by element, converted to fp32 on the way.
template <typename T_, int HD_, int CH_, bool ASYNC>
struct GenericCore {
  using T = T_;
  using S = std::conditional_t<ASYNC, T, float>;  // type of a staged row
  static constexpr int HD = HD_, CH = CH_, COMB = CH_ < 4 ? CH_ : 4, W = 4;
  // 16 tokens where a row of them is short: the fixed steps of a tile weigh less.
  static constexpr int TT = HD * sizeof(S) <= 256 ? 16 : 8, GRAIN = TT, GROUPS = 32 / TT;
  static constexpr int E = 16 / sizeof(S), CHUNKS = HD / E;  // of a row
  static constexpr int STAGE_BYTES = 2 * TT * HD * sizeof(S);
  static constexpr int CTAS = HD <= 128 ? 2 : 1;
  static constexpr int VPL = HD / 32;  // output columns per lane
  static constexpr int STREAM_COST = 6;
  static constexpr int EXTRA_BYTES = W * (CH * HD + TT * CH) * 4;
  // As many stages as leave room for CTAS blocks on an SM, up to six.
  static constexpr int ROOM = (CTAS == 2 ? 115200 : 231000) - W * COMB * ((HD + 4) * 4 + 8) - EXTRA_BYTES;
  static constexpr int STAGES = ROOM / (W * STAGE_BYTES) < 6 ? ROOM / (W * STAGE_BYTES) : 6;
  static_assert(CH <= 8, "");

  float* shared;
  float* q;  // [CH][HD]: the CTA's queries, or this warp's where it is on its own
  float* prob;  // [TT][CH], this warp's
  float scale;
  int heads;
  float m[CH], l[CH], o[CH][VPL];
  float next_q[(CH * HD + W * 32 - 1) / (W * 32)];

  __device__ __forceinline__ GenericCore(const AttnDesc& p, uint8_t* extra)
      : shared(reinterpret_cast<float*>(extra)),
        q(shared),
        prob(q + W * CH * HD + (threadIdx.x >> 5) * TT * CH),
        scale(p.scale * kLog2e) {}

  // Element of chunk c of row r.
  static __device__ __forceinline__ int at(int r, int c) { return r * HD + (c ^ (r & 7)) * E; }

  __device__ __forceinline__ void load(const AttnDesc& p, uint8_t* stage, long long off, int n) const {
    S* k = reinterpret_cast<S*>(stage);
    S* v = k + TT * HD;
    const int lane = threadIdx.x & 31;
    const T* kg = static_cast<const T*>(p.cache.k);
    const T* vg = static_cast<const T*>(p.cache.v);
    // Offset of each row (lane r knows row r's), -1: none.
    if (p.whole_grains) off = off < 0 || (lane & (TT - 1)) >= n ? -1 : off + (lane & (TT - 1)) * p.cache.token_stride;
    if constexpr (ASYNC) {
#pragma unroll
      for (int i = 0; i < TT * CHUNKS / 32; ++i) {
        const int e = i * 32 + lane, r = e / CHUNKS, c = e % CHUNKS;
        const long long row = __shfl_sync(0xffffffffu, off, r);
        if (c * E < p.cache.head_dim) {
          const long long src = row < 0 ? 0 : row + c * E;
          cp_async16_zfill(k + at(r, c), kg + src, row < 0 ? 0 : 16);
          cp_async16_zfill(v + at(r, c), vg + src, row < 0 ? 0 : 16);
        }
      }
    } else {
#pragma unroll 1
      for (int r = 0; r < TT; ++r) {
        const long long row = __shfl_sync(0xffffffffu, off, r);
        for (int d = lane; d < p.cache.head_dim; d += 32) {
          const int dst = at(r, d / E) + d % E;
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
    const S* k = reinterpret_cast<const S*>(stage);
    const S* v = k + TT * HD;
    const int lane = threadIdx.x & 31, r = lane % TT, g = lane / TT;
    float2 pair[CH];  // products go two to an instruction
#pragma unroll
    for (int h = 0; h < CH; ++h) pair[h] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < CHUNKS / GROUPS; ++i) {
      const int c = i * GROUPS + g;
      float kv[E];
      read_row<E>(k + at(r, c), kv);
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        if (h < heads) {
          float qv[E];
          read_row<E>(q + h * HD + c * E, qv);
#pragma unroll
          for (int e = 0; e < E; e += 2)
            pair[h] = fma_f32x2(make_float2(kv[e], kv[e + 1]), make_float2(qv[e], qv[e + 1]), pair[h]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      if (h >= heads) continue;
      float s = pair[h].x + pair[h].y;
#pragma unroll
      for (int d = TT; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s = r < n ? s * scale : kNegInf;
      float top = s;
#pragma unroll
      for (int d = TT / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float now = fmaxf(m[h], top);
      const float base = now == kNegInf ? 0.f : now;  // nothing but -inf so far: every weight is 0
      const float pr = pow2(s - base);
      const float keep = pow2(m[h] - base);
      m[h] = now;
      l[h] = fmaf(l[h], keep, pr);  // this lane's token; the tokens are summed in put
#pragma unroll
      for (int e = 0; e < VPL; e += 2) {
        const float2 w = mul_f32x2(make_float2(o[h][e], o[h][e + 1]), make_float2(keep, keep));
        o[h][e] = w.x;
        o[h][e + 1] = w.y;
      }
      if (g == 0) prob[r * CH + h] = pr;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      // This lane's columns: within one chunk, or whole chunks (fp32, 256 wide).
      float vv[VPL];
      constexpr int PART = VPL < E ? VPL : E;
#pragma unroll
      for (int e = 0; e < VPL; e += PART) {
        float part[PART];
        const int d = lane * VPL + e;
        read_row<PART>(v + at(j, d / E) + d % E, part);
#pragma unroll
        for (int x = 0; x < PART; ++x) vv[e + x] = part[x];
      }
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        if (h >= heads) continue;
        const float pr = prob[j * CH + h];
#pragma unroll
        for (int e = 0; e < VPL; e += 2) {
          const float2 w = fma_f32x2(make_float2(pr, pr), make_float2(vv[e], vv[e + 1]),
                                     make_float2(o[h][e], o[h][e + 1]));
          o[h][e] = w.x;
          o[h][e + 1] = w.y;
        }
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

// Rows on 16-byte boundaries.
bool async_ok(const AttnDesc& p) {
  const CacheDesc& c = p.cache;
  const int e = p.dtype == LORA_DTYPE_BF16 ? 8 : 4;
  const auto low = reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v);
  return (low & 15) == 0 && c.head_dim % e == 0 && c.page_stride % e == 0 && c.token_stride % e == 0 &&
         c.head_stride % e == 0;
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

template <typename T>
size_t most_workspace(const AttnDesc& p) {
  auto of = [&](auto* core) { return workspace_bytes_of(shape_of<std::remove_pointer_t<decltype(core)>>(), p); };
  auto both = [&](auto hd) {
    constexpr int HD = decltype(hd)::value;
    if (p.group == 1) return std::max(of((GenericCore<T, HD, 1, true>*)nullptr), of((GenericCore<T, HD, 1, false>*)nullptr));
    return std::max(of((GenericCore<T, HD, 8, true>*)nullptr), of((GenericCore<T, HD, 8, false>*)nullptr));
  };
  if (p.cache.head_dim <= 64) return both(std::integral_constant<int, 64>());
  if (p.cache.head_dim <= 128) return both(std::integral_constant<int, 128>());
  return both(std::integral_constant<int, 256>());
}

size_t generic_attention_workspace(const AttnDesc& p) {
  return p.dtype == LORA_DTYPE_BF16 ? most_workspace<__nv_bfloat16>(p) : most_workspace<float>(p);
}

cudaError_t launch_attention_generic(const AttnDesc& p, void* workspace, cudaStream_t s) {
  if (p.dtype == LORA_DTYPE_BF16)
    return async_ok(p) ? by_width<__nv_bfloat16, true>(p, workspace, s)
                       : by_width<__nv_bfloat16, false>(p, workspace, s);
  return async_ok(p) ? by_width<float, true>(p, workspace, s) : by_width<float, false>(p, workspace, s);
}

}  // namespace lora
