// attention_mma.cu -- paged decode attention of bf16 caches on the tensor
// cores (mma.sync m16n8k16, fp32 accumulation).  The frame is attention.cuh.
//
// One warp works on a tile of 16 tokens.  The tokens are the 16 rows of the
// product and the query heads that share them its 8 columns, so a group of 8
// heads fills the instruction (the other way round 8 of 16 rows would be
// padding):
//   S^T [16 tokens, 8 heads] = K [16, HD] Q^T       K by ldmatrix, Q in registers
//   O^T [HD, 8 heads]       += V^T [HD, 16] P       V by transposing ldmatrix
// P comes out of the first product with tokens along its rows and is turned
// into the second's operand in registers (movmatrix).  It enters as three bf16
// terms whose sum is p to fp32's own 24 bits: two leave 2^-18, which moves one
// output in some hundreds to the neighbouring bf16 value.  Every term of a
// p > 0 is positive, so an infinite value comes out as that infinity.  The
// second product starts from zero in every tile and O takes it up by rounded
// fused multiply-adds, which hold the softmax's rescaling too: accumulated by
// the instruction itself, long contexts lost a bit of every step (24 of 8192
// to 32768 tokens: 1000 of 196608 outputs not the nearest bf16 to the exact
// result, now 80; the definition in fp32 321).  Four steps of the head go
// together so that their chains overlap (256-wide heads 308 us, one by one 327;
// with 16 heads a group two, 128 wide: 167 and 175).
//
// A call reads 512 bytes of cache per token and key/value head (128 wide) and
// does 4096 flops on them for 8 heads: at memory speed that is some 55
// TFLOP/s, a few percent of what the instruction reaches, so the 128-row
// tcgen05 tiles would buy nothing here and cost the softmax its place in
// registers.  What bounds the kernel is memory.
#include <type_traits>

#include "attention.cuh"

namespace lora {
namespace {

// NT: query heads a stream, in eights.  GRAIN: tokens that lie in one page.
template <int HD_, int NT, int GRAIN_>
struct MmaCore {
  using T = __nv_bfloat16;
  // A stage is 8 KB (16 KB for the widest heads, 4 KB for the narrowest): narrow
  // heads take two blocks of 16 tokens a tile, so the fixed steps of a tile weigh
  // the same.
  static constexpr int BLOCKS = HD_ <= 64 ? 2 : 1, TT = 16 * BLOCKS;
  static constexpr int GRAIN = GRAIN_, GRAINS = TT / GRAIN;
  static constexpr int W = 4, HD = HD_, CH = 8 * NT, COMB = 4;
  static constexpr int STAGE_BYTES = 2 * TT * HD * 2;
  static constexpr int STAGES = HD == 32 ? 6 : 3;
  static constexpr int CTAS = HD <= 128 ? 2 : 1;
  static constexpr int STREAM_COST = 6;
  static constexpr int EXTRA_BYTES = CH * HD * 2;
  static constexpr int KT = HD / 16;  // 16-wide steps of the head

  uint32_t q[KT][NT][2];  // Q^T fragments
  float o[KT][NT][4];     // O^T accumulators: rows 16 k + lane / 4 (+ 8), heads 2 (lane % 4) (+ 1)
  float m[NT][2], l[NT][2];
  float scale;

  uint8_t* q_shared;
  uint4 next_q[(CH * HD / 8 + W * 32 - 1) / (W * 32)];

  __device__ __forceinline__ MmaCore(const AttnDesc& p, uint8_t* extra)
      : scale(p.scale * kLog2e), q_shared(extra) {}

  // Byte offset of 16-byte chunk c of row r: swizzled, so the 8 rows of an
  // ldmatrix block fall on different banks.
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return r * (HD * 2) + ((c ^ (HD >= 64 ? r & 7 : (r >> 1) & 3)) << 4);
  }

  __device__ __forceinline__ void load(const AttnDesc& p, uint8_t* stage, long long off, int n) const {
    constexpr int ROWS = 32 / (HD / 8);  // rows that one copy of the warp covers
    const int lane = threadIdx.x & 31, r0 = lane / (HD / 8), c = lane % (HD / 8);
    const T* kg = static_cast<const T*>(p.cache.k);
    const T* vg = static_cast<const T*>(p.cache.v);
#pragma unroll
    for (int j = 0; j < GRAINS; ++j) {
      const long long first = __shfl_sync(0xffffffffu, off, j);
      if (c * 8 < p.cache.head_dim) {
        long long src = (first < 0 ? 0 : first + r0 * p.cache.token_stride) + c * 8;
        const long long step = first < 0 ? 0 : ROWS * p.cache.token_stride;
        const int live = first < 0 ? 0 : n;
#pragma unroll
        for (int i = 0; i < GRAIN / ROWS; ++i) {
          const int r = j * GRAIN + i * ROWS + r0;
          const uint32_t bytes = r < live ? 16 : 0;
          cp_async16_zfill(stage + at(r, c), kg + src, bytes);
          cp_async16_zfill(stage + TT * HD * 2 + at(r, c), vg + src, bytes);
          src += step;
        }
      }
    }
  }

  // Queries in shared memory: [CH][HD], 16-byte chunks swizzled by the head.
  static constexpr int Q_CHUNKS = CH * HD / 8, Q_PER_THREAD = (Q_CHUNKS + W * 32 - 1) / (W * 32);

  __device__ __forceinline__ void fetch(const AttnDesc& p, int seq, int head0, int heads) {
    const T* src = static_cast<const T*>(p.q.data) + seq * p.q.row_stride + head0 * p.q.head_stride;
#pragma unroll
    for (int i = 0; i < Q_PER_THREAD; ++i) {
      const int e = i * W * 32 + threadIdx.x, h = e / (HD / 8), c = e % (HD / 8);
      next_q[i] = make_uint4(0, 0, 0, 0);
      if (h < heads && c * 8 < p.cache.head_dim)
        next_q[i] = *reinterpret_cast<const uint4*>(src + h * p.q.head_stride + c * 8);
    }
  }

  __device__ __forceinline__ void pass_on() const {
#pragma unroll
    for (int i = 0; i < Q_PER_THREAD; ++i) {
      const int e = i * W * 32 + threadIdx.x, h = e / (HD / 8), c = e % (HD / 8);
      if (Q_CHUNKS % (W * 32) == 0 || e < Q_CHUNKS) *reinterpret_cast<uint4*>(q_shared + at(h, c)) = next_q[i];
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][n][e] = 0.f;
      m[n][0] = m[n][1] = kNegInf;
      l[n][0] = l[n][1] = 0.f;
    }
  }

  __device__ __forceinline__ void begin_solo(const AttnDesc& p, int seq, int head0, int heads) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const T* src = static_cast<const T*>(p.q.data) + seq * p.q.row_stride + head0 * p.q.head_stride;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = n * 8 + g, d = k * 16 + e * 8 + t * 2;
          q[k][n][e] = h < heads && d < p.cache.head_dim
                           ? *reinterpret_cast<const uint32_t*>(src + h * p.q.head_stride + d)
                           : 0u;
        }
    clear();
  }

  __device__ __forceinline__ void begin(const AttnDesc&, int) {
    const int lane = threadIdx.x & 31;
    // Two k steps of 8 heads per load: blocks (chunk 2 k, 2 k + 1, 2 k + 2, 2 k + 3).
    const uint32_t qb = smem_addr(q_shared);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < KT; k += 2)
        ldsm_x4(qb + at(n * 8 + (lane & 7), 2 * k + (lane >> 3)), q[k][n][0], q[k][n][1], q[k + 1][n][0],
                q[k + 1][n][1]);
    clear();
  }

  __device__ __forceinline__ void tile(const AttnDesc& p, const uint8_t* stage, int n_tokens) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const uint32_t kb = smem_addr(stage), vb = kb + TT * HD * 2;
    // Scores: a block's products in two chains (one where there are two
    // blocks), summed below.
    constexpr int CHAINS = BLOCKS == 1 ? 2 : 1;
    float s[BLOCKS][NT][CHAINS][4] = {};
#pragma unroll
    for (int k = 0; k < KT; ++k) {
#pragma unroll
      for (int j = 0; j < BLOCKS; ++j) {
        uint32_t a[4];
        ldsm_x4(kb + at(j * 16 + (lane & 15), 2 * k + (lane >> 4)), a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_bf16_16816(s[j][n][k % CHAINS], a, q[k][n][0], q[k][n][1]);
      }
    }
    uint32_t pt[BLOCKS][NT][2][3];  // P's terms
    float2 kept[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[BLOCKS][4], keep[2];
#pragma unroll
      for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[j][e] = (CHAINS == 2 ? s[j][n][0][e] + s[j][n][CHAINS - 1][e] : s[j][n][0][e]) * scale;
          if (j * 16 + g + (e < 2 ? 0 : 8) >= n_tokens) x[j][e] = kNegInf;
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = fmaxf(x[0][e], x[0][e + 2]);
        if (BLOCKS == 2) top = fmaxf(top, fmaxf(x[BLOCKS - 1][e], x[BLOCKS - 1][e + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float now = fmaxf(m[n][e], top);
        const float base = now == kNegInf ? 0.f : now;  // nothing but -inf so far: every weight is 0
        keep[e] = pow2(m[n][e] - base);
        m[n][e] = now;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j) {
          x[j][e] = pow2(x[j][e] - base);
          x[j][e + 2] = pow2(x[j][e + 2] - base);
          sum += x[j][e] + x[j][e + 2];
        }
        l[n][e] = fmaf(l[n][e], keep[e], sum);  // this lane's tokens; summed over lanes in put
      }
#pragma unroll
      for (int j = 0; j < BLOCKS; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          split3_bf16x2(x[j][2 * e], x[j][2 * e + 1], pt[j][n][e]);
#pragma unroll
          for (int i = 0; i < 3; ++i) pt[j][n][e][i] = transpose_8x8(pt[j][n][e][i]);
        }
      }
      kept[n] = make_float2(keep[0], keep[1]);
    }
    // The instruction cuts what it adds to an accumulator off instead of
    // rounding it, so a tile's products are summed apart and join O rounded.
    constexpr int KG = NT == 1 && KT >= 4 ? 4 : 2;  // steps of the head at a time
#pragma unroll
    for (int k0 = 0; k0 < KT; k0 += KG) {
      float now[KG][NT][4] = {};
#pragma unroll
      for (int j = 0; j < BLOCKS; ++j) {
        uint32_t a[KG][4];
#pragma unroll
        for (int k = 0; k < KG; ++k)
          ldsm_x4_trans(vb + at(j * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * (k0 + k) + ((lane >> 3) & 1)), a[k][0],
                        a[k][1], a[k][2], a[k][3]);
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int k = 0; k < KG; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_bf16_16816(now[k][n], a[k], pt[j][n][0][i], pt[j][n][1][i]);
      }
#pragma unroll
      for (int k = 0; k < KG; ++k)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 sum = fma_f32x2(make_float2(o[k0 + k][n][e], o[k0 + k][n][e + 1]), kept[n],
                                         make_float2(now[k][n][e], now[k][n][e + 1]));
            o[k0 + k][n][e] = sum.x;
            o[k0 + k][n][e + 1] = sum.y;
          }
    }
  }

  __device__ __forceinline__ void put(int part, float* comb, float2* stat) const {
    static_assert(NT <= 2, "");
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool upper = NT > 1 && (part >> 1) != 0;  // picked by selection: the registers stay registers
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = upper ? l[NT - 1][e] : l[0][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (t >> 1 != (part & 1)) continue;  // this lane's heads are in the other half
      const int h = 2 * (t & 1) + e;
      if (g == 0) stat[h] = make_float2(upper ? m[NT - 1][e] : m[0][e], sum);
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        comb[h * (HD + 4) + k * 16 + g] = upper ? o[k][NT - 1][e] : o[k][0][e];
        comb[h * (HD + 4) + k * 16 + g + 8] = upper ? o[k][NT - 1][e + 2] : o[k][0][e + 2];
      }
    }
  }
};

}  // namespace

// Pages hold whole grains of 8 tokens; rows and queries are on 16-byte
// boundaries.
bool mma_attention_ok(const AttnDesc& p) {
  const CacheDesc& c = p.cache;
  const auto low = reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) |
                   reinterpret_cast<uintptr_t>(p.q.data);
  return p.dtype == LORA_DTYPE_BF16 && c.page_size % 8 == 0 && (low & 15) == 0 && c.head_dim % 8 == 0 &&
         c.page_stride % 8 == 0 && c.token_stride % 8 == 0 && c.head_stride % 8 == 0 && p.q.row_stride % 8 == 0 &&
         p.q.head_stride % 8 == 0;
}

// f(a core's type) for the head width, group and page size of p.
template <int GRAIN, class F>
auto with_grain(const AttnDesc& p, F f) {
  const int hd = p.cache.head_dim;
  if (p.group <= 8) {
    if (hd <= 32) return f((MmaCore<32, 1, GRAIN>*)nullptr);
    if (hd <= 64) return f((MmaCore<64, 1, GRAIN>*)nullptr);
    if (hd <= 128) return f((MmaCore<128, 1, GRAIN>*)nullptr);
    return f((MmaCore<256, 1, GRAIN>*)nullptr);
  }
  if (hd <= 32) return f((MmaCore<32, 2, GRAIN>*)nullptr);
  if (hd <= 64) return f((MmaCore<64, 2, GRAIN>*)nullptr);
  if (hd <= 128) return f((MmaCore<128, 2, GRAIN>*)nullptr);
  return f((MmaCore<256, 2, GRAIN>*)nullptr);
}
// Grains of 16 where pages hold them, else of 8: fewer table look-ups and
// offsets a tile (24 contexts of 4000 to 16000 tokens, 256 wide, 16 heads a
// group 233 us against 243 by grains of 8; 256 ragged ones 64 wide 119.5 and
// 121.3; 24 long ones 128 wide 303.4 and 305.1).
template <class F>
auto with_core(const AttnDesc& p, F f) {
  return p.cache.page_size % 16 == 0 ? with_grain<16>(p, f) : with_grain<8>(p, f);
}

CoreShape mma_attention_shape(const AttnDesc& p) {
  return with_core(p, [](auto* core) { return shape_of<std::remove_pointer_t<decltype(core)>>(); });
}

cudaError_t launch_attention_mma(const AttnDesc& p, void* workspace, cudaStream_t s) {
  return with_core(p, [&](auto* core) {
    return launch_core<std::remove_pointer_t<decltype(core)>>(p, workspace, s, LORA_PATH_MMA_ATTENTION);
  });
}

// The workspace is sized for either core, so that it depends on shapes only
// and not on which one the alignments allow.
size_t attention_workspace_bytes(const AttnDesc& p) {
  size_t bytes = generic_attention_workspace(p);
  if (p.dtype == LORA_DTYPE_BF16) bytes = std::max(bytes, workspace_bytes_of(mma_attention_shape(p), p));
  return bytes;
}

cudaError_t launch_attention(const AttnDesc& p, void* workspace, cudaStream_t s) {
  return mma_attention_ok(p) ? launch_attention_mma(p, workspace, s) : launch_attention_generic(p, workspace, s);
}

}  // namespace lora
