// tree_generic.cu -- tree attention in fp32 arithmetic on the CUDA cores: fp32
// caches, and bf16 ones whose shapes or alignments tree_tc.cu does not take.
// The frame is tree.cuh.
//
// A CTA works on a chunk of 32 rows, 8 to a warp, over tiles of 32 tokens in
// shared memory.  In the scores a lane is a token (4 columns of its key against
// 8 broadcast queries: 32 products for 9 loads), the running maximum and sum of
// a row are warp reductions; in the output a lane has HD / 32 columns of 8 rows.
// Several CTAs share an SM, so one's loads run under another's arithmetic.
// Where sequences are short it is bound by waiting, for loads and at barriers (issue
// slots 27% taken, DRAM 4%), and by the join of a stream's many parts: 19 ragged
// trees in fp32 (12 over 4 heads, 80 wide, 1 to 901 tokens) 61 us.
#include "tree.cuh"

namespace lora {
namespace {

constexpr int kGenThreads = 128;
constexpr int kGenRows = 8;  // a warp

template <int HD>
struct GenCfg {
  using S = TreeShape<32, 32, HD, 2>;
  static constexpr int KP = HD + 4;  // pitch of a key: lanes fall on different banks
  static constexpr int PP = S::MR + 4;
  static constexpr int SMEM = (S::TT * KP + S::TT * HD + S::MR * HD + S::TT * PP) * 4;
  static constexpr int CTAS = HD <= 128 ? 4 : 2;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Columns c .. c + 3 of a row of hd columns; zero from hd on.
template <bool VEC, typename T>
__device__ __forceinline__ float4 columns(const T* row, int c, int hd) {
  if constexpr (VEC) {
    return c < hd ? load4(row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = c + e < hd ? load1(row + c + e) : 0.f;
    return make_float4(v[0], v[1], v[2], v[3]);
  }
}

template <int HD, typename T, bool VEC>
__global__ void __launch_bounds__(kGenThreads, GenCfg<HD>::CTAS) tree_generic_kernel(const __grid_constant__ TreeDesc p) {
  using C = GenCfg<HD>;
  using S = typename C::S;
  constexpr int MR = S::MR, TT = S::TT, VPL = HD / 32;
  extern __shared__ __align__(16) float smem[];
  float* sk = smem;                // [TT][KP]
  float* sv = sk + TT * C::KP;     // [TT][HD]
  float* sq = sv + TT * HD;        // [MR][HD]
  float* sp = sq + MR * HD;        // [TT][PP]
  __shared__ long long s_off[2][TT];
  __shared__ TreePiece s_piece;
  __shared__ int s_bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = blockIdx.x;
  const int hd = p.cache.head_dim;
  pdl_launch_dependents();
  if (warp == 0) {
    const TreePiece piece = tree_piece<S>(p, u, u == 0);
    if (lane == 0) {
      s_piece = piece;
      s_bad = 0;
    }
  }
  __syncthreads();
  TreeSegment<S> g;
  g.first(p, s_piece);
  int4 split = make_int4(0, 0, 0, 0);
  const float scale = p.scale * kTreeLog2e;
  // This lane's column e: neighbouring ones in fours (twos for the narrowest heads).
  auto column = [lane](int e) { return (e >> 2) * 128 + (VPL < 4 ? lane * VPL : lane * 4) + (e & 3); };
  while (g.valid) {
    const int kv = g.kv_head(p), row0 = g.chunk() * MR;
    const int rows = (int)min((long long)MR, (long long)g.s.n * p.group - row0);
    for (int e = threadIdx.x; e < MR * (HD / 4); e += kGenThreads) {
      const int r = e / (HD / 4), c = e % (HD / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int i = (row0 + r) / p.group, h = kv * p.group + (row0 + r) % p.group;
        v = columns<VEC>(static_cast<const T*>(p.q.data) + (g.s.row0 + i) * p.q.row_stride + h * p.q.head_stride, c, hd);
      }
      *reinterpret_cast<float4*>(sq + r * HD + c) = v;
    }
    // Where the tokens of a tile are; -1: no token, or its page is not one of
    // the cache's.
    auto locate = [&](int t) {
      if (threadIdx.x < TT) {
        const int j = t * TT + threadIdx.x;
        long long off = -1;
        if (j < g.s.len) {
          const int i = (int)(((unsigned long long)(unsigned)j * p.page_magic) >> p.page_shift);
          const int page = p.tables[g.seq * p.table_stride + i];
          if ((unsigned)page < (unsigned)p.cache.num_pages)
            off = page * p.cache.page_stride + (j - i * p.cache.page_size) * p.cache.token_stride +
                  kv * p.cache.head_stride;
          else s_bad = 1;
        }
        s_off[t & 1][threadIdx.x] = off;
      }
    };
    float m[kGenRows], l[kGenRows], o[kGenRows][VPL];
    int draft[kGenRows];  // the drafted token that each of the warp's rows is
#pragma unroll
    for (int r = 0; r < kGenRows; ++r) {
      m[r] = kTreeNone;
      l[r] = 0.f;
      draft[r] = (int)min((long long)g.s.n - 1, (row0 + (long long)warp * kGenRows + r) / p.group);
#pragma unroll
      for (int e = 0; e < VPL; ++e) o[r][e] = 0.f;
    }
    locate(g.t0);
    __syncthreads();
    for (int t = g.t0; t < g.t1; ++t) {
      for (int e = threadIdx.x; e < TT * (HD / 4); e += kGenThreads) {
        const int r = e / (HD / 4), c = e % (HD / 4) * 4;
        const long long off = s_off[t & 1][r];
        float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
        if (off >= 0) {
          kk = columns<VEC>(static_cast<const T*>(p.cache.k) + off, c, hd);
          vv = columns<VEC>(static_cast<const T*>(p.cache.v) + off, c, hd);
        }
        *reinterpret_cast<float4*>(sk + r * C::KP + c) = kk;
        *reinterpret_cast<float4*>(sv + r * HD + c) = vv;
      }
      if (t + 1 < g.t1) locate(t + 1);
      __syncthreads();
      if (warp * kGenRows < rows) {
        float s[kGenRows] = {};
#pragma unroll 4
        for (int c = 0; c < HD; c += 4) {
          const float4 kk = *reinterpret_cast<const float4*>(sk + lane * C::KP + c);
#pragma unroll
          for (int r = 0; r < kGenRows; ++r) {
            const float4 qq = *reinterpret_cast<const float4*>(sq + (warp * kGenRows + r) * HD + c);
            s[r] = fmaf(qq.x, kk.x, s[r]);
            s[r] = fmaf(qq.y, kk.y, s[r]);
            s[r] = fmaf(qq.z, kk.z, s[r]);
            s[r] = fmaf(qq.w, kk.w, s[r]);
          }
        }
        const int d0 = t * TT - g.s.ctx;  // the tile's first token among the drafted ones
        const bool drafts = d0 + TT > 0;
#pragma unroll
        for (int r = 0; r < kGenRows; ++r) {
          float x = s[r] * scale;
          if (drafts) {
            const unsigned sees = tree_sees(
                p, p.masks ? p.masks + (long long)(g.s.row0 + draft[r]) * p.words : nullptr, draft[r], d0, g.s.n);
            if (!(sees >> lane & 1)) x = kTreeNone;
          }
          float top = x;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          const float now = fmaxf(m[r], top), base = now == kTreeNone ? 0.f : now;
          const float keep = tree_pow2(m[r] - base), w = tree_pow2(x - base);
          m[r] = now;
          float sum = w;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          l[r] = fmaf(l[r], keep, sum);
#pragma unroll
          for (int e = 0; e < VPL; ++e) o[r][e] *= keep;
          sp[lane * C::PP + warp * kGenRows + r] = w;
        }
        __syncwarp();
        const int tokens = min(TT, g.s.len - t * TT);
        // A weight of 0 among drafted tokens may stand for one that the row
        // does not see: its value has no part, be it infinite or NaN.
        auto add = [&](auto guarded) {
#pragma unroll 2
          for (int j = 0; j < tokens; ++j) {
            const float4 a = *reinterpret_cast<const float4*>(sp + j * C::PP + warp * kGenRows);
            const float4 b = *reinterpret_cast<const float4*>(sp + j * C::PP + warp * kGenRows + 4);
            const float w[kGenRows] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            float v[VPL];
#pragma unroll
            for (int e = 0; e < VPL; e += 2) {
              const float2 two = *reinterpret_cast<const float2*>(sv + j * HD + column(e));
              v[e] = two.x;
              v[e + 1] = two.y;
            }
#pragma unroll
            for (int r = 0; r < kGenRows; ++r)
#pragma unroll
              for (int e = 0; e < VPL; ++e)
                if (!decltype(guarded)::value || w[r] != 0.f) o[r][e] = fmaf(w[r], v[e], o[r][e]);
          }
        };
        if (drafts) add(std::true_type{});
        else add(std::false_type{});
      }
      __syncthreads();
    }
    const bool bad = s_bad != 0, whole = g.whole();
    const long long slot = tree_slot<S>(g, u);
    if (warp * kGenRows < rows) {
#pragma unroll
      for (int r = 0; r < kGenRows; ++r) {
        const int row = warp * kGenRows + r;
        if (row >= rows) break;
        const int i = (row0 + row) / p.group, h = kv * p.group + (row0 + row) % p.group;
        T* out = static_cast<T*>(p.out.data) + (g.s.row0 + i) * p.out.row_stride + h * p.out.head_stride;
        const bool none = l[r] == 0.f;  // nothing seen, or -inf alone: 0, whatever the values
        const float inv = 1.f / l[r];
#pragma unroll
        for (int e = 0; e < VPL; ++e) {
          const int d = column(e);
          if (!whole) p.partial[((slot * (HD / 4) + d / 4) * MR + row) * 4 + d % 4] = o[r][e];
          else if (!bad && d < hd) out[d] = [](float v) {
            if constexpr (sizeof(T) == 4) return v;
            else return __float2bfloat16_rn(v);
          }(none ? 0.f : o[r][e] * inv);
        }
        if (lane == 0) {
          if (!whole) p.stats[slot * MR + row] = make_float2(m[r], bad ? -1.f : l[r]);
          else if (bad) atomicOr(p.status, LORA_DEV_BAD_PAGE);
          else if (p.lse) p.lse[(long long)(g.s.row0 + i) * p.num_heads + h] = (m[r] + log2f(l[r])) * kTreeLn2;
        }
      }
    }
    if (g.t0 == 0 && !whole) split = make_int4(g.seq, g.stream, tree_sharers<S>(p, s_piece, g, u), 0);
    __syncthreads();
    if (threadIdx.x == 0) s_bad = 0;
    g.next(p);
    __syncthreads();
  }
  if (threadIdx.x == 0) p.splits[u] = split;
}

template <int HD, typename T, bool VEC>
cudaError_t launch_gen(TreeDesc p, void* workspace, cudaStream_t s) {
  using C = GenCfg<HD>;
  static std::atomic<unsigned long long> done{0};
  tree_fill(tree_sizes<typename C::S>(), p, C::CTAS * std::min(std::max(device_sm_count(), 1), kMaxSmsForWorkspace),
            workspace);
  cudaError_t e = tree_allow_smem(tree_generic_kernel<HD, T, VEC>, C::SMEM, done);
  if (e != cudaSuccess) return e;
  tree_generic_kernel<HD, T, VEC><<<p.pieces, kGenThreads, C::SMEM, s>>>(p);
  if ((e = noted(cudaGetLastError(), LORA_PATH_GENERIC_TREE)) != cudaSuccess) return e;
  return launch_tree_join<typename C::S, T>(p, s);
}

template <int HD>
cudaError_t launch_gen_type(const TreeDesc& p, bool vec, void* workspace, cudaStream_t s) {
  if (p.dtype == LORA_DTYPE_F32)
    return vec ? launch_gen<HD, float, true>(p, workspace, s) : launch_gen<HD, float, false>(p, workspace, s);
  return vec ? launch_gen<HD, __nv_bfloat16, true>(p, workspace, s)
             : launch_gen<HD, __nv_bfloat16, false>(p, workspace, s);
}

}  // namespace

size_t tree_generic_workspace(const TreeDesc& p) {
  auto bytes = [&](auto cfg) {
    using C = decltype(cfg);
    const TreeSizes z = tree_sizes<typename C::S>();
    return tree_bytes(z, tree_pieces(z, p, C::CTAS * kMaxSmsForWorkspace));
  };
  const int hd = p.cache.head_dim;
  return hd <= 64 ? bytes(GenCfg<64>{}) : hd <= 128 ? bytes(GenCfg<128>{}) : bytes(GenCfg<256>{});
}

cudaError_t launch_tree_generic(TreeDesc p, void* workspace, cudaStream_t s) {
  // Four columns at a time where every row starts on such a boundary.
  const CacheDesc& c = p.cache;
  const int es = p.dtype == LORA_DTYPE_F32 ? 4 : 2;
  const auto low = reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) |
                   reinterpret_cast<uintptr_t>(p.q.data);
  const bool vec = low % (4 * es) == 0 && (c.head_dim | c.page_stride | c.token_stride | c.head_stride |
                                           p.q.row_stride | p.q.head_stride) % 4 == 0;
  if (c.head_dim <= 64) return launch_gen_type<64>(p, vec, workspace, s);
  if (c.head_dim <= 128) return launch_gen_type<128>(p, vec, workspace, s);
  return launch_gen_type<256>(p, vec, workspace, s);
}

// The workspace is sized for either kernel, so that it depends on shapes only
// and not on which one the alignments allow.
size_t tree_workspace_bytes(const TreeDesc& p) {
  const size_t bytes = tree_generic_workspace(p);
  return p.dtype == LORA_DTYPE_BF16 ? std::max(bytes, tree_tc_workspace(p)) : bytes;
}

cudaError_t launch_tree(const TreeDesc& p, void* workspace, cudaStream_t s) {
  return tree_tc_ok(p) ? launch_tree_tc(p, workspace, s) : launch_tree_generic(p, workspace, s);
}

}  // namespace lora
