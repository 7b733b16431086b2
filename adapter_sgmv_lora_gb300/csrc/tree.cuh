// tree.cuh -- the frame of tree attention: how drafted tokens and cached ones
// are shared out over the GPU, and how parts are put together again.
//
// Work.  The rows of a stream are (drafted token, query head of the group)
// pairs of one sequence and one key/value head, taken MR at a time (a chunk),
// so all of them share every key and value that is loaded; heads wider than a
// kernel's value part are `parts` streams, one for each part of V.  A stream
// is the ceil(len / TT) tiles of TT cached tokens.  The tiles of all streams,
// stream after stream, form one line, in which a stream also takes COST places
// for its fixed cost; the line is cut into equal pieces, one per CTA, from the
// lengths and row offsets alone.  A piece that holds a whole stream writes the
// result; else it leaves a partial result (running maximum m, sum l,
// unnormalised output O) in the workspace and join_kernel sums the parts in
// the order of the line.  All of it is deterministic.
#pragma once

#include <algorithm>
#include <atomic>
#include <climits>
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace lora {

constexpr float kTreeLog2e = 1.4426950408889634f;
constexpr float kTreeLn2 = 0.6931471805599453f;
constexpr float kTreeNone = -__builtin_huge_valf();

// 2^x, below 2^-126 zero.
__device__ __forceinline__ float tree_pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tree_put4(float* dst, float4 v, int n) {
  if (n >= 4 && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
    *reinterpret_cast<float4*>(dst) = v;
    return;
  }
  const float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) dst[e] = r[e];
}
__device__ __forceinline__ void tree_put4(__nv_bfloat16* dst, float4 v, int n) {
  if (n >= 4 && (reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(round_pack_bf16x2(v.x, v.y), round_pack_bf16x2(v.z, v.w));
    return;
  }
  const float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) dst[e] = __float2bfloat16_rn(r[e]);
}

// Rows of a chunk, tokens of a tile, columns of a value part, places of a
// stream's fixed cost.
template <int MR_, int TT_, int HV_, int COST_>
struct TreeShape {
  static constexpr int MR = MR_, TT = TT_, HV = HV_, COST = COST_;
};

// One sequence.
struct TreeSeq {
  int row0, n, len, ctx;  // first row of q, drafted tokens, cached tokens, tokens before the drafted ones
  int chunks, tiles;      // 0 tiles: nothing to do (no rows, or refused)
  bool bad;               // LORA_DEV_BAD_LENGTH
};

template <class S>
__device__ __forceinline__ TreeSeq tree_seq(const TreeDesc& p, int b) {
  TreeSeq s;
  s.row0 = p.offsets[b];
  s.n = p.offsets[b + 1] - s.row0;
  s.len = p.lengths[b];
  s.ctx = s.len - s.n;
  s.bad = s.n > 0 && (s.len < s.n || s.len > p.max_len || (p.masks && s.n > 64 * p.words));
  const bool live = s.n > 0 && !s.bad;
  s.chunks = live ? (int)(((long long)s.n * p.group + S::MR - 1) / S::MR) : 0;
  s.tiles = live ? (s.len - 1) / S::TT + 1 : 0;
  return s;
}

template <class S>
__device__ __forceinline__ long long tree_places(const TreeDesc& p, const TreeSeq& s) {
  return s.tiles == 0 ? 0 : (long long)p.cache.num_kv_heads * p.parts * s.chunks * (s.tiles + S::COST);
}

// Piece u of the line: [lo, hi), its first sequence and the place where that
// sequence's streams begin; the line's length.  Empty where nothing is computed.
struct TreePiece {
  long long lo, hi, origin, total;
  int seq;
};

__device__ __forceinline__ long long tree_start(long long total, int pieces, int u) {
  const long long base = total / pieces, rest = total - base * pieces;
  return u * base + min((long long)u, rest);
}

// Executed by one full warp; every lane gets the result.  Checks the row
// offsets; with `report` it records what is wrong.
template <class S>
__device__ __forceinline__ TreePiece tree_piece(const TreeDesc& p, int u, bool report) {
  const int lane = threadIdx.x & 31;
  long long total = 0;
  unsigned flags = 0;
  for (int b = lane; b < p.num_seqs; b += 32) {
    const int o0 = p.offsets[b], o1 = p.offsets[b + 1];
    if (o0 < 0 || o1 < o0 || o1 > p.num_rows) {
      flags |= LORA_DEV_BAD_OFFSETS;
      continue;
    }
    const TreeSeq s = tree_seq<S>(p, b);
    if (s.bad) flags |= LORA_DEV_BAD_LENGTH;
    total += tree_places<S>(p, s);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (report && flags && lane == 0)
    atomicOr(p.status, (flags & LORA_DEV_BAD_OFFSETS) ? LORA_DEV_BAD_OFFSETS : flags);
  TreePiece r;
  r.lo = r.hi = r.origin = 0;
  r.total = total;
  r.seq = 0;
  if ((flags & LORA_DEV_BAD_OFFSETS) || total == 0) return r;
  r.lo = tree_start(total, p.pieces, u);
  r.hi = tree_start(total, p.pieces, u + 1);
  if (r.lo >= r.hi) return r;
  long long before = 0;
  for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
    const int b = b0 + lane;
    const long long mine = b < p.num_seqs ? tree_places<S>(p, tree_seq<S>(p, b)) : 0;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    const long long first = before + incl - mine;
    const unsigned who = __ballot_sync(0xffffffffu, r.lo >= first && r.lo < first + mine);
    if (who) {
      const int src = __ffs(who) - 1;
      r.seq = b0 + src;
      r.origin = __shfl_sync(0xffffffffu, first, src);
      return r;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

// Walks the segments of a piece: tiles [t0, t1) of stream `stream` of sequence
// `seq`.  The line goes on behind a sequence's last stream with the next
// sequence that has tiles.
template <class S>
struct TreeSegment {
  TreeSeq s;
  long long at, hi;  // place where the stream begins; end of the piece
  int seq, stream, t0, t1;
  bool valid;

  __device__ __forceinline__ void clip(long long lo) {
    const long long tile0 = at + S::COST;
    t0 = lo > tile0 ? (int)min(lo - tile0, (long long)s.tiles) : 0;
    t1 = hi > tile0 ? (int)min(hi - tile0, (long long)s.tiles) : 0;
  }
  __device__ __forceinline__ void step(const TreeDesc& p) {
    at += s.tiles + S::COST;
    if (++stream == p.cache.num_kv_heads * p.parts * s.chunks) {
      stream = 0;
      do {
        if (++seq >= p.num_seqs) {
          valid = false;
          return;
        }
        s = tree_seq<S>(p, seq);
      } while (s.tiles == 0);
    }
  }
  __device__ __forceinline__ void first(const TreeDesc& p, const TreePiece& r) {
    valid = r.lo < r.hi;
    if (!valid) return;
    hi = r.hi;
    seq = r.seq;
    s = tree_seq<S>(p, seq);
    const long long in = r.lo - r.origin;
    stream = (int)(in / (s.tiles + S::COST));
    at = r.origin + (long long)stream * (s.tiles + S::COST);
    clip(r.lo);
    while (valid && t1 <= t0) {
      step(p);
      if (valid && at < hi) clip(r.lo);
      else valid = false;
    }
  }
  __device__ __forceinline__ void next(const TreeDesc& p) {
    step(p);
    if (!valid) return;
    if (at + S::COST >= hi) {
      valid = false;
      return;
    }
    clip(at);
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == s.tiles; }
  // What the stream is.
  __device__ __forceinline__ int chunk() const { return stream % s.chunks; }
  __device__ __forceinline__ int part(const TreeDesc& p) const { return stream / s.chunks % p.parts; }
  __device__ __forceinline__ int kv_head(const TreeDesc& p) const { return stream / s.chunks / p.parts; }
};

// The partial result of a segment that is not whole.
template <class S>
__device__ __forceinline__ long long tree_slot(const TreeSegment<S>& g, int u) {
  return 2LL * u + (g.t0 == 0 ? 1 : 0);
}

// Pieces that share the stream which piece u begins with segment g.
template <class S>
__device__ __forceinline__ int tree_sharers(const TreeDesc& p, const TreePiece& piece, const TreeSegment<S>& g, int u) {
  const long long end = g.at + S::COST + g.s.tiles;
  const long long base = piece.total / p.pieces, rest = piece.total - base * p.pieces, wide = rest * (base + 1);
  // The first piece that starts at or behind the stream's end.
  const long long next = end <= wide ? (end + base) / (base + 1) : rest + (end - wide + base - 1) / base;
  return (int)(next - u);
}

// Whether a row sees token 32 c + i of the drafted ones: bit i.  d0 = 32 c may
// be below 0 (the context, which every row sees); tokens from n on are none.
__device__ __forceinline__ unsigned tree_sees(const TreeDesc& p, const unsigned long long* mask, int i, int d0, int n) {
  if (d0 + 32 <= 0) return 0xffffffffu;
  if (d0 >= n) return 0u;
  unsigned bits;
  if (!mask) {
    const int upto = i + 1 - d0;  // tokens 0..i
    bits = upto >= 32 ? 0xffffffffu : upto <= 0 ? 0u : (1u << upto) - 1u;
  } else if (d0 < 0) {
    bits = (unsigned)(mask[0] << -d0) | ((1u << -d0) - 1u);
  } else {
    const int w = d0 >> 6, off = d0 & 63;
    unsigned long long v = mask[w] >> off;
    if (off > 32 && w + 1 < p.words) v |= mask[w + 1] << (64 - off);
    bits = (unsigned)v;
  }
  const int left = n - d0;  // > 0
  return left >= 32 ? bits : bits & ((1u << left) - 1u);
}

// Joins the partial results of the stream that piece u begins and others go on
// with: part 0 is slot 2 u + 1, part i the beginning of piece u + i.  A thread
// has four columns of a row; a sum below 0 marks a page outside the cache.
// The partial outputs lie column group by column group, rows side by side.
template <class S, typename T>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ TreeDesc p) {
  pdl_wait();
  const int u = blockIdx.x;
  const int4 split = p.splits[u];  // sequence, stream, parts
  if (split.z == 0) return;
  const TreeSeq s = tree_seq<S>(p, split.x);
  const int chunk = split.y % s.chunks, part = split.y / s.chunks % p.parts, kv = split.y / s.chunks / p.parts;
  const int rows = (int)min((long long)S::MR, (long long)s.n * p.group - (long long)chunk * S::MR);
  for (int e = blockIdx.y * 256 + threadIdx.x; e < S::MR * (S::HV / 4); e += gridDim.y * 256) {
    const int r = e % S::MR, c4 = e / S::MR;
    if (r >= rows || part * S::HV + 4 * c4 >= p.cache.head_dim) continue;
    float m = kTreeNone;
    bool bad = false;
    for (int i = 0; i < split.z; ++i) {
      const float2 st = p.stats[(2LL * (u + i) + (i == 0)) * S::MR + r];
      m = fmaxf(m, st.x);
      bad |= st.y < 0.f;
    }
    if (bad) {
      if (c4 == 0) atomicOr(p.status, LORA_DEV_BAD_PAGE);
      continue;
    }
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < split.z; ++i) {
      const long long slot = 2LL * (u + i) + (i == 0);
      const float2 st = p.stats[slot * S::MR + r];
      const float f = st.x == kTreeNone ? 0.f : tree_pow2(st.x - m);
      const float4 v = reinterpret_cast<const float4*>(p.partial)[(slot * (S::HV / 4) + c4) * S::MR + r];
      l = fmaf(st.y, f, l);
      if (st.x == kTreeNone) continue;  // nothing seen: its output is zero
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    const long long row = (long long)chunk * S::MR + r;
    const int i = (int)(row / p.group), head = kv * p.group + (int)(row % p.group);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int d = part * S::HV + 4 * c4;
    T* out = static_cast<T*>(p.out.data) + (s.row0 + i) * p.out.row_stride + head * p.out.head_stride + d;
    tree_put4(out, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), p.cache.head_dim - d);
    if (d == 0 && p.lse) p.lse[(long long)(s.row0 + i) * p.num_heads + head] = (m + log2f(l)) * kTreeLn2;
  }
}

// ------------------------------------------------------------------- host --

struct TreeSizes {
  int MR, TT, HV, COST;
};
template <class S>
constexpr TreeSizes tree_sizes() {
  return {S::MR, S::TT, S::HV, S::COST};
}

// Pieces: one per resident CTA, or fewer where even the longest sequences
// would not give each a tile.
inline int tree_pieces(const TreeSizes& z, const TreeDesc& p, int most) {
  const int parts = (p.cache.head_dim + z.HV - 1) / z.HV;
  const long long chunks = std::min<long long>((long long)p.num_rows * p.group / z.MR + p.num_seqs, INT_MAX);
  const long long streams = std::min<long long>(chunks * ((long long)p.cache.num_kv_heads * parts), INT_MAX);
  const long long tiles = std::max(1, p.max_len / z.TT + (p.max_len % z.TT != 0));
  return (int)std::max(1LL, std::min<long long>(most, streams * tiles));
}

inline size_t tree_round(size_t n) { return (n + 255) & ~(size_t)255; }
inline size_t tree_stats_at(int pieces) { return tree_round((size_t)pieces * sizeof(int4)); }
inline size_t tree_partial_at(const TreeSizes& z, int pieces) {
  return tree_stats_at(pieces) + tree_round((size_t)2 * pieces * z.MR * sizeof(float2));
}
inline size_t tree_bytes(const TreeSizes& z, int pieces) {
  return tree_partial_at(z, pieces) + tree_round((size_t)2 * pieces * z.MR * z.HV * sizeof(float));
}

// Fills in what the kernels find in p beyond the call itself.
inline void tree_fill(const TreeSizes& z, TreeDesc& p, int most, void* workspace) {
  p.parts = (p.cache.head_dim + z.HV - 1) / z.HV;
  p.pieces = tree_pieces(z, p, most);
  int log = 0;  // page_size <= 2^log: ceil(2^(31 + log) / page_size) is below 2^32 and exact for tokens below 2^31
  while ((1LL << log) < p.cache.page_size) ++log;
  p.page_shift = 31 + log;
  p.page_magic = (unsigned)(((1ULL << p.page_shift) + p.cache.page_size - 1) / p.cache.page_size);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.splits = reinterpret_cast<int4*>(ws);
  p.stats = reinterpret_cast<float2*>(ws + tree_stats_at(p.pieces));
  p.partial = reinterpret_cast<float*>(ws + tree_partial_at(z, p.pieces));
}

template <class S, typename T>
cudaError_t launch_tree_join(const TreeDesc& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.pieces, std::max(1, S::MR * S::HV / 4 / 512));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return noted(cudaLaunchKernelEx(&cfg, tree_join_kernel<S, T>, p), LORA_PATH_JOIN);
}

// Raises a kernel's shared-memory limit, once per device.
template <class Kernel>
cudaError_t tree_allow_smem(Kernel kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// tree_tc.cu: bf16 on tcgen05.  tree_generic.cu: fp32 arithmetic, any type,
// size and alignment.
bool tree_tc_ok(const TreeDesc& p);
size_t tree_tc_workspace(const TreeDesc& p);
cudaError_t launch_tree_tc(TreeDesc p, void* workspace, cudaStream_t s);
size_t tree_generic_workspace(const TreeDesc& p);
cudaError_t launch_tree_generic(TreeDesc p, void* workspace, cudaStream_t s);

}  // namespace lora
