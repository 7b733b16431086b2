// attention.cuh -- the frame of paged decode attention: how the cached tokens
// are shared out over the GPU and how the parts are put together again.  The
// arithmetic of one tile of tokens is a "core" (attention_generic.cu: fp32 on
// the CUDA cores; attention_mma.cu: bf16 on the tensor cores).
//
// Work.  A stream is one sequence with one key/value head (and, for groups
// wider than a core takes, one chunk of the group's query heads): ceil(len /
// TT) tiles of TT tokens, one (empty) tile for an empty sequence.  The tiles
// of all streams, stream after stream, form one line that is cut into equal
// pieces, one per CTA, so the GPU is evenly busy whatever the mix of lengths:
// a single long context is split over every SM and a ragged batch has no
// tail.  Every CTA works the cut out from the lengths alone.
//
// Within a CTA the warps take the tiles of a piece in turn, each through its
// own ring of asynchronous copies; a ring runs ahead across the ends of
// streams, so memory stays busy while results are put together.  Each warp
// keeps a running maximum m, sum l and unnormalised output O of the softmax
// (one pass over the keys): a tile with scores s and values v does
//   m' = max(m, max s), O = O 2^(m-m') + sum 2^(s-m') v, l likewise,
// scores in units of log 2.  At the end of a stream's piece the warps'
// (m, l, O) are joined in shared memory in warp order; if the CTA held the
// whole stream the result is final, else it is a partial result in the
// workspace and join_kernel puts the stream's partial results together in
// order.  All of it is deterministic.
#pragma once

#include <algorithm>
#include <atomic>
#include <climits>
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace lora {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

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

// 2^(a - m) with the convention that a maximum of -inf (nothing seen) weighs
// nothing; an infinite or NaN score stays visible as NaN.
__device__ __forceinline__ float weight_of(float a, float m) { return a == kNegInf ? 0.f : exp2f(a - m); }

// The first n (all, if n >= 4) of four neighbouring outputs; one store where
// they are whole and aligned.
__device__ __forceinline__ void store4(float* dst, float4 v, int n) {
  if (n >= 4 && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
    *reinterpret_cast<float4*>(dst) = v;
    return;
  }
  const float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) dst[e] = r[e];
}
__device__ __forceinline__ void store4(__nv_bfloat16* dst, float4 v, int n) {
  if (n >= 4 && (reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(round_pack_bf16x2(v.x, v.y), round_pack_bf16x2(v.z, v.w));
    return;
  }
  const float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) dst[e] = __float2bfloat16_rn(r[e]);
}

template <int TT>
__device__ __forceinline__ int tiles_of(const AttnDesc& p, int len) {
  if (len < 0 || len > p.max_len) return 0;  // refused: LORA_DEV_BAD_LENGTH
  return len == 0 ? 1 : (len - 1) / TT + 1;
}

// One CTA's piece of the line of tiles, [lo, hi), and the sequence it starts
// in (whose first tile is number base).
struct Piece {
  long long total, lo, hi, base;
  int units, seq;
};

__device__ __forceinline__ long long piece_start(long long total, int units, int u) { return total * u / units; }

// Executed by one full warp (every lane gets the result).
template <int TT, int W>
__device__ __forceinline__ Piece locate_piece(const AttnDesc& p, int u, int max_units) {
  const int lane = threadIdx.x & 31;
  const int streams = p.cache.num_kv_heads * p.chunks;  // per sequence
  long long sum = 0;
  bool bad = false;
  for (int b = lane; b < p.num_seqs; b += 32) {
    const int n = tiles_of<TT>(p, p.lengths[b]);
    bad |= n == 0;
    sum += n;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (u == 0 && bad) atomicOr(p.status, LORA_DEV_BAD_LENGTH);
  Piece r;
  r.total = sum * streams;
  const long long want = (r.total + W - 1) / W;  // a tile for every warp
  r.units = (int)(want < 1 ? 1 : (want < max_units ? want : max_units));
  r.lo = r.hi = r.base = 0;
  r.seq = 0;
  if (u >= r.units || r.total == 0) return r;
  r.lo = piece_start(r.total, r.units, u);
  r.hi = piece_start(r.total, r.units, u + 1);
  const long long want_tile = r.lo / streams;  // in units of one stream's tiles
  long long before = 0;
  for (int c = 0; c < p.num_seqs; c += 32) {
    const int b = c + lane;
    const long long n = b < p.num_seqs ? tiles_of<TT>(p, p.lengths[b]) : 0;
    long long incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    const bool here = n > 0 && want_tile >= before + incl - n && want_tile < before + incl;
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
      const int src = __ffs(who) - 1;
      r.seq = c + src;
      r.base = (before + __shfl_sync(0xffffffffu, incl - n, src)) * streams;
      break;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

// Walks the segments of a piece: the tiles [t0, t1) of stream `stream` of
// sequence `seq` (length len, n tiles).
template <int TT>
struct Segments {
  long long pos, hi;  // next tile of the line after this segment; end of the piece
  int seq, stream, len, n, t0, t1;
  bool valid;

  __device__ __forceinline__ void clip(const AttnDesc& p) {
    const long long room = hi - pos;
    t1 = n - t0 <= room ? n : t0 + (int)room;
    pos += t1 - t0;
  }
  __device__ __forceinline__ void first(const AttnDesc& p, const Piece& r) {
    hi = r.hi;
    pos = r.lo;
    valid = r.lo < r.hi;
    if (!valid) return;
    seq = r.seq;
    len = p.lengths[seq];
    n = tiles_of<TT>(p, len);
    const long long in = r.lo - r.base;
    stream = (int)(in / n);
    t0 = (int)(in - (long long)stream * n);
    clip(p);
  }
  __device__ __forceinline__ void next(const AttnDesc& p) {
    if (pos >= hi) {
      valid = false;
      return;
    }
    if (++stream == p.cache.num_kv_heads * p.chunks) {
      stream = 0;
      do {  // the line has tiles left, so a sequence with tiles follows
        len = p.lengths[++seq];
        n = tiles_of<TT>(p, len);
      } while (n == 0);
    }
    t0 = 0;
    clip(p);
  }
};

// One warp's walk over the tiles it loads, with its lane's token of the tile
// looked up one tile ahead (the block-table read is in flight meanwhile).
template <int TT, int W>
struct TileCursor {
  Segments<TT> seg;
  int tile;
  int page, slot;  // of this lane's token; page -1: no token (slot -1)

  __device__ __forceinline__ void look_up(const AttnDesc& p) {
    const int j = tile * TT + (int)(threadIdx.x & (TT - 1));
    page = -1;
    slot = -1;
    if (j < seg.len) {
      const int i = (unsigned)j / (unsigned)p.cache.page_size;
      slot = j - i * p.cache.page_size;
      page = p.tables[seg.seq * p.table_stride + i];
    }
  }
  __device__ __forceinline__ void settle(const AttnDesc& p, int warp) {
    while (seg.valid && tile >= seg.t1) {
      seg.next(p);
      tile = seg.t0 + warp;
    }
    if (seg.valid) look_up(p);
  }
  __device__ __forceinline__ void first(const AttnDesc& p, const Piece& r, int warp) {
    seg.first(p, r);
    if (!seg.valid) return;
    tile = seg.t0 + warp;
    settle(p, warp);
  }
  __device__ __forceinline__ void next(const AttnDesc& p, int warp) {
    tile += W;
    settle(p, warp);
  }
  // Element offset of this lane's token in the cache (-1: none, or its page
  // is not one of the cache's).  *bad: some lane's page is not.
  __device__ __forceinline__ long long offset(const AttnDesc& p, bool* bad) const {
    const bool none = slot < 0;
    const bool off_cache = !none && (page < 0 || page >= p.cache.num_pages);
    *bad = __any_sync(0xffffffffu, off_cache);
    if (none || off_cache) return -1;
    return page * p.cache.page_stride + slot * p.cache.token_stride +
           (seg.stream / p.chunks) * p.cache.head_stride;
  }
};

// The frame.  Core gives:
//   T, TT (tokens a tile), W (warps), CTAS (resident per SM), HD (padded head
//   width), CH (query heads a stream), COMB (heads joined in shared memory at
//   a time, CH of them in CH / COMB parts), STAGES, STAGE_BYTES (K and V of a
//   tile), EXTRA_BYTES (its own shared memory per CTA)
//   Core(p, extra)            before anything else, all threads
//   load(p, stage, off)       this warp's copies of one tile into a stage
//   fetch(p, seq, head0, heads)  starts loading a stream's queries: this
//                             thread's share, into registers
//   pass_on()                 puts that share into shared memory
//   begin(p, heads)           new stream: its queries are in shared memory
//   tile(p, stage, n)         one tile, its first n tokens
//   put(part, o, s)           this warp's O [COMB][HD + 4] and (m, l) [COMB] of part
template <class Core>
__global__ void __launch_bounds__(Core::W * 32, Core::CTAS) attention_kernel(const __grid_constant__ AttnDesc p) {
  using T = typename Core::T;
  constexpr int TT = Core::TT, W = Core::W, HD = Core::HD, CH = Core::CH, STAGES = Core::STAGES;
  constexpr int COMB = Core::COMB;
  constexpr int PITCH = HD + 4;  // floats per head of the join buffer: its columns fall on different banks
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Piece s_piece;
  uint8_t* ring = smem;
  float* comb = reinterpret_cast<float*>(smem + W * STAGES * Core::STAGE_BYTES);
  float2* stat = reinterpret_cast<float2*>(comb + W * COMB * PITCH);
  uint8_t* extra = reinterpret_cast<uint8_t*>(stat + W * COMB);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = blockIdx.x;
  pdl_launch_dependents();

  if (warp == 0) {
    const Piece r = locate_piece<TT, W>(p, u, gridDim.x);
    if (lane == 0) s_piece = r;
  }
  // Columns past head_dim are never loaded and read as zero.
  if (p.cache.head_dim < HD)
    for (int i = threadIdx.x; i < W * STAGES * Core::STAGE_BYTES / 16; i += W * 32)
      reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  const Piece piece = s_piece;
  if (piece.lo >= piece.hi) return;

  // The next segment's queries travel through registers (each thread a share)
  // into the core's shared buffer while the present segment is worked on.
  auto heads_of = [&](const Segments<TT>& sg, int* head0) {
    const int kv_head = sg.stream / p.chunks;
    const int in_group = (sg.stream - kv_head * p.chunks) * CH;  // first head of the chunk
    *head0 = kv_head * p.group + in_group;
    return min(CH, p.group - in_group);
  };
  Segments<TT> seg;
  seg.first(p, piece);
  Core core(p, extra);
  int head0, heads = heads_of(seg, &head0);
  core.fetch(p, seg.seq, head0, heads);
  uint8_t* my_ring = ring + warp * STAGES * Core::STAGE_BYTES;
  TileCursor<TT, W> cur;
  cur.first(p, piece, warp);
  unsigned bad_stages = 0;
  auto load = [&](int stage) {
    if (cur.seg.valid) {
      bool bad;
      const long long off = cur.offset(p, &bad);
      bad_stages = (bad_stages & ~(1u << stage)) | ((unsigned)bad << stage);
      core.load(p, my_ring + stage * Core::STAGE_BYTES, off);
      cur.next(p, warp);
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int s = 0; s < STAGES; ++s) load(s);

  core.pass_on();
  __syncthreads();
  int stage = 0;
#pragma unroll 1
  while (true) {
    core.begin(p, heads);
    Segments<TT> after = seg;
    after.next(p);
    int after_head0 = 0, after_heads = 0;
    if (after.valid) {
      after_heads = heads_of(after, &after_head0);
      core.fetch(p, after.seq, after_head0, after_heads);
    }
    bool bad = false;
#pragma unroll 1
    for (int t = seg.t0 + warp; t < seg.t1; t += W) {
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      bad |= (bad_stages >> stage) & 1;
      core.tile(p, my_ring + stage * Core::STAGE_BYTES, min(TT, seg.len - t * TT));
      __syncwarp();
      load(stage);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    // Join the warps.  A sum of -1 marks a page outside the cache.
    const bool whole = seg.t0 == 0 && seg.t1 == seg.n;
    const long long slot = 2 * u + (seg.t0 == 0 ? 1 : 0);  // of the workspace
#pragma unroll 1
    for (int part = 0; part < CH / COMB; ++part) {
      const int part_heads = min(COMB, heads - part * COMB);
      if (part_heads <= 0) break;
      if (part > 0) __syncthreads();
      core.put(part, comb + warp * COMB * PITCH, stat + warp * COMB);
      __syncwarp();
      if (bad && lane < COMB) stat[warp * COMB + lane].y = -1.f;
      __syncthreads();
      for (int i = threadIdx.x; i < part_heads * (HD / 4); i += W * 32) {
        const int h = i / (HD / 4), d = (i - h * (HD / 4)) * 4;
        if (d >= p.cache.head_dim) continue;
        float m = kNegInf;
        bool any_bad = false;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float2 st = stat[w * COMB + h];
          m = fmaxf(m, st.x);
          any_bad |= st.y < 0.f;
        }
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float2 st = stat[w * COMB + h];
          const float f = weight_of(st.x, m);
          const float4 v = *reinterpret_cast<const float4*>(comb + (w * COMB + h) * PITCH + d);
          l = fmaf(st.y, f, l);
          o.x = fmaf(v.x, f, o.x);
          o.y = fmaf(v.y, f, o.y);
          o.z = fmaf(v.z, f, o.z);
          o.w = fmaf(v.w, f, o.w);
        }
        const int hc = part * COMB + h;
        if (!whole) {
          *reinterpret_cast<float4*>(p.partial + (slot * CH + hc) * HD + d) = o;
          if (d == 0) p.stats[slot * CH + hc] = make_float2(m, any_bad ? -1.f : l);
        } else if (any_bad) {
          if (d == 0) atomicOr(p.status, LORA_DEV_BAD_PAGE);
        } else {
          T* out = static_cast<T*>(p.out.data) + seg.seq * p.out.row_stride + (head0 + hc) * p.out.head_stride + d;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          store4(out, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), p.cache.head_dim - d);
          if (d == 0 && p.lse) p.lse[(long long)seg.seq * p.num_heads + head0 + hc] = (m + log2f(l)) * kLn2;
        }
      }
    }
    if (!after.valid) break;
    core.pass_on();
    __syncthreads();  // the join's buffer is free, the queries are there
    seg = after;
    head0 = after_head0;
    heads = after_heads;
  }
  cp_async_wait<0>();
}

// Joins the partial results of the streams that several units share.  Block
// (u, h): the stream that unit u starts inside of and unit u - 1 begins, and
// the h-th query head of it; its warps share the partial results out and are
// joined in warp order.  Partial 0 is the end of unit u - 1, partial i the
// beginning of unit u - 1 + i.  Which stream that is follows from the lengths
// alone, so it is found while the units still run; after them the statistics
// and the outputs are one round trip to memory.
constexpr int kJoinWarps = 4, kJoinBatch = 8;

template <class Core>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const __grid_constant__ AttnDesc p) {
  using T = typename Core::T;
  constexpr int TT = Core::TT, HD = Core::HD, CH = Core::CH, VPL = HD / 32;
  __shared__ int4 s_split;
  __shared__ float s_o[kJoinWarps][HD];
  __shared__ float s_l[kJoinWarps];
  const int u = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    const Piece piece = locate_piece<TT, Core::W>(p, u, gridDim.x);
    int4 split = make_int4(0, 0, 0, 0);
    if (piece.lo < piece.hi) {
      Segments<TT> sg;
      sg.first(p, piece);
      const long long begin = piece.lo - sg.t0, end = begin + sg.n;
      if (sg.t0 > 0 && piece_start(piece.total, piece.units, u - 1) <= begin) {
        // First unit that starts at or after the stream's end.
        const long long v = (end * piece.units + piece.total - 1) / piece.total;
        split = make_int4(sg.seq, sg.stream, (int)v - u + 1, 0);
      }
    }
    if (lane == 0) s_split = split;
  }
  __syncthreads();
  pdl_wait();  // every block: the grid must not be over before the units are
  const int4 split = s_split;
  const int kv_head = split.y / p.chunks;
  const int in_group = (split.y - kv_head * p.chunks) * CH;
  if (split.z == 0 || h >= p.group - in_group) return;
  auto slot = [&](int i) { return (long long)(i == 0 ? 2 * (u - 1) + 1 : 2 * (u - 1 + i)) * CH + h; };
  // This warp's first partial results are on their way before the statistics
  // are looked at.
  float v[kJoinBatch][VPL], st_l[kJoinBatch], st_m[kJoinBatch];
  auto load = [&](int from) {
#pragma unroll
    for (int b = 0; b < kJoinBatch; ++b) {
      const int i = from + b * kJoinWarps;
      st_m[b] = kNegInf;
      st_l[b] = 0.f;
#pragma unroll
      for (int e = 0; e < VPL; ++e) v[b][e] = 0.f;
      if (i < split.z) {
        const float2 st = p.stats[slot(i)];
        st_m[b] = st.x;
        st_l[b] = st.y;
        const float* src = p.partial + slot(i) * HD + lane;
#pragma unroll
        for (int e = 0; e < VPL; ++e) v[b][e] = src[e * 32];
      }
    }
  };
  load(warp);
  float m = kNegInf;
  bool bad = false;
  for (int i = lane; i < split.z; i += 32) {
    const float2 st = p.stats[slot(i)];
    m = fmaxf(m, st.x);
    bad |= st.y < 0.f;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (__any_sync(0xffffffffu, bad)) {  // the same in every warp
    if (threadIdx.x == 0) atomicOr(p.status, LORA_DEV_BAD_PAGE);
    return;
  }
  float l = 0.f, o[VPL] = {};
  for (int from = warp; from < split.z; from += kJoinBatch * kJoinWarps) {
    if (from != warp) load(from);
#pragma unroll
    for (int b = 0; b < kJoinBatch; ++b) {
      const float f = weight_of(st_m[b], m);
      l = fmaf(st_l[b], f, l);
#pragma unroll
      for (int e = 0; e < VPL; ++e) o[e] = fmaf(v[b][e], f, o[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < VPL; ++e) s_o[warp][e * 32 + lane] = o[e];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) l += s_l[w];
  const int head = kv_head * p.group + in_group + h;
  T* out = static_cast<T*>(p.out.data) + split.x * p.out.row_stride + head * p.out.head_stride;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int d = threadIdx.x; d < p.cache.head_dim; d += kJoinWarps * 32) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) sum += s_o[w][d];
    out[d] = from_f<T>(sum * inv);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[(long long)split.x * p.num_heads + head] = (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------- host --

// What a core's launch needs; the same numbers size the workspace.
struct CoreShape {
  int TT, W, HD, CH, CTAS;
};

inline int chunks_of(const CoreShape& c, const AttnDesc& p) { return (p.group + c.CH - 1) / c.CH; }

// CTAs of a launch: what fits on the GPU at once, or less when the longest
// sequences the block tables allow would not give every warp a tile.
inline int units_of(const CoreShape& c, const AttnDesc& p, int sms) {
  const long long tiles = std::max(1, p.max_len / c.TT + (p.max_len % c.TT != 0));
  const long long streams = (long long)p.num_seqs * p.cache.num_kv_heads * chunks_of(c, p);
  const long long most = (long long)c.CTAS * std::max(sms, 1);
  if (streams >= most * c.W) return (int)most;
  return (int)std::max(1LL, std::min(most, (tiles * streams + c.W - 1) / c.W));
}

inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

struct WorkspaceParts {
  size_t partial, bytes;  // offset of the outputs (the statistics come first), and the whole
};

inline WorkspaceParts workspace_parts(const CoreShape& c, int units) {
  WorkspaceParts w;
  w.partial = round256((size_t)2 * units * c.CH * sizeof(float2));
  w.bytes = w.partial + round256((size_t)2 * units * c.CH * c.HD * sizeof(float));
  return w;
}

template <class Core>
constexpr CoreShape shape_of() {
  return {Core::TT, Core::W, Core::HD, Core::CH, Core::CTAS};
}

// Raises the kernel's shared-memory limit, once per device.
template <class Core>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(attention_kernel<Core>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

template <class Core>
cudaError_t launch_core(AttnDesc p, void* workspace, cudaStream_t s, unsigned path) {
  constexpr CoreShape c = shape_of<Core>();
  constexpr size_t smem = (size_t)Core::W * Core::STAGES * Core::STAGE_BYTES +
                          (size_t)Core::W * Core::COMB * ((Core::HD + 4) * 4 + 8) + Core::EXTRA_BYTES;
  static_assert(smem <= 227 * 1024 - 256, "a CTA's shared memory");
  p.chunks = chunks_of(c, p);
  const int units = units_of(c, p, std::min(device_sm_count(), kMaxSmsForWorkspace));
  const WorkspaceParts w = workspace_parts(c, units);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.stats = reinterpret_cast<float2*>(ws);
  p.partial = reinterpret_cast<float*>(ws + w.partial);
  cudaError_t e = allow_smem<Core>((int)smem);
  if (e != cudaSuccess) return e;
  attention_kernel<Core><<<units, Core::W * 32, smem, s>>>(p);
  if ((e = noted(cudaGetLastError(), path)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units, std::min(Core::CH, p.group));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return noted(cudaLaunchKernelEx(&cfg, attention_join_kernel<Core>, p), LORA_PATH_JOIN);
}

// attention_mma.cu: bf16 on the tensor cores.  mma_attention_ok: the shapes
// and alignments it takes.
bool mma_attention_ok(const AttnDesc& p);
CoreShape mma_attention_shape(const AttnDesc& p);
cudaError_t launch_attention_mma(const AttnDesc& p, void* workspace, cudaStream_t s);
// attention_generic.cu: fp32 arithmetic, any type, size and alignment.
CoreShape generic_attention_shape(const AttnDesc& p);
cudaError_t launch_attention_generic(const AttnDesc& p, void* workspace, cudaStream_t s);

}  // namespace lora
