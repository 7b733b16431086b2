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
// tail.  Each stream also takes some places of the line for its fixed cost:
// without them a CTA that draws many short streams ends long after the others
// (256 ragged contexts: 25 streams against 4, 194 us against 151).  Every CTA
// works the cut out from the lengths alone.
//
// Where streams are many and short the pieces go to warps instead and a stream
// to the one whose piece holds its first tile: no stream is shared, no warp
// waits for another.  So with up to kSoloTokens tokens a stream and a stream
// for more than every other warp of the GPU (4720 streams of one or two tiles:
// 46.8 us by blocks, 26.0 by warps; 1216 of 14 tiles 32.4 and 28.8; 352 of 3 to
// 6 tiles 16.0 and 18.6, so those stay with blocks), or with one or two tiles
// and more streams than SMs (592 streams of one tile 16.6 and 10.2).  Where
// streams are short and no more than the blocks that fit on the GPU each takes
// one: nothing to join (224 streams of 4 to 7 tiles 20.6 us by even pieces,
// 15.3 so; 128 of up to 16 tiles 14.8 and 13.2).  Past four tiles a warp even
// pieces are as fast or faster (32 of 19 to 38 tiles 13.0 and 16.2).
//
// Within a CTA the warps take the tiles of a piece in turn, each through its
// own ring of asynchronous copies; a ring runs ahead across the ends of
// streams, so memory stays busy while results are put together.  Each step
// commits one group of copies, an empty one where no tile is left.  Each warp
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

// 2^x, below 2^-126 zero.
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(a - m) with the convention that a maximum of -inf (nothing seen) weighs
// nothing; an infinite or NaN score stays visible as NaN.
__device__ __forceinline__ float weight_of(float a, float m) { return a == kNegInf ? 0.f : pow2(a - m); }

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

__device__ __forceinline__ long long divide(long long a, int b) {  // a >= 0, b > 0
  return a >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The line.  A stream takes C places that stand for what a CTA spends on any
// stream it touches (joining its warps, starting the next), then one place a
// tile.  The line is cut into `pieces` even parts.
struct Line {
  long long total, base;  // piece u: base places, the first `rest` pieces one more
  int pieces, rest;
  __device__ __forceinline__ void cut(long long total_, int pieces_) {
    total = total_;
    pieces = pieces_;
    base = divide(total, pieces);
    rest = (int)(total - base * pieces);
  }
  __device__ __forceinline__ long long start(int u) const { return u * base + min(u, rest); }
  // First piece that starts at or after a place.
  __device__ __forceinline__ int first_from(long long place) const {
    const long long wide = rest * (base + 1);
    return place <= wide ? (int)((place + base) / (base + 1)) : rest + (int)((place - wide + base - 1) / base);
  }
};

// One piece of the line, [lo, hi), and the sequence that place lo
// belongs to (whose first place is number origin).
struct Piece {
  long long lo, hi, origin;
  int seq;
};

constexpr int kSoloTokens = 256;
constexpr int kEachTiles = 4;  // tiles a warp

// Sum over the warp of values below 2^32 / of any size.
__device__ __forceinline__ long long warp_sum(unsigned v) {
  return (long long)__reduce_add_sync(0xffffffffu, v & 0xffffu) +
         ((long long)__reduce_add_sync(0xffffffffu, v >> 16) << 16);
}
__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The sequence, of those one lane counted from `seq` on, whose places contain
// `place`; I: wide enough for a place.
template <typename I, int PER>
__device__ __forceinline__ bool find_place(const int (&n)[PER], I mine, I before, I place, int seq, int* found_seq,
                                           I* found_first) {
  const int lane = threadIdx.x & 31;
  I incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const I v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  I first = before + incl - mine;
  const unsigned who = __ballot_sync(0xffffffffu, place >= first && place < first + mine);
  if (!who) return false;
  bool found = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    found = found || place < first + (I)n[i];
    if (!found) {
      first += (I)n[i];
      ++seq;
    }
  }
  const int src = __ffs(who) - 1;
  *found_seq = __shfl_sync(0xffffffffu, seq, src);
  *found_first = __shfl_sync(0xffffffffu, first, src);
  return true;
}

// What one lane counts of sequences [from + 8 lane, from + 8 lane + 8): the
// places of one stream of each.
template <class Core>
struct Count {
  static constexpr int PER = 8, C = Core::STREAM_COST;
  int n[PER];
  unsigned tiles, live;
  int longest;
  bool bad;
  __device__ __forceinline__ void read(const AttnDesc& p, int from) {
    tiles = live = 0;
    longest = 0;
    bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int b = from + (int)(threadIdx.x & 31) * PER + i;
      const int t = b < p.num_seqs ? tiles_of<Core::TT>(p, p.lengths[b]) : 0;
      bad |= t == 0 && b < p.num_seqs;
      n[i] = t > 0 ? t + C : 0;
      longest = max(longest, n[i]);
      tiles += t;
      live += t > 0;
    }
  }
  __device__ __forceinline__ long long places() const { return (long long)tiles + C * live; }
};

// How the whole call is shared out; every warp works it out from the lengths.
// Executed by one full warp (every lane gets the results), as is locate.
template <class Core>
struct Plan {
  static constexpr int CHUNK = 32 * Count<Core>::PER;
  Line line;
  bool solo;   // pieces are for warps, streams are whole
  bool each;   // piece u is stream u: lo is its number in the sequence
  bool small;  // one count covers the sequences, and places fit 32 bits

  // c: the count of the first sequences.
  __device__ __forceinline__ void make(const AttnDesc& p, const Count<Core>& c, bool report) {
    const int streams = p.cache.num_kv_heads * p.chunks;  // per sequence
    const bool once = p.num_seqs <= CHUNK;
    long long tiles, live;
    int longest = c.longest;
    bool bad = c.bad;
    if (once) {
      tiles = warp_sum(c.tiles);
      live = __reduce_add_sync(0xffffffffu, c.live);
    } else {
      tiles = c.tiles;
      live = c.live;
      for (int from = CHUNK; from < p.num_seqs; from += CHUNK) {
        Count<Core> more;
        more.read(p, from);
        tiles += more.tiles;
        live += more.live;
        longest = max(longest, more.longest);
        bad |= more.bad;
      }
      tiles = warp_sum(tiles);
      live = warp_sum(live);
    }
    if (report && bad) atomicOr(p.status, LORA_DEV_BAD_LENGTH);
    longest = __reduce_max_sync(0xffffffffu, longest);
    const long long one = tiles + Core::STREAM_COST * live;
    const long long all = live * streams;
    const int reach = longest - Core::STREAM_COST;  // tiles of the longest stream
    solo = (reach <= kSoloTokens / Core::TT && 2 * all > (long long)Core::CTAS * p.sms * Core::W) ||
           (reach <= 2 && all > p.sms);
    // Else pieces with a tile for every warp.
    const long long want = solo ? all : (tiles * streams + Core::W - 1) / Core::W;
    const long long most = solo ? (long long)p.pieces * Core::W : p.pieces;
    small = once && one < INT_MAX;
    each = !solo && reach <= kEachTiles * Core::W && all <= p.pieces && live == p.num_seqs;
    line.cut(one * streams, (int)(each ? all : want < 1 ? 1 : want < most ? want : most));
  }

  // Piece u.  c: the count of the first sequences.
  __device__ __forceinline__ Piece locate(const AttnDesc& p, Count<Core> c, int u) const {
    const int streams = p.cache.num_kv_heads * p.chunks, lane = threadIdx.x & 31;
    Piece r;
    r.lo = r.hi = r.origin = 0;
    r.seq = 0;
    if (u >= line.pieces || line.total == 0) return r;
    if (each) {
      r.seq = u / streams;
      r.lo = u - r.seq * streams;
      r.hi = r.lo + 1;
      return r;
    }
    r.lo = line.start(u);
    r.hi = line.start(u + 1);
    // The sequence whose one-stream places contain lo / streams.
    const long long place = divide(r.lo, streams);
    if (small) {
      unsigned first = 0;
      find_place<unsigned>(c.n, (unsigned)c.places(), 0u, (unsigned)place, lane * Count<Core>::PER, &r.seq, &first);
      r.origin = (long long)first * streams;
      return r;
    }
    long long before = 0, first = 0;
    for (int from = 0; from < p.num_seqs; from += CHUNK) {
      if (from > 0) c.read(p, from);
      if (find_place<long long>(c.n, c.places(), before, place, from + lane * Count<Core>::PER, &r.seq, &first)) break;
      before += warp_sum(c.places());
    }
    r.origin = first * streams;
    return r;
  }
};

// Key/value head of a stream.
__device__ __forceinline__ int kv_head_of(const AttnDesc& p, int stream) {
  return p.chunks == 1 ? stream : stream / p.chunks;
}

// Walks the segments of a piece: the tiles [t0, t1) of stream `stream` of
// sequence `seq` (length len, n tiles).
template <class Core>
struct Segments {
  long long room;  // places of the piece from this stream's first tile on
  int seq, stream, len, n, t0, t1;
  bool valid, whole;  // whole: streams are not cut

  __device__ __forceinline__ void clip() {
    t1 = n <= room || whole ? n : (int)room;
    valid = room > 0 && t1 > t0;
  }
  __device__ __forceinline__ void first(const AttnDesc& p, const Piece& r, const Plan<Core>& plan) {
    valid = r.lo < r.hi;
    if (!valid) return;
    seq = r.seq;
    len = p.lengths[seq];
    n = tiles_of<Core::TT>(p, len);
    whole = plan.solo || plan.each;
    const long long in = r.lo - r.origin;
    const int places = n + Core::STREAM_COST;
    stream = plan.each ? (int)r.lo : (int)divide(in, places);
    const long long tile0 =  // place of the first tile
        plan.each ? r.lo : r.origin + (long long)stream * places + Core::STREAM_COST;
    t0 = r.lo > tile0 ? (int)(r.lo - tile0) : 0;
    room = r.hi - tile0;
    if (whole && t0 > 0) next(p);  // the stream is the piece's before
    else clip();
  }
  __device__ __forceinline__ void next(const AttnDesc& p) {
    room -= n + Core::STREAM_COST;
    t0 = 0;
    if (room <= 0) {  // the piece ends before the next stream's first tile
      valid = false;
      return;
    }
    if (++stream == p.cache.num_kv_heads * p.chunks) {
      stream = 0;
      do {  // the line goes on, so a sequence with tiles follows
        len = p.lengths[++seq];
        n = tiles_of<Core::TT>(p, len);
      } while (n == 0);
    }
    clip();
  }
};

// A piece that starts inside a stream whose beginning lies in the piece before
// it stands for that stream in the join: {sequence, stream, pieces that share
// it}; others {0, 0, 0}.
template <class Core>
__device__ __forceinline__ int4 split_of(const Line& line, const Piece& piece, const Segments<Core>& first, int u) {
  if (!first.valid || first.t0 == 0) return make_int4(0, 0, 0, 0);  // so where streams are whole
  const long long begin = piece.lo - first.t0, end = begin + first.n;  // places of the stream's tiles
  if (line.start(u - 1) > begin) return make_int4(0, 0, 0, 0);
  return make_int4(first.seq, first.stream, line.first_from(end) - u + 1, 0);
}

// One warp's walk over the tiles it loads: rank, rank + step, ... of each
// segment.  The block-table reads of a tile are made ahead of its load and are
// in flight meanwhile.  Where pages hold whole grains of GRAIN tokens lane i
// looks up grain i of the tile, else token i.
template <class Core>
struct TileCursor {
  static constexpr int GRAINS = Core::TT / Core::GRAIN;
  Segments<Core> seg;
  int tile;
  int page, slot;  // slot: token within the page; below 0: no token

  // No branch per lane: a lane past the end looks its sequence's last token
  // up, so the warp stays together.
  __device__ __forceinline__ void look_up(const AttnDesc& p) {
    const int j = tile * Core::TT + (int)(p.whole_grains ? (threadIdx.x & (GRAINS - 1)) * Core::GRAIN
                                                         : threadIdx.x & (Core::TT - 1));
    page = 0;
    slot = -1;
    if (seg.len > 0) {  // the same on every lane
      const int jj = min(j, seg.len - 1);
      const int i = (int)(((unsigned long long)(unsigned)jj * p.page_magic) >> p.page_shift);
      page = p.tables[seg.seq * p.table_stride + i];
      slot = j < seg.len ? jj - i * p.cache.page_size : -1;
    }
  }
  __device__ __forceinline__ void settle(const AttnDesc& p, int rank) {
    while (seg.valid && tile >= seg.t1) {
      seg.next(p);
      tile = rank;
    }
    if (seg.valid) look_up(p);
  }
  __device__ __forceinline__ void first(const AttnDesc& p, const Segments<Core>& sg, int rank) {
    seg = sg;
    if (!seg.valid) return;
    tile = seg.t0 + rank;
    settle(p, rank);
  }
  __device__ __forceinline__ void next(const AttnDesc& p, int rank, int step) {
    if (!seg.valid) return;
    tile += step;
    settle(p, rank);
  }
  // Element offset in the cache of this lane's grain or token.  -1: none, or
  // its page is not one of the cache's (*bad: some lane's is not).
  __device__ __forceinline__ long long offset(const AttnDesc& p, bool* bad) const {
    const bool off_cache = slot >= 0 && (unsigned)page >= (unsigned)p.cache.num_pages;
    *bad = __any_sync(0xffffffffu, off_cache);
    const long long at = page * p.cache.page_stride + slot * p.cache.token_stride +
                         kv_head_of(p, seg.stream) * p.cache.head_stride;
    return slot < 0 || off_cache ? -1 : at;
  }
  // Tokens of the tile.
  __device__ __forceinline__ int tokens() const { return min(Core::TT, seg.len - tile * Core::TT); }
};

// The frame.  Core gives:
//   T, TT (tokens a tile), W (warps), CTAS (resident per SM), HD (padded head
//   width), CH (query heads a stream), COMB (heads joined in shared memory at
//   a time, CH of them in CH / COMB parts), STAGES, STAGE_BYTES (K and V of a
//   tile), EXTRA_BYTES (its own shared memory per CTA), STREAM_COST (places
//   of the line that stand for a stream's fixed cost), GRAIN (tokens that a
//   load takes from one page where pages allow it)
//   Core(p, extra)            before anything else, all threads
//   load(p, stage, off, n)    this warp's copies of one tile into a stage:
//                             off as TileCursor::offset gives it, n tokens
//   fetch(p, seq, head0, heads)  starts loading a stream's queries: this
//                             thread's share, into registers
//   pass_on()                 puts that share into shared memory
//   begin(p, heads)           new stream: its queries are in shared memory
//   begin_solo(p, seq, head0, heads)  new stream of a warp on its own
//   tile(p, stage, n)         one tile, its first n tokens
//   put(part, o, s)           this warp's O [COMB][HD + 4] and (m, l) [COMB] of part
template <class Core>
__global__ void __launch_bounds__(Core::W * 32, Core::CTAS) attention_kernel(const __grid_constant__ AttnDesc p) {
  using T = typename Core::T;
  constexpr int TT = Core::TT, W = Core::W, HD = Core::HD, CH = Core::CH, STAGES = Core::STAGES;
  constexpr int COMB = Core::COMB;
  constexpr int PITCH = HD + 4;  // floats per head of the join buffer: its columns fall on different banks
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  float* comb = reinterpret_cast<float*>(smem + W * STAGES * Core::STAGE_BYTES);
  float2* stat = reinterpret_cast<float2*>(comb + W * COMB * PITCH);
  uint8_t* extra = reinterpret_cast<uint8_t*>(stat + W * COMB);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();

  Count<Core> count;
  count.read(p, 0);
  Plan<Core> plan;
  plan.make(p, count, blockIdx.x == 0);
  const bool solo = plan.solo;
  const int u = solo ? blockIdx.x * W + warp : blockIdx.x;
  Segments<Core> seg;
  {
    const Piece piece = plan.locate(p, count, u);
    seg.first(p, piece, plan);
    if (p.large && threadIdx.x == 0)
      p.splits[blockIdx.x] = solo ? make_int4(0, 0, 0, 0) : split_of<Core>(plan.line, piece, seg, u);
  }
  if (!seg.valid) return;  // the whole CTA, or a warp on its own
  // The team that works on a segment: the CTA's warps, or one.
  const int team = solo ? 1 : W, rank = solo ? 0 : warp, leader = solo ? warp : 0;
  const int tid = solo ? lane : threadIdx.x;
  auto team_sync = [&] {
    if (solo) __syncwarp();
    else __syncthreads();
  };
  uint8_t* my_ring = ring + warp * STAGES * Core::STAGE_BYTES;
  // Columns past head_dim are never loaded and read as zero.
  if (p.cache.head_dim < HD) {
    for (int i = lane; i < STAGES * Core::STAGE_BYTES / 16; i += 32)
      reinterpret_cast<uint4*>(my_ring)[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  // The next segment's queries travel through registers (each thread a share)
  // into the core's shared buffer while the present segment is worked on.
  auto heads_of = [&](const Segments<Core>& sg, int* head0) {
    const int kv_head = kv_head_of(p, sg.stream);
    const int in_group = (sg.stream - kv_head * p.chunks) * CH;  // first head of the chunk
    *head0 = kv_head * p.group + in_group;
    return min(CH, p.group - in_group);
  };
  Core core(p, extra);
  int head0, heads = heads_of(seg, &head0);
  if (!solo) core.fetch(p, seg.seq, head0, heads);
  TileCursor<Core> cur;
  unsigned bad_stages = 0;
  auto load = [&](int stage, const TileCursor<Core>& c) {
    if (c.seg.valid) {
      bool bad;
      const long long off = c.offset(p, &bad);
      bad_stages = (bad_stages & ~(1u << stage)) | ((unsigned)bad << stage);
      core.load(p, my_ring + stage * Core::STAGE_BYTES, off, c.tokens());
    }
    cp_async_commit();  // of a tile or of nothing: one a step, so the count of groups tells which tile has landed
  };
  {
    // The first tiles' block-table reads all go out before any is waited for.
    TileCursor<Core> ahead[STAGES];
    ahead[0].first(p, seg, rank);
#pragma unroll
    for (int s = 1; s < STAGES; ++s) {
      ahead[s] = ahead[s - 1];
      ahead[s].next(p, rank, team);
    }
    cur = ahead[STAGES - 1];
    cur.next(p, rank, team);
#pragma unroll
    for (int s = 0; s < STAGES; ++s) load(s, ahead[s]);
  }

  if (!solo) {
    core.pass_on();
    __syncthreads();
  }
  int stage = 0;
#pragma unroll 1
  while (true) {
    __syncwarp();  // ldmatrix and mma need the warp's lanes together; a block barrier does not promise that
    if (solo) core.begin_solo(p, seg.seq, head0, heads);
    else core.begin(p, heads);
    Segments<Core> after = seg;
    after.next(p);
    int after_head0 = 0, after_heads = 0;
    if (after.valid) {
      after_heads = heads_of(after, &after_head0);
      if (!solo) core.fetch(p, after.seq, after_head0, after_heads);
    }
    bool bad = false;
#pragma unroll 1
    for (int t = seg.t0 + rank; t < seg.t1; t += team) {
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      bad |= (bad_stages >> stage) & 1;
      core.tile(p, my_ring + stage * Core::STAGE_BYTES, min(TT, seg.len - t * TT));
      __syncwarp();
      load(stage, cur);
      cur.next(p, rank, team);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    // Join the warps.  A sum of -1 marks a page outside the cache.
    const bool whole = seg.t0 == 0 && seg.t1 == seg.n;
    const long long slot = 2 * (long long)u + (seg.t0 == 0 ? 1 : 0);  // of the workspace
#pragma unroll 1
    for (int part = 0; part < CH / COMB; ++part) {
      const int part_heads = min(COMB, heads - part * COMB);
      if (part_heads <= 0) break;
      if (part > 0) team_sync();
      core.put(part, comb + warp * COMB * PITCH, stat + warp * COMB);
      __syncwarp();
      if (bad && lane < COMB) stat[warp * COMB + lane].y = -1.f;
      team_sync();
      for (int i = tid; i < part_heads * (HD / 4); i += team * 32) {
        const int h = i / (HD / 4), d = (i - h * (HD / 4)) * 4;
        if (d >= p.cache.head_dim) continue;
        float m = kNegInf;
        bool any_bad = false;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if (w >= team) break;
          const float2 st = stat[(leader + w) * COMB + h];
          m = fmaxf(m, st.x);
          any_bad |= st.y < 0.f;
        }
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if (w >= team) break;
          const float2 st = stat[(leader + w) * COMB + h];
          const float f = weight_of(st.x, m);
          const float4 v = *reinterpret_cast<const float4*>(comb + ((leader + w) * COMB + h) * PITCH + d);
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
    if (!solo) core.pass_on();
    team_sync();  // the join's buffer is free, the queries are there
    seg = after;
    head0 = after_head0;
    heads = after_heads;
  }
  cp_async_wait<0>();
}

// Joins the partial results of the streams that several pieces share: block u
// those of the stream that piece u starts inside of and piece u - 1 begins.
// Partial 0 is the end of piece u - 1, partial i the beginning of piece
// u - 1 + i; they are summed in a fixed order.
//
// Small calls share few streams among many pieces: a block is one query head,
// its warps share the partial results out.  Which stream it is follows from
// the lengths alone and is found while the pieces still run; after them the
// statistics and the outputs are one round trip to memory (one context of
// 131071 tokens: 25 us of joining before, 5 now).  Calls that may be large
// (large_of) mostly have hundreds of streams shared by two or three pieces and
// no room on the SMs before the pieces are done: there the pieces leave the
// answer in memory and a warp is one head (256 ragged contexts 192.8 us, in
// the small calls' way 195.3; 24 long ones 300.5 and 306.4).
constexpr int kJoinWarps = 4, kJoinBatch = 8;
constexpr int kLargePlaces = 192;  // places a piece, where every sequence fills its table

template <class Core>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const __grid_constant__ AttnDesc p) {
  using T = typename Core::T;
  constexpr int HD = Core::HD, CH = Core::CH, VPL = HD / 32;
  __shared__ int4 s_split;
  __shared__ float s_o[kJoinWarps][HD];
  __shared__ float s_l[kJoinWarps];
  const int u = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The team that joins a head: a warp, or the block's.
  const int team = p.large ? 1 : kJoinWarps, rank = p.large ? 0 : warp, leader = p.large ? warp : 0;
  const int h = p.large ? blockIdx.y * kJoinWarps + warp : blockIdx.y;
  int4 split;
  if (p.large) {
    pdl_wait();
    split = p.splits[u];
  } else {
    if (warp == 0) {
      Count<Core> count;
      count.read(p, 0);
      Plan<Core> plan;
      plan.make(p, count, false);
      const Piece piece = plan.locate(p, count, u);
      Segments<Core> sg;
      sg.first(p, piece, plan);
      split = split_of<Core>(plan.line, piece, sg, u);
      if (lane == 0) s_split = split;
    }
    __syncthreads();
    pdl_wait();  // every block: the grid must not be over before the pieces are
    split = s_split;
  }
  const int kv_head = kv_head_of(p, split.y);
  const int in_group = (split.y - kv_head * p.chunks) * CH;
  if (split.z == 0 || h >= min(CH, p.group - in_group)) return;  // the whole team
  auto slot = [&](int i) { return (long long)(i == 0 ? 2 * (u - 1) + 1 : 2 * (u - 1 + i)) * CH + h; };
  // This warp's first partial results are on their way before the statistics
  // are looked at.
  float v[kJoinBatch][VPL], st_l[kJoinBatch], st_m[kJoinBatch];
  auto load = [&](int from) {
#pragma unroll
    for (int b = 0; b < kJoinBatch; ++b) {
      const int i = from + b * team;
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
  load(rank);
  float m = kNegInf;
  bool bad = false;
  for (int i = lane; i < split.z; i += 32) {
    const float2 st = p.stats[slot(i)];
    m = fmaxf(m, st.x);
    bad |= st.y < 0.f;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (__any_sync(0xffffffffu, bad)) {  // the same in every warp of the team
    if (rank == 0 && lane == 0) atomicOr(p.status, LORA_DEV_BAD_PAGE);
    return;
  }
  float l = 0.f, o[VPL] = {};
  for (int from = rank; from < split.z; from += kJoinBatch * team) {
    if (from != rank) load(from);
#pragma unroll
    for (int b = 0; b < kJoinBatch; ++b) {
      if (from + b * team >= split.z) break;
      const float f = weight_of(st_m[b], m);
      l = fmaf(st_l[b], f, l);
#pragma unroll
      for (int e = 0; e < VPL; ++e) o[e] = fmaf(v[b][e], f, o[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < VPL; ++e) s_o[warp][e * 32 + lane] = o[e];
  if (lane == 0) s_l[warp] = l;
  if (p.large) __syncwarp();
  else __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w)
    if (w < team) l += s_l[leader + w];
  const int head = kv_head * p.group + in_group + h;
  T* out = static_cast<T*>(p.out.data) + split.x * p.out.row_stride + head * p.out.head_stride;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int d = rank * 32 + lane; d < p.cache.head_dim; d += team * 32) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
      if (w < team) sum += s_o[leader + w][d];
    out[d] = from_f<T>(sum * inv);
  }
  if (rank == 0 && lane == 0 && p.lse) p.lse[(long long)split.x * p.num_heads + head] = (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------- host --

// What a core's launch needs; the same numbers size the workspace.
struct CoreShape {
  int TT, W, HD, CH, CTAS, COST;
};

inline int chunks_of(const CoreShape& c, const AttnDesc& p) { return (p.group + c.CH - 1) / c.CH; }

// Streams of a call, and places of its line at most (both saturating): every
// sequence as long as the block tables allow.
inline long long streams_of(const CoreShape& c, const AttnDesc& p) {
  return (long long)p.num_seqs * std::min<long long>((long long)p.cache.num_kv_heads * chunks_of(c, p), INT_MAX);
}
inline long long most_tiles(const CoreShape& c, const AttnDesc& p) {
  return std::max(1, p.max_len / c.TT + (p.max_len % c.TT != 0));
}
inline long long most_places(const CoreShape& c, const AttnDesc& p) {
  return std::min(streams_of(c, p), (long long)INT_MAX) * (most_tiles(c, p) + c.COST);
}

// Pieces the line is cut into at most: what fits on the GPU at once, or less
// when the longest sequences would give every warp a tile with fewer (but one
// for each stream).  The longest the block tables allow: the lengths are on the
// device.  A table wider than need be costs the blocks that find no work, and
// their joins (one context of 517 tokens: 10.5 us with a table of 33 pages,
// 12.6 with one of 8192; 16 of 60 tokens 8.5 and 8.8).
inline int pieces_of(const CoreShape& c, const AttnDesc& p, int sms) {
  const long long most = (long long)c.CTAS * std::max(sms, 1), streams = streams_of(c, p);
  if (streams >= most * c.W) return (int)most;
  // Sure to be a warp each (Plan::make): no blocks beyond those.
  if (most_tiles(c, p) <= 2 && streams > sms) return (int)std::min(most, (streams + c.W - 1) / c.W);
  return (int)std::max(1LL, std::min(most, std::max(std::min(streams, most), (most_tiles(c, p) * streams + c.W - 1) / c.W)));
}
// Whether pieces are long, and streams shared by no more than eight of them,
// where every sequence fills its table.  The lengths may be anything below
// that.  Joining as a large call is no slower then (64 contexts of 200 tokens
// in tables of 2048 pages 22.3 us, in the small calls' way 25.3; 40 of 1000 38.2
// and 40.7; 300 of 64 26.0 and 28.8), unless one context outweighs the others and
// its many parts are a warp's to join (one of 131071 tokens among 39 of 200:
// 103.2 and 101.5).
inline bool large_of(const CoreShape& c, const AttnDesc& p, int sms) {
  const long long most = (long long)c.CTAS * std::max(sms, 1);
  return most_places(c, p) / most >= kLargePlaces && streams_of(c, p) * 8 >= most;
}

inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

struct WorkspaceParts {
  size_t stats, partial, bytes;  // offsets (the splits come first), and the whole
};

inline WorkspaceParts workspace_parts(const CoreShape& c, int pieces) {
  WorkspaceParts w;
  w.stats = round256((size_t)pieces * sizeof(int4));
  w.partial = w.stats + round256((size_t)2 * pieces * c.CH * sizeof(float2));
  w.bytes = w.partial + round256((size_t)2 * pieces * c.CH * c.HD * sizeof(float));
  return w;
}

inline size_t workspace_bytes_of(const CoreShape& c, const AttnDesc& p) {
  return workspace_parts(c, pieces_of(c, p, kMaxSmsForWorkspace)).bytes;
}

template <class Core>
constexpr CoreShape shape_of() {
  return {Core::TT, Core::W, Core::HD, Core::CH, Core::CTAS, Core::STREAM_COST};
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
  // page_size <= 2^log: magic = ceil(2^(31 + log) / page_size) is below 2^32
  // and exact for tokens below 2^31.
  int log = 0;
  while ((1LL << log) < p.cache.page_size) ++log;
  p.page_shift = 31 + log;
  p.page_magic = (unsigned)(((1ULL << p.page_shift) + p.cache.page_size - 1) / p.cache.page_size);
  p.whole_grains = p.cache.page_size % Core::GRAIN == 0;
  const int sms = std::min(device_sm_count(), kMaxSmsForWorkspace);
  p.pieces = pieces_of(c, p, sms);
  p.large = large_of(c, p, sms);
  p.sms = std::max(device_sm_count(), 1);
  const WorkspaceParts w = workspace_parts(c, p.pieces);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.splits = reinterpret_cast<int4*>(ws);
  p.stats = reinterpret_cast<float2*>(ws + w.stats);
  p.partial = reinterpret_cast<float*>(ws + w.partial);
  cudaError_t e = allow_smem<Core>((int)smem);
  if (e != cudaSuccess) return e;
  attention_kernel<Core><<<p.pieces, Core::W * 32, smem, s>>>(p);
  if ((e = noted(cudaGetLastError(), path)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int heads = std::min(Core::CH, p.group);
  cfg.gridDim = dim3(p.pieces, p.large ? (heads + kJoinWarps - 1) / kJoinWarps : heads);
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
size_t generic_attention_workspace(const AttnDesc& p);
cudaError_t launch_attention_generic(const AttnDesc& p, void* workspace, cudaStream_t s);

}  // namespace lora
