// tree_tc.cu -- tree attention of bf16 caches on the tensor cores (tcgen05).
// The frame is tree.cuh.
//
// A chunk is 128 rows, the 128 lanes of TMEM: rows that share a key/value head
// fill an instruction even where each drafted token alone is one row of a
// product, and every key and value is loaded once for all of them.  Tiles of
// TT cached tokens (a stage is 32 KB at most) go through
//   S = Q K^T      [128 x TT]  Q and K in shared memory, S in TMEM
//   P = 2^(S - m)  two threads a row, back into TMEM over S
//   O = P V        [128 x HV]  P from TMEM and shared memory, V as it lies
// S and O have two buffers each: the next scores and the last tile's output are
// under way while a tile's softmax runs.  A thread holds half a row's scores at
// once and half of its running O; the halves exchange their maximum through
// shared memory.  O's tiles are summed apart and taken into registers rounded:
// accumulated by the instruction, which cuts sums off, long contexts lose a bit
// every step, and a rescaling would have to wait for the products.
//
// P enters as three bf16 terms, two cut off and the last rounded, fp32's own 24
// bits together.  Two terms, 16 bits, left 10400 of 2.92 M outputs of 48 ragged
// trees off the bf16 value nearest to the result, three leave 1140 (fp32
// arithmetic 1500), and cost 5 to 20% (94 us, so 99; 24 trees of 64 on the 70B
// attention 431, so 491; 60 tokens against 131012 205, so 248).  What is left
// for the second term is taken from p (1 + 2^-23), a factor that comes off in
// the end, and for the third from (1 + 2^-17) times that (2^-24 p more at most):
// so neither is ever zero, and an infinite value stays one.  The first two lie
// in TMEM over S, which they fill; the third in what else is free there.  At 128
// wide nothing is, and it lies in shared memory, one tile's: its products go
// first, so that it is free again by the time the next is written.
//
// Warps: 0 loads K, 1 loads V, 2 loads Q, 3 issues the products, 4 to 11 are
// the softmax.  K and V come by TMA boxes where a page is whole eights of tokens,
// else by 16-byte asynchronous copies: a page may hold any number of tokens in
// any stride order (boxes: 24 trees of 64 on the 70B attention 697 us, so 499; one
// context of 131072 tokens 313, so 214).  Every wait is bounded.
//
// Those trees (24 contexts of 1024 to 8192 tokens, 64 over 8 heads) take 494 us,
// 473 TFLOP/s counting P once; 60 tokens against 131012 248 us, 2.2 TB/s; 48
// ragged trees over 128 to 2048 tokens 99 us, 2.7 TB/s.  What bounds it is the
// chain of loads, scores, softmax and outputs, whose hand-overs take 150 to 600
// cycles each (read by clocks in the kernel): issue slots are 42% taken, the
// tensor pipe 43%, DRAM 44%, and with two terms products, exponentials or
// loads left out one at a time changed its time by less than a tenth.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "tree.cuh"

namespace lora {
namespace {

constexpr int kTcThreads = 384;
constexpr float kTcLift = 1.f + 1.1920928955078125e-7f;   // 1 + 2^-23
constexpr float kTcLift2 = 1.f + 7.62939453125e-6f;       // 1 + 2^-17

// HK: padded width of Q and K.  HV: columns of V a stream takes.
template <int HK_>
struct TcCfg {
  static constexpr int HK = HK_, HV = HK > 128 ? 128 : HK;
  static constexpr int TT = HK > 128 ? 64 : 128;
  using S = TreeShape<128, TT, HV, 2>;
  static constexpr int Q_BYTES = 128 * HK * 2, K_BYTES = TT * HK * 2, V_BYTES = TT * HV * 2;
  static constexpr bool THIRD_TMEM = HK != 128;    // where P's third terms lie
  static constexpr int P_BYTES = THIRD_TMEM ? 0 : 128 * TT * 2;
  static constexpr int NS = HK == 64 ? 5 : HK == 128 ? 2 : 3;  // stages of K
  static constexpr int NV = HK == 64 ? 5 : 3;                  // of V, which is held longer
  static constexpr int SMEM = Q_BYTES + NS * K_BYTES + NV * V_BYTES + P_BYTES;
};

// Byte offset of 16-byte chunk c of row r in blocks of [rows][64 columns] with
// the 128-byte swizzle.
template <int ROWS>
__device__ __forceinline__ uint32_t tc_at(int r, int c) {
  return (c >> 3) * (ROWS * 128) + r * 128 + ((c & 7) ^ (r & 7)) * 16;
}

// Shared-memory descriptor of an operand whose rows are K and whose columns
// (64 to a 128-byte swizzled row) are the product's: blocks of 64 columns
// `block` bytes apart, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t addr, uint32_t block) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
constexpr uint32_t kTransposeB = 1u << 16;  // instruction descriptor: B's columns are contiguous

// D (+)= A B, A in TMEM.
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// N consecutive columns of this warp's lanes.
template <int N>
__device__ __forceinline__ void tmem_ld_columns(uint32_t taddr, float (&v)[N]) {
  static_assert(N == 32 || N == 64, "");
  uint32_t r[N];
#pragma unroll
  for (int c = 0; c < N; c += 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[c]), "=r"(r[c + 1]), "=r"(r[c + 2]), "=r"(r[c + 3]), "=r"(r[c + 4]), "=r"(r[c + 5]), "=r"(r[c + 6]),
          "=r"(r[c + 7]), "=r"(r[c + 8]), "=r"(r[c + 9]), "=r"(r[c + 10]), "=r"(r[c + 11]), "=r"(r[c + 12]),
          "=r"(r[c + 13]), "=r"(r[c + 14]), "=r"(r[c + 15]), "=r"(r[c + 16]), "=r"(r[c + 17]), "=r"(r[c + 18]),
          "=r"(r[c + 19]), "=r"(r[c + 20]), "=r"(r[c + 21]), "=r"(r[c + 22]), "=r"(r[c + 23]), "=r"(r[c + 24]),
          "=r"(r[c + 25]), "=r"(r[c + 26]), "=r"(r[c + 27]), "=r"(r[c + 28]), "=r"(r[c + 29]), "=r"(r[c + 30]),
          "=r"(r[c + 31])
        : "r"(taddr + c));
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
// What was asked for above is there after this, in the registers that are
// pinned behind it: nothing that uses them moves before the wait.
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void pin(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Moves registers between warpgroups (the launch gives every thread 168).
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Whether a phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// What the upper halves of two floats >= 0 hold, negated.
__device__ __forceinline__ float2 minus_top(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float((a & 0xffff0000u) | 0x80000000u), __uint_as_float((b & 0xffff0000u) | 0x80000000u));
}

// A box of a 4-D tensor map into shared memory; completion counted in bytes.
__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Boxes of 64 columns.  K and V: [page][head][token][column], `rows` tokens a
// box, a power of two that page_size is a multiple of, so that no box crosses
// a page.  Q: [row][head][column], the group's heads of 128 / group rows, where
// group divides 128 (q_boxes).
struct TcMaps {
  CUtensorMap k, v, q;
  int rows;
  int q_boxes;
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// A barrier serves one thread at a time, so one lane speaks for its warp (256
// threads on each of a tile's barriers took most of its time: trees of 64 on
// the 70B attention 460 us, so 420).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  bool ok = false;
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit && !ok; ++i) ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
  return ok;
}

constexpr int kTcFlags = 8;  // tiles whose notes are kept: more than can be in flight

struct TcShared {
  uint64_t kfull[5], kempty[5], vfull[5], vempty[5];
  uint64_t told[2];                // the halves of the rows have said something
  uint64_t land[2];                // V tiles that are looked through before they are handed over
  uint64_t qfull, qempty, sfull[2], pfull[2], pfree, ofull[2], ofree[2], done;
  uint32_t tmem;
  int fail;                        // a wait ran out
  float swap[2][2][128];           // what the halves of a row tell each other, by turns
  int bad[kTcFlags];               // a tile has a page outside the cache
  unsigned odd[kTcFlags][4];       // its drafted tokens whose values are not all finite
  TreePiece piece;
};

// BOXES: K and V come in boxes (pages of a multiple of 8 tokens), else row by row.
template <int HK, bool BOXES>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_tc_kernel(const __grid_constant__ TreeDesc p, const __grid_constant__ TcMaps maps) {
  using C = TcCfg<HK>;
  using S = typename C::S;
  constexpr int TT = C::TT, HV = C::HV, NS = C::NS, NV = C::NV;
  using T = __nv_bfloat16;
  extern __shared__ __align__(1024) uint8_t sq[];  // the swizzle wants whole 1024 bytes
  __shared__ __align__(8) TcShared sh;
  uint8_t* sk = sq + C::Q_BYTES;
  uint8_t* sv = sk + NS * C::K_BYTES;
  uint8_t* sp = sv + NV * C::V_BYTES;  // third terms where they have no TMEM, laid out as Q
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = blockIdx.x;
  const int hd = p.cache.head_dim;
  pdl_launch_dependents();
  if (warp == 0) {
    const TreePiece piece = tree_piece<S>(p, u, u == 0);
    if (lane == 0) {
      sh.piece = piece;
      sh.fail = 0;
      for (int i = 0; i < NS; ++i) {
        mbar_init(&sh.kfull[i], 1);
        mbar_init(&sh.kempty[i], 1);
      }
      for (int i = 0; i < NV; ++i) {
        mbar_init(&sh.vfull[i], 1);
        mbar_init(&sh.vempty[i], 1);
      }
      mbar_init(&sh.qfull, 1);
      mbar_init(&sh.told[0], 8);
      mbar_init(&sh.told[1], 8);
      mbar_init(&sh.land[0], 1);
      mbar_init(&sh.land[1], 1);
      mbar_init(&sh.qempty, 1);
      mbar_init(&sh.pfree, 1);
      mbar_init(&sh.done, 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.sfull[i], 1);
        mbar_init(&sh.pfull[i], 8);
        mbar_init(&sh.ofull[i], 1);
        mbar_init(&sh.ofree[i], 8);
      }
      fence_mbar_init();
    }
  } else if (warp == 3) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh.tmem;
  // TMEM columns: S and P of two tiles, then O of two.  Third terms lie where
  // tiles of 64 tokens or outputs of 64 columns leave room.
  auto s_col = [&](int w) { return tmem + w * 128; };
  auto o_col = [&](int w) { return tmem + 256 + w * 128; };
  auto third_col = [&](int w) { return tmem + w * 128 + (TT == 64 ? 64 : 320); };
  const TreePiece piece = sh.piece;
  TreeSegment<S> g;
  g.first(p, piece);
  bool dead = false;  // a wait ran out: nothing more is waited for
  // 88 x 128 + 208 x 256 = 168 x 384.
  if (warp >= 4) {
    take_registers<208>();
    // ---- softmax: a thread is half a row, tokens and columns of the output
    constexpr int ST = TT / 2, OC = HV / 2;  // of a thread
    const int h = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float scale = p.scale * kTreeLog2e;
    int tile_no = 0;            // of this CTA
    int syncs = 0;              // of the 256 threads
    int4 split = make_int4(0, 0, 0, 0);
    // Tells the other half of the row a value, and learns its own.
    auto tell = [&](float v) {
      sh.swap[syncs & 1][h][row] = v;
      warp_arrive(&sh.told[syncs & 1]);
    };
    auto learn = [&] {
      if (!dead && !warp_wait(&sh.told[syncs & 1], (syncs >> 1) & 1)) dead = true;
      return sh.swap[syncs++ & 1][h ^ 1][row];
    };
    while (g.valid && !dead) {
      const long long crow = (long long)g.chunk() * 128 + row;
      const bool live = crow < (long long)g.s.n * p.group;
      const int draft = live ? (int)(crow / p.group) : g.s.n - 1;
      const int head = g.kv_head(p) * p.group + (int)(live ? crow % p.group : 0);
      const unsigned long long* mask = p.masks ? p.masks + (long long)(g.s.row0 + draft) * p.words : nullptr;
      float m = kTreeNone, l = 0.f;
      const int first_no = tile_no;
      float kept0 = 0.f, kept1 = 0.f;  // what the tiles two and one before scale O by
      float2 o[OC / 2];
#pragma unroll
      for (int e = 0; e < OC / 2; ++e) o[e] = make_float2(0.f, 0.f);
      bool bad = false, strange = false;  // a page outside the cache; values of drafted tokens that are not finite
      // Takes up the output of tile t, number i of this CTA.
      auto fold = [&](float kept, int t, int i) {
        if (dead || !warp_wait(&sh.ofull[i & 1], (i >> 1) & 1)) {
          dead = true;
          return;
        }
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < OC; c += 32) {
          float v[32];
          tmem_ld_columns<32>(o_col(i & 1) + lanes + h * OC + c, v);
          tmem_wait_ld();
          pin(v);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[c / 2 + e] = fma_f32x2(o[c / 2 + e], make_float2(kept, kept), make_float2(v[2 * e], v[2 * e + 1]));
        }
        if (t * TT + TT > g.s.ctx) {
          const unsigned* odd = sh.odd[i % kTcFlags];
          strange |= (odd[0] | odd[1] | odd[2] | odd[3]) != 0;
        }
        tc_fence_before_sync();
        warp_arrive(&sh.ofree[i & 1]);
      };
      // Two steps more than tiles: the output of a tile is taken up two later.
#pragma unroll 1
      for (int t = g.t0; t < g.t1 + 2; ++t) {
        const int b = tile_no & 1, number = first_no + (t - g.t0);
        const bool scores = t < g.t1;
        float s[ST], top = kTreeNone;
        if (scores) {
        if (!warp_wait(&sh.sfull[b], (tile_no >> 1) & 1)) dead = true;
        if (dead) break;
        tc_fence_after_sync();
        bad |= sh.bad[tile_no % kTcFlags] != 0;
        tmem_ld_columns<ST>(s_col(b) + lanes + h * ST, s);
        tmem_wait_ld();
        pin(s);
#pragma unroll
        for (int e = 0; e < ST; e += 2) {
          const float2 x = mul_f32x2(make_float2(s[e], s[e + 1]), make_float2(scale, scale));
          s[e] = x.x;
          s[e + 1] = x.y;
        }
        const int d0 = t * TT + h * ST - g.s.ctx;  // this half's first token among the drafted ones
        if (d0 + ST > 0) {
#pragma unroll
          for (int c = 0; c < ST / 32; ++c) {
            const unsigned sees = tree_sees(p, mask, draft, d0 + c * 32, g.s.n);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(sees >> e & 1)) s[c * 32 + e] = kTreeNone;
          }
        }
        float tops[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int e = 4; e < ST; e += 4)
#pragma unroll
          for (int q = 0; q < 4; ++q) tops[q] = fmaxf(tops[q], s[e + q]);
        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        tell(top);
        }
        if (t >= g.t0 + 2) fold(kept0, t - 2, number - 2);  // until the other half has spoken
        if (dead) break;
        if (!scores) {
          kept0 = kept1;
          continue;
        }
        const float now = fmaxf(m, fmaxf(top, learn())), base = now == kTreeNone ? 0.f : now;
        const float keep = tree_pow2(m - base);
        m = now;
        // The third terms of the tile before have been read.
        if (!C::THIRD_TMEM && tile_no > 0 && !warp_wait(&sh.pfree, (tile_no - 1) & 1)) dead = true;
        if (dead) break;
        float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < ST / 16; ++c) {  // 16 tokens: 8 columns of first terms, 8 of second ones
          uint32_t out[16], third[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float2 x = add_f32x2(make_float2(s[c * 16 + 2 * q], s[c * 16 + 2 * q + 1]), make_float2(-base, -base));
            const float2 w = make_float2(tree_pow2(x.x), tree_pow2(x.y));
            sums[q & 1] = add_f32x2(sums[q & 1], w);
            const uint32_t ab = __float_as_uint(w.x), bb = __float_as_uint(w.y);
            out[q] = __byte_perm(ab, bb, 0x7632);
            const float2 rest = fma_f32x2(w, make_float2(kTcLift, kTcLift), minus_top(ab, bb));
            const uint32_t ar = __float_as_uint(rest.x), br = __float_as_uint(rest.y);
            out[8 + q] = __byte_perm(ar, br, 0x7632);
            const float2 last = fma_f32x2(rest, make_float2(kTcLift2, kTcLift2), minus_top(ar, br));
            third[q] = round_pack_bf16x2(last.x, last.y);
          }
          tmem_st16(s_col(b) + lanes + h * ST + c * 16, out);
          if constexpr (C::THIRD_TMEM) {
            tmem_st8(third_col(b) + lanes + (h * ST + c * 16) / 2, third);
          } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              *reinterpret_cast<uint4*>(sp + tc_at<128>(row, (h * ST + c * 16) / 8 + q)) =
                  make_uint4(third[4 * q], third[4 * q + 1], third[4 * q + 2], third[4 * q + 3]);
          }
        }
        l = fmaf(l, keep, (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y));
        tmem_wait_st();
        tc_fence_before_sync();
        if (!C::THIRD_TMEM) fence_proxy_async_smem();
        warp_arrive(&sh.pfull[b]);
        kept0 = kept1;
        kept1 = keep;
        ++tile_no;
      }
      if (dead) break;
      tell(l);
      l += learn();
      if (dead) break;
      const bool whole = g.whole();
      const long long slot = whole ? 0 : tree_slot<S>(g, u);
      const int part = g.part(p);
      if (!whole) {
        float4* dst = reinterpret_cast<float4*>(p.partial) + (slot * (HV / 4) + h * (OC / 4)) * 128 + row;
#pragma unroll
        for (int e = 0; e < OC / 4; ++e) {
          constexpr float kOff = 1.f / kTcLift;
          dst[e * 128] = make_float4(o[2 * e].x * kOff, o[2 * e].y * kOff, o[2 * e + 1].x * kOff, o[2 * e + 1].y * kOff);
        }
        if (h == 0) p.stats[slot * 128 + row] = make_float2(m, bad ? -1.f : l);
      } else if (live) {
        if (bad) {
          if (h == 0) atomicOr(p.status, LORA_DEV_BAD_PAGE);
        } else {
          const float inv = 1.f / (l * kTcLift);
          const bool none = l == 0.f;  // nothing seen, or -inf alone: 0, whatever the values
          const int col = part * HV + h * OC;
          T* out = static_cast<T*>(p.out.data) + (g.s.row0 + draft) * p.out.row_stride + head * p.out.head_stride + col;
#pragma unroll
          for (int e = 0; e < OC / 8; ++e)
            if (col + 8 * e < hd) {
              const float2* v = o + 4 * e;
              *reinterpret_cast<uint4*>(out + 8 * e) =
                  none ? make_uint4(0, 0, 0, 0)
                       : make_uint4(round_pack_bf16x2(v[0].x * inv, v[0].y * inv), round_pack_bf16x2(v[1].x * inv, v[1].y * inv),
                                    round_pack_bf16x2(v[2].x * inv, v[2].y * inv), round_pack_bf16x2(v[3].x * inv, v[3].y * inv));
            }
          if (h == 0 && part == 0 && p.lse)
            p.lse[(long long)(g.s.row0 + draft) * p.num_heads + head] = (m + log2f(l)) * kTreeLn2;
        }
      }
      if (strange && live && !bad && l != 0.f) {
        // They went into the products as 0: the rows that see them take them
        // now (where every score is -inf they have no weight).
        const int col = part * HV + h * OC;
        for (int j = max(g.s.ctx, g.t0 * TT); j < min(g.s.len, g.t1 * TT); ++j) {
          const int d = j - g.s.ctx;
          if (!(tree_sees(p, mask, draft, d & ~31, g.s.n) >> (d & 31) & 1)) continue;
          const int pg = (int)(((unsigned long long)(unsigned)j * p.page_magic) >> p.page_shift);
          const T* v = static_cast<const T*>(p.cache.v) + p.tables[g.seq * p.table_stride + pg] * p.cache.page_stride +
                       (j - pg * p.cache.page_size) * p.cache.token_stride + g.kv_head(p) * p.cache.head_stride + col;
          T* out = static_cast<T*>(p.out.data) + (g.s.row0 + draft) * p.out.row_stride + head * p.out.head_stride + col;
          float* sum = p.partial + ((slot * (HV / 4) + h * (OC / 4)) * 128 + row) * 4;
          for (int c = 0; c < min(OC, hd - col); ++c) {
            const float x = __bfloat162float(v[c]);
            if (fabsf(x) < __builtin_huge_valf()) continue;
            if (whole) out[c] = __float2bfloat16_rn(__bfloat162float(out[c]) + x);
            else sum[(c >> 2) * 512 + (c & 3)] += x;
          }
        }
      }
      if (g.t0 == 0 && !whole) split = make_int4(g.seq, g.stream, tree_sharers<S>(p, piece, g, u), 0);
      g.next(p);
    }
    if (dead) sh.fail = 1;
    if (h == 0 && row == 0) p.splits[u] = split;
  } else {
    give_registers<88>();
  if (BOXES && warp < 2) {
    // ---- loads of K (warp 0) or V (warp 1), a box a lane
    const bool is_k = warp == 0;
    const int ns = is_k ? NS : NV;
    uint64_t* full = is_k ? sh.kfull : sh.vfull;
    uint64_t* empty = is_k ? sh.kempty : sh.vempty;
    const void* map = is_k ? &maps.k : &maps.v;
    const int box = maps.rows, blocks = (is_k ? HK : HV) / 64;
    int tile_no = 0, looked = 0;
    // A tile of V that is looked through once it has landed: its stage and
    // flag, first drafted token, tokens.
    struct Look {
      int tile, lo, hi;
      bool open;
    } look{};
    auto look_through = [&] {
      if (!look.open) return;
      look.open = false;
      if (!warp_wait(&sh.land[looked & 1], (looked >> 1) & 1)) dead = true;
      ++looked;
      if (dead) return;
      // Drafted tokens' values that are infinite or NaN would reach rows that
      // do not see them (0 times them is NaN): they become 0 here and the rows
      // that see them take them apart.  What lies behind the last token too.
      unsigned* odd = sh.odd[look.tile % kTcFlags];
      if (lane < 4) odd[lane] = 0;
      __syncwarp();
      uint8_t* st = sv + look.tile % NV * C::V_BYTES;
      for (int e = lane; e < (TT - look.lo) * (HV / 8); e += 32) {
        const int r = look.lo + e / (HV / 8);
        uint4* at = reinterpret_cast<uint4*>(st + tc_at<TT>(r, e % (HV / 8)));
        if (r >= look.hi) {
          *at = make_uint4(0, 0, 0, 0);
          continue;
        }
        const uint4 v = *at;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((w[i] & 0x7f80u) == 0x7f80u) {
            w[i] &= 0xffff0000u;
            any = true;
          }
          if ((w[i] & 0x7f800000u) == 0x7f800000u) {
            w[i] &= 0xffffu;
            any = true;
          }
        }
        if (any) {
          *at = make_uint4(w[0], w[1], w[2], w[3]);
          atomicOr(&odd[r >> 5], 1u << (r & 31));
        }
      }
      __syncwarp();
      fence_proxy_async_smem();
      warp_arrive(&full[look.tile % NV]);
    };
    int issued = 0;  // tiles that are looked through, so far issued
    while (g.valid) {
      const int kv = g.kv_head(p), col = is_k ? 0 : g.part(p) * HV;
      const int* table = p.tables + g.seq * p.table_stride;
      auto look_up = [&](int t) {  // the page of this lane's box
        const int j = min(t * TT + min(lane * box, TT - box), g.s.len - 1);
        return table[(int)(((unsigned long long)(unsigned)j * p.page_magic) >> p.page_shift)];
      };
      int page = look_up(g.t0);
      for (int t = g.t0; t < g.t1; ++t) {
        const int j = t * TT + lane * box, tokens = min(TT, g.s.len - t * TT);
        const bool mine = lane * box < tokens;
        const int slot = j - (int)(((unsigned long long)(unsigned)j * p.page_magic) >> p.page_shift) * p.cache.page_size;
        const bool out = mine && (unsigned)page >= (unsigned)p.cache.num_pages;
        const bool bad = __any_sync(0xffffffffu, out);
        const int from = out ? p.cache.num_pages : page;  // behind the last page: zeros
        if (t + 1 < g.t1) page = look_up(t + 1);
        const int stage = tile_no % ns;
        if (tile_no >= ns) {
          const uint32_t turn = (tile_no / ns - 1) & 1;
          // While the stage is still in use, the tile that has landed is looked through.
          if (look.open && !__all_sync(0xffffffffu, mbar_test(&empty[stage], turn))) look_through();
          if (!dead && !warp_wait(&empty[stage], turn)) dead = true;
        }
        if (dead) break;
        if (is_k && lane == 0) sh.bad[tile_no % kTcFlags] = bad;
        const bool through = !is_k && t * TT + TT > g.s.ctx;
        uint64_t* bar = through ? &sh.land[issued & 1] : &full[stage];
        if (lane == 0) mbar_arrive_expect_tx(bar, (tokens + box - 1) / box * box * blocks * 128);
        __syncwarp();
        if (mine) {
          uint8_t* dst = (is_k ? sk + stage * C::K_BYTES : sv + stage * C::V_BYTES) + lane * box * 128;
          for (int b = 0; b < blocks; ++b) tma_load_4d(dst + b * (TT * 128), map, col + b * 64, slot, kv, from, bar);
        }
        look_through();  // the one before, with these on their way
        if (through) {
          look = Look{tile_no, max(0, g.s.ctx - t * TT), tokens, true};
          ++issued;
        }
        ++tile_no;
      }
      if (dead) break;
      g.next(p);
    }
    look_through();
    if (dead) {  // copies in flight land before the block ends
      if (lane == 0) sh.fail = 1;
      if (look.open) (void)mbar_wait(&sh.land[looked & 1], (looked >> 1) & 1);
      for (int i = max(0, tile_no - ns); i < tile_no; ++i) (void)mbar_wait(&full[i % ns], (i / ns) & 1);
    }
  } else if (!BOXES && warp < 2) {
    // ---- loads of K (warp 0) or V (warp 1): a row is C16 chunks of 16 bytes
    constexpr int RPT = TT / 32;  // rows whose offsets a lane looks up
    const bool is_k = warp == 0;
    const int ns = is_k ? NS : NV;
    uint64_t* full = is_k ? sh.kfull : sh.vfull;
    uint64_t* empty = is_k ? sh.kempty : sh.vempty;
    uint8_t* stages = is_k ? sk : sv;
    const T* src = static_cast<const T*>(is_k ? p.cache.k : p.cache.v);
    int tile_no = 0;  // of this CTA
    // Tiles whose copies are on their way, the oldest first: their drafted
    // tokens, the first and the one behind the last.
    int n0 = 0, n1 = 0, n2 = 0, waiting = 0;
    // The oldest has landed: it is made visible and handed over.
    auto hand_over = [&] {
      if (waiting == 3) cp_async_wait<2>();
      else if (waiting == 2) cp_async_wait<1>();
      else cp_async_wait<0>();
      __syncwarp();
      const int handed = tile_no - waiting, draft_lo = n0 & 0xffff, draft_hi = n0 >> 16;
      if (!is_k && draft_hi > draft_lo) {
        // Drafted tokens' values that are infinite or NaN would reach rows
        // that do not see them (0 times them is NaN): they become 0 here and
        // the rows that see them take them apart.
        unsigned* odd = sh.odd[handed % kTcFlags];
        if (lane < 4) odd[lane] = 0;
        __syncwarp();
        uint8_t* st = stages + handed % NV * C::V_BYTES;
        for (int e = lane; e < (draft_hi - draft_lo) * (HV / 8); e += 32) {
          const int r = draft_lo + e / (HV / 8);
          uint4* at = reinterpret_cast<uint4*>(st + tc_at<TT>(r, e % (HV / 8)));
          const uint4 v = *at;
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          bool any = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if ((w[i] & 0x7f80u) == 0x7f80u) {
              w[i] &= 0xffff0000u;
              any = true;
            }
            if ((w[i] & 0x7f800000u) == 0x7f800000u) {
              w[i] &= 0xffffu;
              any = true;
            }
          }
          if (any) {
            *at = make_uint4(w[0], w[1], w[2], w[3]);
            atomicOr(&odd[r >> 5], 1u << (r & 31));
          }
        }
        __syncwarp();
      }
      fence_proxy_async_smem();
      warp_arrive(&full[handed % ns]);
      n0 = n1;
      n1 = n2;
      --waiting;
    };
    while (g.valid) {
      const int kv = g.kv_head(p);
      const long long head = (long long)kv * p.cache.head_stride + (is_k ? 0 : (long long)g.part(p) * HV);
      const int width = is_k ? hd : min(HV, hd - g.part(p) * HV);  // columns that exist
      const int* table = p.tables + g.seq * p.table_stride;
      auto look_up = [&](int t, int (&page)[RPT]) {
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const int j = min(t * TT + i * 32 + lane, g.s.len - 1);
          page[i] = table[(int)(((unsigned long long)(unsigned)j * p.page_magic) >> p.page_shift)];
        }
      };
      int page[RPT];
      look_up(g.t0, page);
      for (int t = g.t0; t < g.t1; ++t) {
        long long off[RPT];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const int j = t * TT + i * 32 + lane;
          const int n = (int)(((unsigned long long)(unsigned)j * p.page_magic) >> p.page_shift);
          const bool none = j >= g.s.len, out = !none && (unsigned)page[i] >= (unsigned)p.cache.num_pages;
          bad |= out;
          off[i] = none || out ? -1
                               : page[i] * p.cache.page_stride + (long long)(j - n * p.cache.page_size) * p.cache.token_stride + head;
        }
        bad = __any_sync(0xffffffffu, bad);
        if (t + 1 < g.t1) look_up(t + 1, page);
        const int stage = tile_no % ns, flag = tile_no % kTcFlags;
        if (tile_no >= ns && !dead) {
          // While the stage is still in use, what has landed is handed over.
          while (waiting > 0 && !__all_sync(0xffffffffu, mbar_test(&empty[stage], (tile_no / ns - 1) & 1))) hand_over();
          if (!warp_wait(&empty[stage], (tile_no / ns - 1) & 1)) dead = true;
        }
        if (dead) {
          if (lane == 0) sh.fail = 1;
          g.valid = false;
          break;
        }
        if (is_k && lane == 0) sh.bad[flag] = bad;
        uint8_t* st = stages + stage * (is_k ? C::K_BYTES : C::V_BYTES);
        auto copy = [&](auto chunks) {
          constexpr int C16 = decltype(chunks)::value, ROWS = 32 / C16;  // chunks of a row, rows a step
          const int c = lane % C16, sub = lane / C16;
          const bool exists = c * 8 < width;
#pragma unroll 8
          for (int i = 0; i < TT / ROWS; ++i) {
            const int r = i * ROWS + sub;
            const long long o = __shfl_sync(0xffffffffu, off[i * ROWS / 32], r & 31);
            const bool in = o >= 0 && exists;
            cp_async16_zfill(st + tc_at<TT>(r, c), src + (in ? o + c * 8 : 0), in ? 16 : 0);
          }
        };
        if constexpr (HK == HV) {
          copy(std::integral_constant<int, HK / 8>());
        } else {
          if (is_k) copy(std::integral_constant<int, HK / 8>());
          else copy(std::integral_constant<int, HV / 8>());
        }
        cp_async_commit();
        const int note = max(0, min(TT, g.s.ctx - t * TT)) | min(TT, g.s.len - t * TT) << 16;
        if (waiting == 0) n0 = note;
        else if (waiting == 1) n1 = note;
        else n2 = note;
        ++tile_no;
        if (++waiting == min(ns, 3)) hand_over();
      }
      if (g.valid) g.next(p);
    }
    while (waiting > 0) hand_over();
    cp_async_wait<0>();
  } else if (warp == 2) {
    // ---- loads of Q: a chunk's rows, once a segment
    int seg_no = 0;
    while (g.valid) {
      if (seg_no > 0 && !warp_wait(&sh.qempty, (seg_no - 1) & 1)) break;
      const int kv = g.kv_head(p);
      if (BOXES && maps.q_boxes) {
        // Rows behind the sequence's are other sequences' or zero: of no effect.
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.qfull, C::Q_BYTES);
          for (int b = 0; b < HK / 64; ++b)
            tma_load_3d(sq + b * (128 * 128), &maps.q, b * 64, kv * p.group, g.s.row0 + g.chunk() * (128 / p.group), &sh.qfull);
        }
        __syncwarp();
        ++seg_no;
        g.next(p);
        continue;
      }
      const long long row0 = (long long)g.chunk() * 128, rows = (long long)g.s.n * p.group - row0;
      constexpr int C16 = HK / 8, ROWS = 32 / C16;
      const int c = lane % C16, sub = lane / C16;
      for (int i = 0; i < 128 / ROWS; ++i) {
        const int r = i * ROWS + sub;
        const bool in = r < rows && c * 8 < hd;
        const T* src = static_cast<const T*>(p.q.data);
        if (in) {
          const int n = (int)((row0 + r) / p.group), h = kv * p.group + (int)((row0 + r) % p.group);
          src += (g.s.row0 + n) * p.q.row_stride + h * p.q.head_stride + c * 8;
        }
        cp_async16_zfill(sq + tc_at<128>(r, c), src, in ? 16 : 0);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      warp_arrive(&sh.qfull);
      ++seg_no;
      g.next(p);
    }
    cp_async_wait<0>();
  } else if (warp == 3) {
    // ---- the products.  The whole warp goes along, so that what the
    // instructions are given is uniform, and one lane issues them.
    constexpr uint32_t s_idesc = idesc_bf16_f32(128, TT), o_idesc = idesc_bf16_f32(128, HV) | kTransposeB;
    const bool leader = elect_one();
    int seg_no = 0, kt = 0, vt = 0;  // segments, tiles of K and of V so far
    bool ok = true;
    const uint64_t qd = sw128_desc(smem_addr(sq)), kd0 = sw128_desc(smem_addr(sk)),
                   vd0 = sw128_desc_mn(smem_addr(sv), TT * 128), pd = sw128_desc(smem_addr(sp));
    while (ok && __shfl_sync(0xffffffffu, (int)g.valid, 0)) {
      const int n = __shfl_sync(0xffffffffu, g.t1 - g.t0, 0);
      if (!(ok = warp_wait(&sh.qfull, seg_no & 1))) break;
#pragma unroll 1
      for (int i = 0; i <= n; ++i) {
        // A tile's scores go out before the output of the tile before, into
        // the columns whose probabilities the products issued last have read.
        if (i < n) {
          const int st = kt % NS;
          if (!(ok = warp_wait(&sh.kfull[st], (kt / NS) & 1))) break;
          tc_fence_after_sync();
          const uint64_t kd = kd0 + st * (C::K_BYTES / 16);
          const uint32_t d = s_col(kt & 1);
          if (leader) {
#pragma unroll
            for (int k = 0; k < HK / 16; ++k)
              tc_mma_bf16(d, qd + ((k >> 2) * (128 * 128) + (k & 3) * 32) / 16,
                          kd + ((k >> 2) * (TT * 128) + (k & 3) * 32) / 16, s_idesc, k > 0);
            tc_commit(&sh.kempty[st]);
            tc_commit(&sh.sfull[kt & 1]);
            if (i + 1 == n) tc_commit(&sh.qempty);
          }
          __syncwarp();
          ++kt;
        }
        if (i == 0) continue;
        const int b = vt & 1, st = vt % NV;
        if (!(ok = warp_wait(&sh.vfull[st], (vt / NV) & 1))) break;
        if (!(ok = warp_wait(&sh.pfull[b], (vt >> 1) & 1))) break;
        if (vt >= 2 && !(ok = warp_wait(&sh.ofree[b], ((vt >> 1) - 1) & 1))) break;
        tc_fence_after_sync();
        const uint64_t vd = vd0 + st * (C::V_BYTES / 16);
        const uint32_t d = o_col(b), a = s_col(b);
        if (leader) {
          // The third terms, whose place is wanted next; then the others in turn.
#pragma unroll
          for (int k = 0; k < TT / 16; ++k)
            if (C::THIRD_TMEM)
              tc_mma_bf16_ts(d, third_col(b) + k * 8, vd + k * (2048 / 16), o_idesc, k > 0);
            else
              tc_mma_bf16(d, pd + ((k >> 2) * (128 * 128) + (k & 3) * 32) / 16, vd + k * (2048 / 16), o_idesc, k > 0);
          if (!C::THIRD_TMEM) tc_commit(&sh.pfree);
#pragma unroll
          for (int k = 0; k < TT / 8; ++k)
            tc_mma_bf16_ts(d, a + k * 8, vd + (k >> 1) * (2048 / 16), o_idesc, 1u);
          tc_commit(&sh.vempty[st]);
          tc_commit(&sh.ofull[b]);
        }
        __syncwarp();
        ++vt;
      }
      if (!ok) break;
      ++seg_no;
      g.next(p);
    }
    if (leader) {
      if (!ok) sh.fail = 1;
      tc_commit(&sh.done);
    }
    __syncwarp();
  }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 3) {
    (void)mbar_wait(&sh.done, 0);  // products in flight end before their columns are released
    if (sh.fail && lane == 0) atomicOr(p.status, LORA_DEV_TIMEOUT);
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 tree_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// The maps of K, V and Q; false: rows are copied one by one.
template <int TT>
bool encode_maps(const TreeDesc& p, TcMaps* m) {
  const CacheDesc& c = p.cache;
  PFN_cuTensorMapEncodeTiled_v12000 enc = tree_encode_fn();
  m->rows = std::min(TT, c.page_size & -c.page_size);
  if (!enc || m->rows < 8) return false;
  // A dimension of one element has any stride; the map wants a legal one.
  auto stride = [](long long elements, long long count) -> cuuint64_t { return count > 1 ? (cuuint64_t)elements * 2 : 16; };
  auto legal = [](cuuint64_t bytes) { return bytes > 0 && bytes % 16 == 0 && bytes < (1ULL << 40); };
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  auto encode = [&](CUtensorMap* map, int rank, void* data, const cuuint64_t* dims, const cuuint64_t* strides,
                    const cuuint32_t* box) {
    for (int i = 0; i + 1 < rank; ++i)
      if (!legal(strides[i])) return false;
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, data, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
  };
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_kv_heads,
                              (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {stride(c.token_stride, c.page_size), stride(c.head_stride, c.num_kv_heads),
                                 stride(c.page_stride, c.num_pages)};
  const cuuint32_t box[4] = {64, (cuuint32_t)m->rows, 1, 1};
  if (!encode(&m->k, 4, c.k, dims, strides, box) || !encode(&m->v, 4, c.v, dims, strides, box)) return false;
  m->q_boxes = 0;
  if (128 % p.group == 0) {
    const cuuint64_t qdims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)p.num_heads, (cuuint64_t)p.num_rows};
    const cuuint64_t qstrides[2] = {stride(p.q.head_stride, p.num_heads), stride(p.q.row_stride, p.num_rows)};
    const cuuint32_t qbox[3] = {64, (cuuint32_t)p.group, (cuuint32_t)(128 / p.group)};
    m->q_boxes = encode(&m->q, 3, p.q.data, qdims, qstrides, qbox);
  }
  return true;
}

template <int HK, bool BOXES>
cudaError_t launch_tc(TreeDesc p, const TcMaps& maps, void* workspace, cudaStream_t s) {
  using C = TcCfg<HK>;
  static std::atomic<unsigned long long> done{0};
  tree_fill(tree_sizes<typename C::S>(), p, std::min(std::max(device_sm_count(), 1), kMaxSmsForWorkspace), workspace);
  cudaError_t e = tree_allow_smem(tree_tc_kernel<HK, BOXES>, C::SMEM, done);
  if (e != cudaSuccess) return e;
  tree_tc_kernel<HK, BOXES><<<p.pieces, kTcThreads, C::SMEM, s>>>(p, maps);
  if ((e = noted(cudaGetLastError(), LORA_PATH_TC_TREE)) != cudaSuccess) return e;
  return launch_tree_join<typename C::S, __nv_bfloat16>(p, s);
}

template <int HK>
cudaError_t launch_tc(const TreeDesc& p, void* workspace, cudaStream_t s) {
  TcMaps maps{};
  return encode_maps<TcCfg<HK>::TT>(p, &maps) ? launch_tc<HK, true>(p, maps, workspace, s)
                                              : launch_tc<HK, false>(p, maps, workspace, s);
}

}  // namespace

// bf16 rows of whole 16-byte chunks on 16-byte boundaries.  A head wider than
// a stream's part of V is read by several CTAs, so its output may not be its
// query.
bool tree_tc_ok(const TreeDesc& p) {
  const CacheDesc& c = p.cache;
  const auto low = reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) |
                   reinterpret_cast<uintptr_t>(p.q.data) | reinterpret_cast<uintptr_t>(p.out.data);
  return p.dtype == LORA_DTYPE_BF16 && (low & 15) == 0 && c.head_dim % 8 == 0 && c.page_stride % 8 == 0 &&
         c.token_stride % 8 == 0 && c.head_stride % 8 == 0 && p.q.row_stride % 8 == 0 && p.q.head_stride % 8 == 0 &&
         p.out.row_stride % 8 == 0 && p.out.head_stride % 8 == 0 && !(c.head_dim > 128 && p.q.data == p.out.data);
}

size_t tree_tc_workspace(const TreeDesc& p) {
  auto bytes = [&](auto cfg) {
    const TreeSizes z = tree_sizes<typename decltype(cfg)::S>();
    return tree_bytes(z, tree_pieces(z, p, kMaxSmsForWorkspace));
  };
  const int hd = p.cache.head_dim;
  return hd <= 64 ? bytes(TcCfg<64>{}) : hd <= 128 ? bytes(TcCfg<128>{}) : bytes(TcCfg<256>{});
}

cudaError_t launch_tree_tc(TreeDesc p, void* workspace, cudaStream_t s) {
  if (p.cache.head_dim <= 64) return launch_tc<64>(p, workspace, s);
  if (p.cache.head_dim <= 128) return launch_tc<128>(p, workspace, s);
  return launch_tc<256>(p, workspace, s);
}

}  // namespace lora
