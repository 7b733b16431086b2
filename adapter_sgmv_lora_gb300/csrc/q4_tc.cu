// q4_tc.cu -- the 4-bit base projection on tcgen05, for batches of more rows
// than q4.cu's kernels take at their best.
//
// A CTA has 128 outputs (the lanes of TMEM) and up to 128 rows of the batch
// (columns).  Weights are unpacked once for all of them into bf16 code - zero,
// which is exact, in the swizzled layout the products read; x comes beside them
// by asynchronous copies.  A group's sum (or every 128 inputs') goes through
//   S = (code - zero) x^T   into one of two TMEM buffers
//   y += scale S            in registers, fp32: an output is a lane, so its
//                           scale is one number a thread
// so a weight is never rounded.  The delta is more of the same: 32 ranks of a
// slot's B beside themselves against u as two bf16 terms, scale 1, taken over by
// the columns of the slot's rows alone, so that what other slots hold cannot
// reach them.  Against u's second term, which may be zero or of the other sign,
// an element of B that is not finite counts as zero: against the first it gives
// its infinity or NaN.
//
// Warps 0 to 7 hold y, 8 to 15 load and unpack, 16 issues the products, 17 loads
// x.  The unpacking warps work in pairs, each pair on every fourth block: a
// block's copies, waits and barriers take longer than its arithmetic, so several
// are under way (all eight on one block at a time: gate and up of the 8B model,
// 28672 outputs of 4096 inputs, 128 rows, 146 us, so 119; the delta's planes
// summed by all of them and one thread issuing the products: 92).  Every wait is
// bounded.
//
// Gate and up take 82 us for 64 rows, 96 for 128, 143 for 256; q4.cu's tiles
// 122, 229 and 441.  What bounds it is the way of a block through the barriers,
// some 800 cycles whatever the rows: leaving out the unpacking saves 8%, with
// three of four products and of the stores 15%, the scaling or x nothing.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "ptx.cuh"
#include "q4.cuh"
#include "tiles.cuh"

namespace lora {
namespace {

constexpr int kOuts = 128, kRowsMost = 128, kK = 64, kStagesMost = 8;
constexpr int kFold = 8, kProd = 8, kGroups = 4, kThreads = (kFold + kProd + 2) * 32;
constexpr int kWBytes = kOuts * kK * 2;
constexpr int kRaw = 3, kRawBytes = kOuts * kK / 2;  // a pair's blocks of packed weights on their way
constexpr int kRing = kGroups * kRaw * kRawBytes, kSmemMost = 225 * 1024;  // beside 2 KB that are not dynamic

struct Shared {
  uint64_t full[kStagesMost], empty[kStagesMost], sum[2], taken[2], done;
  uint32_t tmem;
  int ok, fail, runs;
  int slot[kRowsMost];
  int begin[kRowsMost + 1];  // runs of rows of one slot
  int ranks[kRowsMost];      // theirs; 0 without adapter
};

// The delta's blocks in order: 32 ranks of a run of rows, the ranks in spans of
// kSpan, whose part of u the unpacking warps sum into shared memory first.
constexpr int kSpan = 64;
template <typename F>
__device__ __forceinline__ void delta_blocks(const Shared& sh, int span, F&& f) {
#pragma unroll 1
  for (int run = 0; run < sh.runs; ++run) {
    const int end = min(sh.ranks[run], span + kSpan);
#pragma unroll 1
    for (int k0 = span; k0 < end; k0 += 32)
      if (!f(run, k0)) return;
  }
}

static_assert(sizeof(Shared) <= 2048 && kRowsMost * (kSpan + 4) * 4 <= kRing, "shared memory");

// One lane speaks for its warp; all of it waits.
__device__ __forceinline__ void arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ bool wait(uint64_t* bar, int use) {
  bool ok = false;
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit && !ok; ++i) ok = __all_sync(0xffffffffu, mbar_try_wait(bar, use & 1));
  return ok;
}

__device__ __forceinline__ void loaders_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kProd * 32) : "memory"); }

// 16-byte chunk c of row r of a block of 64 columns, 128-byte swizzle.
__device__ __forceinline__ int at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// A word's 8 codes in order; low: 128 + zero, twice.
__device__ __forceinline__ uint4 unpack_in_order(uint32_t w, uint32_t low) {
  const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
  auto pair = [&](uint32_t order) {
    return sub_bf16x2((__byte_perm(even, odd, order) & 0x000f000fu) | 0x43004300u, low);
  };
  return make_uint4(pair(0x4400), pair(0x5511), pair(0x6622), pair(0x7733));
}

// Zero in the place of what is infinite or NaN.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v) {
  const uint32_t none = sub_bf16x2(v, v);  // 0, or NaN
  return v & __heq2_mask(*reinterpret_cast<const __nv_bfloat162*>(&none), __nv_bfloat162(0.f, 0.f));
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// FOLD: blocks of 64 inputs whose products are summed before they are scaled.
template <int FOLD>
__global__ void __launch_bounds__(kThreads, 1)
    q4_tc_kernel(const __grid_constant__ ProblemDesc p, const __grid_constant__ Q4Weights wts,
                 const __grid_constant__ Q4Work w, const __grid_constant__ CUtensorMap xmap, int tile_rows, int stages,
                 const float* __restrict__ u) {
  using T = __nv_bfloat16;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Shared sh;
  uint8_t* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  const int stage_bytes = kWBytes + tile_rows * kK * 2;
  uint8_t* ring = smem + stages * stage_bytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (w.wait_first) pdl_wait();
  int j = 0;
  while (j + 1 < p.n_slices && (int)blockIdx.x >= w.blk_begin[j + 1]) ++j;
  const SliceDesc& sl = p.sl[j];
  const Q4Desc& d = wts.w[j];
  const int o0 = (blockIdx.x - w.blk_begin[j]) * kOuts, t0 = blockIdx.y * tile_rows;
  const int rows = min(tile_rows, p.num_tokens - t0), cols = (rows + 15) & ~15;
  const int nb = (p.in_dim + kK - 1) / kK;

  // The packed weights need nobody: their copies start first.  A thread unpacks
  // what it copies: two outputs' 64 inputs, 64 outputs apart.
  const int pair = (warp - kFold) >> 1, r = threadIdx.x & 63;
  const long long out[2] = {min(o0 + r, sl.out_dim - 1), min(o0 + r + 64, sl.out_dim - 1)};
  uint8_t* mine = ring + (pair * kRaw * 4 * 64 + r) * 16;
  auto load_q = [&](int b, int slot) {
    if (b < nb) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool in = b * kK + (c & 1) * 32 < p.in_dim;
        const uint8_t* q = d.q + out[c >> 1] * d.q_stride;
        cp_async16_zfill(mine + (slot * 4 + c) * 1024, in ? q + b * (kK / 2) + (c & 1) * 16 : q, in ? 16 : 0);
      }
    }
    cp_async_commit();
  };
  const bool loads = warp >= kFold && warp < kFold + kProd;
  if (loads)
    for (int n = 0; n < kRaw - 1; ++n) load_q(pair + n * kGroups, n);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sh.full[i], 3);  // a pair of warps, and x's loader
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sum[i], 1);
      mbar_init(&sh.taken[i], kFold);
    }
    mbar_init(&sh.done, 1);
    fence_mbar_init();
    sh.fail = 0;
  }
  const int routed = min(max(p.end - t0, 0), rows);
  if (warp == 1) {
    const bool ok = p.G == 0 || warp_check_routing(p);
    if (lane == 0) sh.ok = ok;
  } else if (warp == kFold + kProd) {
    tmem_alloc(&sh.tmem, 256);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const bool good = sh.ok;
  if (threadIdx.x < kRowsMost)
    sh.slot[threadIdx.x] = good && (int)threadIdx.x < routed ? p.lora_ids[group_of_row(p, t0 + threadIdx.x)] : -1;
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int c = 0; c < kRowsMost; c += 32) {
      const int row = c + lane;
      const bool starts = row < routed && (row == 0 || sh.slot[row] != sh.slot[row - 1]);
      const unsigned all = __ballot_sync(0xffffffffu, starts);
      if (starts) {
        const int i = n + __popc(all & ((1u << lane) - 1)), slot = sh.slot[row];
        sh.begin[i] = row;
        sh.ranks[i] = slot >= 0 ? slot_kmax(p, slot) : 0;
      }
      n += __popc(all);
    }
    if (lane == 0) {
      sh.begin[n] = routed;
      sh.runs = n;
    }
  }
  __syncthreads();
  const uint32_t tmem = sh.tmem;
  bool ok = good;

  if (loads) {
    const bool wide_b = p.R % 8 == 0 && ((reinterpret_cast<uintptr_t>(sl.B) | (uintptr_t)(sl.B_slot_stride * 2)) & 15) == 0;
    auto zero_of = [&](int i, int b) { return d.zeros && b < nb ? d.zeros[out[i] * d.z_stride + b * kK / d.group] : 8; };
    int coming[2] = {zero_of(0, pair), zero_of(1, pair)};
    int slot = 0;
#pragma unroll 1
    for (int b = pair; b < nb && ok; b += kGroups) {
      load_q(b + (kRaw - 1) * kGroups, slot == 0 ? kRaw - 1 : slot - 1);
      const int zero[2] = {coming[0], coming[1]};
#pragma unroll
      for (int i = 0; i < 2; ++i) coming[i] = zero_of(i, b + kGroups);
      const int use = b / stages, st = b - use * stages;
      if (use > 0) ok = wait(&sh.empty[st], use - 1);
      if (!ok) break;
      cp_async_wait<kRaw - 1>();
      uint8_t* dst = smem + st * stage_bytes;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int near = min(zero[c >> 1], 127), rest = zero[c >> 1] - near;
        const uint32_t low = small_bf16(128 + near) * 0x10001u;
        const uint4 q = *reinterpret_cast<const uint4*>(mine + (slot * 4 + c) * 1024);
        const uint32_t words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 v = unpack_in_order(words[e], low);
          if (rest) {  // a zero past 127
            const uint32_t far = small_bf16(rest) * 0x10001u;
            v = make_uint4(sub_bf16x2(v.x, far), sub_bf16x2(v.y, far), sub_bf16x2(v.z, far), sub_bf16x2(v.w, far));
          }
          *reinterpret_cast<uint4*>(dst + at(r + (c >> 1) * 64, (c & 1) * 4 + e)) = v;
        }
      }
      fence_proxy_async_smem();
      arrive(&sh.full[st]);
      slot = slot == kRaw - 1 ? 0 : slot + 1;
    }
    cp_async_wait<0>();
    // The delta's blocks.
    if (!w.wait_first) pdl_wait();  // u comes from the shrink
    int i = nb;
    float* s_u = reinterpret_cast<float*>(ring);  // [rows][kSpan + 4]; the copies through it are over
    constexpr int pitch = kSpan + 4;
    for (int span = 0; span < p.R && routed > 0 && good; span += kSpan) {
      loaders_sync();
      const float* ur = u + ((long long)t0 * p.n_slices + j) * p.R + span;
      const int ranks = min(kSpan, p.R - span);
#pragma unroll 4
      for (int e = threadIdx.x - kFold * 32; e < routed * ranks; e += kProd * 32) {
        const int row = e / ranks, k = e - row * ranks;
        const float* from = ur + (long long)row * p.n_slices * p.R + k;
        float v = 0.f;
#pragma unroll 4
        for (int c = 0; c < w.nsplit; ++c) v += __ldcg(from + c * w.plane_stride);
        s_u[row * pitch + k] = v;
      }
      loaders_sync();
      if (!ok) continue;
      delta_blocks(sh, span, [&](int run, int k0) {
        if (i % kGroups != pair) {
          ++i;
          return true;
        }
        const int first = sh.begin[run], last = sh.begin[run + 1], ranks = sh.ranks[run];
        const int use = i / stages, st = i - use * stages;
        if (use > 0) ok = wait(&sh.empty[st], use - 1);
        if (!ok) return false;
        uint8_t* dst = smem + st * stage_bytes;
        const T* slot_b = static_cast<const T*>(sl.B) + sh.slot[first] * sl.B_slot_stride;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int k = k0 + (c & 3) * 8;
          const T* b = slot_b + out[c >> 2] * p.R + k;
          uint4 v;
          if (wide_b && k + 8 <= ranks) {
            v = __ldg(reinterpret_cast<const uint4*>(b));
          } else {
            uint32_t bits[4] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (k + e < ranks) bits[e / 2] |= (uint32_t)__bfloat16_as_ushort(b[e]) << (e % 2 * 16);
            v = make_uint4(bits[0], bits[1], bits[2], bits[3]);
          }
          *reinterpret_cast<uint4*>(dst + at(r + (c >> 2) * 64, c & 3)) = v;
          *reinterpret_cast<uint4*>(dst + at(r + (c >> 2) * 64, 4 + (c & 3))) =
              make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z), finite_bf16x2(v.w));
        }
        // u as two terms, of rows outside the run zero.
        const int k = k0 + (r & 3) * 8;
#pragma unroll 1
        for (int row = r >> 2; row < cols; row += 16) {
          uint32_t hi[4] = {}, lo[4] = {};
          if (row >= first && row < last) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float v = k + e < ranks ? s_u[row * pitch + k - span + e] : 0.f;
              const __nv_bfloat16 top = __float2bfloat16_rn(v);
              const float back = __bfloat162float(top);  // infinite or NaN: no second term
              const __nv_bfloat16 rest = __float2bfloat16_rn(isfinite(back) ? v - back : 0.f);
              hi[e / 2] |= (uint32_t)__bfloat16_as_ushort(top) << (e % 2 * 16);
              lo[e / 2] |= (uint32_t)__bfloat16_as_ushort(rest) << (e % 2 * 16);
            }
          }
          *reinterpret_cast<uint4*>(dst + kWBytes + at(row, r & 3)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(dst + kWBytes + at(row, 4 + (r & 3))) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        arrive(&sh.full[st]);
        ++i;
        return true;
      });
    }
    if (!ok && good && lane == 0) sh.fail = 1;
  } else if (warp == kFold + kProd + 1) {
    if (good && lane == 0) {
      const uint32_t bytes = tile_rows * kK * 2;
      const uint64_t policy = policy_evict_last();
      int st = 0, use = 0;
      auto free_stage = [&] { return use == 0 || mbar_wait(&sh.empty[st], (use - 1) & 1); };
      auto next = [&] {
        if (++st == stages) {
          st = 0;
          ++use;
        }
      };
      for (int i = 0; i < nb && (ok = free_stage()); ++i) {
        mbar_arrive_expect_tx(&sh.full[st], bytes);
        tma_load_2d_hint(smem + st * stage_bytes + kWBytes, &xmap, i * kK, t0, &sh.full[st], policy);
        next();
      }
      // The delta's blocks come whole from the other warps.
      for (int span = 0; span < p.R && ok; span += kSpan)
        delta_blocks(sh, span, [&](int, int) {
          if ((ok = free_stage())) {
            mbar_arrive(&sh.full[st]);
            next();
          }
          return ok;
        });
      if (!ok) {  // a bounded wait for the copies in flight
        sh.fail = 1;
        const int last = st == 0 ? stages - 1 : st - 1;
        (void)mbar_wait(&sh.full[last], (st == 0 ? use - 1 : use) & 1);
      }
    }
    __syncwarp();
  } else if (warp == kFold + kProd) {
    const uint32_t idesc = idesc_bf16_f32(kOuts, 16) - ((16u >> 3) << 17) + ((uint32_t)(cols >> 3) << 17);
    int i = 0, m = 0;  // block, sum
    int stage = 0, turn = 0;
    const uint64_t a0 = sw128_desc(smem_addr(smem)), x0 = sw128_desc(smem_addr(smem) + kWBytes);
    uint64_t a = a0, x = x0;
    auto block = [&](bool first, bool last) {
      if (first && m >= 2) ok = mbar_wait(&sh.taken[m & 1], ((m >> 1) - 1) & 1);
      ok = ok && mbar_wait(&sh.full[stage], turn);
      if (!ok) return;
      tc_fence_after_sync();
      const uint32_t to = tmem + (m & 1) * 128;
      tc_mma_bf16(to, a, x, idesc, first ? 0u : 1u);
#pragma unroll
      for (int ks = 1; ks < kK / 16; ++ks) tc_mma_bf16(to, a + ks * 2, x + ks * 2, idesc, 1u);
      tc_commit(&sh.empty[stage]);
      if (last) tc_commit(&sh.sum[m & 1]);
      ++i;
      m += last;
      a += stage_bytes >> 4;
      x += stage_bytes >> 4;
      if (++stage == stages) {
        stage = 0;
        turn ^= 1;
        a = a0;
        x = x0;
      }
    };
    // An elected thread, not lane 0: the products' operands are then known to be
    // the warp's (trees on the 70B qkv 191 us, so 172).
    if (elect_one()) {
      while (i < nb && ok) block(i % FOLD == 0, i % FOLD == FOLD - 1 || i == nb - 1);
      for (int span = 0; span < p.R && ok; span += kSpan)
        delta_blocks(sh, span, [&](int, int) {
          block(true, true);
          return ok;
        });
      if (!ok && good) sh.fail = 1;
      tc_commit(&sh.done);
    }
    __syncwarp();
  } else {
    // Two warps share a quarter of the outputs: sixteens of columns by turns.
    const int half = warp >> 2, o = o0 + (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const uint16_t* scales = static_cast<const uint16_t*>(d.scales) + min(o, sl.out_dim - 1) * d.s_stride;
    // The slots' B rows of these outputs are wanted at the end: into L2 now.
    for (int run = warp; run < sh.runs; run += kFold)
      if (sh.ranks[run] > 0) {
        const char* b = static_cast<const char*>(sl.B) + (sh.slot[sh.begin[run]] * sl.B_slot_stride + (long long)o0 * p.R) * 2;
        const int bytes = min(kOuts, sl.out_dim - o0) * p.R * 2;
        for (int e = lane * 128; e < bytes; e += 32 * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(b + e));
      }
    float y[kRowsMost / 2] = {};
    const int units = (nb + FOLD - 1) / FOLD;
    // Scales are read four sums ahead of their use.
    auto scale_of = [&](int m) { return m < units ? __ldg(scales + m * FOLD * kK / d.group) : (uint16_t)0; };
    uint16_t ahead[4] = {scale_of(0), scale_of(1), scale_of(2), scale_of(3)};
    int m = 0;
#pragma unroll 1
    for (int m0 = 0; m0 < units && ok; m0 += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (m >= units || !ok) break;
        const float scale = __uint_as_float((uint32_t)ahead[i] << 16);
        ahead[i] = scale_of(m + 4);
        if (!(ok = wait(&sh.sum[m & 1], m / 2))) break;
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < kRowsMost / 32; ++c) {
          const int col = (2 * c + half) * 16;
          if (col < cols) {
            float s[16];
            tmem_ld16(lanes + (m & 1) * 128 + col, s);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[c * 16 + e] = fmaf(scale, s[e], y[c * 16 + e]);
          }
        }
        tc_fence_before_sync();
        arrive(&sh.taken[m & 1]);
        ++m;
      }
    }
    for (int span = 0; span < p.R && ok; span += kSpan)
      delta_blocks(sh, span, [&](int run, int) {
        const int first = sh.begin[run], last = sh.begin[run + 1];
        if (!(ok = wait(&sh.sum[m & 1], m / 2))) return false;
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < kRowsMost / 32; ++c) {
          const int col = (2 * c + half) * 16;
          if (col < last && col + 16 > first) {
            float s[16];
            tmem_ld16(lanes + (m & 1) * 128 + col, s);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (col + e >= first && col + e < last) y[c * 16 + e] += s[e];
          }
        }
        tc_fence_before_sync();
        arrive(&sh.taken[m & 1]);
        ++m;
        return true;
      });
    if (!ok && good && lane == 0) sh.fail = 1;
    if (ok && o < sl.out_dim) {
      if (!w.wait_first) pdl_wait();
      T* dst = static_cast<T*>(sl.y) + (long long)t0 * sl.y_row_stride + o;
      const T* bias = sl.bias ? static_cast<const T*>(sl.bias) + o : nullptr;
#pragma unroll
      for (int c = 0; c < kRowsMost / 32; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int row = (2 * c + half) * 16 + e;
          if (row >= rows) continue;
          float v = y[c * 16 + e];
          if (bias && sh.slot[row] >= 0) v += __bfloat162float(bias[sh.slot[row] * sl.bias_slot_stride]);
          dst[row * sl.y_row_stride] = __float2bfloat16_rn(v);
        }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kFold + kProd) {
    (void)mbar_wait(&sh.done, 0);  // products in flight end before their columns are released
    if (sh.fail && lane == 0) atomicOr(p.status, LORA_DEV_TIMEOUT);
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 256);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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

template <int FOLD>
cudaError_t launch(const ProblemDesc& p, const Q4Weights& wts, const Q4Work& w, const float* u, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(q4_tc_kernel<FOLD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
  }
  const int tiles = (p.num_tokens + kRowsMost - 1) / kRowsMost;
  const int tile_rows = ((p.num_tokens + tiles - 1) / tiles + 15) / 16 * 16;
  const int stage_bytes = kWBytes + tile_rows * kK * 2;
  const int stages = std::min(kStagesMost, (kSmemMost - 1024 - kRing) / stage_bytes);
  // x as boxes of 64 inputs by a tile's rows; rows and inputs past the last are zero.
  CUtensorMap xmap;
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  const cuuint64_t dims[2] = {(cuuint64_t)p.in_dim, (cuuint64_t)p.num_tokens};
  const cuuint64_t stride[1] = {(cuuint64_t)p.x_row_stride * 2};
  const cuuint32_t box[2] = {kK, (cuuint32_t)tile_rows}, ones[2] = {1, 1};
  if (!enc || stride[0] >= (1ULL << 40) ||
      enc(&xmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p.x), dims, stride, box, ones,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(w.blk_begin[p.n_slices], (p.num_tokens + tile_rows - 1) / tile_rows);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = stages * stage_bytes + kRing + 1024;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return noted(cudaLaunchKernelEx(&cfg, q4_tc_kernel<FOLD>, p, wts, w, xmap, tile_rows, stages, u), LORA_PATH_TC_Q4);
}

}  // namespace

bool q4_tc_ok(const ProblemDesc& p, const Q4Weights& w) {
  const long long row_tiles = (p.num_tokens + kRowsMost - 1) / kRowsMost, sms = std::max(device_sm_count(), 1);
  if (row_tiles > 65535 || p.in_dim < kK || p.x_row_stride < p.in_dim) return false;
  long long tiles = 0, small = 0;
  for (int j = 0; j < p.n_slices; ++j) {
    if (w.w[j].group < p.in_dim && w.w[j].group % kK != 0) return false;
    tiles += (p.sl[j].out_dim + kOuts - 1) / kOuts;
    small += (p.sl[j].out_dim + 31) / 32;
  }
  // A wave of this kernel takes what two and a half of q4.cu's 32 x 32 tiles do,
  // two to an SM.  us here and there, 4096 inputs, rank 32: 4096 outputs 54
  // and 46 (128 rows), 47 and 59 (160), 55 and 151 (512); 10240 outputs 42 and 54
  // (48), 65 and 108 (128), 175 and 387 (512); 28672 outputs 80 and 68 (32), 81
  // and 121 (48), 119 and 272 (128), 375 and 1052 (512).
  const long long waves = (tiles * row_tiles + sms - 1) / sms;
  const long long there = (small * ((p.num_tokens + 31) / 32) + 2 * sms - 1) / (2 * sms);
  return p.num_tokens > 16 && 2 * there > 5 * waves;
}

cudaError_t launch_q4_tc(const ProblemDesc& p, const Q4Weights& wts, Q4Work w, const float* u, cudaStream_t s) {
  int blocks = 0;
  bool wide = true;  // groups of whole 128s: twice the products before a sum is scaled
  for (int j = 0; j < p.n_slices; ++j) {
    w.blk_begin[j] = blocks;
    blocks += (p.sl[j].out_dim + kOuts - 1) / kOuts;
    wide = wide && (wts.w[j].group >= p.in_dim || wts.w[j].group % (2 * kK) == 0);
  }
  w.blk_begin[p.n_slices] = blocks;
  return wide ? launch<2>(p, wts, w, u, s) : launch<1>(p, wts, w, u, s);
}

}  // namespace lora
