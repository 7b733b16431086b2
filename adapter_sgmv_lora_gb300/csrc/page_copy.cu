// page_copy.cu -- copies listed pages of every layer's K and V
// (lora_kv_copy_pages).  Bounded by memory: each byte is read once and
// written once.
//
// The list of pages and the layers' pointers travel as launch parameters (no
// upload, so a call is one launch per table-full of copies).  A page is
// `outer` x `mid` runs of `run` contiguous units: its three inner dimensions,
// merged where one continues the other, so a dense page is a single run.
//
// Stores are streaming (evicted first), so they do not push a forked source
// out of L2 between its copies: 192 copies of 12 pages in 32 layers 71.7 us
// against 77.6 (5.97 TB/s; the counters show DRAM 72% busy, 5.1 TB/s of writes),
// 900 moves in 32 layers 543 us either way (6.95 TB/s).
#include <algorithm>
#include <cuda_bf16.h>
#include <utility>

#include "internal.h"

namespace lora {
namespace {

constexpr int kMaxTensors = 128;  // K and V of 64 layers a launch
constexpr int kMaxCopies = 1024;  // pages a launch
constexpr int kFewCopies = 32;    // a short list goes in a small launch parameter
constexpr int kThreads = 256;
constexpr int kUnroll = 4;        // units in flight per thread

template <int COPIES>
struct CopyTable {
  void* tensor[kMaxTensors];
  int2 page[COPIES];  // source, destination
};

struct PageShape {  // in units of the copy
  long long page_stride, outer_stride, mid_stride;
  long long outer, mid, run;
};

// grid.x: chunks of a page; grid.y: tensors; grid.z: pages, `together` of them
// to a block where they are small (an eighth of a block's threads had work on
// pages of one token: 2617 of them in 5 layers 29 us, together 19).
// DENSE: the page is one run.  I: the index type within a page (32 bits unless
// the page has more units).
template <typename U, bool DENSE, typename I, int COPIES>
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyTable<COPIES> table,
                                                              const __grid_constant__ PageShape g, int pages,
                                                              int together) {
  U* base = static_cast<U*>(table.tensor[blockIdx.y]);
  const int page0 = blockIdx.z * together;
  const I run = (I)g.run, per_outer = (I)(g.mid * g.run), total = (I)(g.outer * g.mid * g.run);
  const I all = total * (I)min(together, pages - page0);
  const I first = (I)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  U v[kUnroll];
  U* dst[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    I e = first + i * kThreads;
    if (e < all) {
      int n = page0;
      if (together > 1) {
        n += (int)(e / total);
        e -= (I)(n - page0) * total;
      }
      long long at = e;
      if constexpr (!DENSE) {
        const I o = e / per_outer, r = e - o * per_outer, m = r / run;
        at = o * g.outer_stride + m * g.mid_stride + (r - m * run);
      }
      const int2 page = table.page[n];
      v[i] = base[page.x * g.page_stride + at];
      dst[i] = base + page.y * g.page_stride + at;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i)
    if (first + i * kThreads < all) __stcs(dst[i], v[i]);
}

template <typename U, int COPIES>
cudaError_t run(const CopyTable<COPIES>& t, const PageShape& g, int tensors, int pages, cudaStream_t s) {
  const long long total = g.outer * g.mid * g.run, chunk = (long long)kThreads * kUnroll;
  const int together = (int)std::max(1LL, chunk / total);
  const dim3 grid((unsigned)((total + chunk - 1) / chunk), tensors, (pages + together - 1) / together);
  const bool dense = g.outer * g.mid == 1;
  if (total > (1LL << 31)) copy_pages_kernel<U, false, long long, COPIES><<<grid, kThreads, 0, s>>>(t, g, pages, 1);
  else if (dense) copy_pages_kernel<U, true, unsigned, COPIES><<<grid, kThreads, 0, s>>>(t, g, pages, together);
  else copy_pages_kernel<U, false, unsigned, COPIES><<<grid, kThreads, 0, s>>>(t, g, pages, together);
  return noted(cudaGetLastError(), LORA_PATH_PAGES);
}

// One launch: np copies in nc layers.
template <int COPIES>
cudaError_t launch_table(const PageShape& g, int unit, const lora_kv_cache_t* caches, int nc, const int* src,
                         const int* dst, int np, cudaStream_t s) {
  CopyTable<COPIES> t;
  for (int i = 0; i < nc; ++i) {
    t.tensor[2 * i] = caches[i].k;
    t.tensor[2 * i + 1] = caches[i].v;
  }
  for (int i = 0; i < np; ++i) t.page[i] = make_int2(src[i], dst[i]);
  switch (unit) {
    case 16: return run<uint4>(t, g, 2 * nc, np, s);
    case 8: return run<uint2>(t, g, 2 * nc, np, s);
    case 4: return run<unsigned>(t, g, 2 * nc, np, s);
    default: return run<unsigned short>(t, g, 2 * nc, np, s);
  }
}

}  // namespace

cudaError_t launch_copy_pages(const CacheDesc& c, int dtype, const lora_kv_cache_t* caches, int num_caches,
                              const int* src, const int* dst, int n, cudaStream_t s) {
  // Inner dimensions of a page in bytes, smallest stride first; merged while
  // contiguous.
  const long long es = dtype == LORA_DTYPE_BF16 ? 2 : 4;
  std::pair<long long, int> a{c.token_stride * es, c.page_size}, b{c.head_stride * es, c.num_kv_heads};
  if (a.second == 1) std::swap(a, b);  // b is the dimension of one, if any is
  if (b.second > 1 && b.first < a.first) std::swap(a, b);
  long long run_bytes = c.head_dim * es;
  if (a.second > 1 && a.first == run_bytes) {
    run_bytes *= a.second;
    a = b;
    b = {0, 1};
    if (a.second > 1 && a.first == run_bytes) {
      run_bytes *= a.second;
      a = {0, 1};
    }
  }
  const long long page_bytes = c.page_stride * es;
  // The widest unit that every address and length is a multiple of.
  unsigned long long low = (unsigned long long)run_bytes | (a.second > 1 ? a.first : 0) | (b.second > 1 ? b.first : 0) |
                           (c.num_pages > 1 ? page_bytes : 0) | 16;
  for (int i = 0; i < num_caches; ++i)
    low |= reinterpret_cast<unsigned long long>(caches[i].k) | reinterpret_cast<unsigned long long>(caches[i].v);
  const long long unit = (long long)(low & (~low + 1));
  const PageShape g{page_bytes / unit, b.first / unit, a.first / unit, b.second, a.second, run_bytes / unit};
  for (int c0 = 0; c0 < num_caches; c0 += kMaxTensors / 2) {
    const int nc = std::min(num_caches - c0, kMaxTensors / 2);
    for (int p0 = 0; p0 < n; p0 += kMaxCopies) {
      const int np = std::min(n - p0, kMaxCopies);
      const cudaError_t e =
          np <= kFewCopies ? launch_table<kFewCopies>(g, (int)unit, caches + c0, nc, src + p0, dst + p0, np, s)
                           : launch_table<kMaxCopies>(g, (int)unit, caches + c0, nc, src + p0, dst + p0, np, s);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace lora
