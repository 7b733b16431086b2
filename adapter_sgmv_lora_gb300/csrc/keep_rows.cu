// keep_rows.cu -- moves the cache rows of an accepted branch of drafted tokens
// up behind the context, in every layer's K and V (lora_kv_keep_rows).  Each
// moved byte is read once and written once.
//
// A path ascends, so row context + path[k] never lies before row context + k:
// moving in the order of k, a row is overwritten only after it was read.  A
// thread moves its own column (one unit of a row) of every row of the path, a
// batch of rows at a time with the loads ahead of the stores, so no two
// threads touch the same address and nothing has to be synchronised.  Seven of 8
// to 40 drafted tokens of 64 sequences in 32 layers, 8 x 128 wide: 14.5 us, 4.1
// TB/s (start, path and table take 4 of them: one sequence 4.9 us).
#include <algorithm>
#include <cuda_bf16.h>

#include "internal.h"

namespace lora {
namespace {

constexpr int kMaxTensors = 128;  // K and V of 64 layers a launch
constexpr int kThreads = 128;
constexpr int kBatch = 8;         // rows in flight per thread

struct KeepTable {
  void* tensor[kMaxTensors];
};

// grid.x: sequences; grid.y: tensors; grid.z: shares of a row's units.
// per_head: units of a head; strides in units.
template <typename U>
__global__ void __launch_bounds__(kThreads) keep_rows_kernel(const __grid_constant__ KeepTable table,
                                                             const __grid_constant__ KeepDesc p, int per_head,
                                                             long long page_stride, long long token_stride,
                                                             long long head_stride, int report) {
  __shared__ long long s_src[LORA_MAX_KEPT], s_dst[LORA_MAX_KEPT];
  __shared__ unsigned s_bad;
  __shared__ int s_kept;
  const int b = blockIdx.x;
  const int len = p.lengths[b], first = p.offsets[b];
  const long long n = (long long)p.offsets[b + 1] - first;
  const int* path = p.path + b * p.path_stride;
  if (threadIdx.x == 0) {
    // Without drafted tokens nothing is read, whatever the length, and the length stays.
    s_bad = (first < 0 || n < 0 || (n > 0 && (len < n || len > p.max_len))) ? LORA_DEV_BAD_LENGTH : 0u;
    s_kept = p.max_kept;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < p.max_kept; k += kThreads)
    if (path[k] == -1) atomicMin(&s_kept, k);
  __syncthreads();
  const int kept = s_kept;
  const long long ctx = len - n;
  if (s_bad == 0) {  // the same for the whole block: set before the barriers
    unsigned bad = 0;
    for (int k = threadIdx.x; k < kept; k += kThreads) {
      const int node = path[k];
      if (node < 0 || node >= n || (k > 0 && path[k - 1] >= node)) {
        bad |= LORA_DEV_BAD_ROW;
        continue;
      }
      const long long src = ctx + node, dst = ctx + k;
      const int* row = p.tables + b * p.table_stride;
      const int sp = row[src / p.cache.page_size], dp = row[dst / p.cache.page_size];
      if ((unsigned)sp >= (unsigned)p.cache.num_pages || (unsigned)dp >= (unsigned)p.cache.num_pages)
        bad |= LORA_DEV_BAD_PAGE;
      s_src[k] = sp * page_stride + (src % p.cache.page_size) * token_stride;
      s_dst[k] = dp * page_stride + (dst % p.cache.page_size) * token_stride;
    }
    __syncthreads();
    if (bad) atomicOr(&s_bad, bad);
  }
  __syncthreads();
  if (s_bad) {
    if (threadIdx.x == 0 && report && blockIdx.y == 0 && blockIdx.z == 0) atomicOr(p.status, s_bad);
    return;
  }
  if (threadIdx.x == 0 && report && blockIdx.y == 0 && blockIdx.z == 0 && p.new_lengths)
    p.new_lengths[b] = (int)(ctx + kept);
  U* base = static_cast<U*>(table.tensor[blockIdx.y]);
  const int units = p.cache.num_kv_heads * per_head;
  for (int e = blockIdx.z * kThreads + threadIdx.x; e < units; e += gridDim.z * kThreads) {
    const int h = e / per_head;
    U* col = base + h * head_stride + (e - h * per_head);
    for (int k0 = 0; k0 < kept; k0 += kBatch) {
      U v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (k0 + i < kept && s_src[k0 + i] != s_dst[k0 + i]) v[i] = col[s_src[k0 + i]];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (k0 + i < kept && s_src[k0 + i] != s_dst[k0 + i]) col[s_dst[k0 + i]] = v[i];
    }
  }
}

template <typename U>
cudaError_t run(const KeepTable& t, const KeepDesc& p, int es, int tensors, bool report, cudaStream_t s) {
  const long long unit = sizeof(U);
  const int per_head = (int)((long long)p.cache.head_dim * es / unit);
  const long long units = (long long)per_head * p.cache.num_kv_heads;
  const dim3 grid(p.num_seqs, tensors,
                  (unsigned)std::max(1LL, std::min((units + kThreads - 1) / kThreads, 64LL)));
  keep_rows_kernel<U><<<grid, kThreads, 0, s>>>(t, p, per_head, p.cache.page_stride * es / unit,
                                                p.cache.token_stride * es / unit, p.cache.head_stride * es / unit,
                                                report);
  return noted(cudaGetLastError(), LORA_PATH_KEEP);
}

}  // namespace

cudaError_t launch_keep_rows(const KeepDesc& p, int dtype, const lora_kv_cache_t* caches, int num_caches,
                             cudaStream_t s) {
  const int es = dtype == LORA_DTYPE_BF16 ? 2 : 4;
  const CacheDesc& c = p.cache;
  // The widest unit that every address and length is a multiple of.
  unsigned long long low = (unsigned long long)c.head_dim * es | 16;
  if (c.num_pages > 1) low |= (unsigned long long)c.page_stride * es;
  if (c.page_size > 1) low |= (unsigned long long)c.token_stride * es;
  if (c.num_kv_heads > 1) low |= (unsigned long long)c.head_stride * es;
  for (int i = 0; i < num_caches; ++i)
    low |= reinterpret_cast<unsigned long long>(caches[i].k) | reinterpret_cast<unsigned long long>(caches[i].v);
  const int unit = (int)(low & (~low + 1));
  for (int c0 = 0; c0 < num_caches; c0 += kMaxTensors / 2) {
    const int nc = std::min(num_caches - c0, kMaxTensors / 2);
    KeepTable t;
    for (int i = 0; i < nc; ++i) {
      t.tensor[2 * i] = caches[c0 + i].k;
      t.tensor[2 * i + 1] = caches[c0 + i].v;
    }
    cudaError_t e;
    switch (unit) {
      case 16: e = run<uint4>(t, p, es, 2 * nc, c0 == 0, s); break;
      case 8: e = run<uint2>(t, p, es, 2 * nc, c0 == 0, s); break;
      case 4: e = run<unsigned>(t, p, es, 2 * nc, c0 == 0, s); break;
      default: e = run<unsigned short>(t, p, es, 2 * nc, c0 == 0, s); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace lora
