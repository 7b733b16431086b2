// attention_api.cu -- the extern "C" entry points between the projections
// (rotation + cache append, paged attention, page copies): argument
// validation and dispatch.  The host bookkeeping of pages is in pages.cpp.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstdlib>
#include <utility>

#include "internal.h"

namespace lora {
namespace {

lora_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA; }

bool dtype_ok(int t) { return t == LORA_DTYPE_F32 || t == LORA_DTYPE_BF16; }

// Natural alignment: what the element-wise kernels need (16-byte alignment
// only decides which kernel runs).
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }
int elem_bytes(int dtype) { return dtype == LORA_DTYPE_BF16 ? 2 : 4; }

// Whether `counts` elements at `strides`, each a run of `run` addresses,
// are all apart: from the smallest stride up, each dimension must step over
// everything below it.
template <int N>
bool disjoint(std::pair<int64_t, int64_t> (&dims)[N], int64_t run) {
  std::sort(dims, dims + N);
  int64_t extent = run;
  for (const auto& [stride, count] : dims) {
    if (stride < 0) return false;
    if (count <= 1) continue;
    if (stride < extent) return false;
    if (stride > (INT64_MAX / 2 - extent) / count) return false;
    extent += stride * (count - 1);
  }
  return true;
}

lora_status_t validate_cache(const lora_kv_cache_t* c) {
  if (!c) return LORA_ERR_NULL;
  if (!dtype_ok(c->dtype)) return LORA_ERR_DTYPE;
  if (c->num_pages < 1 || c->page_size < 1 || c->num_kv_heads < 1 || c->head_dim < 1 ||
      c->head_dim > LORA_MAX_HEAD_DIM)
    return LORA_ERR_SHAPE;
  if ((int64_t)c->num_pages * c->page_size > INT32_MAX) return LORA_ERR_SHAPE;
  if (!c->k || !c->v) return LORA_ERR_NULL;
  std::pair<int64_t, int64_t> dims[3] = {{c->page_stride, c->num_pages},
                                         {c->token_stride, c->page_size},
                                         {c->head_stride, c->num_kv_heads}};
  if (!disjoint(dims, c->head_dim)) return LORA_ERR_SHAPE;
  return aligned(c->k, elem_bytes(c->dtype)) && aligned(c->v, elem_bytes(c->dtype)) ? LORA_OK : LORA_ERR_ALIGN;
}

// Inputs may repeat addresses (a stride of 0 broadcasts).
lora_status_t validate_input(const lora_heads_t& h, int dtype) {
  if (!h.data) return LORA_ERR_NULL;
  const int64_t most = INT64_MAX >> 32;
  if (h.row_stride < 0 || h.head_stride < 0 || h.row_stride > most || h.head_stride > most) return LORA_ERR_SHAPE;
  return aligned(h.data, elem_bytes(dtype)) ? LORA_OK : LORA_ERR_ALIGN;
}

// `in` is the view that `out` may be written over: with the same strides,
// where they reach anything.
lora_status_t validate_output(const lora_heads_t& out, const lora_heads_t& in, int64_t rows, int64_t heads,
                              int64_t head_dim, int dtype) {
  if (!out.data) return LORA_ERR_NULL;
  if (!aligned(out.data, elem_bytes(dtype))) return LORA_ERR_ALIGN;
  std::pair<int64_t, int64_t> dims[2] = {{out.row_stride, rows}, {out.head_stride, heads}};
  if (!disjoint(dims, head_dim)) return LORA_ERR_SHAPE;
  if (out.data == in.data && ((rows > 1 && out.row_stride != in.row_stride) ||
                              (heads > 1 && out.head_stride != in.head_stride)))
    return LORA_ERR_SHAPE;
  return LORA_OK;
}

HeadsDesc heads(const lora_heads_t& h) { return {h.data, (long long)h.row_stride, (long long)h.head_stride}; }

CacheDesc cache_desc(const lora_kv_cache_t* c) {
  return {c->k,           c->v,         (long long)c->page_stride, (long long)c->token_stride, (long long)c->head_stride,
          c->num_pages,   c->page_size, c->num_kv_heads,           c->head_dim};
}

lora_status_t validate_attention(const lora_attention_t* a, const lora_kv_cache_t* c) {
  if (!a) return LORA_ERR_NULL;
  lora_status_t st = validate_cache(c);
  if (st != LORA_OK) return st;
  if (a->num_seqs < 0 || a->num_heads < 1 || a->num_heads % c->num_kv_heads != 0) return LORA_ERR_SHAPE;
  if (a->max_pages < 0 || a->table_stride < 0 || (a->num_seqs > 1 && a->table_stride < a->max_pages))
    return LORA_ERR_SHAPE;
  if (a->num_seqs == 0) return LORA_OK;  // nothing is read or written
  if ((st = validate_input(a->q, c->dtype)) != LORA_OK) return st;
  if ((st = validate_output(a->out, a->q, a->num_seqs, a->num_heads, c->head_dim, c->dtype)) != LORA_OK) return st;
  if (!a->lengths || (a->max_pages > 0 && !a->block_tables)) return LORA_ERR_NULL;
  if (!aligned(a->lengths, 4) || !aligned(a->block_tables, 4) || !aligned(a->lse, 4)) return LORA_ERR_ALIGN;
  return LORA_OK;
}

AttnDesc attention_desc(const lora_attention_t* a, const lora_kv_cache_t* c) {
  AttnDesc d{};
  d.dtype = c->dtype;
  d.num_seqs = a->num_seqs;
  d.num_heads = a->num_heads;
  d.group = a->num_heads / c->num_kv_heads;
  d.q = heads(a->q);
  d.out = heads(a->out);
  d.cache = cache_desc(c);
  d.tables = a->block_tables;
  d.table_stride = (long long)a->table_stride;
  d.max_pages = a->max_pages;
  // A token's number plus a tile stays within 32 bits.
  d.max_len = (int)std::min<int64_t>((int64_t)a->max_pages * c->page_size, INT32_MAX - 256);
  d.lengths = a->lengths;
  d.scale = a->scale;
  d.lse = a->lse;
  return d;
}

// Whether src and dst lists are within [0, num_pages), no destination is
// listed twice and no page is on both sides.  Short lists pairwise, long ones
// with two bits a page.
lora_status_t check_copies(const int32_t* src, const int32_t* dst, int32_t n, int32_t num_pages) {
  for (int32_t i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= num_pages || dst[i] < 0 || dst[i] >= num_pages) return LORA_ERR_SHAPE;
  if (n <= 16) {
    for (int32_t i = 0; i < n; ++i)
      for (int32_t j = 0; j < n; ++j)
        if (src[j] == dst[i] || (j < i && dst[j] == dst[i])) return LORA_ERR_SHAPE;
    return LORA_OK;
  }
  uint8_t* mark = static_cast<uint8_t*>(std::calloc(((size_t)num_pages + 3) / 4, 1));
  if (!mark) return LORA_ERR_WORKSPACE;
  lora_status_t st = LORA_OK;
  for (int32_t i = 0; i < n; ++i) mark[src[i] >> 2] |= 1u << (2 * (src[i] & 3));
  for (int32_t i = 0; i < n && st == LORA_OK; ++i) {
    const int shift = 2 * (dst[i] & 3);
    if ((mark[dst[i] >> 2] >> shift) & 3) st = LORA_ERR_SHAPE;
    mark[dst[i] >> 2] |= 2u << shift;
  }
  std::free(mark);
  return st;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" lora_status_t lora_rope_append(const lora_rope_t* r, const lora_kv_cache_t* cache, lora_stream_t stream) {
  begin_call();
  if (!r) return LORA_ERR_NULL;
  if (!dtype_ok(r->dtype)) return LORA_ERR_DTYPE;
  if (r->num_tokens < 0 || r->num_heads < 0 || r->num_kv_heads < 0 || r->num_heads + (int64_t)r->num_kv_heads < 1 ||
      r->head_dim < 1 || r->head_dim > LORA_MAX_HEAD_DIM)
    return LORA_ERR_SHAPE;
  if (r->num_heads > (1 << 20) || r->num_kv_heads > (1 << 20)) return LORA_ERR_SHAPE;
  if (r->rotary_dim < 0 || r->rotary_dim % 2 != 0 || r->rotary_dim > r->head_dim) return LORA_ERR_SHAPE;
  if (r->layout != LORA_ROPE_HALVES && r->layout != LORA_ROPE_INTERLEAVED) return LORA_ERR_SHAPE;
  if (r->num_tokens == 0) return LORA_OK;  // nothing is read or written
  if (r->rotary_dim > 0 && (!r->turns || !r->positions)) return LORA_ERR_NULL;
  if ((cache == nullptr) != (r->cache_rows == nullptr)) return LORA_ERR_NULL;
  if (!aligned(r->turns, 8) || !aligned(r->positions, 4) || !aligned(r->cache_rows, 4) ||
      !aligned(r->q_weight, elem_bytes(r->dtype)) || !aligned(r->k_weight, elem_bytes(r->dtype)))
    return LORA_ERR_ALIGN;
  lora_status_t st;
  if (r->num_heads > 0) {
    if ((st = validate_input(r->q, r->dtype)) != LORA_OK) return st;
    if ((st = validate_output(r->q_out, r->q, r->num_tokens, r->num_heads, r->head_dim, r->dtype)) != LORA_OK) return st;
  }
  if (r->num_kv_heads > 0) {
    if ((st = validate_input(r->k, r->dtype)) != LORA_OK) return st;
    if (!cache && !r->k_out.data) return LORA_ERR_NULL;  // k would go nowhere
    if (r->k_out.data &&
        (st = validate_output(r->k_out, r->k, r->num_tokens, r->num_kv_heads, r->head_dim, r->dtype)) != LORA_OK)
      return st;
  }
  if (cache) {
    if ((st = validate_cache(cache)) != LORA_OK) return st;
    if (cache->dtype != r->dtype) return LORA_ERR_DTYPE;
    if (cache->num_kv_heads != r->num_kv_heads || cache->head_dim != r->head_dim) return LORA_ERR_SHAPE;
    if ((st = validate_input(r->v, r->dtype)) != LORA_OK) return st;
  }
  RopeDesc d{};
  d.dtype = r->dtype;
  d.T = r->num_tokens;
  d.H = r->num_heads;
  d.Hk = r->num_kv_heads;
  d.hd = r->head_dim;
  d.rot = r->rotary_dim;
  d.layout = r->layout;
  d.attention_scale = r->attention_scale;
  d.eps = r->eps;
  d.turns = reinterpret_cast<const unsigned long long*>(r->turns);
  d.positions = r->positions;
  d.q = heads(r->q);
  d.k = heads(r->k);
  d.v = heads(r->v);
  d.q_out = heads(r->q_out);
  d.k_out = heads(r->k_out);
  d.q_weight = r->q_weight;
  d.k_weight = r->k_weight;
  d.cache_rows = r->cache_rows;
  if (cache) d.cache = cache_desc(cache);
  if (!(d.status = status_ptr())) return LORA_ERR_CUDA;
  return cuda_status(launch_rope(d, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" size_t lora_attention_workspace_bytes(const lora_attention_t* attention, const lora_kv_cache_t* cache) {
  if (validate_attention(attention, cache) != LORA_OK) return 0;
  return attention_workspace_bytes(attention_desc(attention, cache));
}

extern "C" lora_status_t lora_paged_attention(const lora_attention_t* attention, const lora_kv_cache_t* cache,
                                              void* workspace, size_t workspace_bytes, lora_stream_t stream) {
  begin_call();
  const lora_status_t st = validate_attention(attention, cache);
  if (st != LORA_OK) return st;
  if (attention->num_seqs == 0) return LORA_OK;
  AttnDesc d = attention_desc(attention, cache);
  if (!workspace || workspace_bytes < attention_workspace_bytes(d)) return LORA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0) return LORA_ERR_ALIGN;
  if (!(d.status = status_ptr())) return LORA_ERR_CUDA;
  return cuda_status(launch_attention(d, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" lora_status_t lora_kv_copy_pages(const lora_kv_cache_t* caches, int32_t num_caches, const int32_t* src,
                                            const int32_t* dst, int32_t num_copies, lora_stream_t stream) {
  begin_call();
  if (num_caches < 0 || num_copies < 0) return LORA_ERR_SHAPE;
  if (num_caches == 0) return LORA_OK;
  if (!caches || (num_copies > 0 && (!src || !dst))) return LORA_ERR_NULL;
  lora_status_t st;
  if ((st = validate_cache(&caches[0])) != LORA_OK) return st;
  for (int32_t i = 1; i < num_caches; ++i) {
    const lora_kv_cache_t &a = caches[i], &b = caches[0];
    const bool same = a.num_pages == b.num_pages && a.page_size == b.page_size && a.num_kv_heads == b.num_kv_heads &&
                      a.head_dim == b.head_dim && a.page_stride == b.page_stride &&
                      a.token_stride == b.token_stride && a.head_stride == b.head_stride;
    // A layer like the first has its pointers left to check.
    if (same && a.dtype == b.dtype && a.k && a.v && aligned(a.k, elem_bytes(a.dtype)) &&
        aligned(a.v, elem_bytes(a.dtype)))
      continue;
    if ((st = validate_cache(&a)) != LORA_OK) return st;
    return a.dtype != b.dtype ? LORA_ERR_DTYPE : LORA_ERR_SHAPE;
  }
  if ((st = check_copies(src, dst, num_copies, caches[0].num_pages)) != LORA_OK) return st;
  if (num_copies == 0) return LORA_OK;
  return cuda_status(launch_copy_pages(cache_desc(&caches[0]), caches[0].dtype, caches, num_caches, src, dst,
                                       num_copies, reinterpret_cast<cudaStream_t>(stream)));
}
