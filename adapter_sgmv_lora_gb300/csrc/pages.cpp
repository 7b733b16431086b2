// pages.cpp -- host side of the paged cache: the frequency table of the
// position rotation (lora_build_rope), the masks of a tree of drafted tokens
// (lora_build_tree) and the bookkeeping of a cache's pages (lora_pages_*) in
// arrays that the caller owns.  Nothing here allocates, so
// nothing here can throw.
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/lora_sgmv.h"

extern "C" lora_status_t lora_build_rope(int32_t rotary_dim, double theta, lora_rope_scaling_t scaling, double factor,
                                         int32_t original_max_positions, double low_turns, double high_turns,
                                         const double* frequencies, uint64_t* turns) {
  constexpr double kTwoPi = 6.283185307179586476925;
  if (!turns) return LORA_ERR_NULL;
  if (rotary_dim < 2 || rotary_dim > LORA_MAX_HEAD_DIM || rotary_dim % 2 != 0) return LORA_ERR_SHAPE;
  if (!frequencies && !(theta > 0.0 && std::isfinite(theta))) return LORA_ERR_SHAPE;
  switch (scaling) {
    case LORA_ROPE_NONE: break;
    case LORA_ROPE_NTK:
      if (frequencies || rotary_dim < 4) return LORA_ERR_SHAPE;
      break;
    case LORA_ROPE_LINEAR: break;
    case LORA_ROPE_PARTS:
      if (original_max_positions < 1 || !(high_turns > low_turns) || !std::isfinite(high_turns - low_turns))
        return LORA_ERR_SHAPE;
      break;
    default: return LORA_ERR_SHAPE;
  }
  if (scaling != LORA_ROPE_NONE && !(factor > 0.0 && std::isfinite(factor))) return LORA_ERR_SHAPE;
  const int32_t n = rotary_dim / 2;
  if (frequencies)
    for (int32_t i = 0; i < n; ++i)
      if (!std::isfinite(frequencies[i])) return LORA_ERR_SHAPE;
  double base = theta;
  if (scaling == LORA_ROPE_NTK) base = theta * std::pow(factor, rotary_dim / (rotary_dim - 2.0));
  if (!frequencies && !(base > 0.0 && std::isfinite(base))) return LORA_ERR_SHAPE;
  double scaled[LORA_MAX_HEAD_DIM / 2];
  for (int32_t i = 0; i < n; ++i) {
    double f = frequencies ? frequencies[i] : std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == LORA_ROPE_LINEAR) f /= factor;
    if (scaling == LORA_ROPE_PARTS) {
      const double over = original_max_positions * f / kTwoPi;
      double g = (over - low_turns) / (high_turns - low_turns);
      g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
      f = g * f + (1.0 - g) * f / factor;
    }
    if (!std::isfinite(f)) return LORA_ERR_SHAPE;
    scaled[i] = f;
  }
  for (int32_t i = 0; i < n; ++i) {
    double t = scaled[i] / kTwoPi;
    t -= std::floor(t);  // [0, 1]: a tiny negative turn rounds up to 1, the same angle as 0
    turns[i] = t < 1.0 ? static_cast<uint64_t>(std::ldexp(t, 64)) : 0;
  }
  return LORA_OK;
}

extern "C" lora_status_t lora_build_tree(int32_t num_nodes, const int32_t* parents, int32_t mask_words,
                                         uint64_t* masks, int32_t* depths) {
  if (num_nodes < 0 || mask_words < 1 || mask_words > LORA_MAX_MASK_WORDS || num_nodes > 64 * mask_words)
    return LORA_ERR_SHAPE;
  if (num_nodes > 0 && !parents) return LORA_ERR_NULL;
  for (int32_t i = 0; i < num_nodes; ++i)
    if (parents[i] < -1 || parents[i] >= i) return LORA_ERR_SHAPE;
  for (int32_t i = 0; i < num_nodes; ++i) {
    const int32_t p = parents[i];
    if (depths) depths[i] = p < 0 ? 0 : depths[p] + 1;
    if (!masks) continue;
    uint64_t* row = masks + (int64_t)i * mask_words;
    for (int32_t w = 0; w < mask_words; ++w) row[w] = p < 0 ? 0 : masks[(int64_t)p * mask_words + w];
    row[i >> 6] |= 1ull << (i & 63);
  }
  return LORA_OK;
}

namespace {

lora_status_t check(const lora_pages_t* p) {
  if (!p || !p->tables || !p->lengths || !p->refs || !p->free_pages) return LORA_ERR_NULL;
  if (p->num_pages < 1 || p->page_size < 1 || p->max_seqs < 1 || p->max_pages < 1) return LORA_ERR_SHAPE;
  if (static_cast<int64_t>(p->num_pages) * p->page_size > INT32_MAX) return LORA_ERR_SHAPE;
  return LORA_OK;
}

int32_t* table_of(const lora_pages_t* p, int32_t seq) { return p->tables + static_cast<int64_t>(seq) * p->max_pages; }

int32_t pages_for(const lora_pages_t* p, int64_t tokens) {
  return static_cast<int32_t>((tokens + p->page_size - 1) / p->page_size);
}

}  // namespace

extern "C" lora_status_t lora_pages_init(lora_pages_t* pages) {
  const lora_status_t st = check(pages);
  if (st != LORA_OK) return st;
  const int64_t entries = static_cast<int64_t>(pages->max_seqs) * pages->max_pages;
  for (int64_t i = 0; i < entries; ++i) pages->tables[i] = -1;
  for (int32_t s = 0; s < pages->max_seqs; ++s) pages->lengths[s] = 0;
  for (int32_t g = 0; g < pages->num_pages; ++g) {
    pages->refs[g] = 0;
    pages->free_pages[g] = pages->num_pages - 1 - g;  // the lowest page is taken first
  }
  pages->num_free = pages->num_pages;
  return LORA_OK;
}

extern "C" lora_status_t lora_pages_append(lora_pages_t* pages, int32_t seq, int32_t num_tokens, int32_t* rows,
                                           int32_t* copy_src, int32_t* copy_dst) {
  const lora_status_t st = check(pages);
  if (st != LORA_OK) return st;
  if (!copy_src || !copy_dst || (num_tokens > 0 && !rows)) return LORA_ERR_NULL;
  if (seq < 0 || seq >= pages->max_seqs || num_tokens < 0) return LORA_ERR_SHAPE;
  const int32_t len = pages->lengths[seq];
  const int32_t ps = pages->page_size;
  const int64_t total = static_cast<int64_t>(len) + num_tokens;
  if ((total + ps - 1) / ps > pages->max_pages) return LORA_ERR_SHAPE;
  int32_t* table = table_of(pages, seq);
  const int32_t have = pages_for(pages, len), need = pages_for(pages, total);
  const bool copy = num_tokens > 0 && len % ps != 0 && pages->refs[table[have - 1]] > 1;
  if (need - have + (copy ? 1 : 0) > pages->num_free) return LORA_ERR_NO_PAGES;
  *copy_src = *copy_dst = -1;
  if (copy) {
    const int32_t fresh = pages->free_pages[--pages->num_free];
    *copy_src = table[have - 1];
    *copy_dst = fresh;
    --pages->refs[table[have - 1]];
    pages->refs[fresh] = 1;
    table[have - 1] = fresh;
  }
  for (int32_t i = have; i < need; ++i) {
    table[i] = pages->free_pages[--pages->num_free];
    pages->refs[table[i]] = 1;
  }
  for (int32_t i = 0; i < num_tokens; ++i) rows[i] = table[(len + i) / ps] * ps + (len + i) % ps;
  pages->lengths[seq] = static_cast<int32_t>(total);
  return LORA_OK;
}

extern "C" lora_status_t lora_pages_fork(lora_pages_t* pages, int32_t parent, int32_t child, int32_t num_tokens) {
  const lora_status_t st = check(pages);
  if (st != LORA_OK) return st;
  if (parent < 0 || parent >= pages->max_seqs || child < 0 || child >= pages->max_seqs) return LORA_ERR_SHAPE;
  if (pages->lengths[child] != 0 || num_tokens < 0 || num_tokens > pages->lengths[parent]) return LORA_ERR_SHAPE;
  const int32_t n = pages_for(pages, num_tokens);
  const int32_t* from = table_of(pages, parent);
  int32_t* to = table_of(pages, child);
  for (int32_t i = 0; i < n; ++i) {
    to[i] = from[i];
    ++pages->refs[from[i]];
  }
  pages->lengths[child] = num_tokens;
  return LORA_OK;
}

extern "C" lora_status_t lora_pages_trim(lora_pages_t* pages, int32_t seq, int32_t num_tokens) {
  const lora_status_t st = check(pages);
  if (st != LORA_OK) return st;
  if (seq < 0 || seq >= pages->max_seqs) return LORA_ERR_SHAPE;
  if (num_tokens < 0 || num_tokens > pages->lengths[seq]) return LORA_ERR_SHAPE;
  int32_t* table = table_of(pages, seq);
  const int32_t keep = pages_for(pages, num_tokens);
  for (int32_t i = pages_for(pages, pages->lengths[seq]) - 1; i >= keep; --i) {
    if (--pages->refs[table[i]] == 0) pages->free_pages[pages->num_free++] = table[i];
    table[i] = -1;
  }
  pages->lengths[seq] = num_tokens;
  return LORA_OK;
}

extern "C" lora_status_t lora_pages_compact(lora_pages_t* pages, int32_t* src, int32_t* dst, int32_t* num_copies) {
  const lora_status_t st = check(pages);
  if (st != LORA_OK) return st;
  if (!src || !dst || !num_copies) return LORA_ERR_NULL;
  const int32_t used = pages->num_pages - pages->num_free;
  int32_t n = 0, to = 0;
  for (int32_t from = used; from < pages->num_pages; ++from) {
    if (pages->refs[from] == 0) continue;
    while (pages->refs[to] != 0) ++to;  // below `used` there is a free page for each used one above it
    src[n] = from;
    dst[n] = to;
    ++n;
    pages->refs[to] = pages->refs[from];
    pages->refs[from] = 0;
  }
  if (n > 0) {
    for (int32_t s = 0; s < pages->max_seqs; ++s) {
      int32_t* table = table_of(pages, s);
      const int32_t have = pages_for(pages, pages->lengths[s]);
      for (int32_t i = 0; i < have; ++i) {
        if (table[i] < used) continue;
        int32_t lo = 0, hi = n - 1;  // src ascends: find the entry's move
        while (lo < hi) {
          const int32_t mid = (lo + hi) / 2;
          if (src[mid] < table[i]) lo = mid + 1;
          else hi = mid;
        }
        table[i] = dst[lo];
      }
    }
  }
  for (int32_t i = 0; i < pages->num_free; ++i) pages->free_pages[i] = pages->num_pages - 1 - i;
  *num_copies = n;
  return LORA_OK;
}
