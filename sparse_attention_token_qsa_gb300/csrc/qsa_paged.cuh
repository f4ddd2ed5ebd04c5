// What the kernels that read or move a paged K/V cache share: the division of
// a token by the page size, a token's pool row, the sequences' rows, and the
// drafted tokens a row of a tree sees.
#pragma once

#include <stdint.h>

#include "qsa_device.cuh"

namespace qsa {

// t / d for 0 <= t < 2^31 as a multiply-high and a shift (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994):
// with l = ceil(log2 d), p = 31 + l and m = ceil(2^p / d) < 2^32, t / d is
// (t * m) >> p, since t * (m d - 2^p) < 2^31 d <= 2^p keeps the error below
// 1/d.  d = 1 has no such m (shift < 0: the quotient is t).
struct FastDiv {
  uint32_t mul;
  int32_t shift, d;
};

inline FastDiv make_fast_div(int32_t d) {
  if (d == 1) return FastDiv{1u, -1, 1};
  int l = 0;
  while ((1ll << l) < d) ++l;
  const int p = 31 + l;
  return FastDiv{(uint32_t)((((uint64_t)1 << p) + (uint64_t)d - 1) / (uint64_t)d), p - 32, d};
}

__device__ __forceinline__ int32_t fast_div(const FastDiv &f, int32_t t) {
  return f.shift < 0 ? t : (int32_t)(__umulhi((uint32_t)t, f.mul) >> f.shift);
}

// The cached sequences of one call and the rows that read them.
struct CachedSeqs {
  int32_t pool_pages;
  FastDiv page;
  const int32_t *table;
  int32_t table_len;
  int64_t table_cols;
  const int32_t *ctx_len;
  const int32_t *row_start;
  int32_t n_seqs, n_rows;
  const uint32_t *mask;  // nullptr: drafted row j sees the drafted tokens k <= j
  int32_t mask_words;
};

struct SeqView {
  int32_t row0, rows, ctx;  // rows 0 for a sequence that is skipped
  bool ok;
};

// What the arrays say of sequence s.
struct SeqRaw {
  int32_t r0, r1, ctx;
};
__device__ __forceinline__ SeqRaw read_seq(const CachedSeqs &c, int32_t s) {
  return SeqRaw{c.row_start[s], c.row_start[s + 1], c.ctx_len[s]};
}

// Its rows and its context length, rows 0 (and ok false) where they contradict
// the row count, the mask's width or the table.
__device__ __forceinline__ SeqView view_seq(const CachedSeqs &c, const SeqRaw &raw) {
  SeqView v;
  v.row0 = raw.r0;
  v.ctx = raw.ctx;
  const bool range = raw.r0 >= 0 && raw.r1 >= raw.r0 && raw.r1 <= c.n_rows && raw.ctx >= 0;
  v.rows = range ? raw.r1 - raw.r0 : 0;
  v.ok = range && (int64_t)v.ctx + v.rows <= (int64_t)c.table_len * c.page.d &&
         (c.mask == nullptr || v.rows <= (int64_t)32 * c.mask_words);
  if (!v.ok) v.rows = 0;
  return v;
}
__device__ __forceinline__ SeqView view_seq(const CachedSeqs &c, int32_t s) {
  return view_seq(c, read_seq(c, s));
}

// Pool row (slot) of token t >= 0 of sequence s, or -1 where the table's entry
// is outside the pool.  t must lie inside the table.
__device__ __forceinline__ int64_t token_slot(const CachedSeqs &c, int32_t s, int32_t t) {
  const int32_t pg = fast_div(c.page, t);
  const int32_t phys = c.table[(int64_t)s * c.table_cols + pg];
  if (phys < 0 || phys >= c.pool_pages) return -1;
  return (int64_t)phys * c.page.d + (t - pg * c.page.d);
}

// Whether drafted row j (its mask words at mrow) sees drafted token k < rows.
__device__ __forceinline__ bool sees_draft(const uint32_t *mrow, int32_t j, int32_t k) {
  return mrow == nullptr ? k <= j : (mrow[k >> 5] >> (k & 31)) & 1u;
}

// The sequence whose rows hold `row` where the starts ascend: the last s with
// row_start[s] <= row.
__device__ __forceinline__ int32_t seq_of_row(const CachedSeqs &c, int32_t row) {
  int32_t lo = 0, hi = c.n_seqs;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (c.row_start[mid] <= row) lo = mid; else hi = mid;
  }
  return lo;
}

// A CTA's (or team's) share of a list of `total` tiles cut into equal runs.
struct TileShare {
  int64_t per, first, n;
};

__device__ __forceinline__ TileShare tile_share(int64_t total, uint32_t sharers, uint32_t at) {
  TileShare h;
  h.per = (total >> 31) == 0 ? (int64_t)(((uint32_t)total + sharers - 1u) / sharers) : (total + sharers - 1) / sharers;
  h.first = h.per * at;
  h.n = max((int64_t)0, min(h.per, total - h.first));
  return h;
}

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

}  // namespace qsa
