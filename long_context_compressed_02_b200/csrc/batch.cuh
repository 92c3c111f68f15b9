// The ragged batch of a serving step, as kernels see it: n_seq sequences whose
// new tokens are rows cu_q[b] .. cu_q[b+1] - 1 of the batch, at positions
// q_pos[b], q_pos[b] + 1, ...; and the pages of a cache.
#pragma once
#include <cstdint>

namespace csa {

// Sequence of token i, found by a whole warp: 32 probes a step, so up to 32
// sequences take one step and 1024 two (a load latency each, against
// log2(n_seq) of a search by one thread).  Returns -1 for tokens before the
// first or behind the last sequence.  Ends for any contents of cu_q: each step
// keeps at most 1/32 of the range, rounded up, and stops at one.
__device__ __forceinline__ int find_seq_warp(const int32_t* cu_q, int n_seq, int64_t i, int lane) {
  if (i < cu_q[0] || i >= cu_q[n_seq]) return -1;
  int lo = 0, len = n_seq;                      // the last b in [lo, lo + len) with cu_q[b] <= i
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const int64_t off = (int64_t)(lane + 1) * step;
    const bool le = off < len && cu_q[lo + off] <= i;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    lo += k * step;
    len = min(step, len - k * step);
  }
  return lo;
}

// Tokens of sequence b that are rows of the batch, whatever cu_q holds.
__device__ __forceinline__ int seq_len(const int32_t* cu_q, int b, int64_t n_tok) {
  const int c0 = cu_q[b];
  return c0 < 0 ? 0 : (int)max((int64_t)0, min((int64_t)cu_q[b + 1], n_tok) - c0);
}

// One paged cache: block_table [n_seq, max_pages] of page numbers, pages of
// 2^ps_log2 rows.
struct PageTable {
  const int32_t* table;
  int64_t n_pages;
  int max_pages, ps_log2;
};

// Row of the page store ([n_pages * page_size] rows) that holds row `row` of
// sequence b, or -1 if the table has no page for it.  row >= 0.
__device__ __forceinline__ int64_t page_row(const PageTable& t, int b, int64_t row) {
  const int64_t j = row >> t.ps_log2;
  if (j >= t.max_pages) return -1;
  const int32_t pg = __ldg(t.table + (int64_t)b * t.max_pages + j);
  if (pg < 0 || pg >= t.n_pages) return -1;
  return ((int64_t)pg << t.ps_log2) + (row & ((1 << t.ps_log2) - 1));
}

}  // namespace csa
