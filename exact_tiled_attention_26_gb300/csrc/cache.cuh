// The paged key/value cache as the kernels see it, shared by the cache kernels and the
// attention over the cache.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace fa {

// Pages of `page` rows; row s of head h of page p lies at ((p * Hk + h) * page + s) * d.
// Sequence b's row j is in page table[b * table_stride + j / page], slot j % page.
struct CacheView {
  uint8_t *K, *V;            // bf16, or e4m3 with one exponent byte per row in Ke, Ve
  uint8_t *Ke, *Ve;
  const int* table;
  long long table_stride;
  const int* lens;           // [B]
  const int* n_new;          // [B], or null: every sequence has all T new tokens
  int cols, pages, Hk, page, page_shift, T;
};

// Exponent bytes stand for the power of two 2^(byte - 127); 255 marks a row that holds
// an infinity or a NaN and reads back as NaN.
constexpr int kExpNaN = 255;
// 2^-100 is the least scale: smaller rows lose bits instead (their values are below
// 2^-91), and every scale, its inverse and every value in between stays a normal fp32
// number.
constexpr int kExpMin = 27;
constexpr int kExpMax = 247;  // the scale of the largest bf16 numbers

// Keys of a sequence: its length, clamped to what the table can hold.
FA_DEV int clamp_len(const CacheView& c, int n) {
  const int cap = c.cols << c.page_shift;  // at most 2^30 (make_cache_view)
  return min(max(n, 0), cap);
}
FA_DEV int seq_len(const CacheView& c, int b) { return clamp_len(c, c.lens[b]); }
// New tokens of a sequence.
FA_DEV int clamp_new(const CacheView& c, int n) { return min(max(n, 0), c.T); }
FA_DEV int seq_new(const CacheView& c, int b) { return c.n_new == nullptr ? c.T : clamp_new(c, c.n_new[b]); }
// Position of the first new token (negative when a length is smaller than the number of
// new tokens: the tokens at negative positions do not exist).
FA_DEV int seq_prefix(const CacheView& c, int b) { return max(c.lens[b], 0) - seq_new(c, b); }
// Page of row j of sequence b, or -1 where the table has none (an entry outside
// [0, pages)).  j must be in [0, cols * page).
FA_DEV int page_of(const CacheView& c, int b, int j) {
  const int p = c.table[b * c.table_stride + (j >> c.page_shift)];
  return p >= 0 && p < c.pages ? p : -1;
}

// The table's entry for row j, whatever j is (beyond the table: its last column); to be
// compared with [0, pages) by the caller.  Needs cols > 0; j up to 2^30 + 2^26.
FA_DEV int table_entry(const CacheView& c, int b, int j) {
  return c.table[b * c.table_stride + min(j >> c.page_shift, c.cols - 1)];
}

// Host side: checks a cache and a table (fa.h states the rules) and fills the view.
fa_status make_cache_view(const fa_cache* c, const int* table, int cols, long long table_stride, const int* lens,
                          const int* n_new, int B, int T, CacheView* out);

}  // namespace fa
