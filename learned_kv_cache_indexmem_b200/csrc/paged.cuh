// paged.cuh -- device helpers of the paged cache: a sequence's new tokens and
// cached length, and the cache row of a position, all bounds-checked.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace imem {

struct SeqInfo {
  int tok0;   // first new token (row of the packed token axis)
  int n;      // new tokens
  int len;    // cached tokens, the new ones included
  int bad;    // a length or token range outside what the call was given
};

// Token range and length of sequence s. Malformed values are held inside the
// buffers (and flagged), so that nothing derived from them leaves them.
__device__ __forceinline__ SeqInfo seq_info(int s, int batch, int n_tokens, const int32_t* start,
                                            const PagedView& pg) {
  SeqInfo q;
  q.bad = 0;
  if (start) {
    const int a = start[s], b = start[s + 1];
    q.tok0 = min(max(a, 0), n_tokens);
    const int end = min(max(b, q.tok0), n_tokens);
    q.n = end - q.tok0;
    q.bad = a < 0 || b < a || b > n_tokens;
  } else {
    q.n = n_tokens / batch;
    q.tok0 = s * q.n;
  }
  // 2^30 tokens at most: positions and rounded-up key counts stay ints
  const long long cap = min((long long)pg.max_pages << pg.page_log, 1LL << 30);
  const int len = pg.len[s];
  q.len = (int)min((long long)max(len, 0), cap);
  q.bad |= len != q.len;
  return q;
}

// Cache row (page * page_size + slot) of position pos >= 0 of a sequence whose
// table row is `table`; -1 if the page is not one of the cache's.
__device__ __forceinline__ long long cache_row(const PagedView& pg, const int32_t* table, int pos) {
  const int page = table[pos >> pg.page_log];
  if (page < 0 || page >= pg.n_pages) return -1;
  return ((long long)page << pg.page_log) + (pos & ((1 << pg.page_log) - 1));
}

// ln of the sum of exponentials from a row's maximum in log2 units and its sum
// relative to that. +inf, a score of the row, is the result; a NaN stays one; a
// sum of 0 (nothing seen, or scores of -inf alone) gives -inf.
__device__ __forceinline__ float lse_of(float m2, float sum) {
  if (m2 == INFINITY) return m2;
  return sum != 0.f ? (m2 + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace imem
