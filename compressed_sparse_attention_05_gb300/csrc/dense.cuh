// What the kernels over the whole compressed cache share (readings R14, R15):
// the arguments, and which keys a query token sees.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace csa2 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Entries present in sequence b that the call may read: n_entries[b], bounded by
// the caller's max_entries and by the page-table row.
__device__ __forceinline__ int dense_entries(const DenseArgs& a, int b) {
  const int64_t room = min((int64_t)a.max_entries, (int64_t)a.max_pages * kPage);
  const int n = a.n_entries[b];
  return n < 0 ? 0 : (int)min((int64_t)n, room);
}
__device__ __forceinline__ bool dense_count_bad(const DenseArgs& a, int b) {
  const int n = a.n_entries[b];
  return n < 0 || n > min((int64_t)a.max_entries, (int64_t)a.max_pages * kPage) || (a.shift && a.shift[b] < 0);
}

// Entries evicted from sequence b so far: without entry_pos, entry j's last token is at
// raw position 4 (j + shift) + 3.
__device__ __forceinline__ int64_t dense_shift(const DenseArgs& a, int b) {
  const int s = a.shift ? a.shift[b] : 0;
  return s > 0 ? s : 0;
}

// What one query token sees.
struct DenseRow {
  int t;          // raw position
  int nv;         // entries j < nv whose last token is at or before `last` (without entry_pos: all of them)
  int last;       // and, with a document mask, whose first token is at or after doc
  int doc;        // raw position at which the token's document starts
  int w_lo, w_n;  // window rows: raw positions w_lo .. w_lo + w_n - 1
};

__device__ __forceinline__ DenseRow dense_row(const DenseArgs& a, int b, int i, int n_ent, int64_t shift, int pos0) {
  DenseRow r;
  const int64_t row = (int64_t)b * a.Tq + i;
  r.t = a.q_pos[row];
  r.doc = a.doc_start ? max(0, a.doc_start[row]) : 0;
  int64_t last = (int64_t)r.t + 1;   // tokens the row may see
  if (a.prefix_len && r.t >= 0) last = max(last, (int64_t)a.prefix_len[b]);
  // Evictions fill holes with newer entries, so that with entry_pos an index says nothing about the position.
  const int64_t v = a.entry_pos ? n_ent : (last < 0 ? 0 : last >> 2) - shift;
  r.nv = (int)max((int64_t)0, min(v, (int64_t)n_ent));
  r.last = (int)min(last - 1, (int64_t)INT_MAX);
  if (r.t < 0) {
    r.nv = 0;
    r.last = INT_MIN;
  }
  const int64_t lo = max(max((int64_t)r.doc, (int64_t)r.t - a.W + 1), (int64_t)max(pos0, 0));
  const int64_t hi = min((int64_t)r.t, (int64_t)pos0 + a.swa_cap - 1);
  r.w_lo = (int)lo;
  r.w_n = (r.t >= 0 && a.W > 0 && a.swa_cap > 0) ? (int)max((int64_t)0, hi - lo + 1) : 0;
  return r;
}

// First entry index that a document mask can let through (without entry_pos the
// entries are in position order: entry j's first token is at 4 (j + shift)).
__device__ __forceinline__ int dense_first(const DenseArgs& a, int doc, int64_t shift) {
  return a.entry_pos ? 0 : (int)max((int64_t)0, (((int64_t)doc + 3) >> 2) - shift);
}

}  // namespace csa2
