// Packed rows of a batch (eagle_rows): which request a row belongs to, and
// the bounds of a request's rows.
#pragma once
#include "internal.h"
#include "common.cuh"

namespace eagle {

struct PackedRows {
  const int32_t* start;   // [B + 1]
  int n_rows, B;
};

// Rows [lo, hi) of request b, by its own two starts; none (and false) when they
// break 0 <= lo <= hi <= n_rows.
__device__ __forceinline__ bool request_rows(const PackedRows& r, int b, int& lo, int& hi) {
  lo = r.start[b];
  hi = r.start[b + 1];
  if (lo >= 0 && lo <= hi && hi <= r.n_rows) return true;
  hi = lo = 0;
  return false;
}

// The request that holds packed row `row` (every lane of a warp calls it; the
// result is the same in all), or -1: the first whose end passes the row, by
// a 32-way search of the ends, confirmed against that request's bounds.  Where
// starts out of order mislead the search, a row may have a request that it
// does not find.  The place it arrives at never goes back as the row goes up,
// so a request it finds for its first and last row it finds for all between.
__device__ __forceinline__ int request_of_row(const PackedRows& r, int row, int lane) {
  int lo = 0, n = r.B;    // the answer is in [lo, lo + n], r.B when no end passes the row
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int probe = lo + min((lane + 1) * step, n) - 1;
    const bool in = lane * step < n;
    const unsigned below = __ballot_sync(0xffffffffu, in && r.start[probe + 1] <= row);
    const int c = __popc(below);              // whole steps whose last end does not pass the row
    const int next = min(lo + c * step, lo + n);
    n = step == 1 ? 0 : min(step - 1, lo + n - next);
    lo = next;
  }
  if (lo >= r.B) return -1;
  int a, z;
  return request_rows(r, lo, a, z) && row >= a && row < z ? lo : -1;
}

// The first request that holds a row by its own two starts, or -1, whatever
// the others are.
__device__ __forceinline__ int first_request_of_row(const PackedRows& r, int row, int lane) {
  for (int b0 = 0; b0 < r.B; b0 += 32) {
    int a = 0, z = 0;
    if (b0 + lane < r.B) request_rows(r, b0 + lane, a, z);
    const unsigned who = __ballot_sync(0xffffffffu, row >= a && row < z);
    if (who) return b0 + __ffs(who) - 1;
  }
  return -1;
}

// Whether a cache takes n more rows of request b at length L: within cap and,
// when paged, in allocated blocks, the first of which (where the counts are
// given) no other table entry maps; none, whatever the length (every lane of a
// warp calls it; the result is the same in all).
__device__ __forceinline__ bool cache_takes(const PagedKv& pg, int cap, int b, int L, int n, int lane) {
  if (n == 0) return true;
  if (L < 0 || static_cast<long long>(L) + n > cap) return false;
  bool ok = true;
  if (pg.table) {
    const int last = (L + n - 1) >> pg.shift;
    for (int c = (L >> pg.shift) + lane; c <= last; c += 32) {
      const int blk = pg.table[static_cast<size_t>(b) * pg.per_req + c];
      ok = ok && blk >= 0 && blk < pg.n_blocks;
    }
    if (pg.ref) ok = ok && !block_shared(pg, b, L);
  }
  return __all_sync(0xffffffffu, ok);
}

}  // namespace eagle
