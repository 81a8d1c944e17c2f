// A paged KV cache: pages of `1 << shift` slots of every KV head, k and v
// [pages][Hkv][slots of a page][D], and a block table whose row b names the
// pages of request b in the order of its slots.
#pragma once

#include "common.cuh"

namespace spec {

struct PageTable {
  const int32_t *table;    // [B][max_pages]
  int max_pages, pages, shift;
  int32_t *status;         // the call's, for the bounds-checked build

  // Slots of a request, which are counted in 32 bits (with room for a tile).
  __device__ __forceinline__ int capacity() const {
    return static_cast<int>(min(static_cast<long long>(max_pages) << shift, 0x7FFFFFFFll - 4096));
  }
  // The page of request b's slots [i << shift, (i + 1) << shift), or -1 for an id
  // outside the pool (i below max_pages).
  __device__ __forceinline__ int page(int b, int i) const {
    if (!in_bounds(i, max_pages, status, b)) return -1;
    const int id = __ldg(table + static_cast<size_t>(b) * max_pages + i);
    return static_cast<unsigned>(id) < static_cast<unsigned>(pages) ? id : -1;
  }
  // Whether `n` rows from `row` on lie in a pool of `heads` KV heads (bounds-checked
  // build; true in the normal one).
  __device__ __forceinline__ bool holds(long long row, long long n, int heads, int b) const {
    return range_in_bounds(row, n, static_cast<long long>(pages) * heads << shift, status, b);
  }
};

// Whether one of the pages of slots [from, to) of request b lies outside the
// pool; by one warp, which looks at the `part`-th of `parts` shares of them.
__device__ __forceinline__ bool warp_finds_bad_page(const PageTable &p, int b, int from, int to, int lane,
                                                    int part = 0, int parts = 1) {
  if (to <= from) return false;
  const int end = static_cast<int>((static_cast<unsigned>(to) - 1u) >> p.shift) + 1;
  bool bad = false;
#pragma unroll 8
  for (int i = (from >> p.shift) + 32 * part + lane; i < end; i += 32 * parts) bad |= p.page(b, i) < 0;
  return __any_sync(0xffffffffu, bad);
}

// Host-side checks of a pool's sizes; the shift of its page size in *shift.
inline int check_pages(int pages, int page_size, int max_pages, int *shift) {
  if (pages < 1 || max_pages < 1 || page_size < 8 || page_size > 4096 || (page_size & (page_size - 1)))
    return SPEC_ERR_SHAPE;
  int s = 3;
  while ((1 << s) < page_size) ++s;
  *shift = s;
  return SPEC_OK;
}

// Rows of a ragged batch: request b's rows are [offsets[b], offsets[b+1]).
struct RowRange {
  int lo, n, err;
};
__device__ __forceinline__ RowRange row_range(const int32_t *offsets, int b, int T) {
  RowRange r;
  r.lo = __ldg(offsets + b);
  const int hi = __ldg(offsets + b + 1);
  r.n = hi - r.lo;
  r.err = r.lo < 0 || hi > T || hi < r.lo ? SPEC_ERR_TREE_TOO_LARGE : 0;
  return r;
}

// find_request by a warp: 32 places are looked at in every step, so that a
// batch of up to 32 requests takes one load, one of 1024 two (a bisection 5 and
// 10, each 0.4 us of latency).  -1 when no request holds row t.
__device__ __forceinline__ int warp_find_request(const int32_t *off, int B, int t, int lane) {
  int lo = 0, n = B;          // the request is among [lo, lo + n)
  while (n > 32) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool below = at < lo + n && __ldg(off + at) <= t;
    const int last = 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, below) | 1u));
    n = min(step, lo + n - (lo + last * step));
    lo += last * step;
  }
  const int b = lo + lane;
  const bool mine = lane < n && __ldg(off + b) <= t && t < __ldg(off + b + 1);
  const uint32_t who = __ballot_sync(0xffffffffu, mine);
  return who ? lo + __ffs(static_cast<int>(who)) - 1 : -1;
}

}  // namespace spec
