// Pieces shared by the kernels of attention over a paged cache: which block of
// rows a CTA has, and what a row sees.
#pragma once

#include "attn_common.cuh"
#include "paged.cuh"

namespace spec {

struct PagedAttnArgs {
  AttnArgs a;          // k, v: the pools; S_cap: a request's slots
  PageTable pages;
  int causal;          // rows are runs of tokens, not trees
};

// Rows, prefix and errors of request b.
__device__ __forceinline__ ReqGeom paged_geometry(const PagedAttnArgs &p, int b) {
  ReqGeom g;
  g.L = __ldg(p.a.prefix_lens + b);
  const RowRange r = row_range(p.a.offsets, b, p.a.T);
  g.lo = r.lo;
  g.n = r.n;
  g.err = r.err;
  if (!g.err && !p.causal && (g.n < 1 || g.n > SPEC_MAX_TREE_NODES)) g.err = SPEC_ERR_TREE_TOO_LARGE;
  if (!g.err && (g.L < 0 || g.L > p.a.S_cap - g.n)) g.err = SPEC_ERR_PREFIX_RANGE;
  g.keys = g.err ? 0 : g.L + g.n;
  return g;
}

// One block of at most ROWS query rows (node-major, head-minor) of a request.
struct RowBlock {
  int b;               // -1: none
  int row0, rows;      // of the request's n x G rows
  int keys;            // cache slots that some row of the block sees: [0, keys)
  ReqGeom R;
};

// The j-th block of the batch; by one warp, 32 requests a step, whose three
// loads are under way at once.  The host knows only how many rows there are in
// all, so a launch has blocks for the worst split of them over the requests;
// those left over find none, and requests in error have none.  The last blocks
// of a run of tokens, which see most, come first.
template <int ROWS>
__device__ __forceinline__ RowBlock find_block(const PagedAttnArgs &p, int j, int lane) {
  const int G = p.a.G;
  RowBlock w;
  w.b = -1;
  w.row0 = w.rows = w.keys = 0;
  w.R = {0, 0, 0, 0, 0};
  for (int b0 = 0; b0 < p.a.B; b0 += 32) {
    ReqGeom mine = {0, 0, 0, 0, 0};
    if (b0 + lane < p.a.B) mine = paged_geometry(p, b0 + lane);
    const int blocks = mine.err ? 0 : (mine.n * G + ROWS - 1) / ROWS;
    int up_to = blocks;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, up_to, d);
      if (lane >= d) up_to += x;
    }
    const int total = __shfl_sync(0xffffffffu, up_to, 31);
    if (j >= total) {
      j -= total;
      continue;
    }
    const int at = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, j < up_to))) - 1;
    const int count = __shfl_sync(0xffffffffu, blocks, at);
    int i = j - (__shfl_sync(0xffffffffu, up_to, at) - count);
    if (p.causal) i = count - 1 - i;
    w.b = b0 + at;
    w.R.lo = __shfl_sync(0xffffffffu, mine.lo, at);
    w.R.n = __shfl_sync(0xffffffffu, mine.n, at);
    w.R.L = __shfl_sync(0xffffffffu, mine.L, at);
    w.R.keys = w.R.L + w.R.n;
    w.row0 = i * ROWS;
    w.rows = min(ROWS, w.R.n * G - w.row0);
    w.keys = p.causal ? w.R.L + (w.row0 + w.rows - 1) / G + 1 : w.R.keys;
    break;
  }
  return w;
}

// The first 4 KB of the block table on their way into L1 before it is known
// which entries are wanted: that takes a load of its own.  By one warp.
__device__ __forceinline__ void touch_table(const PagedAttnArgs &p, int lane) {
  if (32ll * lane >= static_cast<long long>(p.a.B) * p.pages.max_pages) return;
  int unused;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(unused) : "l"(p.pages.table + 32 * lane));
}

// Blocks that find_block may have to tell apart.
template <int ROWS>
inline long long most_blocks(const AttnArgs &a) {
  return (static_cast<long long>(a.T) * a.G - (a.B < a.T ? a.B : a.T)) / ROWS + (a.B < a.T ? a.B : a.T);
}

// Every request's error, reported once (those in error have no block); by one
// warp of the launch's first CTA.
__device__ __forceinline__ void report_bad_requests(const PagedAttnArgs &p, int lane) {
  for (int b = lane; b < p.a.B; b += 32) {
    const ReqGeom g = paged_geometry(p, b);
    if (g.err) report(p.a.status, b, g.err);
  }
}

// What one row sees: slots [0, until), and the tree nodes in `tree`, node 0 at
// slot L.
struct RowSees {
  int until;
  uint4 tree;
};

__device__ __forceinline__ uint32_t low_ones(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// Which of the 32 slots from k0 on a row sees, as bits.
__device__ __forceinline__ uint32_t sees_32(const RowSees &r, int k0, int L) {
  const uint32_t near = low_ones(r.until - k0);
  const int o = k0 - L;            // first slot's node
  const uint4 m = r.tree;
  if (o <= -32) return near;
  if (o < 0) return near | (m.x << -o);
  const int w = o >> 5;
  const uint32_t lo = w == 0 ? m.x : w == 1 ? m.y : w == 2 ? m.z : w == 3 ? m.w : 0u;
  const uint32_t hi = w == 0 ? m.y : w == 1 ? m.z : w == 2 ? m.w : 0u;
  return near | __funnelshift_r(lo, hi, o & 31);
}

int launch_attn_paged_f32(const PagedAttnArgs &p, int max_prefix, void *stream);

}  // namespace spec
