// Pieces shared by the kernels of attention over a paged cache: which block of
// rows a CTA has, and what a row sees.
#pragma once

#include "attn_kv4.cuh"
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

// Up to this many requests their blocks are counted 32 requests a step, which leaves
// none without rows in between; beyond, a request's first block follows from its
// offset alone.  (bf16, a token each of 256, 1024 and 4096 requests behind 200 slots,
// 8 heads, the form with an SM to itself: 106, 420 and 1711 us; counted, 114, 628 and
// 6365.)
constexpr int kCounted = 64;

// What block i of a request with geometry R, of `count`, has.
template <int ROWS>
__device__ __forceinline__ void set_block(const PagedAttnArgs &p, RowBlock &w, int i, int count) {
  const int G = p.a.G;
  if (p.causal) i = count - 1 - i;
  w.row0 = i * ROWS;
  w.rows = min(ROWS, w.R.n * G - w.row0);
  w.keys = p.causal ? w.R.L + (w.row0 + w.rows - 1) / G + 1 : w.R.keys;
}

// Block j of many requests: request b's blocks start at (offsets[b] G + (ROWS - 1) b)
// / ROWS, which leaves room for ceil(n_b G / ROWS) of them, so that a search finds b.
// Blocks in between have no rows.
template <int ROWS>
__device__ __forceinline__ RowBlock find_block_of_many(const PagedAttnArgs &p, int j, int lane) {
  auto first = [&](int b) {
    return (static_cast<long long>(__ldg(p.a.offsets + b)) * p.a.G + (ROWS - 1ll) * b) / ROWS;
  };
  RowBlock w;
  w.b = -1;
  w.row0 = w.rows = w.keys = 0;
  w.R = {0, 0, 0, 0, 0};
  int lo = 0, n = p.a.B;      // as warp_find_request
  while (n > 32) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool below = at < lo + n && first(at) <= j;
    const int last = 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, below) | 1u));
    n = min(step, lo + n - (lo + last * step));
    lo += last * step;
  }
  const int mine = lo + lane;
  const uint32_t who = __ballot_sync(0xffffffffu, lane < n && first(mine) <= j && j < first(mine + 1));
  if (!who) return w;
  const int b = lo + __ffs(static_cast<int>(who)) - 1;
  w.R = paged_geometry(p, b);
  const long long i = j - first(b);      // from 0 on; beyond 32 bits where offsets are anything
  const int count = w.R.err ? 0 : (w.R.n * p.a.G + ROWS - 1) / ROWS;
  if (i >= count) return w;
  w.b = b;
  set_block<ROWS>(p, w, static_cast<int>(i), count);
  return w;
}

// The j-th block of the batch; by one warp, 32 requests a step, whose three
// loads are under way at once.  The host knows only how many rows there are in
// all, so a launch has blocks for the worst split of them over the requests;
// those left over find none, and requests in error have none.  The last blocks
// of a run of tokens, which see most, come first.
template <int ROWS>
__device__ __forceinline__ RowBlock find_block(const PagedAttnArgs &p, int j, int lane) {
  if (p.a.B > kCounted) return find_block_of_many<ROWS>(p, j, lane);
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
    const int i = j - (__shfl_sync(0xffffffffu, up_to, at) - count);
    w.b = b0 + at;
    w.R.lo = __shfl_sync(0xffffffffu, mine.lo, at);
    w.R.n = __shfl_sync(0xffffffffu, mine.n, at);
    w.R.L = __shfl_sync(0xffffffffu, mine.L, at);
    w.R.keys = w.R.L + w.R.n;
    set_block<ROWS>(p, w, i, count);
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
  if (a.B > kCounted) return (static_cast<long long>(a.T) * a.G + (ROWS - 1ll) * a.B) / ROWS;
  return (static_cast<long long>(a.T) * a.G - (a.B < a.T ? a.B : a.T)) / ROWS + (a.B < a.T ? a.B : a.T);
}

// Blocks of requests alike, by which launches are planned.
template <int ROWS>
inline long long likely_blocks(const AttnArgs &a) {
  return (static_cast<long long>(mean_nodes(a)) * a.G + ROWS - 1) / ROWS * (a.B < a.T ? a.B : a.T);
}

// Every request's error, reported once (those in error have no block); by one
// warp each of the first head's CTAs.
__device__ __forceinline__ void report_bad_requests(const PagedAttnArgs &p, int lane) {
  const long long step = 32ll * gridDim.x;
  for (long long b = 32ll * blockIdx.x + lane; b < p.a.B; b += step) {
    const ReqGeom g = paged_geometry(p, static_cast<int>(b));
    if (g.err) report(p.a.status, static_cast<int>(b), g.err);
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

// The output of a block whose keys are not split: rows as merge_splits takes them,
// eight dims a thread.  (128-node trees x 4, 64 heads on 8, behind 8192 keys: 137
// to 141 us, with the merge's loop 143; prompts of 128 tokens x 64, 74 and 81.)
template <int D, int THREADS, typename E, typename OutRow>
__device__ __forceinline__ void write_rows(int tid, int rows, const float *so, OutRow out_row) {
  __syncthreads();
#pragma unroll 4
  for (int idx = tid; idx < rows * (D / 8); idx += THREADS) {
    const int r = idx / (D / 8), c = idx % (D / 8) * 8;
    const float *from = so + r * (D + 4);
    const float total = from[D + 1];
    const float4 x = *reinterpret_cast<const float4 *>(from + c), y = *reinterpret_cast<const float4 *>(from + c + 4);
    E *dst = out_row(r);
    if (total < 0.f || !dst) continue;
    const float inv = total == 0.f ? 0.f : __fdividef(1.f, total);
    if constexpr (sizeof(E) == 4) {
      *reinterpret_cast<float4 *>(dst + c) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
      *reinterpret_cast<float4 *>(dst + c + 4) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
    } else {
      const __nv_bfloat162 h[4] = {__floats2bfloat162_rn(x.x * inv, x.y * inv), __floats2bfloat162_rn(x.z * inv, x.w * inv),
                                   __floats2bfloat162_rn(y.x * inv, y.y * inv), __floats2bfloat162_rn(y.z * inv, y.w * inv)};
      const uint32_t *u = reinterpret_cast<const uint32_t *>(h);
      *reinterpret_cast<uint4 *>(dst + c) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
}

// Merge of a block's rows over the splits of its keys, and the output, by all
// THREADS threads of the CTA.  Each CTA of the cluster has its rows in
// so[rows][D + 4] (shared memory, at the same place in all): the weighted sum,
// the reference, the sum of weights (below zero: this CTA's are not to be used).
// CTA q merges rows [q share, (q + 1) share): every CTA sends it those, in one
// copy that completes on its barrier, to recv[split][share][D + 4] behind `so`.
// (Pieces read from the peers, or stored to them, by the threads themselves: 1000
// cycles and more for each round of them.)  Code that runs once costs more in
// instruction fetches than in work here, so the loop is one for all splits, and
// kept small: factors worked out once a row, unrolled, took 1000 cycles longer.
template <int D>
constexpr int merge_bytes(int rows) { return (2 * rows + kMaxSplits) * (D + 4) * 4; }      // so and recv

// False: a peer's rows did not arrive in time, and none are written.
template <int D, int THREADS, typename E, typename OutRow>
__device__ __forceinline__ bool merge_splits(int tid, int CS, int split, int rows, float *so, uint64_t *bar,
                                             OutRow out_row) {
  if (CS == 1) {
    write_rows<D, THREADS, E>(tid, rows, so, out_row);
    return true;
  }
  constexpr int kStride = D + 4;
  const int share = (rows + CS - 1) / CS;
  const int from = min(rows, split * share), n = min(rows, from + share) - from;
  float *recv = so + rows * kStride;
  bool ok = true;
  fence_proxy_async_smem();
  cluster_sync_all();      // every CTA's rows are there, and room for its peers'
  if (tid < CS) {
    const int r0 = min(rows, tid * share), rn = min(rows, r0 + share) - r0;
    if (rn > 0)
      bulk_copy_s2s(peer_addr(recv + split * share * kStride, tid), smem_addr(so + r0 * kStride),
                    static_cast<uint32_t>(rn * kStride * 4), peer_addr(bar, tid));
  }
  if (n > 0) {
    if (tid == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(CS * n * kStride * 4));
    ok = mbar_wait(bar, 0);      // (every CTA sends, also after a time-out: none may leave before)
  }
#pragma unroll 1
  for (int idx = tid; idx < n * (D / 4) && ok; idx += THREADS) {
    const int r = idx / (D / 4), c = idx % (D / 4) * 4;
    const float *part = recv + r * kStride;
    float top = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool void_part = false;
#pragma unroll 1
    for (int q = 0; q < CS; ++q, part += share * kStride) {
      const float2 m = *reinterpret_cast<const float2 *>(part + D);
      const float4 v = *reinterpret_cast<const float4 *>(part + c);
      const float next = fmaxf(top, m.x), zero = next == -INFINITY ? 0.f : next;
      const float f0 = fast_exp2(top - zero), f1 = fast_exp2(m.x - zero);
      top = next;
      void_part |= m.y < 0.f;
      sum = fmaf(f1, m.y, sum * f0);
      acc.x = fmaf(f1, v.x, acc.x * f0);
      acc.y = fmaf(f1, v.y, acc.y * f0);
      acc.z = fmaf(f1, v.z, acc.z * f0);
      acc.w = fmaf(f1, v.w, acc.w * f0);
    }
    E *dst = out_row(from + r);
    if (void_part || !dst) continue;
    const float inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
    store_row4(dst + c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
  cluster_arrive_relaxed();      // no CTA leaves while a copy may still read its rows
  cluster_wait();
  return ok;
}

int launch_attn_paged_f32(const PagedAttnArgs &p, int max_prefix, void *stream);

}  // namespace spec
