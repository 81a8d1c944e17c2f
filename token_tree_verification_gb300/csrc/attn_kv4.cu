// Tree attention over the 4-bit KV cache, with an optional sliding window.
//
// For node i of request b and query head h of KV head g:
//   o[i][h] = sum_j softmax_j(s q . k_j) v_j  over the keys j that i sees,
// k_j and v_j the values of slot j's record (kv4.cuh).  A node sees the prefix
// and its ancestors; with a window w, of those only positions p_j > p_i - w or
// p_j < sinks, where a prefix key's position is its slot and a tree node's is
// the prefix length plus its depth.
#include <type_traits>

#include "attn_kv4.cuh"

namespace spec {

namespace {

// ---------------------------------------------------------------- mma.sync path
// Few rows on each key: every warp decodes records in registers, straight into
// the fragments of mma.m16n8k16, and no tile passes through shared memory
// twice.  Both products are taken transposed, keys (then dimensions) along M
// and rows along N, so that eight rows cost eight, not sixteen or 128:
//   S^T = K Q^T   A: 16 keys x 16 dims of K,   B: 16 dims x 8 rows of Q
//   O^T = V^T P^T A: 16 dims x 16 keys of V^T, B: 16 keys x 8 rows of P
// The order of dims inside a contraction is free, so lane (g, t) = (lane / 4,
// lane % 4) takes D/4 consecutive dims of key g as they lie in the record (one
// 16-byte load at D = 128), and D/8 consecutive dims of each of its V keys.
// S^T's accumulators hold (key g, rows 2t and 2t + 1); movmatrix turns a pair
// of them into P's fragment (row g, keys 2t and 2t + 1).
//
// Which key of a group of 16 is fragment row n is free as well (one order for
// both products).  key_of spreads the loads over the banks: the record's
// stride is 4 (D = 128: 36) or 20 words modulo 32, and with this order the
// eight 16-byte pieces of K, or the sixteen 8-byte pieces of V, that go in one
// pass hit 32 different banks.
//
// Each warp has a ring of its own, tiles of 32 keys brought by one bulk copy
// each, so warps never wait for one another until the end.
//
// What bounds it: every key is decoded by one warp, about 330 instructions per
// tile of 32 keys at D = 128, so long prefixes run at the issue rate just below
// the memory's.  8 requests x 32 heads x 6 rows behind 27000 to 32768 keys:
// 1.10 GB in 182 us, 6.1 TB/s, 0.89 of what a copy reaches.  Short ones are bound
// by latency: one token of 8 query heads x 4 requests x 8 KV heads behind 8192
// keys (38 MB) 15.3 us, of which set-up, first tile and merge are about 10; 8
// rows of one request behind 128 keys, fp32, 4.9 us.  fp32 calls of more rows
// decode every key for each block of up to 32: 256 units behind 4096 keys take 45
// us for 8 rows, 66 for 16, 118 for 32; 1024 rows of 32 units behind 8192 718 us.
constexpr int kFewTile = 32;       // keys of a stage
constexpr int kFewStages = 2;

template <int D, int NT, int W, bool F32>
struct FewCfg {
  static constexpr int kWarps = W;
  static constexpr int kRows = 8 * NT;
  static constexpr int R = kv4_record_bytes(D);
  static constexpr int kSteps = D / 16;               // k steps of S^T, m tiles of O^T
  static constexpr int kParts = F32 ? 2 : 1;          // halves per fp32 query and weight
  static constexpr bool kQInRegs = NT * kParts <= 2;
  static constexpr int kStageBytes = kFewTile * R;
  static constexpr int kRing = kWarps * kFewStages * kStageBytes;
  static constexpr int kOStride = D + 4;
  static constexpr int kMerge = kWarps * kRows * kOStride * 4;
  static constexpr int kQBytes = kQInRegs ? 0 : kParts * kSteps * NT * 32 * 8;
  static constexpr int kOffQ = kRing > kMerge ? kRing : kMerge;
  static constexpr int kOffRecv = kOffQ + kQBytes;    // what the peers of a cluster send
  static constexpr int kSmem = kOffRecv + (kRows * D + 4 * kMaxSplits) * 4;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero.
__device__ __forceinline__ void mma_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Key (0 .. 15) of fragment row n (0 .. 7); row n + 8 is the key after it.
__device__ __forceinline__ int key_of(int n) {
  const int t = n >> 1, o = n & 1;
  return t < 2 ? 2 * t + 4 * o : 8 + 2 * t - 4 * o;
}

template <int D, int NT, int W, bool F32>
__global__ void __launch_bounds__(32 * W, NT == 1 ? 16 / W : NT == 2 ? 2 : 1)
tree_attn_kv4_few_kernel(const Kv4AttnArgs p) {
  using C = FewCfg<D, NT, W, F32>;
  constexpr int kFewWarps = W, kFewThreads = 32 * W;
  using E = typename std::conditional<F32, float, __nv_bfloat16>::type;
  constexpr int R = C::R, KS = C::kSteps, NP = C::kParts;
  constexpr int kWords = D / 32;                  // code words of one lane's share of a key
  const AttnArgs &a = p.a;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar_full[kFewWarps][kFewStages];
  __shared__ uint4 s_tree[C::kRows];
  __shared__ int s_first[C::kRows];
  __shared__ float s_m[kFewWarps][C::kRows], s_l[kFewWarps][C::kRows];
  __shared__ float2 s_ml[kMaxSplits][C::kRows];
  __shared__ int s_par[SPEC_MAX_TREE_NODES];
  __shared__ int s_timeout;
  const int CS = static_cast<int>(gridDim.x), split = static_cast<int>(blockIdx.x);
  const int b = blockIdx.z / a.Hkv, g_kv = blockIdx.z % a.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

  pdl_trigger();
  if (lane == 0) {
    for (int s = 0; s < kFewStages; ++s) mbar_init(&bar_full[warp][s], 1);
    fence_barrier_init();
  }
  if (tid == 0) s_timeout = 0;
  __syncwarp();
  pdl_wait();

  const ReqGeom G = kv4_geometry(a, b);
  if (G.err) {      // the same for the whole cluster
    if (tid == 0 && split == 0 && blockIdx.y == 0 && g_kv == 0) report(a.status, b, G.err);
    return;
  }
  const TileList<kFewTile> tiles(G.L, G.keys, p.window, p.sinks);
  const int per = (tiles.count + CS - 1) / CS;
  const int t_end = min(tiles.count, (split + 1) * per);
  const int t_begin = split * per + warp;             // this warp's tiles: t_begin, + kFewWarps, ...
  const uint8_t *kv = static_cast<const uint8_t *>(a.k) + (static_cast<size_t>(b) * a.Hkv + g_kv) * a.S_cap * R;
  uint8_t *ring = smem + warp * kFewStages * C::kStageBytes;

  auto request = [&](int i, int st) {     // lane 0: tile i into stage st
    const int key0 = tiles.key0(i);
    const int n = min(kFewTile, G.keys - key0);
    if (!range_in_bounds(key0, n, a.S_cap, a.status, b)) {
      mbar_arrive(&bar_full[warp][st]);
      return;
    }
    mbar_arrive_expect_tx(&bar_full[warp][st], static_cast<uint32_t>(n * R));
    bulk_copy_g2s(smem_addr(ring + st * C::kStageBytes), kv + static_cast<size_t>(key0) * R,
                  static_cast<uint32_t>(n * R), &bar_full[warp][st]);
  };
  // A cluster takes every gridDim.y-th block of its request's rows: the grid is
  // sized by the mean number of rows, which the host knows, and a request with
  // more than that takes more turns.
  const int rows_total = G.n * a.G;
  bool ok = true;
  int st = 0, phase = 0;
  for (int row0 = static_cast<int>(blockIdx.y) * C::kRows; row0 < rows_total;
       row0 += static_cast<int>(gridDim.y) * C::kRows) {
    const int rows_here = min(C::kRows, rows_total - row0);
    if (CS > 1) cluster_arrive_relaxed();   // this CTA runs, and has read what it was sent before
    if (lane == 0)
      for (int s = 0; s < kFewStages; ++s)
        if (t_begin + s * kFewWarps < t_end) request(t_begin + s * kFewWarps, (st + s) % kFewStages);

    // ---- the rows: what each sees, and its query as halves
    if (!a.mask && row0 == static_cast<int>(blockIdx.y) * C::kRows) {
      for (int i = tid; i < G.n; i += kFewThreads)
        s_par[i] = in_bounds(G.lo + i, a.T, a.status, b) ? __ldg(a.parents + G.lo + i) : -2;
      __syncthreads();
    }
    // (the mask's load is under way while the queries are taken)
    uint4 row_mask = make_uint4(0u, 0u, 0u, 0u);
    const int row_node = (row0 + tid) / a.G;
    if (a.mask && tid < rows_here && in_bounds(G.lo + row_node, a.T, a.status, b))
      row_mask = __ldg(a.mask + G.lo + row_node);
    uint32_t qf[C::kQInRegs ? NP : 1][C::kQInRegs ? KS : 1][C::kQInRegs ? NT : 1][2];
    uint2 *sq = reinterpret_cast<uint2 *>(smem + C::kOffQ);   // [part][step][tile][lane]
    float c_row[NT][2];                                       // score factor of rows 2t, 2t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g, node = (row0 + r) / a.G;
      float x[D / 4];
      const bool live = r < rows_here && in_bounds(G.lo + node, a.T, a.status, b);
      const E *src = static_cast<const E *>(a.q) +
                     (static_cast<size_t>(G.lo + node) * a.Hq + g_kv * a.G + (row0 + r) % a.G) * D + t * (D / 4);
#pragma unroll
      for (int c = 0; c < D / 4; c += 16 / static_cast<int>(sizeof(E))) {
        const uint4 w = live ? __ldg(reinterpret_cast<const uint4 *>(src + c)) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (F32) {
            x[c + e] = __uint_as_float(u[e]);
          } else {
            x[c + 2 * e] = __uint_as_float(u[e] << 16);
            x[c + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
          }
        }
      }
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < D / 4; ++c) top = fmaxf(top, fabsf(x[c]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int up = row_exponent(top);
      const float grow = power_of_two(up);
      // (a factor of zero would make NaN of a masked score; one this small hides all)
      const float c = fmaxf(a.scale_log2 * power_of_two(-up), power_of_two(-126));
      c_row[nt][0] = __shfl_sync(0xffffffffu, c, 8 * t);
      c_row[nt][1] = __shfl_sync(0xffffffffu, c, 8 * t + 4);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int part = 0; part < NP; ++part) {
          uint32_t h[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y0 = x[4 * s + 2 * e] * grow, y1 = x[4 * s + 2 * e + 1] * grow;
            h[e] = pack_half2(y0, y1);
            if (part) {
              const float2 f = unpack_half2(h[e]);
              h[e] = pack_half2(y0 - f.x, y1 - f.y);
            }
          }
          if constexpr (C::kQInRegs) {
            qf[part][s][nt][0] = h[0];
            qf[part][s][nt][1] = h[1];
          } else if (nt % kFewWarps == warp) {      // NT <= 4: each tile of rows by one warp
            sq[((part * KS + s) * NT + nt) * 32 + lane] = make_uint2(h[0], h[1]);
          }
        }
    }
    if (tid < C::kRows) {
      if (a.mask) {
        row_mask = clip_mask(row_mask, G.n);
      } else if (tid < rows_here) {
        bool bad = false;
        row_mask = ancestor_mask([&](int i) { return s_par[i]; }, row_node, &bad);
        if (bad) report(a.status, b, SPEC_ERR_BAD_PARENT);
      }
      const RowKeys see = row_keys(row_mask, G.L, p.window, p.sinks);
      s_tree[tid] = see.tree;
      s_first[tid] = see.first;
    }
    __syncthreads();

    // ---- the keys
    float o[NT][KS][4];
    // a row's reference as 8 - reference, how large a score may come against it (-inf:
    // there is no reference yet), and its sum of weights
    float nbase[NT][2], limit[NT][2], l_row[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        nbase[nt][e] = kWeightLog2;
        limit[nt][e] = -INFINITY;
        l_row[nt][e] = 0.f;
      }
    }
    const int kn = key_of(g);                                 // this lane's K rows: kn, kn + 1
    const int kv0 = key_of(2 * t), kv1 = key_of(2 * t + 1);   // its V keys: these and the ones after
    for (int i = t_begin; i < t_end; i += kFewWarps) {
      if (ok && !mbar_await(&bar_full[warp][st], phase)) {
        ok = false;       // no more copies; those in flight get as long again to land
#pragma unroll 1
        for (int s = st; s < st + kFewStages && i + (s - st) * kFewWarps < t_end; ++s)
          mbar_wait(&bar_full[warp][s % kFewStages], s < kFewStages ? phase : phase ^ 1);
      }
      const int key0 = tiles.key0(i);
      uint8_t *tile = ring + st * C::kStageBytes;
      // keys that some row may not see: the tree, and the window's borders.  Those
      // that none sees lose their value scales where they lie (a test at each use
      // took 5% more time of long prefixes).
      const bool whole = key0 + kFewTile <= G.L &&
                         (p.window == 0 || key0 + kFewTile <= p.sinks || key0 >= G.L + G.n - p.window);
      if (!whole) {
        if (!LiveKeys(G.L, G.keys, p.window, p.sinks)(key0 + lane)) {
          uint32_t *scales = reinterpret_cast<uint32_t *>(tile + lane * R + D + D / 16);
#pragma unroll
          for (int e = 0; e < D / 64; ++e) scales[e] = 0u;
        }
        fence_proxy_async_smem();       // before the stage's next copy
        __syncwarp();
      }
      float sc[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t kw[2][kWords], ks[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint8_t *rec = tile + (16 * mt + kn + e) * R;
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(rec + 16 * t);
            kw[e][0] = w.x; kw[e][1] = w.y; kw[e][2] = w.z; kw[e][3] = w.w;
            ks[e] = *reinterpret_cast<const uint16_t *>(rec + D + 2 * t);
          } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(rec + 8 * t);
            kw[e][0] = w.x; kw[e][1] = w.y;
            ks[e] = rec[D + t];
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          uint32_t h0[4], h1[4];
          kv4_codes_to_half2(kw[0][w], h0);
          kv4_codes_to_half2(kw[1][w], h1);
          const uint32_t s0 = kv4_scale_half2(w < 2 ? ks[0] & 0xFFu : ks[0] >> 8);
          const uint32_t s1 = kv4_scale_half2(w < 2 ? ks[1] & 0xFFu : ks[1] >> 8);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h0[e] = mul_half2(h0[e], s0);
            h1[e] = mul_half2(h1[e], s1);
          }
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int part = 0; part < NP; ++part)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const int s = 2 * w + half;
                uint2 q;
                if constexpr (C::kQInRegs) q = make_uint2(qf[part][s][nt][0], qf[part][s][nt][1]);
                else q = sq[((part * KS + s) * NT + nt) * 32 + lane];
                if (s == 0 && part == 0)
                  mma_16816_first(sc[mt][nt], h0[0], h1[0], h0[1], h1[1], q.x, q.y);
                else
                  mma_16816(sc[mt][nt], h0[2 * half], h1[2 * half], h0[2 * half + 1], h1[2 * half + 1], q.x, q.y);
              }
        }
      }
      if (!whole) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 8 * nt + 2 * t + e;
            const RowKeys see = {p.window ? p.sinks : 0, s_first[r], s_tree[r]};
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (!row_sees(see, key0 + 16 * mt + kn + k, G.L, G.keys)) sc[mt][nt][2 * k + e] = -INFINITY;
          }
      }
      // x = score - reference + 8, in powers of two, and whether a reference moves
      float pw[2][NT][4], mx[NT][2];
      bool want = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              pw[mt][nt][2 * k + e] = fmaf(sc[mt][nt][2 * k + e], c_row[nt][e], nbase[nt][e]);
          mx[nt][e] = fmaxf(fmaxf(pw[0][nt][e], pw[0][nt][2 + e]), fmaxf(pw[1][nt][e], pw[1][nt][2 + e]));
          want |= mx[nt][e] > limit[nt][e];
        }
      // The weights, in fp32 calls at the present references, which hardly ever
      // move, before the vote on them (16 rows, 256 units behind 4096: 65.7 -> 62.8
      // us; bf16 calls have little to overlap: 178 -> 180 us on long prefixes)
      auto weigh = [&] {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) pw[mt][nt][e] = fast_exp2(pw[mt][nt][e]);
      };
      if (F32) weigh();
      if (__any_sync(0xffffffffu, want)) {
        bool again = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = mx[nt][e];
#pragma unroll
            for (int x = 4; x < 32; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            if (m > limit[nt][e]) {
              const bool fresh = limit[nt][e] == -INFINITY, far = far_above(m, nbase[nt][e], fresh);
              const Move move(m, nbase[nt][e], fresh);        // (far: a factor of 0)
              l_row[nt][e] *= move.factor;
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                o[nt][j][e] *= move.factor;
                o[nt][j][2 + e] *= move.factor;
              }
              nbase[nt][e] = far ? kWeightLog2 : move.next;
              limit[nt][e] = far ? -INFINITY : kWeightLog2 + kMoveLog2;
              again |= far;
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float x = fmaf(sc[mt][nt][2 * k + e], c_row[nt][e], move.base) - move.less;
                  pw[mt][nt][2 * k + e] = F32 ? fast_exp2(x) : x;
                }
            }
          }
        if (__any_sync(0xffffffffu, again)) {
          i -= kFewWarps;
          continue;
        }
      }
      if (!F32) weigh();
      // ---- weights, and their product with V
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t pf[NP][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float p0 = pw[mt][nt][2 * k], p1 = pw[mt][nt][2 * k + 1];
            l_row[nt][0] += p0;
            l_row[nt][1] += p1;
            const uint32_t h = pack_half2(p0, p1);
            pf[0][nt][k] = movmatrix(h);
            if constexpr (F32) {
              const float2 f = unpack_half2(h);
              pf[1][nt][k] = movmatrix(pack_half2(p0 - f.x, p1 - f.y));
            }
          }
        // keys kv0, kv1 (k index 2t, 2t + 1), and the ones after them (+ 8)
        uint32_t vw[4][D / 64];
        uint32_t vs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 16 * mt + ((e & 1) ? kv1 : kv0) + (e >> 1);
          const uint8_t *rec = tile + key * R;
          if constexpr (D == 128) {
            const uint2 w = *reinterpret_cast<const uint2 *>(rec + D / 2 + 8 * g);
            vw[e][0] = w.x; vw[e][1] = w.y;
            vs[e] = rec[D + D / 16 + g];
          } else {
            vw[e][0] = *reinterpret_cast<const uint32_t *>(rec + D / 2 + 4 * g);
            vs[e] = rec[D + D / 16 + g / 2];
          }
        }
        const uint32_t sa = (vs[0] << 7) | (vs[1] << 23), sb = (vs[2] << 7) | (vs[3] << 23);
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint32_t ae[4], ao[4], be[4], bo[4];   // even and odd dims of the first and second key pair
          kv4_codes_to_half2((vw[0][w] & 0x0F0F0F0Fu) | ((vw[1][w] << 4) & 0xF0F0F0F0u), ae);
          kv4_codes_to_half2(((vw[0][w] >> 4) & 0x0F0F0F0Fu) | (vw[1][w] & 0xF0F0F0F0u), ao);
          kv4_codes_to_half2((vw[2][w] & 0x0F0F0F0Fu) | ((vw[3][w] << 4) & 0xF0F0F0F0u), be);
          kv4_codes_to_half2(((vw[2][w] >> 4) & 0x0F0F0F0Fu) | (vw[3][w] & 0xF0F0F0F0u), bo);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a0 = mul_half2(ae[e], sa), a1 = mul_half2(ao[e], sa);
            const uint32_t a2 = mul_half2(be[e], sb), a3 = mul_half2(bo[e], sb);
#pragma unroll
            for (int part = 0; part < NP; ++part)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16816(o[nt][4 * w + e], a0, a1, a2, a3, pf[part][nt][0], pf[part][nt][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0 && ok && i + kFewStages * kFewWarps < t_end) request(i + kFewStages * kFewWarps, st);
      if (++st == kFewStages) {
        st = 0;
        phase ^= 1;
      }
    }
    if (!ok && lane == 0) s_timeout = 1;

    // ---- the warps' parts of each row, then the splits'
    __syncthreads();     // every ring is read; no copy is in flight unless a wait ran out
    const bool timed_out = s_timeout != 0;
    if (timed_out && tid == 0) report(a.status, b, SPEC_ERR_TIMEOUT);
    float *so = reinterpret_cast<float *>(smem);      // [warp][row][kOStride]
    if (!timed_out) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nt + 2 * t + e;
          float l = l_row[nt][e];
#pragma unroll
          for (int x = 4; x < 32; x *= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
          if (g == 0) {
            s_m[warp][r] = limit[nt][e] == -INFINITY ? -INFINITY : kWeightLog2 - nbase[nt][e];
            s_l[warp][r] = l;
          }
          float *dst = so + (warp * C::kRows + r) * C::kOStride + (D / 8) * g;
#pragma unroll
          for (int j = 0; j < KS; ++j)
            *reinterpret_cast<float2 *>(dst + 2 * j) = make_float2(o[nt][j][e], o[nt][j][2 + e]);
        }
    }
    __syncthreads();
    auto out_row = [&](int r) -> E * {
      const int node = (row0 + r) / a.G;
      if (!in_bounds(G.lo + node, a.T, a.status, b)) return nullptr;
      return static_cast<E *>(a.o) + (static_cast<size_t>(G.lo + node) * a.Hq + g_kv * a.G + (row0 + r) % a.G) * D;
    };
    if (!merge_rows<D, kFewWarps, C::kRows, kFewThreads, E>(
            tid, CS, split, rows_here, timed_out, so, s_m, s_l, s_ml, reinterpret_cast<float4 *>(smem + C::kOffRecv),
            [] { cluster_wait(); }, out_row))
      return;
    fence_proxy_async_smem();
    __syncthreads();    // all is read, before this CTA's next arrival says so and the ring is filled again
  }
}

// Up to 8 rows: eight warps a CTA where CTAs are few, else four.
inline bool few_narrow(long long units, int cs) { return units * cs > 2 * sm_count(); }

template <int D, int NT, int W, bool F32>
struct FewKernel {
  static KernelState state;
};
template <int D, int NT, int W, bool F32>
KernelState FewKernel<D, NT, W, F32>::state;

// A launch of `cs` splits (a cluster) of every unit, a unit being one block of
// rows of one (request, KV head).
template <int D, int NT, int W, bool F32>
int launch_few(const Kv4AttnArgs &p, int blocks, int cs, int dev, void *stream) {
  using C = FewCfg<D, NT, W, F32>;
  auto kernel = tree_attn_kv4_few_kernel<D, NT, W, F32>;
  if (!allow_clusters(kernel, C::kSmem, dev, &FewKernel<D, NT, W, F32>::state)) return SPEC_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, cs, 32 * W, C::kSmem);
  cfg.gridDim = dim3(cs, static_cast<unsigned>(blocks), static_cast<unsigned>(p.a.B * p.a.Hkv));
  cfg.stream = static_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// Splits of the keys, by the time they are expected to take, fitted to forced
// splits of 3 to 200 units behind 500 to 32000 keys.
//
// Fewer units than SMs: a warp's tile of 32 keys takes kTile[0] us while an SM has
// one CTA of W warps, kTile[1] where two fill it; clusters of three and more are
// placed unevenly, so that the step between the two begins early.  kFixed: set-up,
// first tile and output, without and with a merge of splits.  (One token, 8 query
// heads, 40 and 76 units behind 4000 keys 12.3 -> 10.8 and 19.9 -> 15.5 us against
// a plan for evenly filled SMs; 16 fp32 rows, 40 units 28.3 -> 18.8.)
//
// More units: CTAs follow one another, and what counts is the SM's issue slots,
// 0.47 us a tile and CTA of four warps.
template <int D, int NT, bool F32>
int few_splits(const Kv4AttnArgs &p, long long units, int max_prefix, int dev) {
  constexpr int W = NT == 1 ? 8 : 4;
  using C = FewCfg<D, NT, W, F32>;
  auto kernel = tree_attn_kv4_few_kernel<D, NT, W, F32>;
  KernelState *state = &FewKernel<D, NT, W, F32>::state;
  if (!allow_clusters(kernel, C::kSmem, dev, state)) return 0;
  constexpr double kTile[2] = {NT == 1 ? 1.0 : NT == 2 ? 1.2 : 1.9, NT == 1 ? 1.88 : NT == 2 ? 2.0 : 3.5};
  constexpr double kFixed[2] = {NT == 1 ? 4.4 : NT == 2 ? 4.4 : 10.0, NT == 1 ? 5.2 : NT == 2 ? 6.5 : 11.8};
  long long keys = static_cast<long long>(max_prefix) + mean_nodes(p.a);
  if (p.window) {
    const long long near = static_cast<long long>(p.window) + p.sinks + mean_nodes(p.a) + 2 * kFewTile;
    if (near < keys) keys = near;
  }
  const long long tiles = (keys + kFewTile - 1) / kFewTile, sms = sm_count();
  int best = 1;
  double least = -1;
  for (const int cs : {1, 2, 3, 4, 6, 8, 16}) {
    if (cs > 1 && tiles < 4 * cs) break;
    double us;
    if (units < sms) {
      const int at_once = clusters_at_once(kernel, cs, 32 * W, C::kSmem, dev, state);     // two CTAs on an SM
      if (at_once < 1) continue;
      const bool narrow = NT == 1 && few_narrow(units, cs);      // CTAs of half the warps
      const int warps = cs * (narrow ? W / 2 : W);
      const double fill = static_cast<double>(units) / (narrow ? at_once : 0.5 * at_once);     // 2: full
      const double step = cs <= 2 ? (fill > 1 ? 1.0 : 0.0) : fill < 0.4 ? 0.0 : fill > 1 ? 1.0 : (fill - 0.4) / 0.6;
      const double waves = fill <= 2 ? 1.0 : ceil(0.5 * fill);
      us = waves * (static_cast<double>((tiles + warps - 1) / warps) * (kTile[0] + step * (kTile[1] - kTile[0])) +
                    kFixed[cs > 1]);
    } else {
      if (cs > 8 || cs % 3 == 0) continue;       // (200 units: 35.6 us with 3 splits, 33.0 with 1 or 2)
      const double per_sm = static_cast<double>((units * cs + sms - 1) / sms);
      const double per_tile = 0.47 * per_sm > 1.0 ? 0.47 * per_sm : 1.0;
      const double fixed = (cs > 1 ? 4.5 : 3.0) * (per_sm > 4 ? per_sm / 4 : 1.0);
      us = static_cast<double>((tiles + 4 * cs - 1) / (4 * cs)) * per_tile + fixed;
    }
    if (least < 0 || us < least) {
      least = us;
      best = cs;
    }
  }
  return best;
}

template <int D, int NT, bool F32>
int split_few(const Kv4AttnArgs &p, int blocks, int max_prefix, void *stream) {
  const int dev = current_device();
  if (dev < 0) return SPEC_ERR_CUDA;
  const long long units = static_cast<long long>(p.a.B) * p.a.Hkv * blocks;
  const int cs = few_splits<D, NT, F32>(p, units, max_prefix, dev);
  if (cs < 1) return SPEC_ERR_CUDA;
  if constexpr (NT == 1)
    return few_narrow(units, cs) ? launch_few<D, 1, 4, F32>(p, blocks, cs, dev, stream)
                                 : launch_few<D, 1, 8, F32>(p, blocks, cs, dev, stream);
  else return launch_few<D, NT, 4, F32>(p, blocks, cs, dev, stream);
}

template <int D, bool F32>
int attn_few(const Kv4AttnArgs &p, int max_prefix, void *stream) {
  const int rows = mean_nodes(p.a) * p.a.G;
  if constexpr (F32) {      // (bf16 has other kernels for more than 8 rows)
    if (rows > 16) return split_few<D, 4, true>(p, (rows + 31) / 32, max_prefix, stream);
    if (rows > 8) return split_few<D, 2, true>(p, 1, max_prefix, stream);
  }
  return split_few<D, 1, F32>(p, 1, max_prefix, stream);
}

// Slots, and the ends of the tiles that hold them, are counted in 32 bits.
constexpr int kMaxSlots = 0x7FFFFFFF - 1024;

// Which bf16 kernel: by the mean number of rows on each key (a request with
// more takes more turns).  Measured, 256 units (32 heads x 8 requests) behind 8192
// and 2048 keys, D = 128 | 64, us; in brackets the kernels not taken, of which
// mma.sync takes 9 rows and along N 33 rows as two blocks:
//    8 rows  mma.sync 62.4, 22.0 | 43.9, 15.2    (along N 81.1, 30.5 | 70.6, 27.4)
//    9 rows  along N  81.2, 30.9 | 70.5, 27.4    (mma.sync 117, 39.0 | 79.3, 26.4)
//   32 rows  along N  101, 36.7 | 94.1, 32.9     (along M 133, 45.9 | 120, 40.6)
//   33 rows  along M  133, 46.0 | 121, 41.1      (along N 200, 70.2 | 183, 63.5)
// Short calls at D = 64 are the exception: 9 rows behind 512 keys take 15.8 us along
// N and 12.2 in mma.sync, in a window of 1024 21.6 and 17.2.
template <int D>
int attn_bf16(const Kv4AttnArgs &p, int max_prefix, void *stream) {
  const int rows = mean_nodes(p.a) * p.a.G;
  if (rows <= 8) return attn_few<D, false>(p, max_prefix, stream);
  return rows <= 32 ? launch_kv4_tc(p, max_prefix, stream) : launch_kv4_rows(p, max_prefix, stream);
}

}  // namespace

}  // namespace spec

extern "C" int spec_tree_attn_kv4(const void *q, const void *kv_cache, void *o, int dtype, int B, int T,
                                  int Hq, int Hkv, int D, int S_cap, int max_prefix,
                                  const int32_t *prefix_lens, const int32_t *tree_offsets,
                                  const uint32_t *mask, const int32_t *parents, float softmax_scale,
                                  int window, int sinks, int32_t *status, void *stream) {
  using namespace spec;
  if (!q || !kv_cache || !o || !prefix_lens || !tree_offsets || (!mask && !parents) || !status)
    return SPEC_ERR_NULL;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  if (B < 1 || T < 1 || T > static_cast<long long>(B) * SPEC_MAX_TREE_NODES || Hq < 1 || Hkv < 1 || Hq % Hkv ||
      Hq / Hkv > 128 || S_cap < 1 || max_prefix < 0 || window < 0 || sinks < 0)
    return SPEC_ERR_SHAPE;
  if (D != 64 && D != 128) return SPEC_ERR_SHAPE;
  if (S_cap > kMaxSlots || static_cast<long long>(B) * Hkv > 65535) return SPEC_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(kv_cache) | reinterpret_cast<uintptr_t>(o) |
       reinterpret_cast<uintptr_t>(mask)) & 15)
    return SPEC_ERR_ALIGNMENT;
  Kv4AttnArgs p = {};
  p.a.q = q;
  p.a.k = kv_cache;
  p.a.o = o;
  p.a.prefix_lens = prefix_lens;
  p.a.offsets = tree_offsets;
  p.a.mask = reinterpret_cast<const uint4 *>(mask);
  p.a.parents = mask ? nullptr : parents;
  p.a.status = status;
  p.a.B = B;
  p.a.T = T;
  p.a.Hq = Hq;
  p.a.Hkv = Hkv;
  p.a.G = Hq / Hkv;
  p.a.D = D;
  p.a.S_cap = S_cap;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf(static_cast<float>(D));
  p.a.scale_log2 = scale * 1.4426950408889634f;
  // positions stay below S_cap: a window that large hides nothing
  p.window = window < S_cap ? window : S_cap;
  p.sinks = sinks < S_cap ? sinks : S_cap;
  if (dtype == SPEC_BF16)
    return D == 128 ? attn_bf16<128>(p, max_prefix, stream) : attn_bf16<64>(p, max_prefix, stream);
  return D == 128 ? attn_few<128, true>(p, max_prefix, stream) : attn_few<64, true>(p, max_prefix, stream);
}
