// Attention of trees and chunks over a paged cache, fp32 throughout.
//
// One CTA = one split of the keys x one block of query rows (node-major, head-minor)
// of one request and KV head.  Products go two at a time (fma.rn.f32x2).
//
// Blocks of 4 or 8 rows: a warp takes 8 or 4 keys at a time, straight from memory into
// registers, and nothing but the weights passes through shared memory.  Memory bounds
// it: a token of 4 query heads each, D = 128, of 64 requests x 8 heads behind 1000 keys
// 87 us (6.1 TB/s, 0.9 of a copy), of 1024 behind 200 323; of 4 requests behind 4096
// 27.  (Tiles of 32 keys in shared memory for 16 rows, whose products read their
// operands there: 248, 620 and 77.)
//
// Blocks of 64 rows: sixteen threads share four rows; of a tile of 32 keys each has the
// scores of two, and of the output eight dims, so that a row's maximum, sum and weights
// stay within half a warp.  Keys and values arrive by asynchronous copies, the keys of
// the next tile beside the output's products and its values beside the scores'.
// Products and shared memory bound it (a chunk of 512 rows x 32 heads behind 4096 keys,
// D = 128: 1.17 ms, 32 TFLOP/s).
#include "attn_paged.cuh"

namespace spec {

namespace {

constexpr int kKeys = 32;      // of a tile

__device__ __forceinline__ void copy_16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int left>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(left) : "memory");
}

// acc += a b, two at once.
__device__ __forceinline__ void madd2(float2 &acc, float2 a, float2 b) {
  asm("{\n\t.reg .b64 s, x, y;\n\t"
      "mov.b64 s, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "fma.rn.f32x2 s, x, y, s;\n\tmov.b64 {%0, %1}, s;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
}

template <int D>
struct F32Cfg {
  static constexpr int R = 64, kTile = kKeys;
  static constexpr int kMine = 4;             // rows of a thread
  static constexpr int kThreads = R / kMine * 16, kCost = 9;
  static constexpr int kRow = D + 4;          // floats of a row of q, keys or the result: sixteen rows on all banks
  static constexpr int kP = kKeys + 4;
  static constexpr int kOffK = R * kRow, kOffV = kOffK + kKeys * kRow, kOffP = kOffV + kKeys * D;
  static constexpr int kEnd = kOffP + R * kP;
  // (the result's rows take the place of all)
  static constexpr int kSmem = kEnd * 4 > merge_bytes<D>(R) ? kEnd * 4 : merge_bytes<D>(R);
};

template <int D>
__global__ void __launch_bounds__(F32Cfg<D>::kThreads)
tree_attn_paged_f32_kernel(const PagedAttnArgs p, const int CS) {
  using C = F32Cfg<D>;
  constexpr int R = C::R, kMine = C::kMine;
  constexpr int kDims = D / 16;               // of a thread: kDims / 4 groups of four
  const AttnArgs &a = p.a;
  extern __shared__ __align__(16) float sm[];
  __shared__ uint64_t s_bar;
  __shared__ long long s_slot[2][kKeys];
  __shared__ long long s_row[R];
  __shared__ int s_par[SPEC_MAX_TREE_NODES];
  const int split = static_cast<int>(blockIdx.x) % CS, block = static_cast<int>(blockIdx.x) / CS;
  const int g_kv = static_cast<int>(blockIdx.y), tid = threadIdx.x, lane = tid & 31;
  const int tx = tid & 15, r0 = (tid >> 4) * kMine;    // this thread's keys tx and tx + 16, and its rows from r0 on
  pdl_trigger();
  if (tid == 0) {
    mbar_init(&s_bar, 1);
    fence_barrier_init();
  }
  pdl_wait();
  if (tid < 32) touch_table(p, lane);
  const RowBlock w = find_block<R>(p, block, lane);
  if (g_kv == 0 && tid < 32) report_bad_requests(p, lane);
  if (w.b < 0) return;       // the same for every CTA of the cluster
  const int b = w.b, L = w.R.L;
  const int all = (w.keys + kKeys - 1) / kKeys, per = (all + CS - 1) / CS, t0 = split * per;
  const int ntiles = max(0, min(t0 + per, all) - t0);
  const uint32_t sb = smem_addr(sm);

  bool bad = false;                      // a page outside the pool, anywhere in the request
  const int pages = (w.R.keys + (1 << p.pages.shift) - 1) >> p.pages.shift;
#pragma unroll 4
  for (int i = tid; i < pages; i += C::kThreads) bad |= p.pages.page(b, i) < 0;

  // where the slots of tile i lie in the pools (first element; -1: no key), a tile
  // ahead of the copies: a look-up per copy took longer than the products
  auto look_up = [&](int i) {
    if (tid >= kKeys) return;
    const int key = (t0 + i) * kKeys + tid;
    long long at = -1;
    if (i < ntiles && key < w.keys) {
      const int page = max(0, p.pages.page(b, key >> p.pages.shift));
      at = ((static_cast<long long>(page) * a.Hkv + g_kv) << p.pages.shift) + (key & ((1 << p.pages.shift) - 1));
      at = p.pages.holds(at, 1, a.Hkv, b) ? at * D : -1;
    }
    s_slot[i & 1][tid] = at;
  };
  auto bring = [&](int i, const void *pool, int off, int stride) {
    if (i < ntiles) {
#pragma unroll 4
      for (int u = tid; u < kKeys * (D / 4); u += C::kThreads) {
        const int r = u / (D / 4), c = u % (D / 4) * 4;
        const long long slot = s_slot[i & 1][r];
        copy_16(sb + (off + r * stride + c) * 4, static_cast<const float *>(pool) + (slot < 0 ? 0 : slot) + c, slot >= 0);
      }
    }
    copies_end();
  };
  look_up(0);
  __syncthreads();
  bring(0, a.k, C::kOffK, C::kRow);
  bring(0, a.v, C::kOffV, D);

  // ---- Q, and what the rows see
  auto first_of = [&](int r) -> long long {
    const int node = (w.row0 + r) / a.G;
    if (r >= w.rows || !in_bounds(w.R.lo + node, a.T, a.status, b)) return -1;
    return (static_cast<long long>(w.R.lo + node) * a.Hq + g_kv * a.G + (w.row0 + r) - node * a.G) * D;
  };
  for (int r = tid; r < R; r += C::kThreads) s_row[r] = first_of(r);
  if (a.parents)
    for (int i = tid; i < w.R.n; i += C::kThreads)
      s_par[i] = in_bounds(w.R.lo + i, a.T, a.status, b) ? __ldg(a.parents + w.R.lo + i) : -2;
  __syncthreads();
  for (int i = tid; i < R * (D / 4); i += C::kThreads) {
    const int r = i / (D / 4), c = i % (D / 4);
    const float4 q = s_row[r] < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                  : __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + s_row[r]) + c);
    *reinterpret_cast<float4 *>(sm + r * C::kRow + 4 * c) = q;
  }
  RowSees see[kMine];
#pragma unroll
  for (int r = 0; r < kMine; ++r) {
    const int node = (w.row0 + r0 + r) / a.G;
    see[r].until = p.causal ? L + node + 1 : L;
    see[r].tree = make_uint4(0u, 0u, 0u, 0u);
    if (p.causal || s_row[r0 + r] < 0) continue;
    if (a.mask) {
      see[r].tree = clip_mask(__ldg(a.mask + w.R.lo + node), w.R.n);
    } else {
      bool wrong = false;
      see[r].tree = ancestor_mask([&](int i) { return s_par[i]; }, node, &wrong);
      if (wrong) report(a.status, b, SPEC_ERR_BAD_PARENT);
    }
  }
  const int all_see = p.causal ? L + w.row0 / a.G + 1 : L;

  float2 o[kMine][kDims / 2] = {};
  float ref[kMine], sum[kMine];      // references in powers of two; sums of this thread's keys
#pragma unroll
  for (int r = 0; r < kMine; ++r) {
    ref[r] = -INFINITY;
    sum[r] = 0.f;
  }
  const float c2 = a.scale_log2;
  for (int i = 0; i < ntiles; ++i) {
    const int key0 = (t0 + i) * kKeys;
    copies_wait<1>();
    __syncthreads();
    look_up(i + 1);
    // ---- scores: the thread's rows x two keys, even and odd dims apart
    float s[kMine][2];
    {
      const float *q = sm + r0 * C::kRow, *k = sm + C::kOffK + tx * C::kRow;
      float2 dot[kMine][2] = {};
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 k0 = *reinterpret_cast<const float4 *>(k + d);
        const float4 k1 = *reinterpret_cast<const float4 *>(k + 16 * C::kRow + d);
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
          const float4 x = *reinterpret_cast<const float4 *>(q + r * C::kRow + d);
          madd2(dot[r][0], make_float2(x.x, x.y), make_float2(k0.x, k0.y));
          madd2(dot[r][1], make_float2(x.x, x.y), make_float2(k1.x, k1.y));
          madd2(dot[r][0], make_float2(x.z, x.w), make_float2(k0.z, k0.w));
          madd2(dot[r][1], make_float2(x.z, x.w), make_float2(k1.z, k1.w));
        }
      }
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
        s[r][0] = dot[r][0].x + dot[r][0].y;
        s[r][1] = dot[r][1].x + dot[r][1].y;
      }
    }
    __syncthreads();
    bring(i + 1, a.k, C::kOffK, C::kRow);
    // ---- weights
#pragma unroll
    for (int r = 0; r < kMine; ++r) {
      if (key0 + kKeys > all_see) {
        const uint32_t sees = sees_32(see[r], key0, L);
        if (!((sees >> tx) & 1u)) s[r][0] = -INFINITY;
        if (!((sees >> tx >> 16) & 1u)) s[r][1] = -INFINITY;
      }
      float top = fmaxf(s[r][0], s[r][1]);
#pragma unroll
      for (int d = 8; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      top = fmaxf(ref[r], top * c2);
      const float factor = ref[r] == top ? 1.f : ref[r] == -INFINITY ? 0.f : exp2f(ref[r] - top);
      ref[r] = top;
      const float base = top == -INFINITY ? 0.f : -top;
      // one rounding of s c - ref, but for references without places behind the
      // point, where the largest score's own rounding has to cancel
      const bool steep = !(fabsf(base) < 16777216.f);
      float weight[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        weight[e] = fast_exp2(steep ? __fadd_rn(__fmul_rn(s[r][e], c2), base) : fmaf(s[r][e], c2, base));
      sum[r] = sum[r] * factor + weight[0] + weight[1];
#pragma unroll
      for (int d = 0; d < kDims / 2; ++d) {
        o[r][d].x *= factor;
        o[r][d].y *= factor;
      }
      sm[C::kOffP + (r0 + r) * C::kP + tx] = weight[0];
      sm[C::kOffP + (r0 + r) * C::kP + tx + 16] = weight[1];
    }
    copies_wait<1>();
    __syncthreads();
    // ---- output: the thread's rows x eight dims (four at D = 64)
#pragma unroll 2
    for (int j = 0; j < kKeys; j += 4) {
      float4 weight[kMine];
#pragma unroll
      for (int r = 0; r < kMine; ++r)
        weight[r] = *reinterpret_cast<const float4 *>(sm + C::kOffP + (r0 + r) * C::kP + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int g = 0; g < kDims / 4; ++g) {
          const float4 v = *reinterpret_cast<const float4 *>(sm + C::kOffV + (j + e) * D + 64 * g + 4 * tx);
#pragma unroll
          for (int r = 0; r < kMine; ++r) {
            const float x = (&weight[r].x)[e];
            madd2(o[r][2 * g], make_float2(x, x), make_float2(v.x, v.y));
            madd2(o[r][2 * g + 1], make_float2(x, x), make_float2(v.z, v.w));
          }
        }
      }
    }
    __syncthreads();
    bring(i + 1, a.v, C::kOffV, D);
  }
  copies_wait<0>();
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) report(a.status, b, SPEC_ERR_PAGE);
  // ---- the rows take q's place
#pragma unroll
  for (int r = 0; r < kMine; ++r) {
#pragma unroll
    for (int d = 8; d; d /= 2) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], d);
    if (tx == 0) *reinterpret_cast<float2 *>(sm + (r0 + r) * C::kRow + D) = make_float2(ref[r], bad ? -1.f : sum[r]);
#pragma unroll
    for (int g = 0; g < kDims / 4; ++g)
      *reinterpret_cast<float4 *>(sm + (r0 + r) * C::kRow + 64 * g + 4 * tx) =
          make_float4(o[r][2 * g].x, o[r][2 * g].y, o[r][2 * g + 1].x, o[r][2 * g + 1].y);
  }
  auto out_row = [&](int r) { return s_row[r] < 0 ? nullptr : static_cast<float *>(a.o) + s_row[r]; };
  if (!merge_splits<D, C::kThreads, float>(tid, CS, split, w.rows, sm, &s_bar, out_row) && tid == 0)
    report(a.status, b, SPEC_ERR_TIMEOUT);
}

// Few rows (R of them, 4 or 8): a warp takes K = 32 / R keys at a time, a lane D / 32
// dims of each, straight from memory; rows of Q, the weighted sum and the loads under
// way are registers.  The 32 products of a step are summed over the lanes so that
// lane r K + j is left with row r's score of key j.  K keys that start at a multiple of
// K lie in one page.
template <int D, int kR>
struct FewCfg {
  static constexpr int R = kR, kCost = 2;
  static constexpr int kWarps = 8, kThreads = 32 * kWarps, kStep = 32 / R, kTile = kWarps * kStep;
  static constexpr int kPart = merge_bytes<D>(R) / 4;      // floats: the merge's rows, then the warps'
  static constexpr int kSmem = (kPart + kWarps * R * (D + 4)) * 4;
};

template <int V>
struct Dims {
  float2 x[V / 2];
};

template <int V>
__device__ __forceinline__ Dims<V> load_dims(const float *p) {
  Dims<V> d;
  if constexpr (V == 4) {
    const float4 v = __ldcs(reinterpret_cast<const float4 *>(p));
    d.x[0] = make_float2(v.x, v.y);
    d.x[1] = make_float2(v.z, v.w);
  } else {
    d.x[0] = __ldcs(reinterpret_cast<const float2 *>(p));
  }
  return d;
}

template <int D, int R>
__global__ void __launch_bounds__(FewCfg<D, R>::kThreads, 2)
tree_attn_paged_f32_few_kernel(const PagedAttnArgs p, const int CS) {
  using C = FewCfg<D, R>;
  constexpr int K = C::kStep, V = D / 32;
  const AttnArgs &a = p.a;
  extern __shared__ __align__(16) float sm[];
  __shared__ uint64_t s_bar;
  __shared__ long long s_row[R];
  __shared__ int s_par[SPEC_MAX_TREE_NODES];
  __shared__ __align__(16) float s_weight[C::kWarps][32];
  const int split = static_cast<int>(blockIdx.x) % CS, block = static_cast<int>(blockIdx.x) / CS;
  const int g_kv = static_cast<int>(blockIdx.y), tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int r_mine = lane / K, j_mine = lane % K;      // this lane's score: row and key of a step
  pdl_trigger();
  if (tid == 0) {
    mbar_init(&s_bar, 1);
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == 0) touch_table(p, lane);
  const RowBlock w = find_block<R>(p, block, lane);
  if (g_kv == 0 && warp == 0) report_bad_requests(p, lane);
  if (w.b < 0) return;       // the same for every CTA of the cluster
  const int b = w.b, L = w.R.L;
  const int all = (w.keys + C::kTile - 1) / C::kTile, per = (all + CS - 1) / CS, t0 = split * per;
  const int ntiles = max(0, min(t0 + per, all) - t0);

  // where this warp's keys of tile i start in the pools (any page will do for an id
  // outside the pool: no row is written)
  auto look_up = [&](int i) -> long long {
    const int key = (t0 + i) * C::kTile + warp * K;
    if (i >= ntiles || key >= w.keys) return 0;
    const long long page = max(0, p.pages.page(b, key >> p.pages.shift));
    const long long row = ((page * a.Hkv + g_kv) << p.pages.shift) + (key & ((1 << p.pages.shift) - 1));
    return (p.pages.holds(row, min(K, w.keys - key), a.Hkv, b) ? row * D : 0) + lane * V;
  };
  long long at = look_up(0);

  // ---- Q, and what this lane's row sees
  auto first_of = [&](int r) -> long long {
    const int node = (w.row0 + r) / a.G;
    if (r >= w.rows || !in_bounds(w.R.lo + node, a.T, a.status, b)) return -1;
    return (static_cast<long long>(w.R.lo + node) * a.Hq + g_kv * a.G + (w.row0 + r) - node * a.G) * D;
  };
  if (tid < R) s_row[tid] = first_of(tid);
  if (a.parents)
    for (int i = tid; i < w.R.n; i += C::kThreads)
      s_par[i] = in_bounds(w.R.lo + i, a.T, a.status, b) ? __ldg(a.parents + w.R.lo + i) : -2;
  __syncthreads();
  Dims<V> q[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    q[r] = Dims<V>{};
    if (s_row[r] >= 0) q[r] = load_dims<V>(static_cast<const float *>(a.q) + s_row[r] + lane * V);
  }
  RowSees see;
  {
    const int node = (w.row0 + r_mine) / a.G;
    see.until = p.causal ? L + node + 1 : L;
    see.tree = make_uint4(0u, 0u, 0u, 0u);
    if (!p.causal && s_row[r_mine] >= 0) {
      if (a.mask) {
        see.tree = clip_mask(__ldg(a.mask + w.R.lo + node), w.R.n);
      } else {
        bool wrong = false;
        see.tree = ancestor_mask([&](int i) { return s_par[i]; }, node, &wrong);
        if (wrong) report(a.status, b, SPEC_ERR_BAD_PARENT);
      }
    }
  }
  const int all_see = p.causal ? L + w.row0 / a.G + 1 : L;

  Dims<V> o[R] = {};
  float ref = -INFINITY, sum = 0.f;      // this lane's row's reference, in powers of two; its weights' sum
  const float c2 = a.scale_log2;
  for (int i = 0; i < ntiles; ++i) {
    const int key0 = (t0 + i) * C::kTile + warp * K;
    if (key0 >= w.keys) break;
    const int n = min(K, w.keys - key0);
    Dims<V> k[K], v[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      k[j] = Dims<V>{};
      if (j < n) k[j] = load_dims<V>(static_cast<const float *>(a.k) + at + j * D);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      v[j] = Dims<V>{};
      if (j < n) v[j] = load_dims<V>(static_cast<const float *>(a.v) + at + j * D);
    }
    at = look_up(i + 1);
    // ---- scores: of the lane's dims, then summed over the lanes
    float s[32];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < K; ++j) {
        float2 dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int d = 0; d < V / 2; ++d) madd2(dot, q[r].x[d], k[j].x[d]);
        s[r * K + j] = dot.x + dot.y;
      }
#pragma unroll
    for (int round = 0; round < 5; ++round) {
      const int half = 16 >> round;
      const bool upper = lane & half;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e >= half) break;
        const float keep = upper ? s[e + half] : s[e], send = upper ? s[e] : s[e + half];
        s[e] = keep + __shfl_xor_sync(0xffffffffu, send, half);
      }
    }
    float score = s[0];
    // ---- weights
    const int key = key0 + j_mine;
    if (key0 + K > all_see && !(sees_32(see, key, L) & 1u)) score = -INFINITY;
    float top = score;
#pragma unroll
    for (int d = K / 2; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    top *= c2;
    // a reference moves when a score passes it by more than 2^8
    if (__any_sync(0xffffffffu, top > ref + 8.f)) {
      const float next = top > ref + 8.f ? top : ref;
      const float factor = next == ref ? 1.f : ref == -INFINITY ? 0.f : exp2f(ref - next);
      sum *= factor;
      ref = next;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = __shfl_sync(0xffffffffu, factor, r * K);
#pragma unroll
        for (int d = 0; d < V / 2; ++d) {
          o[r].x[d].x *= f;
          o[r].x[d].y *= f;
        }
      }
    }
    const float base = ref == -INFINITY ? 0.f : -ref;
    // one rounding of s c - ref, but for references without places behind the
    // point, where the largest score's own rounding has to cancel
    const bool steep = !(fabsf(base) < 16777216.f);
    const float weight = fast_exp2(steep ? __fadd_rn(__fmul_rn(score, c2), base) : fmaf(score, c2, base));
    sum += weight;
    s_weight[warp][lane] = weight;
    __syncwarp();
    // ---- output
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < K; j += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(&s_weight[warp][r * K + j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = (&x.x)[e];
#pragma unroll
          for (int d = 0; d < V / 2; ++d) madd2(o[r].x[d], make_float2(y, y), v[j + e].x[d]);
        }
      }
    __syncwarp();
  }
  bool bad = false;                      // a page outside the pool, anywhere in the request
  const int pages = (w.R.keys + (1 << p.pages.shift) - 1) >> p.pages.shift;
#pragma unroll 4
  for (int i = tid; i < pages; i += C::kThreads) bad |= p.pages.page(b, i) < 0;
  // ---- the warps' rows, then the CTA's
#pragma unroll
  for (int d = K / 2; d; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  float *part = sm + C::kPart + warp * R * (D + 4);
  if (j_mine == 0) *reinterpret_cast<float2 *>(part + r_mine * (D + 4) + D) = make_float2(ref, sum);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int d = 0; d < V / 2; ++d) *reinterpret_cast<float2 *>(part + r * (D + 4) + lane * V + 2 * d) = o[r].x[d];
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) report(a.status, b, SPEC_ERR_PAGE);
  for (int idx = tid; idx < R * (D / 4); idx += C::kThreads) {
    const int r = idx / (D / 4), c = idx % (D / 4) * 4;
    const float *from = sm + C::kPart + r * (D + 4);
    float most = -INFINITY;
#pragma unroll
    for (int u = 0; u < C::kWarps; ++u) most = fmaxf(most, from[u * R * (D + 4) + D]);
    const float zero = most == -INFINITY ? 0.f : most;
    float total = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < C::kWarps; ++u) {
      const float2 m = *reinterpret_cast<const float2 *>(from + u * R * (D + 4) + D);
      const float4 x = *reinterpret_cast<const float4 *>(from + u * R * (D + 4) + c);
      const float f = fast_exp2(m.x - zero);
      total = fmaf(f, m.y, total);
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    }
    *reinterpret_cast<float4 *>(sm + r * (D + 4) + c) = acc;
    if (c == 0) *reinterpret_cast<float2 *>(sm + r * (D + 4) + D) = make_float2(most, bad ? -1.f : total);
  }
  auto out_row = [&](int r) { return s_row[r] < 0 ? nullptr : static_cast<float *>(a.o) + s_row[r]; };
  if (!merge_splits<D, C::kThreads, float>(tid, CS, split, w.rows, sm, &s_bar, out_row) && tid == 0)
    report(a.status, b, SPEC_ERR_TIMEOUT);
}

struct Plan {
  int splits;
  long long cost;      // waves x (tiles of a CTA + its set-up and merge, in tiles); -1: not to be had
};

// As many splits of the keys as cost least.  (Device us by splits 1, 2, 3, 5 and 8 of
// 64 rows of 32 heads behind 2048 keys, D = 128, tiles of 32 keys x 64 rows: 315, 201,
// 162, 121 and 83.)
template <typename C, typename Kernel>
Plan plan(Kernel kernel, KernelState &state, const PagedAttnArgs &p, int max_prefix, int dev) {
  const long long units = likely_blocks<C::R>(p.a) * p.a.Hkv;
  const long long tiles = (static_cast<long long>(max_prefix) + mean_nodes(p.a) + C::kTile - 1) / C::kTile;
  Plan best = {1, -1};
  if (!allow_clusters(kernel, C::kSmem, dev, &state)) return best;
  for (int n = 1; n <= kMaxSplits; n = n == 8 ? kMaxSplits : n + 1) {
    if (n > 1 && tiles < n) break;
    const int slots = clusters_at_once(kernel, n, C::kThreads, C::kSmem, dev, &state);
    if (slots < 1) continue;
    const long long waves = (units + slots - 1) / slots;
    const long long cost = waves * ((tiles + n - 1) / n + (n > 1 ? 5 : 3));
    if (best.cost < 0 || cost < best.cost) best = {n, cost};
  }
  return best;
}

template <typename C, typename Kernel>
int launch(Kernel kernel, const Plan &plan, const PagedAttnArgs &p, void *stream) {
  if (plan.cost < 0) return SPEC_ERR_CUDA;
  const long long blocks = most_blocks<C::R>(p.a);
  if (blocks * plan.splits > 0x7FFFFFFFll) return SPEC_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, plan.splits, C::kThreads, C::kSmem);
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * plan.splits), static_cast<unsigned>(p.a.Hkv), 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, kernel, p, plan.splits) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// Up to 4 rows a request and KV head: blocks of 4.  More: blocks of 8, or of 64 where
// a tile of those, which takes 4.5 times as long, makes the launch shorter.
template <int D>
int launch_by_rows(const PagedAttnArgs &p, int max_prefix, void *stream) {
  static KernelState of_4, of_8, of_64;
  const int dev = current_device();
  if (dev < 0) return SPEC_ERR_CUDA;
  const long long rows = mean_nodes(p.a) * static_cast<long long>(p.a.G);
  if (rows <= 4) {
    const auto kernel = tree_attn_paged_f32_few_kernel<D, 4>;
    return launch<FewCfg<D, 4>>(kernel, plan<FewCfg<D, 4>>(kernel, of_4, p, max_prefix, dev), p, stream);
  }
  const auto kernel = tree_attn_paged_f32_few_kernel<D, 8>;
  const Plan few = plan<FewCfg<D, 8>>(kernel, of_8, p, max_prefix, dev);
  if (rows > 8) {
    const auto tiles = tree_attn_paged_f32_kernel<D>;
    const Plan many = plan<F32Cfg<D>>(tiles, of_64, p, max_prefix, dev);
    if (many.cost >= 0 && (few.cost < 0 || F32Cfg<D>::kCost * many.cost < FewCfg<D, 8>::kCost * few.cost))
      return launch<F32Cfg<D>>(tiles, many, p, stream);
  }
  return launch<FewCfg<D, 8>>(kernel, few, p, stream);
}

}  // namespace

int launch_attn_paged_f32(const PagedAttnArgs &p, int max_prefix, void *stream) {
  return p.a.D == 128 ? launch_by_rows<128>(p, max_prefix, stream) : launch_by_rows<64>(p, max_prefix, stream);
}

}  // namespace spec
