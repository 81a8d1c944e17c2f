// Attention of trees and chunks over a paged cache, fp32 throughout.
//
// One CTA = one split of the keys x one block of R query rows (node-major,
// head-minor) of one request and KV head.  Sixteen threads share four rows (two
// for R = 16): of a tile of 32 keys each has the scores of two, and of the output
// eight dims, so that a row's maximum, sum and weights stay within half a warp.
// Products go two at a time (fma.rn.f32x2).  Keys and values arrive by asynchronous
// copies, the keys of the next tile beside the output's products and its values
// beside the scores'.  R = 16 for few rows, where what 64 would multiply in vain
// costs more than reading the keys; there the copies' latency bounds it (2 us a
// tile and CTA), for many rows the products and shared memory (a chunk of 512 rows
// x 32 heads behind 4096 keys, D = 128: 1.11 ms, 33 TFLOP/s).
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

template <int D, int R>
struct F32Cfg {
  static constexpr int kMine = R == 64 ? 4 : 2;      // rows of a thread
  static constexpr int kThreads = R / kMine * 16;
  static constexpr int kRow = D + 4;          // floats of a row of q, keys or the result: sixteen rows on all banks
  static constexpr int kP = kKeys + 4;
  static constexpr int kOffK = R * kRow, kOffV = kOffK + kKeys * kRow, kOffP = kOffV + kKeys * D;
  static constexpr int kEnd = kOffP + R * kP;
  // (the result's rows take the place of all)
  static constexpr int kSmem = kEnd * 4 > merge_bytes<D>(R) ? kEnd * 4 : merge_bytes<D>(R);
};

template <int D, int R>
__global__ void __launch_bounds__(F32Cfg<D, R>::kThreads)
tree_attn_paged_f32_kernel(const PagedAttnArgs p, const int CS) {
  using C = F32Cfg<D, R>;
  constexpr int kMine = C::kMine;
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
      at = (((static_cast<long long>(page) * a.Hkv + g_kv) << p.pages.shift) + (key & ((1 << p.pages.shift) - 1))) * D;
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

// As many splits of the keys as make waves x (tiles of a CTA + its set-up and
// merge, in tiles) least.  (Device us by splits 1, 2, 3, 5 and 8: 8 rows of 4 heads
// behind 128 keys, D = 64, 12.2, 9.4, 7.7, 6.1 and 6.3; 64 rows of 32 heads behind
// 2048, D = 128, 315, 201, 162, 121 and 83.)
template <int D, int R>
int launch(const PagedAttnArgs &p, int max_prefix, void *stream) {
  using C = F32Cfg<D, R>;
  auto kernel = tree_attn_paged_f32_kernel<D, R>;
  static KernelState state;
  const int dev = current_device();
  if (dev < 0 || !allow_clusters(kernel, C::kSmem, dev, &state)) return SPEC_ERR_CUDA;
  const long long blocks = most_blocks<R>(p.a), units = likely_blocks<R>(p.a) * p.a.Hkv;
  const long long tiles = (static_cast<long long>(max_prefix) + mean_nodes(p.a) + kKeys - 1) / kKeys;
  int cs = 1;
  long long best = -1;
  for (int n = 1; n <= kMaxSplits; n = n == 8 ? kMaxSplits : n + 1) {
    if (n > 1 && tiles < n) break;
    const int slots = clusters_at_once(kernel, n, C::kThreads, C::kSmem, dev, &state);
    if (slots < 1) continue;
    const long long waves = (units + slots - 1) / slots;
    const long long cost = waves * ((tiles + n - 1) / n + (n > 1 ? 5 : 3));
    if (best < 0 || cost < best) {
      best = cost;
      cs = n;
    }
  }
  if (blocks * cs > 0x7FFFFFFFll) return SPEC_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, cs, C::kThreads, C::kSmem);
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * cs), static_cast<unsigned>(p.a.Hkv), 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, kernel, p, cs) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

int launch_attn_paged_f32(const PagedAttnArgs &p, int max_prefix, void *stream) {
  const bool few = mean_nodes(p.a) * static_cast<long long>(p.a.G) <= 16;
  if (p.a.D == 128) return few ? launch<128, 16>(p, max_prefix, stream) : launch<128, 64>(p, max_prefix, stream);
  return few ? launch<64, 16>(p, max_prefix, stream) : launch<64, 64>(p, max_prefix, stream);
}

}  // namespace spec
