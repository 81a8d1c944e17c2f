// Attention of trees and chunks over a paged cache, fp32 throughout.
//
// One CTA = one split of the keys x one block of R query rows (node-major,
// head-minor) of one request and KV head, 4 R threads.  Sixteen threads share
// four rows: of a tile of 32 keys each has the scores of two (all four rows),
// and of the output eight dims, so that a row's maximum, sum and weights stay
// within half a warp, and 32 products follow six (scores) or three (output)
// 16-byte loads from shared memory.  The products bound it: there is no tensor
// core for fp32's 24 bits.  Keys and values arrive by asynchronous copies, the
// keys of the next tile beside the output's products and its values beside the
// scores'.  R = 16 for few rows, where what 64 would multiply in vain costs more
// than reading the keys.
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

template <int D, int R>
struct F32Cfg {
  static constexpr int kThreads = 4 * R;
  static constexpr int kRow = D + 4;          // floats of a row of q, keys or the result: sixteen rows on all banks
  static constexpr int kP = kKeys + 4;
  static constexpr int kOffK = R * kRow, kOffV = kOffK + kKeys * kRow, kOffP = kOffV + kKeys * D;
  static constexpr int kEnd = kOffP + R * kP;
  // (the result's rows take the place of all)
  static constexpr int kSmem = kEnd * 4 > merge_bytes<D>(R) ? kEnd * 4 : merge_bytes<D>(R);
};

template <int D, int R>
__global__ void __launch_bounds__(4 * R)
tree_attn_paged_f32_kernel(const PagedAttnArgs p, const int CS) {
  using C = F32Cfg<D, R>;
  constexpr int kDims = D / 16;               // of a thread: kDims / 4 groups of four
  const AttnArgs &a = p.a;
  extern __shared__ __align__(16) float sm[];
  __shared__ uint64_t s_bar;
  __shared__ long long s_row[R];
  __shared__ int s_par[SPEC_MAX_TREE_NODES];
  const int split = static_cast<int>(blockIdx.x) % CS, block = static_cast<int>(blockIdx.x) / CS;
  const int g_kv = static_cast<int>(blockIdx.y), tid = threadIdx.x, lane = tid & 31;
  const int tx = tid & 15, r0 = (tid >> 4) * 4;        // this thread's keys tx and tx + 16, and rows r0 .. r0 + 3
  pdl_trigger();
  if (tid == 0) {
    mbar_init(&s_bar, 1);
    fence_barrier_init();
  }
  pdl_wait();
  if (tid < 32) touch_table(p, lane);
  const RowBlock w = find_block<R>(p, block, lane);
  if (blockIdx.x == 0 && g_kv == 0 && tid < 32) report_bad_requests(p, lane);
  if (w.b < 0) return;       // the same for every CTA of the cluster
  const int b = w.b, L = w.R.L;
  const int all = (w.keys + kKeys - 1) / kKeys, per = (all + CS - 1) / CS, t0 = split * per;
  const int ntiles = max(0, min(t0 + per, all) - t0);
  const uint32_t sb = smem_addr(sm);

  bool bad = false;                      // a page outside the pool, anywhere in the request
  const int pages = (w.R.keys + (1 << p.pages.shift) - 1) >> p.pages.shift;
#pragma unroll 4
  for (int i = tid; i < pages; i += C::kThreads) bad |= p.pages.page(b, i) < 0;

  auto bring = [&](int i, const void *pool, int off, int stride) {
    if (i < ntiles) {
      const int key0 = (t0 + i) * kKeys;
#pragma unroll
      for (int u = 0; u < kKeys * (D / 4) / C::kThreads; ++u) {
        const int at = tid + u * C::kThreads, r = at / (D / 4), c = at % (D / 4), key = key0 + r;
        const bool there = key < w.keys;
        const int page = there ? max(0, p.pages.page(b, key >> p.pages.shift)) : 0;
        const size_t slot = ((static_cast<size_t>(page) * a.Hkv + g_kv) << p.pages.shift) +
                            (there ? key & ((1 << p.pages.shift) - 1) : 0);
        copy_16(sb + (off + r * stride + 4 * c) * 4, static_cast<const float *>(pool) + slot * D + 4 * c, there);
      }
    }
    copies_end();
  };
  bring(0, a.k, C::kOffK, C::kRow);
  bring(0, a.v, C::kOffV, D);

  // ---- Q, and what the rows see
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
  for (int i = tid; i < R * (D / 4); i += C::kThreads) {
    const int r = i / (D / 4), c = i % (D / 4);
    const float4 q = s_row[r] < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                  : __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + s_row[r]) + c);
    *reinterpret_cast<float4 *>(sm + r * C::kRow + 4 * c) = q;
  }
  RowSees see[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
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

  float o[4][kDims] = {}, ref[4], sum[4];      // references in powers of two; sums of this thread's keys
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    ref[r] = -INFINITY;
    sum[r] = 0.f;
  }
  const float c2 = a.scale_log2;
  for (int i = 0; i < ntiles; ++i) {
    const int key0 = (t0 + i) * kKeys;
    copies_wait<1>();
    __syncthreads();
    // ---- scores: four rows x two keys
    float s[4][2] = {};
    {
      const float *q = sm + r0 * C::kRow, *k = sm + C::kOffK + tx * C::kRow;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 k0 = *reinterpret_cast<const float4 *>(k + d);
        const float4 k1 = *reinterpret_cast<const float4 *>(k + 16 * C::kRow + d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 x = *reinterpret_cast<const float4 *>(q + r * C::kRow + d);
          s[r][0] = fmaf(x.w, k0.w, fmaf(x.z, k0.z, fmaf(x.y, k0.y, fmaf(x.x, k0.x, s[r][0]))));
          s[r][1] = fmaf(x.w, k1.w, fmaf(x.z, k1.z, fmaf(x.y, k1.y, fmaf(x.x, k1.x, s[r][1]))));
        }
      }
    }
    __syncthreads();
    bring(i + 1, a.k, C::kOffK, C::kRow);
    // ---- weights
#pragma unroll
    for (int r = 0; r < 4; ++r) {
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
      for (int d = 0; d < kDims; ++d) o[r][d] *= factor;
      sm[C::kOffP + (r0 + r) * C::kP + tx] = weight[0];
      sm[C::kOffP + (r0 + r) * C::kP + tx + 16] = weight[1];
    }
    copies_wait<1>();
    __syncthreads();
    // ---- output: four rows x eight dims (four at D = 64)
#pragma unroll 2
    for (int j = 0; j < kKeys; j += 4) {
      float4 weight[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        weight[r] = *reinterpret_cast<const float4 *>(sm + C::kOffP + (r0 + r) * C::kP + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int g = 0; g < kDims / 4; ++g) {
          const float4 v = *reinterpret_cast<const float4 *>(sm + C::kOffV + (j + e) * D + 64 * g + 4 * tx);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float x = (&weight[r].x)[e];
            o[r][4 * g] = fmaf(x, v.x, o[r][4 * g]);
            o[r][4 * g + 1] = fmaf(x, v.y, o[r][4 * g + 1]);
            o[r][4 * g + 2] = fmaf(x, v.z, o[r][4 * g + 2]);
            o[r][4 * g + 3] = fmaf(x, v.w, o[r][4 * g + 3]);
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
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int d = 8; d; d /= 2) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], d);
    if (tx == 0) *reinterpret_cast<float2 *>(sm + (r0 + r) * C::kRow + D) = make_float2(ref[r], bad ? -1.f : sum[r]);
#pragma unroll
    for (int g = 0; g < kDims / 4; ++g)
      *reinterpret_cast<float4 *>(sm + (r0 + r) * C::kRow + 64 * g + 4 * tx) =
          make_float4(o[r][4 * g], o[r][4 * g + 1], o[r][4 * g + 2], o[r][4 * g + 3]);
  }
  auto out_row = [&](int r) { return s_row[r] < 0 ? nullptr : static_cast<float *>(a.o) + s_row[r]; };
  if (!merge_splits<D, C::kThreads, float>(tid, CS, split, w.rows, sm, &s_bar, out_row) && tid == 0)
    report(a.status, b, SPEC_ERR_TIMEOUT);
}

// As many splits of the keys as make waves x (tiles of a CTA + its set-up and
// merge, in tiles) least.
template <int D, int R>
int launch(const PagedAttnArgs &p, int max_prefix, void *stream) {
  using C = F32Cfg<D, R>;
  auto kernel = tree_attn_paged_f32_kernel<D, R>;
  static KernelState state;
  const int dev = current_device();
  if (dev < 0 || !allow_clusters(kernel, C::kSmem, dev, &state)) return SPEC_ERR_CUDA;
  const long long blocks = most_blocks<R>(p.a), units = blocks * p.a.Hkv;
  const long long tiles = (static_cast<long long>(max_prefix) + mean_nodes(p.a) + kKeys - 1) / kKeys;
  int cs = 1;
  long long best = -1;
  for (int n = 1; n <= kMaxSplits; n = n == 8 ? kMaxSplits : n + 1) {
    if (n > 1 && tiles < 2 * n) break;
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
