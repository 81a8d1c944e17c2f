// Pieces shared by the three kernels of tree attention over the 4-bit cache:
// what a row sees, which tiles that takes, and the merge of the key splits.
#pragma once

#include "attn_common.cuh"
#include "kv4.cuh"

namespace spec {

struct Kv4AttnArgs {
  AttnArgs a;          // k: the cache; v unused
  int window, sinks;   // window 0: none
};

// What one row sees: prefix keys [0, sinks) and [first, L), and the tree nodes
// in `tree`.
struct RowKeys {
  int sinks, first;
  uint4 tree;
};

// A node's ancestors lie on one path, so the r-th lowest bit of its set is the
// ancestor of depth r, and its own depth is the number of set bits less one.
__device__ __forceinline__ RowKeys row_keys(uint4 m, int L, int window, int sinks) {
  RowKeys r;
  r.tree = m;
  r.sinks = 0;
  r.first = 0;
  if (window == 0) return r;
  const int depth = max(0, __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w) - 1);
  r.sinks = sinks;
  r.first = max(0, L + depth - window + 1);
  // ancestors of depth [sinks - L, depth - window] are out of sight
  const int from = max(0, sinks - L), to = depth - window;
  uint32_t *w = &r.tree.x;
  int rank = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t left = w[i];
    while (left && rank <= to) {
      const uint32_t low = left & (0u - left);
      if (rank >= from) w[i] &= ~low;
      left ^= low;
      ++rank;
    }
  }
  return r;
}

__device__ __forceinline__ bool row_sees(const RowKeys &r, int key, int L, int keys) {
  if (key < L) return key < r.sinks || key >= r.first;
  return key_visible(key, L, keys, r.tree);
}

// The slots that some row may see.  The others in a tile, behind the last or left
// behind by the window, may hold anything, and their values are taken as zeros:
// a weight of zero does not hide a NaN.
struct LiveKeys {
  int from, sinks;
  uint32_t span;         // keys from `from` on
  __device__ __forceinline__ LiveKeys(int L, int keys, int window, int sinks_)
      : from(window ? max(0, L - window + 1) : 0), sinks(window ? min(sinks_, keys) : 0) {
    span = static_cast<uint32_t>(keys - from);
  }
  __device__ __forceinline__ bool operator()(int key) const {
    return static_cast<uint32_t>(key - from) < span || key < sinks;
  }
};

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

// Global to shared bulk copy (16-byte aligned, a multiple of 16 bytes),
// completing on `bar`.
__device__ __forceinline__ void bulk_copy_g2s(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

template <typename E>
__device__ __forceinline__ void store_row4(E *dst, float4 v) {
  if constexpr (sizeof(E) == 4) {
    *reinterpret_cast<float4 *>(dst) = v;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  }
}

// mbar_wait for roles that wait long and often: the thread is suspended up to
// 10 us a try (3.8 us, measured) instead of polling through the issue slots of the
// working warps.  The limit is a number of tries, 3.8 s of them and at most 10 s,
// never less than kWaitLimitNs while a try takes 2 us: a look at a clock, whichever
// way, costs the loops that wait 1 to 2% (128-node trees 135.7 -> 137.5 us and
// more).  (`bar` is a shared-memory address.)
constexpr uint32_t kSleepTries = 1000000;
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 10000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Whether the phase is over, without waiting.
__device__ __forceinline__ bool mbar_over(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// -DSPEC_WAIT_POLLS=n (the failure test's build): waits give up after n looks.
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity, uint32_t tries = kSleepTries) {
#ifdef SPEC_WAIT_POLLS
  tries = SPEC_WAIT_POLLS;
#endif
#pragma unroll 1
  for (uint32_t it = 0; it < tries; ++it) {
#ifdef SPEC_WAIT_POLLS
    if (mbar_over(bar, parity)) return true;
#else
    if (mbar_try(bar, parity)) return true;
#endif
  }
  return false;
}
// For warps that are to go on at once: mbar_wait.
__device__ __forceinline__ bool mbar_await(uint64_t *bar, uint32_t parity) {
#ifdef SPEC_WAIT_POLLS
  return mbar_sleep(smem_addr(bar), parity);
#else
  return mbar_wait(bar, parity);
#endif
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A place in a ring of n stages and the phase of its barriers.
template <int n>
struct Ring {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if constexpr (n == 2) {
      at ^= 1;
      phase ^= at ^ 1;
    } else if (++at == n) {
      at = 0;
      phase ^= 1;
    }
  }
};

// Which tiles of `TILE` keys a row block reads: all, or with a window those
// that hold the first `sinks` slots, then those from the root's window on.
template <int TILE>
struct TileList {
  int head, skip, count;
  __device__ __forceinline__ TileList(int L, int keys, int window, int sinks) {
    const int all = (keys + TILE - 1) / TILE;
    head = 0;
    skip = 0;
    if (window > 0) {
      head = (min(sinks, keys) + TILE - 1) / TILE;
      const int from = max(0, L - window + 1) / TILE;
      skip = max(0, from - head);
    }
    count = all - skip;
  }
  __device__ __forceinline__ int key0(int i) const { return (i < head ? i : i + skip) * TILE; }
};

// The weights' halves are scaled by 2^8 at the reference, a whole number at or
// above the largest score so far, which moves only when a score passes it by
// more than 7: they stay below 2^15 (a half ends at 2^16), and the row's
// largest is at least 2^7, 2^32 times half the step of the smallest halves.
// Whole references make 8 - m and the factors 2^(m - m') exact.
constexpr float kWeightLog2 = 8.f;
constexpr float kMoveLog2 = 7.f;

// A move of a row's reference: `most` is the row's largest x = score - reference
// + 8 (score, all in powers of two, being s c) and `old` the present 8 -
// reference.  From 2^24 on fp32 does not hold every whole number, and s c + (8 -
// reference) may miss the range of halves either way: at 2^27 the steps are 16.
// There x keeps its rounding at the old reference and is brought to the new one by
// a subtraction, which leaves the largest score a weight of at least 1.
//
// A score that far above a reference so low has lost its last places in x, and what
// is summed is nothing beside it (2^-1024): the row starts again without a
// reference, and its tile is taken once more (`far`).
constexpr float kWholeEnd = 16777216.f, kFarStep = 1024.f, kFarBase = 4096.f;
__device__ __forceinline__ float reference_step(float most) {
  return fabsf(most) < kWholeEnd ? ceilf(most - kWeightLog2) : most;
}
__device__ __forceinline__ bool far_above(float most, float old, bool fresh) {
  return !fresh && most >= kFarStep && fabsf(old) >= kFarBase;
}
struct Move {
  float factor, next;       // of what is summed; the new 8 - reference
  float base, less;         // x = s c + base - less
  __device__ __forceinline__ explicit Move(float old) : factor(1.f), next(old), base(old), less(0.f) {}   // none
  __device__ __forceinline__ Move(float most, float old, bool fresh) {
    const float by = reference_step(most);
    factor = fresh ? 0.f : exp2f(-by);
    next = old - by;
    const bool steep = !(fabsf(next) < kWholeEnd);
    base = steep ? old : next;
    less = steep ? by : 0.f;
  }
};

constexpr int kMaxSplits = 16;

// A row's query is taken as halves: scaled by 2^up so that its largest finite
// element is near 2^13, which the score factor takes back.  bf16 elements are
// exact down to 2^-27 of the largest; below, the half's smallest step takes at
// most 2^-38 of it, far under what the sums of the scores round.  (A row below
// 2^-113 stays that much smaller: its scores vanish either way.)
__device__ __forceinline__ int row_exponent(float top) {
  return top > 0.f && top < INFINITY ? min(13 + 127 - (__float_as_int(top) >> 23), 126) : 0;
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }

// Merge of a block's rows over the CTA's own parts and the cluster's splits,
// and the output, by THREADS threads of the CTA (`tid` among them; any others
// run the two cluster barriers of a split block, ready()'s and the one here)
// with W parts per row in
// so[W][ROWS][D + 4] (weighted sums), s_m[W][ROWS] (references) and
// s_l[W][ROWS] (sums of weights), or with `timed_out`.  Without splits the
// merged piece of four dims is the result; else it goes to the CTA of the
// cluster that merges it (CTA q has pieces [q share, (q + 1) share)), and
// every CTA gets each row's reference and sum: stores that nothing waits for.
// ready() returns once every CTA's `recv` and `s_ml` may be written.  Returns
// false when a CTA of the cluster timed out (nothing is written then).
template <int D, int W, int ROWS, int THREADS, typename E, typename Ready, typename OutRow>
__device__ __forceinline__ bool merge_rows(int tid, int CS, int split, int rows_here, bool timed_out, float *so,
                                           const float (*s_m)[ROWS], const float (*s_l)[ROWS],
                                           float2 (*s_ml)[ROWS], float4 *recv, Ready ready, OutRow out_row) {
  constexpr int kStride = D + 4;
  const int pieces = rows_here * (D / 4);
  const int share = (pieces + CS - 1) / CS;
  // the factors of a row's W parts, and its merged reference and sum
  auto part_factors = [&](int r, float (&f)[W], float &M, float &L) {
    M = s_m[0][r];
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, s_m[w][r]);
    const float base = M == -INFINITY ? 0.f : M;
    L = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      f[w] = fast_exp2(s_m[w][r] - base);
      L = fmaf(f[w], s_l[w][r], L);
    }
  };
  auto add_piece = [](float4 &acc, float f, float4 v) {
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  };
  auto finish = [&](int r, int c, float4 acc, float L) {
    const float inv = L == 0.f ? 0.f : 1.f / L;
    E *dst = out_row(r);
    if (dst) store_row4(dst + c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  };
  float per_share = 0.f;
  if (CS > 1) {
    per_share = 1.f / static_cast<float>(share);
    ready();
    for (int i = tid; i < rows_here * kMaxSplits; i += THREADS) {
      const int r = i / kMaxSplits, q = i % kMaxSplits;
      if (q >= CS) continue;
      float f[W], M, L;
      part_factors(r, f, M, L);
      const uint32_t dst = peer_addr(&s_ml[split][r], q);
      st_peer_f32(dst, timed_out ? INFINITY : M);
      st_peer_f32(dst + 4, timed_out ? -1.f : L);      // no sum of weights is negative
    }
  }
  if (!timed_out) {
#pragma unroll 2
    for (int idx = tid; idx < pieces; idx += THREADS) {
      const int r = idx / (D / 4), c = idx % (D / 4) * 4;
      float f[W], M, L;
      part_factors(r, f, M, L);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w)
        add_piece(acc, f[w], *reinterpret_cast<const float4 *>(so + (w * ROWS + r) * kStride + c));
      if (CS > 1) {
        // (idx and share are far below 2^22: the quotient is exact)
        const int q = static_cast<int>((static_cast<float>(idx) + 0.5f) * per_share);
        st_peer_f32x4(peer_addr(recv + split * share + idx - q * share, q), acc);
      } else {
        finish(r, c, acc, L);
      }
    }
  }
  if (CS == 1) return !timed_out;
  cluster_sync_all();
  bool any_timeout = false;
  for (int q = 0; q < CS; ++q) any_timeout |= s_ml[q][0].y < 0.f;
  if (any_timeout) return false;      // every CTA of the cluster sees the same
  for (int i = tid; i < min(share, pieces - split * share); i += THREADS) {
    const int idx = split * share + i, r = idx / (D / 4), c = idx % (D / 4) * 4;
    float M = -INFINITY;
#pragma unroll 4
    for (int q = 0; q < CS; ++q) M = fmaxf(M, s_ml[q][r].x);
    const float base = M == -INFINITY ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
#pragma unroll 4
    for (int q = 0; q < CS; ++q) {
      const float2 ml = s_ml[q][r];
      const float f = fast_exp2(ml.x - base);
      L = fmaf(f, ml.y, L);
      add_piece(acc, f, recv[q * share + i]);
    }
    finish(r, c, acc, L);
  }
  return true;
}

// The host does not know the requests' tree sizes; launches are sized by their
// mean, rounded up.
inline int mean_nodes(const AttnArgs &a) { return 1 + (a.T - 1) / a.B; }

// What the launches keep of a kernel, per device.
struct KernelState {
  std::atomic<size_t> granted[kMaxDevices];
  std::atomic<bool> wide[kMaxDevices], fits[kMaxDevices];
  std::atomic<int> at_once[kMaxDevices][kMaxSplits + 1];    // clusters of each size that run at once, plus one
};

// Allows the kernel its shared memory, and clusters beyond the portable 8.
template <typename Kernel>
bool allow_clusters(Kernel kernel, size_t smem, int dev, KernelState *state) {
  if (!allow_dynamic_smem(kernel, smem, state->granted)) return false;
  if (state->wide[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return false;
  state->wide[dev].store(true, std::memory_order_release);
  return true;
}

inline void cluster_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int cs, int threads,
                           size_t smem) {
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  pdl_attribute(attr[1]);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

// Clusters of `cs` CTAs that run at once: fewer than SMs / cs, since a cluster
// stays within one of the GPU's groups of SMs.  0 when it cannot be said now: the
// next launch asks again (and no later call of the program meets the error).
template <typename Kernel>
int clusters_at_once(Kernel kernel, int cs, int threads, size_t smem, int dev, KernelState *state) {
  const int known = state->at_once[dev][cs].load(std::memory_order_relaxed);
  if (known) return known - 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, cs, threads, smem);
  cfg.gridDim = dim3(cs, 1, 1);
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 0) {
    cudaGetLastError();
    return 0;
  }
  state->at_once[dev][cs].store(n + 1, std::memory_order_relaxed);
  return n;
}

// The tensor-core paths, bf16 only: rows along N (attn_kv4_tc.cu) and along M
// (attn_kv4_rows.cu).
int launch_kv4_tc(const Kv4AttnArgs &p, int max_prefix, void *stream);
int launch_kv4_rows(const Kv4AttnArgs &p, int max_prefix, void *stream);

}  // namespace spec
