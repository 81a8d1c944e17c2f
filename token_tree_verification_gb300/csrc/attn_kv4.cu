// Tree attention over the 4-bit KV cache, with an optional sliding window.
//
// For node i of request b and query head h of KV head g:
//   o[i][h] = sum_j softmax_j(s q . k_j) v_j  over the keys j that i sees,
// k_j and v_j the values of slot j's record (kv4.cuh).  A node sees the prefix
// and its ancestors; with a window w, of those only positions p_j > p_i - w or
// p_j < sinks, where a prefix key's position is its slot and a tree node's is
// the prefix length plus its depth.
#include "attn_common.cuh"
#include "kv4.cuh"

namespace spec {

namespace {

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
  const int depth = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w) - 1;
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

// ---------------------------------------------------------------- CUDA cores
constexpr int kSimpleThreads = 128;

// One CTA per (node, query head), a key per thread and round.
template <int D, typename E>
__global__ void __launch_bounds__(kSimpleThreads)
tree_attn_kv4_kernel(const Kv4AttnArgs p) {
  constexpr int R = kv4_record_bytes(D);
  const AttnArgs &a = p.a;
  __shared__ float qs[D];
  __shared__ float ps[kSimpleThreads];
  __shared__ float red[kSimpleThreads / 32];
  const int h = blockIdx.x, t = blockIdx.y, tid = threadIdx.x;
  if (h == 0 && t == 0)
    for (int i = tid; i < a.B; i += kSimpleThreads) {
      const ReqGeom r = request_geometry(a, i);
      if (r.err) report(a.status, i, r.err);
    }
  const int b = find_request(a.offsets, a.B, t);
  if (b < 0) return;
  const ReqGeom G = request_geometry(a, b);
  if (G.err) return;
  const RowKeys see = row_keys(node_mask(a, G, b, t), G.L, p.window, p.sinks);
  const E *q = static_cast<const E *>(a.q) + (static_cast<size_t>(t) * a.Hq + h) * D;
  const uint8_t *kv = static_cast<const uint8_t *>(a.k) +
                      (static_cast<size_t>(b) * a.Hkv + h / a.G) * a.S_cap * R;
  if (tid < D) qs[tid] = static_cast<float>(q[tid]);
  __syncthreads();
  float m_run = -INFINITY, l_run = 0.f, acc = 0.f;
  for (int c0 = 0; c0 < G.keys; c0 += kSimpleThreads) {
    const int key = c0 + tid;
    float sc = -INFINITY;
    if (key < G.keys && row_sees(see, key, G.L, G.keys)) {
      const uint8_t *rec = kv + static_cast<size_t>(key) * R;
      float dot = 0.f;
      for (int w = 0; w < D / 8; ++w) {
        uint32_t x[4];
        kv4_codes_to_half2(reinterpret_cast<const uint32_t *>(rec)[w], x);
        const uint32_t s = kv4_scale_half2(rec[D + w / 2]);
        for (int i = 0; i < 4; ++i) {
          const uint32_t y = mul_half2(x[i], s);
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y));
          dot = fmaf(qs[8 * w + 2 * i], f.x, dot);
          dot = fmaf(qs[8 * w + 2 * i + 1], f.y, dot);
        }
      }
      sc = dot * a.scale_log2;
    }
    float mx = sc;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = red[0];
    for (int w = 1; w < kSimpleThreads / 32; ++w) mx = fmaxf(mx, red[w]);
    const float m_new = fmaxf(m_run, mx);
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = m_run == -INFINITY ? 0.f : exp2f(m_run - base);
    const float w = exp2f(sc - base);
    ps[tid] = w;
    float sum = w;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < kSimpleThreads / 32; ++i) sum += red[i];
    l_run = l_run * alpha + sum;
    m_run = m_new;
    if (tid < D) {
      float part = 0.f;
      const int nk = min(kSimpleThreads, G.keys - c0);
      for (int j = 0; j < nk; ++j) {
        if (ps[j] == 0.f) continue;
        const uint8_t *rec = kv + static_cast<size_t>(c0 + j) * R;
        uint32_t x[4];
        kv4_codes_to_half2(rec[D / 2 + tid / 2], x);
        const uint32_t y = mul_half2(x[0], kv4_scale_half2(rec[D + D / 16 + tid / 16]));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y));
        part = fmaf(ps[j], tid & 1 ? f.y : f.x, part);
      }
      acc = acc * alpha + part;
    }
    __syncthreads();
  }
  if (tid < D)
    static_cast<E *>(a.o)[(static_cast<size_t>(t) * a.Hq + h) * D + tid] =
        static_cast<E>(l_run == 0.f ? 0.f : acc / l_run);
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(Hq), static_cast<unsigned>(T), 1);
  if (dtype == SPEC_BF16) {
    if (D == 128) tree_attn_kv4_kernel<128, __nv_bfloat16><<<grid, kSimpleThreads, 0, st>>>(p);
    else tree_attn_kv4_kernel<64, __nv_bfloat16><<<grid, kSimpleThreads, 0, st>>>(p);
  } else {
    if (D == 128) tree_attn_kv4_kernel<128, float><<<grid, kSimpleThreads, 0, st>>>(p);
    else tree_attn_kv4_kernel<64, float><<<grid, kSimpleThreads, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
