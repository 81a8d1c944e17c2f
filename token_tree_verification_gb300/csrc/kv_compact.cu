// The depth-first KV-cache update after verification.
//
// SpecInfer news write-up, "Token 樹驗證器": the verifier's KV cache is
// updated depth-first, so the accepted path becomes the next step's prefix
// without extra storage.  Slot L + j receives the old slot L + path[j]
// (j = 1 .. acc) in the K and V caches of every KV head.
//
// One CTA per (KV head, request): every accepted row of K and V is read into
// shared memory first and written back after one barrier (a destination slot
// may be the source of a later path entry), in 16-byte chunks.  The 4-bit
// cache is one array whose rows are the slots' records, so the same kernel
// moves it (kv4.cuh).
#include "kv4.cuh"

namespace spec {

namespace {

constexpr int kKvThreads = 256;

struct KvArgs {
  uint8_t *k, *v;           // v: null when key and value share a row
  int arrays, row_bytes;    // 2 (K and V) or 1
  int B, H, S_cap, W;
  const int32_t *prefix, *offsets, *path, *accept;
  int32_t *new_prefix, *status;
};

__global__ void __launch_bounds__(kKvThreads)
kv_compact_kernel(const KvArgs a) {
  extern __shared__ __align__(16) uint4 rows[];   // [2][acc][row chunks]
  __shared__ int s_ok, s_acc, s_L;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  if (tid == 0) {
    const int L = __ldg(a.prefix + b);
    int ok = __ldcg(a.status + b) == 0;
    int acc = 0;
    if (ok) {
      const int n = __ldg(a.offsets + b + 1) - __ldg(a.offsets + b);
      acc = __ldg(a.accept + b);
      const int32_t *pn = a.path + static_cast<size_t>(b) * a.W;
      int err = 0;
      if (L < 0 || static_cast<long long>(L) + n > a.S_cap) {
        err = SPEC_ERR_PREFIX_RANGE;
      } else if (acc < 0 || acc + 1 > a.W) {
        err = SPEC_ERR_TREE_TOO_LARGE;
      } else {
        int prev = __ldg(pn);
        if (prev != 0) err = SPEC_ERR_BAD_PARENT;
        for (int j = 1; j <= acc && !err; ++j) {
          const int x = __ldg(pn + j);
          if (x <= prev || x >= n) err = SPEC_ERR_BAD_PARENT;
          prev = x;
        }
      }
      if (err) {
        if (h == 0) report(a.status, b, err);
        ok = 0;
      }
    }
    if (h == 0) a.new_prefix[b] = ok ? L + 1 + acc : L;
    s_ok = ok;
    s_acc = ok ? acc : 0;
    s_L = L;
  }
  __syncthreads();
  const int acc = s_acc;
  if (!s_ok || acc == 0) return;
  const int L = s_L;
  const int32_t *pn = a.path + static_cast<size_t>(b) * a.W;
  const int chunks = a.row_bytes / 16;                // 16-byte chunks per row
  const size_t row_bytes = static_cast<size_t>(a.row_bytes);
  const size_t head = (static_cast<size_t>(b) * a.H + h) * a.S_cap;
  const int total = a.arrays * acc * chunks;
  for (int i = tid; i < total; i += kKvThreads) {
    const int kv = i / (acc * chunks), rem = i % (acc * chunks);
    const int j = rem / chunks, c = rem % chunks;
    const int x = __ldg(pn + j + 1);
    const uint8_t *src = (kv ? a.v : a.k) + (head + L + x) * row_bytes;
    rows[i] = in_bounds(L + x, a.S_cap, a.status, b) ? __ldcs(reinterpret_cast<const uint4 *>(src) + c)
                                                      : make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  for (int i = tid; i < total; i += kKvThreads) {
    const int kv = i / (acc * chunks), rem = i % (acc * chunks);
    const int j = rem / chunks, c = rem % chunks;
    uint8_t *dst = (kv ? a.v : a.k) + (head + L + 1 + j) * row_bytes;
    if (in_bounds(L + 1 + j, a.S_cap, a.status, b)) reinterpret_cast<uint4 *>(dst)[c] = rows[i];
  }
}

// Checks shared by the dense and the 4-bit call, and the launch.
int compact_rows(KvArgs args, int max_depth_plus1, void *stream) {
  if (!args.prefix || !args.offsets || !args.path || !args.accept || !args.new_prefix || !args.status)
    return SPEC_ERR_NULL;
  if (args.B < 1 || args.H < 1 || args.S_cap < 1 || max_depth_plus1 < 1 ||
      max_depth_plus1 > SPEC_MAX_TREE_NODES || args.B > 65535)
    return SPEC_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(args.k) & 15) || (reinterpret_cast<uintptr_t>(args.v) & 15))
    return SPEC_ERR_ALIGNMENT;
  // room for every row an accepted path can move (acc <= max_depth_plus1 - 1)
  const size_t smem = static_cast<size_t>(args.arrays) * (max_depth_plus1 - 1) * args.row_bytes;
  if (smem > 200 * 1024) return SPEC_ERR_SHAPE;
  static std::atomic<size_t> granted[kMaxDevices];
  if (smem > 48 * 1024 && !allow_dynamic_smem(kv_compact_kernel, smem, granted)) return SPEC_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(args.H), static_cast<unsigned>(args.B), 1);
  cfg.blockDim = dim3(kKvThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_compact_kernel, args) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

}  // namespace spec

extern "C" int spec_kv_compact(void *k_cache, void *v_cache, int dtype, int B, int Hkv, int D,
                               int S_cap, const int32_t *prefix_lens,
                               const int32_t *tree_offsets, const int32_t *path_nodes,
                               const int32_t *accept_len, int max_depth_plus1,
                               int32_t *new_prefix_lens, int32_t *status, void *stream) {
  using namespace spec;
  if (!k_cache || !v_cache || !prefix_lens || !tree_offsets || !path_nodes || !accept_len ||
      !new_prefix_lens || !status)
    return SPEC_ERR_NULL;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  const int es = dtype == SPEC_F32 ? 4 : 2;
  if (D < 8 || (D * es) % 16 != 0) return SPEC_ERR_SHAPE;
  const KvArgs args = {static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), 2, D * es, B, Hkv, S_cap,
                       max_depth_plus1, prefix_lens, tree_offsets, path_nodes, accept_len, new_prefix_lens, status};
  return compact_rows(args, max_depth_plus1, stream);
}

extern "C" int spec_kv4_compact(void *kv_cache, int B, int Hkv, int D, int S_cap,
                                const int32_t *prefix_lens, const int32_t *tree_offsets,
                                const int32_t *path_nodes, const int32_t *accept_len,
                                int max_depth_plus1, int32_t *new_prefix_lens, int32_t *status,
                                void *stream) {
  using namespace spec;
  if (!kv_cache) return SPEC_ERR_NULL;
  if (D != 64 && D != 128) return SPEC_ERR_SHAPE;
  // the CTAs of a request read its length while one of them writes the new one
  if (new_prefix_lens && new_prefix_lens == prefix_lens) return SPEC_ERR_SHAPE;
  const KvArgs args = {static_cast<uint8_t *>(kv_cache), nullptr, 1, kv4_record_bytes(D), B, Hkv, S_cap,
                       max_depth_plus1, prefix_lens, tree_offsets, path_nodes, accept_len, new_prefix_lens, status};
  return compact_rows(args, max_depth_plus1, stream);
}
