// The depth-first KV-cache update after verification, on a paged cache: slot
// L + j receives the old slot L + path[j] (j = 1 .. acc) in K and V of every KV
// head, wherever the block table puts the two.
//
// One CTA per (KV head, request).  A destination may be a later source, so every
// accepted row is read before the first is written: into registers, four
// 16-byte pieces a thread, or for paths that are longer into shared memory.
// The call is a chain of loads, each some 0.4 us behind the one before: lengths;
// path; pages; rows.  The path is looked up and checked by 128 threads at once,
// an entry each.  (One path of 32 heads, D = 128: 2.1 us; of 16 requests 3.4, 0.8
// TB/s.)
#include "paged.cuh"

namespace spec {

namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;          // of a thread, in registers

struct CompactArgs {
  uint8_t *k, *v;
  PageTable pages;
  int row_bytes, H, W;
  const int32_t *prefix, *offsets, *path, *accept;
  int32_t *new_prefix, *status;
};

__global__ void __launch_bounds__(kThreads)
kv_compact_paged_kernel(const CompactArgs a) {
  extern __shared__ __align__(16) uint4 s_rows[];                  // rows beyond the registers' share
  __shared__ long long s_src[SPEC_MAX_TREE_NODES], s_dst[SPEC_MAX_TREE_NODES];   // rows of the pools
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int L = __ldg(a.prefix + b), lo = __ldg(a.offsets + b), hi = __ldg(a.offsets + b + 1);
  const int accepted = __ldg(a.accept + b);
  const int32_t *path = a.path + static_cast<size_t>(b) * a.W;
  // (the first entries' loads do not wait for the path's length)
  const int x = tid < a.W ? __ldg(path + tid) : 0, before = tid > 0 && tid < a.W ? __ldg(path + tid - 1) : -1;
  const bool skipped = __ldcg(a.status + b) != 0;      // another call's error, or this one's found by another head
  const int n = hi - lo;
  int err = 0;
  if (L < 0 || lo < 0 || n < 1 || n > SPEC_MAX_TREE_NODES || static_cast<long long>(L) + n > a.pages.capacity())
    err = n < 1 || n > SPEC_MAX_TREE_NODES || lo < 0 ? SPEC_ERR_TREE_TOO_LARGE : SPEC_ERR_PREFIX_RANGE;
  else if (accepted < 0 || accepted >= a.W)
    err = SPEC_ERR_TREE_TOO_LARGE;
  // each thread's path entry: the root first, then increasing nodes of the tree.  Entry
  // j of such a path is node j or a later one; asked of every entry by itself, that
  // keeps the slots that a thread looks up within [L, L + n) whatever the others hold.
  if (!skipped && !err && tid <= accepted) {
    if (tid == 0 ? x != 0 : x <= before || x < tid || x >= n) {
      err = SPEC_ERR_BAD_PARENT;
    } else {
      const int src = L + x, dst = L + tid, size = 1 << a.pages.shift;
      const int ps = a.pages.page(b, src >> a.pages.shift), pd = a.pages.page(b, dst >> a.pages.shift);
      if (ps < 0 || pd < 0) err = SPEC_ERR_PAGE;
      s_src[tid] = (static_cast<long long>(ps) * a.H + h) * size + (src & (size - 1));
      s_dst[tid] = (static_cast<long long>(pd) * a.H + h) * size + (dst & (size - 1));
      if (!err && !(a.pages.holds(s_src[tid], 1, a.H, b) && a.pages.holds(s_dst[tid], 1, a.H, b))) err = SPEC_ERR_INDEX;
    }
  }
  // every thread has the same view of what does not depend on its entry; entries
  // that are no path come before pages that are not there
  const bool bad_path = __syncthreads_or(err == SPEC_ERR_BAD_PARENT);
  const bool bad_page = __syncthreads_or(err == SPEC_ERR_PAGE);
  if (bad_path) err = SPEC_ERR_BAD_PARENT;
  else if (bad_page) err = SPEC_ERR_PAGE;
  const bool ok = __syncthreads_and(!skipped && !err);
  if (tid == 0 && h == 0) {
    if (err && !skipped) report(a.status, b, err);
    a.new_prefix[b] = ok ? L + 1 + accepted : L;
  }
  if (!ok || accepted == 0) return;

  const int chunks = a.row_bytes / 16;
  const int half = accepted * chunks, total = 2 * half;
  auto piece = [&](int i, const long long *rows) -> uint4 * {
    const int kv = i >= half, rem = i - kv * half, j = rem / chunks;
    return reinterpret_cast<uint4 *>(kv ? a.v : a.k) + rows[j + 1] * chunks + (rem - j * chunks);
  };
  uint4 held[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u)
    if (tid + u * kThreads < total) held[u] = __ldcs(piece(tid + u * kThreads, s_src));
  for (int i = tid + kPieces * kThreads; i < total; i += kThreads)
    s_rows[i - kPieces * kThreads] = __ldcs(piece(i, s_src));
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kPieces; ++u)
    if (tid + u * kThreads < total) *piece(tid + u * kThreads, s_dst) = held[u];
  for (int i = tid + kPieces * kThreads; i < total; i += kThreads)
    *piece(i, s_dst) = s_rows[i - kPieces * kThreads];
}

}  // namespace

}  // namespace spec

extern "C" int spec_kv_compact_paged(void *k_pages, void *v_pages, int dtype, int B, int Hkv, int D, int num_pages,
                                     int page_size, const int32_t *block_table, int max_pages,
                                     const int32_t *prefix_lens, const int32_t *tree_offsets,
                                     const int32_t *path_nodes, const int32_t *accept_len, int max_depth_plus1,
                                     int32_t *new_prefix_lens, int32_t *status, void *stream) {
  using namespace spec;
  if (!k_pages || !v_pages || !block_table || !prefix_lens || !tree_offsets || !path_nodes || !accept_len ||
      !new_prefix_lens || !status)
    return SPEC_ERR_NULL;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  CompactArgs a = {};
  const int rc = check_pages(num_pages, page_size, max_pages, &a.pages.shift);
  if (rc != SPEC_OK) return rc;
  // (the CTAs of a request read its length while one of them writes the new one)
  if (B < 1 || B > 65535 || Hkv < 1 || (D != 64 && D != 128) || max_depth_plus1 < 1 ||
      max_depth_plus1 > SPEC_MAX_TREE_NODES || (new_prefix_lens < prefix_lens + B && prefix_lens < new_prefix_lens + B))
    return SPEC_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15) return SPEC_ERR_ALIGNMENT;
  a.k = static_cast<uint8_t *>(k_pages);
  a.v = static_cast<uint8_t *>(v_pages);
  a.pages.table = block_table;
  a.pages.max_pages = max_pages;
  a.pages.pages = num_pages;
  a.pages.status = status;
  a.row_bytes = D * (dtype == SPEC_F32 ? 4 : 2);
  a.H = Hkv;
  a.W = max_depth_plus1;
  a.prefix = prefix_lens;
  a.offsets = tree_offsets;
  a.path = path_nodes;
  a.accept = accept_len;
  a.new_prefix = new_prefix_lens;
  a.status = status;
  const int most = 2 * (max_depth_plus1 - 1) * a.row_bytes, held = kPieces * kThreads * 16;
  const size_t smem = most > held ? static_cast<size_t>(most - held) : 0;
  static std::atomic<size_t> granted[kMaxDevices];
  if (smem > 40 * 1024 && !allow_dynamic_smem(kv_compact_paged_kernel, smem, granted)) return SPEC_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(Hkv), static_cast<unsigned>(B), 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_compact_paged_kernel, a) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
