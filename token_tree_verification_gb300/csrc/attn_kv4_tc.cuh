// Pieces shared by the two tensor-core kernels of tree attention over the
// 4-bit cache: register budgets, packed arithmetic, and the decoding of a
// tile's records.
#pragma once

#include "attn_kv4.cuh"
#include "tcgen05.cuh"

namespace spec {

namespace tc {

// An MN-major operand of 32 or 16 16-bit elements along M/N, rows of K packed
// one after another and swizzled over their own width (64 or 32 bytes: layouts
// 4 and 6); the stride offset is that of 8 rows.
template <int N>
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
  static_assert(N == 32 || N == 16, "one swizzle atom wide");
  constexpr uint64_t layout = N == 32 ? 4 : 6;
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(1) << 16 |
         static_cast<uint64_t>(8 * N * 2 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | layout << 61;
}

// idesc_bf16_f32 for half-precision A and B (format 0): kind::f16 takes both
// operands in bf16 or both in half, as the descriptor says, so the bf16 MMAs
// serve for halves too.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}

// One lane of a converged warp (the same one every time).  A warp that loops
// as a whole, with only the MMAs themselves under this branch, keeps its
// descriptors in uniform registers: an M = 128, N = 16 MMA then issues every 18
// cycles, N = 64 every 33 (the tensor cores' own rate), against 46 for both
// from a loop that a single lane runs.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

}  // namespace tc

constexpr int kTile = 128;            // keys of a tile

template <int regs>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(regs));
}
template <int regs>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(regs));
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}
// The largest of n values (NaN is passed over).
template <int n>
__device__ __forceinline__ float max_of(const float (&x)[n]) {
  static_assert(n % 8 == 0, "pairs of four chains");
  float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int j = 4; j + 4 < n; j += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = max3(m[e], x[j + e], x[j + 4 + e]);
  return max3(max3(m[0], m[1], x[n - 1]), max3(m[2], m[3], x[n - 2]), fmaxf(x[n - 3], x[n - 4]));
}

__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[8]) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(v[i]);
  tc::st8(taddr, u);
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Reduction of n values (a power of two) over the warp's lanes: lane l returns
// value l % n reduced over all of them.  Each round exchanges half of the
// values with the lane across and keeps the other half.
template <int n, typename Op>
__device__ __forceinline__ float reduce_scatter(const float (&x)[n], int lane, Op op) {
  float v[n];
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = x[i];
#pragma unroll
  for (int h = n / 2; h >= 1; h /= 2) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? v[i] : v[i + h];
      const float keep = up ? v[i + h] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, h));
    }
  }
#pragma unroll
  for (int h = n; h < 32; h *= 2) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], h));
  return v[0];
}

// One lane's key of a tile of records: its D codes and scales, from a stage
// of the ring; zeros for one that is not live.
template <int D>
struct KeyCodes {
  uint4 code[D / 32];
  uint32_t scale[D / 64];

  __device__ __forceinline__ KeyCodes(const uint8_t *rec, bool of_v, bool live) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      code[c] = *reinterpret_cast<const uint4 *>(rec + (of_v ? D / 2 : 0) + 16 * c);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      scale[c] = *reinterpret_cast<const uint32_t *>(rec + D + (of_v ? D / 16 : 0) + 4 * c);
      if (!live) scale[c] = 0u;
    }
  }

  // put(g, h): the 16 dims of group g as eight half pairs
  template <typename Put>
  __device__ __forceinline__ void decode(Put put) const {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const uint32_t word[4] = {code[c].x, code[c].y, code[c].z, code[c].w};
#pragma unroll
      for (int q = 0; q < 2; ++q) {       // a group: two words
        uint32_t h[8];
        kv4_codes_to_half2(word[2 * q], *reinterpret_cast<uint32_t(*)[4]>(h));
        kv4_codes_to_half2(word[2 * q + 1], *reinterpret_cast<uint32_t(*)[4]>(h + 4));
        const uint32_t s = kv4_scale_half2(__byte_perm(scale[c / 2], 0, 0x4440 + 2 * (c & 1) + q));
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = mul_half2(h[e], s);
        put(2 * c + q, h);
      }
    }
  }
};

// A group's place in a 128-byte-swizzled operand of [keys][64 dims] boxes:
// `row` is the key's row of the first box with the key's swizzle in bits 4-6.
template <int kBoxBytes>
__device__ __forceinline__ void put_swizzled(uint32_t row, int g, const uint32_t (&h)[8]) {
  const uint32_t at = row + (g >> 2) * kBoxBytes, piece = (g & 3) << 5;
  st_shared_v4(at ^ piece, h[0], h[1], h[2], h[3]);
  st_shared_v4(at ^ (piece + 16), h[4], h[5], h[6], h[7]);
}

// Whether the kernel was compiled to launch with the registers that its roles
// divide: with fewer, the roles that take more would wait for ever.
template <typename Kernel>
bool has_registers(Kernel kernel, int regs, int dev, KernelState *state) {
  if (state->fits[dev].load(std::memory_order_acquire)) return true;
  cudaFuncAttributes f;
  if (cudaFuncGetAttributes(&f, kernel) != cudaSuccess || f.numRegs < regs) return false;
  state->fits[dev].store(true, std::memory_order_release);
  return true;
}

// Launch of a kernel that takes one CTA per SM: `blocks` row blocks (the grid's
// y) of every (request, KV head), and as many splits of the keys (a cluster) as
// make waves x (tiles of a CTA + its set-up, first tile and merge, in tiles)
// least.  (24 and 64 rows behind 4000 keys, by splits: 19 units 11.8 and 14.9 us
// with 6, 19.6 and 24.7 with 8, of which 19 do not run at once; 40 units 15.2 and
// 19.3 with 3, 24.4 and 31.4 with 4; 6 units behind 500 9.0 and 11.1 with 2, 9.3
// and 12.3 without.)
template <typename Kernel>
int launch_kv4_tiles(Kernel kernel, const Kv4AttnArgs &p, int threads, int regs, size_t smem, int blocks,
                     int max_prefix, KernelState *state, void *stream) {
  const AttnArgs &a = p.a;
  const int dev = current_device();
  if (dev < 0 || !has_registers(kernel, regs, dev, state) || !allow_clusters(kernel, smem, dev, state))
    return SPEC_ERR_CUDA;
  const int nodes = mean_nodes(a);
  long long keys = static_cast<long long>(max_prefix) + nodes;
  if (p.window) {
    const long long near = static_cast<long long>(p.window) + p.sinks + nodes + 2 * kTile;
    if (near < keys) keys = near;
  }
  const long long tiles = (keys + kTile - 1) / kTile;
  const long long pairs = static_cast<long long>(a.B) * a.Hkv;
  const long long units = pairs * blocks;
  int cs = 1;
  long long best = -1;
  for (int c = 1; c <= kMaxSplits; c = c == 8 ? kMaxSplits : c + 1) {
    if (c > 1 && tiles < 2 * c) break;
    const int slots = clusters_at_once(kernel, c, threads, smem, dev, state);
    if (slots < 1) continue;
    const long long waves = (units + slots - 1) / slots;
    const long long cost = waves * (2 * ((tiles + c - 1) / c) + (c > 1 ? 19 : 16));     // in half tiles
    if (best < 0 || cost < best) {
      best = cost;
      cs = c;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, cs, threads, smem);
  cfg.gridDim = dim3(cs, static_cast<unsigned>(blocks), static_cast<unsigned>(pairs));
  cfg.stream = static_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace spec
