// Tree attention over the 4-bit KV cache on the 5th-generation tensor cores,
// bf16 queries, for blocks of up to 128 rows of one KV head: large trees,
// and trees with several query heads per KV head.
//
// With that many rows the products are bound by the softmax and the decoding,
// not by what a row costs the tensor cores, so the rows lie along M here:
//   S[rows][keys] = Q K^T   A = Q (TMEM),  B = K (keys x dims, shared memory, K-major)
//   O[rows][dims] = P V     A = P (TMEM),  B = V (keys x dims, shared memory, MN-major)
// A softmax thread then has one row, whose reference, sum and factor are
// registers, and its weights go to TMEM as they are; decoded records serve 128
// rows instead of 32.  (attn_kv4_tc.cu has the form for fewer rows, where the
// cost is the decoding of each key.)
//
// One CTA = one split of the keys x one block of 128 rows x one (request, KV
// head).  Warp roles:
//   warp 0      brings tiles of 128 records, one bulk copy each
//   warp 1      allocates TMEM and issues S_i, the two halves of the tile's keys apart
//   warp 2      issues O += P_i V_i, the halves apart
//   warps 4-11  softmax: a TMEM lane quarter's two warps hold the same 32 rows, each
//               one half of the tile's keys, with references, sums and an O of its
//               own, merged at the end like splits of the keys: no warp waits for
//               another.  A tile's weights are taken at the reference that the row
//               has; the rare tile that moves it reads S again
//   warps 12-15 decode keys, warps 16-19 values (one key per lane: loads of records
//               36 words apart and swizzled stores of rows 128 bytes apart are both
//               free of bank conflicts); with the softmax warps they merge the rows
// (Sixteen softmax warps, a quarter of the keys each, met at a barrier per tile
// that two of them shared: 142 us for the 128-node trees below, 129 at D = 64.
// Warps whose rows are no node's go along: leaving the work out took 2% longer.)
// What passes through shared memory comes next to the softmax in cost: 36 KB of
// records in and out, 64 KB of decoded operands in and 64 KB out per tile, 1300
// cycles at 128 bytes each.  (Q as a shared-memory operand, read for each half
// of the keys, added 64 KB.)
//
// Measured, D = 128: 4 requests x 8 KV heads x 1024 rows behind 8192 keys take
// 135 us, 1.04 PFLOP/s, 0.55 of the measured bf16 rate (256 CTAs are two waves on
// 152 SMs, of which the second is two thirds full; with all arithmetic taken out
// the copies, products and waits alone take 100 us), at D = 64 122 us.  A tree of
// 64 nodes on 32 heads behind 2048 keys, five tiles a CTA: 13.9 us, nearly all
// latency (set-up 3, first tile 2, loop 4, merge 3).
#include <type_traits>

#include "attn_kv4_tc.cuh"

namespace spec {

namespace {

constexpr int kRows = 128;
constexpr int kSoftFirst = 4;         // warps: four issuers, then the softmax, then the decoders
constexpr int kSoftWarps = 8;
constexpr int kDecodeFirst = kSoftFirst + kSoftWarps;
constexpr int kDecodeWarps = 4;       // for keys, and as many for values
constexpr int kThreads = 32 * (kDecodeFirst + 2 * kDecodeWarps);
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kHalf = kTile / 2;      // keys of one softmax thread
constexpr int kMergeThreads = kSoftThreads + 32 * 2 * kDecodeWarps;     // softmax and decoders
// Registers: 20 warps launch with 96 a thread; the softmax warps take 152, the
// decoders keep 64 and the issuers 40.
constexpr int kLaunchRegs = 96, kSoftRegs = 152, kDecodeRegs = 64, kIssueRegs = 40;
static_assert(kSoftWarps * kSoftRegs + 2 * kDecodeWarps * kDecodeRegs + kSoftFirst * kIssueRegs <=
                  (kSoftFirst + kSoftWarps + 2 * kDecodeWarps) * kLaunchRegs,
              "register split");

template <int D>
struct Kv4Rows128 {
  static constexpr int R = kv4_record_bytes(D);
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTile * 128;             // 128 rows of 64 halves, K and V alike
  static constexpr int kOpBytes = kBoxes * kBoxBytes;
  static constexpr int kRaw = 2;                            // stages of records (3: 140 us in place of 136)
  static constexpr int kRawBytes = kTile * R;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + 2 * kOpBytes;
  static constexpr int kOffRaw = kOffV + 2 * kOpBytes;
  // after the loop: the rows of both halves, the ones received, and their
  // references and sums
  static constexpr int kOffRecv = 2 * kRows * (D + 4) * 4;
  static constexpr int kOffMl = kOffRecv + (kRows * D + 4 * kMaxSplits) * 4;
  static constexpr int kEnd = kOffRaw + kRaw * kRawBytes;
  static constexpr int kMerge = kOffMl + kMaxSplits * kRows * 8;
  static constexpr int kSmem = (kEnd > kMerge ? kEnd : kMerge) + 1024;
  // TMEM: S, O of both halves, P (a pair of keys per column), Q (a pair of dims)
  static constexpr uint32_t kColO = kTile, kColP = kColO + 256, kColQ = kColP + kTile / 2, kTmemCols = 512;
  static_assert(kSmem <= 227 * 1024 - 8192, "shared memory budget");
};

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// Which of the 32 keys from k0 on a row sees, as bits.
__device__ __forceinline__ uint32_t sees32(const RowKeys &r, int k0, int L, int window) {
  uint32_t prefix = low_bits(L - k0);
  if (window) prefix &= low_bits(r.sinks - k0) | ~low_bits(r.first - k0);
  const int o = k0 - L;            // first key's node
  const uint4 m = r.tree;
  if (o <= -32) return prefix;
  if (o < 0) return prefix | (m.x << -o);
  const int w = o >> 5;
  const uint32_t lo = w == 0 ? m.x : w == 1 ? m.y : w == 2 ? m.z : w == 3 ? m.w : 0u;
  const uint32_t hi = w == 0 ? m.y : w == 1 ? m.z : w == 2 ? m.w : 0u;
  return __funnelshift_r(lo, hi, o & 31);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_attn_kv4_rows_kernel(const Kv4AttnArgs p) {
  using C = Kv4Rows128<D>;
  constexpr int R = C::R, kRaw = C::kRaw;
  const AttnArgs &a = p.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ struct {
    uint64_t raw_full[kRaw], raw_empty[kRaw];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], s_empty[2], p_full[2], o_done[2], q_full;     // [half of the keys]
    uint64_t drained[2];
  } bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_timeout;
  __shared__ int s_par[SPEC_MAX_TREE_NODES];
  __shared__ long long s_row[kRows];          // a row's first element of o
  __shared__ float s_top[2][kRows];           // [half of the dims][row]: largest magnitude of q
  __shared__ float s_ref[2][kRows], s_sum[2][kRows];

  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
  float2 (*s_ml)[kRows] = reinterpret_cast<float2 (*)[kRows]>(smem + C::kOffMl);
  const uint32_t raw_full = smem_addr(bars.raw_full), raw_empty = smem_addr(bars.raw_empty);
  const uint32_t s_full = smem_addr(bars.s_full), s_empty = smem_addr(bars.s_empty);
  const uint32_t p_full = smem_addr(bars.p_full), o_done = smem_addr(bars.o_done);
  const int CS = static_cast<int>(gridDim.x), split = static_cast<int>(blockIdx.x);
  const int b = blockIdx.z / a.Hkv, g_kv = blockIdx.z % a.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(&bars.raw_full[s], 1);
      mbar_init(&bars.raw_empty[s], 2 * kDecodeWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.k_full[s], kDecodeWarps);
      mbar_init(&bars.v_full[s], kDecodeWarps);
      mbar_init(&bars.k_empty[s], 1);
      mbar_init(&bars.v_empty[s], 1);
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.s_empty[s], kSoftWarps / 2);
      mbar_init(&bars.p_full[s], kSoftWarps / 2);
      mbar_init(&bars.o_done[s], 1);
      mbar_init(&bars.drained[s], 1);
    }
    mbar_init(&bars.q_full, kSoftWarps);
    fence_barrier_init();
    s_timeout = 0;
  }
  if (warp == 1) {
    tc::tmem_alloc(&s_tmem, C::kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  pdl_wait();

  const ReqGeom G = request_geometry(a, b);
  const int rows_total = G.err ? 0 : G.n * a.G;
  if (G.err && tid == 0 && split == 0 && blockIdx.y == 0 && g_kv == 0) report(a.status, b, G.err);
  const TileList<kTile> tiles(G.L, G.keys, p.window, p.sinks);
  const int per = (tiles.count + CS - 1) / CS;
  const int t0 = split * per;
  const int ntiles = max(0, min(t0 + per, tiles.count) - t0);

  // Each role runs the turns (row blocks) of this CTA on its own, its places
  // in the rings going on from turn to turn, and meets the others at their
  // ends, where the softmax warps merge the rows.  A wait that runs out clears
  // ok: the role stops waiting, and all return after the turn.  (The
  // products go on, on whatever is there: no lane leaves a loop in which its warp
  // meets.)
  bool ok = true;
  auto turns = [&](auto &&work, auto &&finish) {
    for (int row0 = static_cast<int>(blockIdx.y) * kRows; row0 < rows_total;
         row0 += static_cast<int>(gridDim.y) * kRows) {
      work(row0);
      if (!ok) s_timeout = 1;
      __syncwarp();
      tc::fence_before_sync();
      __syncthreads();
      tc::fence_after_sync();
      const bool done = finish(row0);
      // (the next turn's records and operands take the staged rows' place)
      if (!done) break;
      fence_proxy_async_smem();
      __syncthreads();
    }
  };
  // A split block's CTAs arrive twice at the cluster's barrier: when a thread's
  // work on the turn is done (then peers may write here), and when the rows
  // have been sent.
  auto wait_merge = [&](int) {       // the other roles while rows are merged
    if (CS == 1) return s_timeout == 0;
    cluster_arrive_relaxed();
    cluster_wait();
    cluster_sync_all();
    bool done = true;
    for (int q = 0; q < CS; ++q) done &= !(s_ml[q][0].y < 0.f);
    return done;
  };

  // The softmax warps' rows, staged, and the decoders' hands.
  auto merge = [&](int row0, int thread) {
    const bool timed_out = s_timeout != 0;
    if (timed_out && thread == 0) report(a.status, b, SPEC_ERR_TIMEOUT);
    auto out_row = [&](int r) { return s_row[r] < 0 ? nullptr : static_cast<__nv_bfloat16 *>(a.o) + s_row[r]; };
    return merge_rows<D, 2, kRows, kMergeThreads, __nv_bfloat16>(
        thread, CS, split, min(kRows, rows_total - row0), timed_out, reinterpret_cast<float *>(smem), s_ref, s_sum,
        s_ml, reinterpret_cast<float4 *>(smem + C::kOffRecv), [] { cluster_wait(); }, out_row);
  };

  // (each group of four warps has one register budget)
  if (warp < kSoftFirst) {
    give_registers<kIssueRegs>();
    if (warp == 0) {
      // ------------------------------------------------------------ records
      const uint8_t *kv = static_cast<const uint8_t *>(a.k) + (static_cast<size_t>(b) * a.Hkv + g_kv) * a.S_cap * R;
      Ring<kRaw> raw;
      raw.phase = 1;      // every stage is free at first
      turns([&](int) {
        if (lane != 0) return;
        for (int i = 0; i < ntiles && ok; ++i, raw.next()) {
          // (decoders that gave up free a stage whose last copy has not landed: nothing
          // may be announced on a barrier that still awaits bytes)
          ok = mbar_sleep(raw_empty + 8 * raw.at, raw.phase) && mbar_over(raw_full + 8 * raw.at, raw.phase);
          if (!ok) break;
          const int key0 = tiles.key0(t0 + i), count = min(kTile, G.keys - key0);
          const uint32_t bytes = static_cast<uint32_t>(count * R);
          if (range_in_bounds(key0, count, a.S_cap, a.status, b)) {
            mbar_arrive_expect_tx(&bars.raw_full[raw.at], bytes);
            bulk_copy_g2s(sb + C::kOffRaw + raw.at * C::kRawBytes, kv + static_cast<size_t>(key0) * R, bytes,
                          &bars.raw_full[raw.at]);
          } else {
            mbar_arrive(&bars.raw_full[raw.at]);
          }
        }
      }, wait_merge);
      // (of a stage that has had no copy the phase before is over)
      if (s_timeout != 0 && lane == 0)
        for (uint32_t st = 0; st < kRaw; ++st) mbar_wait(&bars.raw_full[st], st < raw.at ? raw.phase ^ 1 : raw.phase);
    } else if (warp == 1) {
      // ------------------------------------------------------------ S = Q K^T
      constexpr uint32_t id = tc::idesc_f16_f32(kRows, kTile / 2, 0, 0);
      const uint64_t kd0 = tc::smem_desc_sw128(sb + C::kOffK, 16, 1024);
      const uint32_t k_full = smem_addr(bars.k_full);
      Ring<2> kr;
      const bool leader = tc::elect_one();
      uint32_t phase = 1;        // of the S buffer: free at first
      uint32_t q_phase = 0;
      turns([&](int) {
        if (ntiles == 0) return;
        ok = mbar_sleep(smem_addr(&bars.q_full), q_phase);
        q_phase ^= 1;
        for (int i = 0; i < ntiles; ++i, kr.next(), phase ^= 1) {
          ok = ok && mbar_sleep(k_full + 8 * kr.at, kr.phase);
          for (int half = 0; half < 2; ++half) {
            ok = ok && mbar_sleep(s_empty + 8 * half, phase);
            tc::fence_after_sync();
            const uint64_t kd = kd0 + static_cast<uint64_t>((kr.at * C::kOpBytes + half * (kTile / 2 * 128)) >> 4);
            if (leader) {
  #pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t at = ((ks >> 2) * C::kBoxBytes + (ks & 3) * 32) >> 4;
                tc::mma_bf16_ts(tmem + half * (kTile / 2), tmem + C::kColQ + ks * 8, kd + at, id, ks > 0);
              }
              tc::commit(&bars.s_full[half]);
              if (half) tc::commit(&bars.k_empty[kr.at]);
            }
            __syncwarp();
          }
        }
      }, wait_merge);
    } else if (warp == 2) {
      // ------------------------------------------------------------ O += P V
      constexpr uint32_t id = tc::idesc_f16_f32(kRows, D, 0, 1);
      const uint64_t vd0 = tc::smem_desc_sw128(sb + C::kOffV, C::kBoxBytes, 1024);
      const uint32_t v_full = smem_addr(bars.v_full);
      Ring<2> vr;
      const bool leader = tc::elect_one();
      uint32_t phase = 0;        // of P
      turns([&](int) {
        for (int i = 0; i < ntiles; ++i, vr.next(), phase ^= 1) {
          ok = ok && mbar_sleep(v_full + 8 * vr.at, vr.phase);
          for (int half = 0; half < 2; ++half) {
            ok = ok && mbar_sleep(p_full + 8 * half, phase);
            tc::fence_after_sync();
            const uint64_t vd = vd0 + static_cast<uint64_t>((vr.at * C::kOpBytes + half * (kTile / 2 * 128)) >> 4);
            const uint32_t pt = tmem + C::kColP + half * (kTile / 4);
            if (leader) {
  #pragma unroll
              for (int kk = 0; kk < kTile / 32; ++kk)
                tc::mma_bf16_ts(tmem + C::kColO + half * 128, pt + kk * 8, vd + (kk * 16 * 128 >> 4), id, (i | kk) != 0);
              tc::commit(&bars.o_done[half]);
              if (half) tc::commit(&bars.v_empty[vr.at]);
            }
            __syncwarp();
          }
        }
      }, wait_merge);
    } else {
      turns([](int) {}, wait_merge);
    }
  } else if (warp >= kDecodeFirst) {
    // ------------------------------------------------------------ decode
    give_registers<kDecodeRegs>();
    const bool of_v = warp >= kDecodeFirst + kDecodeWarps;
    const int key = (warp & 3) * 32 + lane;
    const uint32_t full = smem_addr(of_v ? bars.v_full : bars.k_full);
    const uint32_t empty = smem_addr(of_v ? bars.v_empty : bars.k_empty);
    const uint8_t *rec0 = smem + C::kOffRaw + key * R;
    const uint32_t row = sb + (of_v ? C::kOffV : C::kOffK) + key * 128 + ((key & 7) << 4);
    const LiveKeys live(G.L, G.keys, p.window, p.sinks);
    Ring<kRaw> raw;
    Ring<2> op;
    turns([&](int) {
      for (int i = 0; i < ntiles; ++i, raw.next(), op.next()) {
        ok = ok && mbar_sleep(raw_full + 8 * raw.at, raw.phase);
        const KeyCodes<D> codes(rec0 + raw.at * C::kRawBytes, of_v, live(tiles.key0(t0 + i) + key));
        ok = ok && mbar_sleep(empty + 8 * op.at, op.phase ^ 1);
        const uint32_t dst = row + op.at * C::kOpBytes;
        codes.decode([&](int g, const uint32_t(&h)[8]) { put_swizzled<C::kBoxBytes>(dst, g, h); });
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_at(full + 8 * op.at);
          mbar_arrive_at(raw_empty + 8 * raw.at);
        }
      }
    }, [&](int row0) {
      if (CS > 1) cluster_arrive_relaxed();
      return merge(row0, tid - 32 * kSoftFirst);
    });
  } else {
    // ------------------------------------------------------------ softmax
    take_registers<kSoftRegs>();
    const int quad = warp & 3, half = (warp - kSoftFirst) >> 2;
    const int soft = tid - 32 * kSoftFirst;            // 0 .. 255
    const int row = quad * 32 + lane;                  // and TMEM lane
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_col = trow + half * kHalf, o_col = trow + C::kColO + half * 128;
    const uint32_t p_col = trow + C::kColP + half * (kHalf / 2);
    const uint32_t s_full_h = s_full + 8 * half, s_empty_h = s_empty + 8 * half, p_full_h = p_full + 8 * half,
                   o_done_h = o_done + 8 * half;
    uint32_t phase = 0;      // of S, P and the products: flips with every tile
    turns([&](int row0) {
      const int rows_here = min(kRows, rows_total - row0);
      const bool live = row < rows_here;
      // ---- Q as halves: this thread's row, half of its dims.  Every load of
      //      the set-up is under way before the first is used.
      const int node = (row0 + row) / a.G;
      const bool mine = live && in_bounds(G.lo + node, a.T, a.status, b);
      const long long first =
          (static_cast<long long>(G.lo + node) * a.Hq + g_kv * a.G + (row0 + row) - node * a.G) * D;
      const uint4 *src =
          reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + first + half * (D / 2));
      uint4 x4[D / 16], m = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) x4[c] = mine ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
      if (a.mask) {
        if (mine) m = __ldg(a.mask + G.lo + node);
      } else if (row0 == static_cast<int>(blockIdx.y) * kRows) {
        for (int i = soft; i < G.n; i += kSoftThreads)
          s_par[i] = in_bounds(G.lo + i, a.T, a.status, b) ? __ldg(a.parents + G.lo + i) : -2;
      }
      if (half == 0) s_row[row] = mine ? first : -1;
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint32_t u[4] = {x4[c].x, x4[c].y, x4[c].z, x4[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = max3(top, fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xFFFF0000u)));
      }
      s_top[half][row] = top;
      named_bar_sync(1, kSoftThreads);
      const int up = row_exponent(fmaxf(s_top[0][row], s_top[1][row]));
      const float grow = power_of_two(up), c = a.scale_log2 * power_of_two(-up);
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t u = (&x4[2 * q + (e >> 2)].x)[e & 3];
          h[e] = pack_half2(__uint_as_float(u << 16) * grow, __uint_as_float(u & 0xFFFF0000u) * grow);
        }
        tc::st8(trow + C::kColQ + half * (D / 4) + 8 * q, h);
      }
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(smem_addr(&bars.q_full));
      // ---- what this thread's row sees
      if (a.mask) {
        m = clip_mask(m, G.n);
      } else if (live) {
        bool bad = false;
        m = ancestor_mask([&](int i) { return s_par[i]; }, node, &bad);
        if (bad) report(a.status, b, SPEC_ERR_BAD_PARENT);
      }
      const RowKeys see = row_keys(m, G.L, p.window, p.sinks);
      float ref = live ? -INFINITY : 0.f;      // rows of no node need no reference
      float sum = 0.f;
      float shift = kWeightLog2;               // 8 - reference (8 while there is none)

      for (int i = 0; i < ntiles; ++i, phase ^= 1) {
        const int key0 = tiles.key0(t0 + i), k0 = key0 + half * kHalf;
        const bool whole = k0 + kHalf <= G.L && (p.window == 0 || k0 + kHalf <= p.sinks || k0 >= G.L + G.n - p.window);
        ok = ok && mbar_sleep(s_full_h, phase);
        __syncwarp();
        tc::fence_after_sync();
        // The tile's weights at the present reference and their sum, and the
        // largest score - reference + 8, in powers of two.  (S is read again when
        // the reference moves, which it hardly ever does.)
        uint32_t h[kHalf / 16][8];
        float tile_sum, most;
        auto weigh = [&](auto exponents) {
          float x[2][32];
          tc::ld32(s_col, x[0]);
          tc::ld32(s_col + 32, x[1]);
          tc::wait_ld();
          float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
          most = -INFINITY;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            exponents(x[part]);
            if (!whole) {
              const uint32_t sees = sees32(see, k0 + 32 * part, G.L, p.window);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((sees >> j) & 1u)) x[part][j] = -INFINITY;
            }
            most = fmaxf(most, max_of(x[part]));
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float p0 = fast_exp2(x[part][j]), p1 = fast_exp2(x[part][j + 1]);
              const float p2 = fast_exp2(x[part][j + 2]), p3 = fast_exp2(x[part][j + 3]);
              add2(s0, s1, p0, p1);
              add2(s2, s3, p2, p3);
              h[2 * part + j / 16][j / 2 % 8] = pack_half2(p0, p1);
              h[2 * part + j / 16][j / 2 % 8 + 1] = pack_half2(p2, p3);
            }
          }
          add2(s0, s1, s2, s3);
          tile_sum = s0 + s1;
        };
        weigh([&](float(&x)[32]) {
#pragma unroll
          for (int j = 0; j < 32; j += 2) fma2(x[j], x[j + 1], c, c, shift, shift);
        });
        const bool fresh = ref == -INFINITY;
        const bool moves = most > (fresh ? -INFINITY : kWeightLog2 + kMoveLog2);
        if (__any_sync(0xffffffffu, moves)) {
          Move move(shift);
          const bool far = moves && far_above(most, shift, fresh);
          if (far) {
            move.factor = 0.f;
            shift = kWeightLog2;
            ref = -INFINITY;
          } else if (moves) {
            move = Move(most, shift, fresh);
            shift = move.next;
            ref = kWeightLog2 - shift;
          }
          if (i > 0) {
            // O holds the products of this turn's earlier tiles
            ok = ok && mbar_sleep(o_done_h, phase ^ 1);
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll 1
            for (int j = 0; j < D; j += 8) {
              float o[8];
              tc::ld8(o_col + j, o);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= move.factor;
              tmem_st(o_col + j, o);
            }
            tc::wait_st();
          }
          sum *= move.factor;
          if (__any_sync(0xffffffffu, far)) {
            --i;
            phase ^= 1;
            continue;
          }
          const bool steep = __any_sync(0xffffffffu, move.less != 0.f);
          weigh([&](float(&x)[32]) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) fma2(x[j], x[j + 1], c, c, move.base, move.base);
            if (steep) {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] -= move.less;
            }
          });
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(s_empty_h);
        sum += tile_sum;
        // ---- the weights' place is free once the last tile's product is done (most
        //      often it is: the test spares the wait's 115 cycles)
        ok = ok && (mbar_over(o_done_h, phase ^ 1) || mbar_sleep(o_done_h, phase ^ 1));
        __syncwarp();
        tc::fence_after_sync();
#pragma unroll
        for (int q = 0; q < kHalf / 16; ++q) tc::st8(p_col + 8 * q, h[q]);
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(p_full_h);
      }
      // ---- the block's rows out of TMEM.  Their place in shared memory is free
      //      once the last products of both halves are done.
      if (ntiles > 0) ok = ok && mbar_sleep(o_done_h, phase ^ 1);
      if (CS > 1) cluster_arrive_relaxed();
      __syncwarp();
      tc::fence_after_sync();
      if (!ok) s_timeout = 1;
      named_bar_sync(1, kSoftThreads);
      if (s_timeout == 0) {
        s_sum[half][row] = sum;
        s_ref[half][row] = ntiles > 0 ? ref : -INFINITY;
        const uint32_t so = sb + (half * kRows + row) * (D + 4) * 4;
#pragma unroll
        for (int j = 0; j < D; j += 32) {
          float o[32] = {};
          if (ntiles > 0) {
            tc::ld32(o_col + j, o);
            tc::wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            st_shared_v4(so + (j + e) * 4, __float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]),
                         __float_as_uint(o[e + 3]));
        }
      }
    }, [&](int row0) { return merge(row0, soft); });
  }
  __syncwarp();
  // A turn that was given up may leave products under way (and copies, see warp 0):
  // the warps that issued them wait, with a limit, before the CTA gives up its memory.
  if (s_timeout != 0 && (warp == 1 || warp == 2)) {
    if (tc::elect_one()) tc::commit(&bars.drained[warp - 1]);
    __syncwarp();
    mbar_wait(&bars.drained[warp - 1], 0);
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace

int launch_kv4_rows(const Kv4AttnArgs &p, int max_prefix, void *stream) {
  const int blocks = (mean_nodes(p.a) * p.a.G + kRows - 1) / kRows;
  static KernelState state[2];
  if (p.a.D == 128)
    return launch_kv4_tiles(tree_attn_kv4_rows_kernel<128>, p, kThreads, kLaunchRegs, Kv4Rows128<128>::kSmem, blocks,
                            max_prefix, &state[0], stream);
  return launch_kv4_tiles(tree_attn_kv4_rows_kernel<64>, p, kThreads, kLaunchRegs, Kv4Rows128<64>::kSmem, blocks,
                          max_prefix, &state[1], stream);
}

}  // namespace spec
