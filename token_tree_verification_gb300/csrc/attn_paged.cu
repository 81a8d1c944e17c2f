// Attention of trees and chunks over a paged cache on the 5th-generation
// tensor cores, bf16 in, fp32 accumulate.
//
// One CTA = one split of the keys x one block of 128 query rows (node-major,
// head-minor) of one request and KV head, so that a tile of keys and values
// serves every query head of its KV head.  Rows lie along M:
//   S[rows][keys] = Q K^T   A = Q (TMEM),  B = K (keys x dims, shared memory, K-major)
//   O[rows][dims] = P V     A = P (TMEM),  B = V (keys x dims, shared memory, MN-major)
// P enters its product as a bf16 high part and a bf16 remainder, some 16
// significant bits of each weight: with the high part alone elements of a
// hundredth of the output's largest come out wrong by a tenth (their terms
// cancel).  That makes a tile's tensor work 3/2 of the least: 512 cycles for S
// and 1024 for O per 128 keys at D = 128.
//
// Warp roles:
//   warps 0, 3  bring tiles of 128 keys and of 128 values into rings of their own;
//               a lane copies one box, 64 dims of one page's slots (of 128 at most),
//               whose page it looked up a tile ahead.  (A box is some 60 cycles of
//               the warp's time; with one warp for both, pages of 16 slots took 3000
//               a tile.)  Warp 3 then looks through the request's whole page table:
//               a request that names a page outside the pool gets no output
//   warp 1      allocates TMEM and issues S_u, for 64 keys (half a tile) at a time
//   warp 2      issues O += P_u V_u
//   warps 4-11  softmax, in two groups that take the halves in turn; a thread
//               has a row (a TMEM lane) and the 64 keys of a half
// That is the whole form, which has an SM to itself.  A launch of many blocks with
// few keys each is set-up for the most part (offsets, page, keys: three loads one
// behind the other; output), and takes the small form: half an SM, one softmax group,
// one tile of keys and one of values, so that a CTA's set-up hides behind another's
// tiles.  At D = 128 its Q lies in shared memory, which leaves TMEM for the scores of
// two halves (one: 121 in place of 107 us for single tokens of 256 requests behind 500
// keys; at D = 64 there is room for both and it gains nothing).  launch_bf16 says which
// form is taken and what both take.
// TMEM holds the scores of five halves, and P takes the place of S, so that the
// products of one half run beside the softmax of two others.  A row's reference
// is shared by the groups, which decide on it in the order of the halves (a
// barrier per lane quarter and group passes the turn); it moves when a score passes
// it by more than 2^8, which is rare behind the first keys, and O is then rescaled
// in place.  A quarter without rows leaves the softmax out.
//
// The tensor cores' queue is short: what an issuing warp does between two batches
// of products (tests of barriers at 36 cycles, waits at 70, descriptors) is time
// lost unless the other issuing warp fills it.  Hence two of them; one that issued
// both kinds took 2750 cycles a tile in place of 1900, 2350 with the tests placed
// between its products.
//
// Measured, device times: 128-node trees of 4 requests, 64 heads on 8, behind 8192
// keys: 138 to 141 us, 1.0 PFLOP/s and with the remainders' products 1.5; the tensor pipe
// is busy for 0.8 of an SM's time, for all but 0.04 of the busiest's, which has two of
// 256 CTAs where an even share is 1.7.  A
// chunk of 2048 tokens behind 16384, 64 heads on 8: 0.97 to 1.02 ms, 1.17 PFLOP/s, with
// the remainders' 1.75, near what a library product sustains.  6-node chains of 8
// requests, 32 heads, behind 27000 to 32768 keys: 564 us, 7.0 TB/s, a copy's rate.
// One token of 4 requests behind 8192 keys, 64 heads on 8: 27 us, 5 TB/s; 64-node
// tree, 32 heads, behind 2048: 14.9 us, of them 2.5 to the first key tile, 7 of tiles
// and 4 of output and merge.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_kv4_tc.cuh"
#include "attn_paged.cuh"

namespace spec {

namespace {

constexpr int kRows = 128;
constexpr int kSoftFirst = 4;         // warps: issuers and the page check, then the softmax
constexpr int kHalf = kTile / 2;      // keys of a product, and of one softmax thread
constexpr float kPass = 8.f;          // powers of two by which a score may pass its row's reference

// A wait that is over already, most often.
__device__ __forceinline__ bool mbar_now(uint64_t *bar, uint32_t parity) {
  return mbar_over(smem_addr(bar), parity) || mbar_sleep(smem_addr(bar), parity);
}

// The whole form has an SM to itself; the small one (kSmall) half of it: one softmax
// group, a stage of keys and of values, half of TMEM, and no splits.
template <int D, bool kSmall>
struct PagedCfg {
  static constexpr int kGroups = kSmall ? 1 : 2;            // of four softmax warps
  static constexpr int kSoftThreads = 128 * kGroups;
  static constexpr int kThreads = 32 * kSoftFirst + kSoftThreads;
  static constexpr int kCtas = kSmall ? 2 : 1;              // of an SM
  static constexpr int kBufs = kSmall ? 2 : 5;             // halves' scores and weights in TMEM
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTile * 128;             // 128 slots of 64 dims
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kStages = (kSmall ? 1 : 3) * 128 / D;      // of keys, and as many of values
  static constexpr int kOffK = 0, kOffV = kStages * kTileBytes;
  static constexpr bool kQSmem = kSmall && D == 128;        // Q lies in shared memory, as keys do
  static constexpr int kOffQ = 2 * kStages * kTileBytes;
  static constexpr int kRings = kOffQ + (kQSmem ? D / 64 * kRows * 128 : 0), kMerge = kSmall ? kRows * (D + 4) * 4 : merge_bytes<D>(kRows);
  // (the rows take the rings' place after the loop)
  static constexpr int kSmem = (kRings > kMerge ? kRings : kMerge) + 1024;
  // TMEM: the halves' S, and P in their place (a pair of keys per column, remainders
  // behind the high parts), Q (a pair of dims), O
  static constexpr uint32_t kColQ = kBufs * kHalf, kColO = kColQ + (kQSmem ? 0 : 64), kTmemCols = 512 / kCtas;
  static_assert(kColO + D <= kTmemCols, "tensor memory");
  static_assert(kCtas * (kSmem + 8192) <= 227 * 1024, "shared memory budget");
};

// What rounding to bf16 took from y0 and y1 (`top` holds the two, y0's low), exactly.
__device__ __forceinline__ void minus_bf16x2(float y0, float y1, uint32_t top, float &r0, float &r1) {
  asm("{\n\t.reg .b16 t0, t1, m;\n\t"
      "mov.b32 {t0, t1}, %2;\n\tmov.b16 m, 0xBF80;\n\t"
      "fma.rn.f32.bf16 %0, t0, m, %3;\n\tfma.rn.f32.bf16 %1, t1, m, %4;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "r"(top), "f"(y0), "f"(y1));
}

template <int D, bool kSmall>
__global__ void __launch_bounds__(PagedCfg<D, kSmall>::kThreads, PagedCfg<D, kSmall>::kCtas)
tree_attn_paged_kernel(const PagedAttnArgs p, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const int splits) {
  using C = PagedCfg<D, kSmall>;
  constexpr int NS = C::kStages, kGroups = C::kGroups, kBufs = C::kBufs, kSoftThreads = C::kSoftThreads;
  const int CS = kSmall ? 1 : splits;
  const AttnArgs &a = p.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ struct {
    uint64_t k_full[NS], k_empty[NS], v_full[NS], v_empty[NS];
    uint64_t q_full, s_full[kBufs], p_full[kBufs], o_done[kBufs], turn[4][kGroups], drained[2], merge;
  } bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_timeout, s_bad_page;
  __shared__ int s_par[SPEC_MAX_TREE_NODES];
  __shared__ long long s_row[kRows];          // a row's first element of o
  __shared__ float s_ref[kRows], s_part[kGroups][kRows];

  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sb = __shfl_sync(0xffffffffu, smem_addr(smem), 0);
  const int split = static_cast<int>(blockIdx.x) % CS, block = static_cast<int>(blockIdx.x) / CS;
  const int g_kv = static_cast<int>(blockIdx.y);
  // (a shuffle tells the compiler that a value is the same in all lanes: the products'
  // operands then stay in uniform registers)
  auto uniform = [](auto x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  if (!kSmall) pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars.k_full[s], 1);
      mbar_init(&bars.k_empty[s], 1);
      mbar_init(&bars.v_full[s], 1);
      mbar_init(&bars.v_empty[s], 1);
    }
    mbar_init(&bars.q_full, 4 * kGroups);
    for (int s = 0; s < kBufs; ++s) {
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.p_full[s], 4);
      mbar_init(&bars.o_done[s], 1);
    }
    for (int s = 0; s < 4 * kGroups; ++s) mbar_init(&bars.turn[0][0] + s, 1);
    mbar_init(&bars.merge, 1);
    mbar_init(&bars.drained[0], 1);
    mbar_init(&bars.drained[1], 1);
    fence_barrier_init();
    s_timeout = 0;
    s_bad_page = 0;
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  // The small form leaves room for CTAs of the launches before and after: it must
  // take its TMEM neither before those in front have done with theirs, nor after
  // those behind, which would wait for it with TMEM in hand.
  if (kSmall) pdl_wait();
  if (warp == 1) {
    tc::tmem_alloc(&s_tmem, C::kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(s_tmem);
  if (kSmall) pdl_trigger();
  else pdl_wait();

  if (warp == 0) touch_table(p, lane);
  const RowBlock w = find_block<kRows>(p, block, lane);
  if (g_kv == 0 && warp == 3) report_bad_requests(p, lane);
  if (w.b < 0) {       // the same for every CTA of the cluster
    if (warp == 1) {
      __syncwarp();
      tc::tmem_dealloc(tmem, C::kTmemCols);
    }
    return;
  }
  const int b = w.b, L = w.R.L;
  const int all = (w.keys + kTile - 1) / kTile;
  const int per = (all + CS - 1) / CS;
  const int t0 = split * per;
  const int ntiles = uniform(max(0, min(t0 + per, all) - t0));
  const int halves = uniform(max(0, min(2 * ntiles, (w.keys - t0 * kTile + kHalf - 1) / kHalf)));      // that hold a key
  bool ok = true;      // cleared by a wait that ran out: the role goes on without waiting, and no row is written

  Ring<NS> copies;     // of the copying warps
  copies.phase = 1;    // every stage is free at first
  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ keys and values
    const bool of_v = warp == 3;
    uint64_t *full = of_v ? bars.v_full : bars.k_full, *empty = of_v ? bars.v_empty : bars.k_empty;
    const CUtensorMap *map = of_v ? &tmv : &tmk;
    uint8_t *ring = smem + (of_v ? C::kOffV : C::kOffK);
    const int shift = min(p.pages.shift, 7), box_slots = 1 << shift;
    const int place = lane / C::kBoxes, bx = lane % C::kBoxes;           // a lane's box: page and half of D
    const int in_page = (1 << p.pages.shift) - 1;
    auto boxes = [&](int i) {      // of tile i that hold a key
      return (min(kTile, w.keys - (t0 + i) * kTile) + box_slots - 1) >> shift;
    };
    auto look_up = [&](int i) {    // (an id outside the pool: any page will do, no row is written)
      if (i >= ntiles || place >= boxes(i)) return 0;
      return max(0, p.pages.page(b, ((t0 + i) * kTile + (place << shift)) >> p.pages.shift));
    };
    int page = look_up(0);
    for (int i = 0; i < ntiles; ++i) {
      const int next = look_up(i + 1);
      const int n = boxes(i), slot = ((t0 + i) * kTile + (place << shift)) & in_page;
      // (a consumer that gave up frees a stage whose last copy has not landed: nothing
      // may be announced on a barrier that still awaits bytes)
      ok = ok && mbar_now(&empty[copies.at], copies.phase) && mbar_over(smem_addr(&full[copies.at]), copies.phase);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[copies.at], static_cast<uint32_t>(n * C::kBoxes * box_slots * 128));
      __syncwarp();
      if (place < n)
        tma_load_4d(ring + copies.at * C::kTileBytes + bx * C::kBoxBytes + (place << shift) * 128, map, &full[copies.at],
                    bx * 64, slot, g_kv, page);
      copies.next();
      page = next;
    }
    if (of_v && warp_finds_bad_page(p.pages, b, 0, w.R.keys, lane) && lane == 0) s_bad_page = 1;
  } else if (warp == 1) {
    // ------------------------------------------------------------ S = Q K^T
    constexpr uint32_t id = tc::idesc_bf16_f32(kRows, kHalf, 0, 0);
    const uint64_t kd0 = tc::smem_desc_sw128(sb + C::kOffK, 16, 1024);
    [[maybe_unused]] const uint64_t qd = tc::smem_desc_sw128(sb + C::kOffQ, 16, 1024);
    Ring<NS> ring;
    Ring<kBufs> buf;
    buf.phase = 1;             // free at first, then when what is in it has been multiplied
    const bool leader = tc::elect_one();
    if (halves > 0) ok = mbar_sleep(smem_addr(&bars.q_full), 0);
    for (int u = 0; u < halves; ++u, buf.next()) {
      const int h = u & 1;
      if (h == 0) ok = ok && mbar_now(&bars.k_full[ring.at], ring.phase);
      ok = ok && mbar_now(&bars.o_done[buf.at], buf.phase);
      tc::fence_after_sync();
      const uint64_t kd = kd0 + static_cast<uint64_t>((ring.at * C::kTileBytes + h * (kHalf * 128)) >> 4);
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t at = ((ks >> 2) * C::kBoxBytes + (ks & 3) * 32) >> 4;
          if constexpr (C::kQSmem)
            tc::mma_bf16(tmem + buf.at * kHalf, qd + at, kd + at, id, ks > 0);
          else
            tc::mma_bf16_ts(tmem + buf.at * kHalf, tmem + C::kColQ + ks * 8, kd + at, id, ks > 0);
        }
        tc::commit(&bars.s_full[buf.at]);
        if (h) tc::commit(&bars.k_empty[ring.at]);
      }
      __syncwarp();
      if (h) ring.next();
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ O += P V
    constexpr uint32_t id = tc::idesc_bf16_f32(kRows, D, 0, 1);
    const uint64_t vd0 = tc::smem_desc_sw128(sb + C::kOffV, C::kBoxBytes, 1024);
    Ring<NS> ring;
    Ring<kBufs> buf;
    const bool leader = tc::elect_one();
    for (int u = 0; u < halves; ++u, buf.next()) {
      const int h = u & 1;
      if (h == 0) ok = ok && mbar_now(&bars.v_full[ring.at], ring.phase);
      ok = ok && mbar_now(&bars.p_full[buf.at], buf.phase);
      tc::fence_after_sync();
      const uint64_t vd = vd0 + static_cast<uint64_t>((ring.at * C::kTileBytes + h * (kHalf * 128)) >> 4);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < kHalf / 16; ++kk) {
          const uint32_t pt = tmem + buf.at * kHalf + kk * 8;
          const uint64_t v = vd + (kk * 16 * 128 >> 4);
          tc::mma_bf16_ts(tmem + C::kColO, pt, v, id, (u | kk) != 0);
          tc::mma_bf16_ts(tmem + C::kColO, pt + kHalf / 2, v, id, true);
        }
        tc::commit(&bars.o_done[buf.at]);
        if (h) tc::commit(&bars.v_empty[ring.at]);
      }
      __syncwarp();
      if (h) ring.next();
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3, group = (warp - kSoftFirst) >> 2;
    const int soft = tid - 32 * kSoftFirst;
    const int row = quad * 32 + lane;                  // and TMEM lane
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // decisions on the row's reference: this group's, and the one that goes before
    const uint32_t turn = smem_addr(&bars.turn[quad][group]);
    const uint32_t turn_before = smem_addr(&bars.turn[quad][(group + kGroups - 1) % kGroups]);
    uint32_t round = group > 0 ? 0 : 1;      // of the one before, for the group's next half
    const bool busy = quad * 32 < w.rows;              // (a quarter without rows only keeps the barriers going)
    const bool live = row < w.rows;
    // ---- Q: this thread's row, its group's share of the dims
    constexpr int kDims = D / kGroups;
    const int node = (w.row0 + row) / a.G;
    const bool mine = live && in_bounds(w.R.lo + node, a.T, a.status, b);
    const long long first =
        (static_cast<long long>(w.R.lo + node) * a.Hq + g_kv * a.G + (w.row0 + row) - node * a.G) * D;
    const uint4 *src =
        reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + first + group * kDims);
    uint4 m = make_uint4(0u, 0u, 0u, 0u);
    if (a.mask && mine) m = clip_mask(__ldg(a.mask + w.R.lo + node), w.R.n);
    if (busy) {
      uint4 x4[kDims / 8];
#pragma unroll
      for (int c = 0; c < kDims / 8; ++c) x4[c] = mine ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
      if constexpr (C::kQSmem) {
#pragma unroll
        for (int q = 0; q < kDims / 8; ++q)
          st_shared_v4(sb + C::kOffQ + (q >> 3) * C::kBoxBytes + row * 128 + ((q ^ row) & 7) * 16, x4[q].x, x4[q].y,
                       x4[q].z, x4[q].w);
        fence_proxy_async_smem();
      } else {
#pragma unroll
        for (int q = 0; q < kDims / 16; ++q) {
          const uint4 x = x4[2 * q], y = x4[2 * q + 1];
          const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
          tc::st8(trow + C::kColQ + group * (kDims / 2) + 8 * q, u);
        }
        tc::wait_st();
      }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive_at(smem_addr(&bars.q_full));
    if (group == 0) s_row[row] = mine ? first : -1;
    // ---- what this thread's row sees
    if (a.parents) {
      for (int i = soft; i < w.R.n; i += kSoftThreads)
        s_par[i] = in_bounds(w.R.lo + i, a.T, a.status, b) ? __ldg(a.parents + w.R.lo + i) : -2;
      named_bar_sync(1, kSoftThreads);
      bool bad = false;
      if (live) m = ancestor_mask([&](int i) { return s_par[i]; }, node, &bad);
      if (bad) report(a.status, b, SPEC_ERR_BAD_PARENT);
    }
    const RowSees see = {p.causal ? L + node + 1 : L, m};
    const int all_see = p.causal ? L + w.row0 / a.G + 1 : L;       // what every row of the block sees: [0, all_see)
    const float c = a.scale_log2;
    float ref = -INFINITY, sum = 0.f;      // in powers of two; of this thread's weights 2^(score - ref)
    if (group == 0) s_ref[row] = -INFINITY;
    named_bar_sync(1, kSoftThreads);

    Ring<kBufs> buf, before;               // of this half, and of the one before
    for (int v = 0; v < group; ++v) {
      before = buf;
      buf.next();
    }
    for (int u = group; u < halves; u += kGroups) {
      const int k0 = t0 * kTile + u * kHalf;
      const uint32_t s_col = trow + buf.at * kHalf;
      ok = ok && mbar_now(&bars.s_full[buf.at], buf.phase);
      __syncwarp();
      tc::fence_after_sync();
      if (busy) {
        float x[2][32];
        tc::ld32(s_col, x[0]);
        tc::ld32(s_col + 32, x[1]);
        tc::wait_ld();
        if (k0 + kHalf > all_see) {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint32_t sees = sees_32(see, k0 + 32 * v, L);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((sees >> j) & 1u)) x[v][j] = -INFINITY;
          }
        }
        const float most = fmaxf(max_of(x[0]), max_of(x[1])) * c;
        // The halves take turns at the row's reference: the other group's decision
        // on the half before was long ago, most often.
        if (u > 0) ok = ok && (mbar_over(turn_before, round) || mbar_sleep(turn_before, round));
        round ^= 1;
        __syncwarp();
        const float now = s_ref[row];
        if (__any_sync(0xffffffffu, now != ref || most > now + kPass)) {
          const float next = most > now + kPass ? most : now;
          if (__any_sync(0xffffffffu, next != now)) {
            if (u > 0) {
              // O holds the products of the halves before
              const float factor = next == now ? 1.f : now == -INFINITY ? 0.f : exp2f(now - next);
              ok = ok && mbar_sleep(smem_addr(&bars.o_done[before.at]), before.phase);
              __syncwarp();
              tc::fence_after_sync();
#pragma unroll 1
              for (int j = 0; j < D; j += 16) {
                float o[16];
                tc::ld16(trow + C::kColO + j, o);
                tc::wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= factor;
                tc::st16(trow + C::kColO + j, o);
              }
              tc::wait_st();
            }
            s_ref[row] = next;
          }
          if (next != ref) sum *= ref == -INFINITY ? 0.f : exp2f(ref - next);
          ref = next;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_at(turn);
        // weights 2^(s c - ref): one rounding of the difference, except where the
        // reference has no places behind the point left; there the largest score's
        // own rounding must cancel, or its weight could pass fp32's range
        const float base = ref == -INFINITY ? 0.f : -ref;
        const bool steep = !(fabsf(base) < kWholeEnd);
        const float cs = steep ? 1.f : c;
        if (__any_sync(0xffffffffu, steep)) {
          const float pre = steep ? c : 1.f;
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int j = 0; j < 32; ++j) x[v][j] = __fmul_rn(x[v][j], pre);
        }
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              float *y = &x[v][16 * part + j];
              fma2(y[0], y[1], cs, cs, base, base);
              fma2(y[2], y[3], cs, cs, base, base);
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = fast_exp2(y[e]);
              add2(s0, s1, y[0], y[1]);
              add2(s2, s3, y[2], y[3]);
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y[e], y[e + 1]);
                const uint32_t top = *reinterpret_cast<const uint32_t *>(&h);
                float r0, r1;
                minus_bf16x2(y[e], y[e + 1], top, r0, r1);
                const __nv_bfloat162 l = __floats2bfloat162_rn(r0, r1);
                hi[(j + e) / 2] = top;
                lo[(j + e) / 2] = *reinterpret_cast<const uint32_t *>(&l);
              }
            }
            tc::st8(s_col + 16 * v + 8 * part, hi);
            tc::st8(s_col + kHalf / 2 + 16 * v + 8 * part, lo);
          }
        add2(s0, s1, s2, s3);
        sum += s0 + s1;
      }
      if (k0 + kHalf > w.keys) {
        // slots behind the last key may hold anything: a weight of zero does not
        // hide a NaN
        const int at = (u >> 1) % NS;
        ok = ok && mbar_sleep(smem_addr(&bars.v_full[at]), ((u >> 1) / NS) & 1);
        const int valid = w.keys - k0, pieces = (kHalf - valid) * C::kBoxes * 8;
        for (int z = soft & 127; z < pieces; z += 128) {
          const int r = (u & 1) * kHalf + valid + z / (C::kBoxes * 8), rest = z % (C::kBoxes * 8);
          st_shared_v4(sb + C::kOffV + at * C::kTileBytes + (rest >> 3) * C::kBoxBytes + r * 128 + (rest & 7) * 16, 0u,
                       0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      if (busy) tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(smem_addr(&bars.p_full[buf.at]));
#pragma unroll
      for (int v = 0; v < kGroups; ++v) {
        before = buf;
        buf.next();
      }
    }
    // ---- the block's rows out of TMEM.  Their place in shared memory is free
    //      once the last products of both groups are done.
    //      (One after the other from the group's own last half on: a barrier that is
    //      two phases behind looks done.)
    int u = halves > group ? halves - 1 - (halves - 1 - group) % kGroups : 0;
    buf = Ring<kBufs>();
    for (int v = 0; v < u; ++v) buf.next();
    for (; u < halves; ++u, buf.next()) ok = ok && mbar_sleep(smem_addr(&bars.o_done[buf.at]), buf.phase);
    __syncwarp();
    tc::fence_after_sync();
    if (busy && halves > 0)
      ok = ok && mbar_sleep(smem_addr(&bars.turn[quad][(halves - 1) % kGroups]), (halves - 1) / kGroups & 1);
    __syncwarp();
    const float now = s_ref[row];
    if (now != ref) sum *= ref == -INFINITY ? 0.f : exp2f(ref - now);
    s_part[group][row] = sum;
    if (!ok) s_timeout = 1;
    named_bar_sync(1, kSoftThreads);
    if (busy && s_timeout == 0) {
      float *staged = reinterpret_cast<float *>(smem) + row * (D + 4);
      if (group == 0) {
        for (int q = 1; q < kGroups; ++q) sum += s_part[q][row];
        *reinterpret_cast<float2 *>(staged + D) = make_float2(now, sum);
      }
      const uint32_t so = smem_addr(staged + group * kDims);
#pragma unroll
      for (int j = 0; j < kDims; j += 32) {
        float o[32] = {};
        if (halves > 0) {
          tc::ld32(trow + C::kColO + group * kDims + j, o);
          tc::wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          st_shared_v4(so + (j + e) * 4, __float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]),
                       __float_as_uint(o[e + 3]));
      }
    }
  }
  if (!ok) s_timeout = 1;
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const bool timed_out = s_timeout != 0, bad_page = s_bad_page != 0;
  if (timed_out) {
    // What was given up may leave copies and products under way: the warps that
    // issued them wait, with a limit.  (Of a stage that has had no copy the phase
    // before is over.)
    if (tid == 0) report(a.status, b, SPEC_ERR_TIMEOUT);
    if (lane == 0 && (warp == 0 || warp == 3))
      for (uint32_t st = 0; st < NS; ++st)
        mbar_wait(warp == 3 ? &bars.v_full[st] : &bars.k_full[st], st < copies.at ? copies.phase ^ 1 : copies.phase);
    if (warp == 1 || warp == 2) {
      if (tc::elect_one()) tc::commit(&bars.drained[warp - 1]);
      __syncwarp();
      mbar_wait(&bars.drained[warp - 1], 0);
    }
    __syncthreads();
  }
  if (bad_page && tid == 0) report(a.status, b, SPEC_ERR_PAGE);
  if (warp == 1) {
    __syncwarp();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
  float *so = reinterpret_cast<float *>(smem);
  if ((timed_out || bad_page) && tid < kRows) so[tid * (D + 4) + D + 1] = -1.f;
  auto out_row = [&](int r) { return s_row[r] < 0 ? nullptr : static_cast<__nv_bfloat16 *>(a.o) + s_row[r]; };
  if (!merge_splits<D, C::kThreads, __nv_bfloat16>(tid, CS, split, w.rows, so, &bars.merge, out_row) && tid == 0)
    report(a.status, b, SPEC_ERR_TIMEOUT);
}

// ---------------------------------------------------------------- host side
using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;

EncodeFn tensor_map_encoder() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(f);
  });
  return fn;
}

// 4-D map over a pool [pages][Hkv][slots][D]: a box is 64 dims of a page's
// slots, 128 at most, loaded with 128-byte swizzle.  (Boxes of eight slots and
// up start on the 1024 bytes over which the swizzle repeats.)
bool encode_pool(CUtensorMap *m, const void *base, const PageTable &pages, int Hkv, int D) {
  const EncodeFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t slots = 1ull << pages.shift;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), slots, static_cast<cuuint64_t>(Hkv),
                              static_cast<cuuint64_t>(pages.pages)};
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  const cuuint64_t strides[3] = {row, slots * row, static_cast<cuuint64_t>(Hkv) * slots * row};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(slots < kTile ? slots : kTile), 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// As many splits of the keys (a cluster) as make waves x (tiles of a CTA + its
// set-up, first tile and merge, which grows with the rows, in half tiles) least; or
// the small form, whose tiles, two CTAs side by side, cost 4.5 half tiles (3 at D = 64).
// (Device us by splits 1, 2, 3, 4, 5 and 8: 32 rows of 8 heads behind 500 keys 9.5,
// 9.1, 8.1, 8.1, 7.5 and 7.6; 128 rows of 32 heads behind 300 12.3, 13.2, 13.2, 13.5;
// one token x 4 x 8 heads behind 8192 58, 34, 26.9, 26.2, 39 and 45.  Whole and small
// form, 8 heads of 4 query heads each: a token of 256 requests behind 60, 500, 1000,
// 1500, 2000 and 3000 keys 77 and 39, 144 and 107, 215 and 187, 283 and 261, 350 and
// 338, 486 and 484; at D = 64 behind 60, 500, 1500 and 3000 72 and 34, 118 and 71, 210
// and 147, 336 and 256 (60 keys of all lie in L2; from memory the small form takes 43
// and, at D = 64, 38); prompts of 512 tokens x 8, 80 and 50.  128-node trees x 4, 64
// heads on 8, behind 8192: 137 and 149, at D = 64 118 and 112; chains of 6 x 8, 32
// heads, behind 27000 to 32768: 562 and 610.  The occupancy calculator says one CTA an
// SM for the small form, but two run.)
template <int D>
int launch_bf16(const PagedAttnArgs &p, int max_prefix, void *stream) {
  using C = PagedCfg<D, false>;
  auto kernel = tree_attn_paged_kernel<D, false>;
  static KernelState state;
  const int dev = current_device();
  if (dev < 0 || !allow_clusters(kernel, C::kSmem, dev, &state)) return SPEC_ERR_CUDA;
  CUtensorMap tmk, tmv;
  if (!encode_pool(&tmk, p.a.k, p.pages, p.a.Hkv, D) || !encode_pool(&tmv, p.a.v, p.pages, p.a.Hkv, D))
    return SPEC_ERR_CUDA;
  const long long blocks = most_blocks<kRows>(p.a), units = likely_blocks<kRows>(p.a) * p.a.Hkv;
  const long long keys = static_cast<long long>(max_prefix) + mean_nodes(p.a);
  const long long tiles = (keys + kTile - 1) / kTile;
  const long long mean_tiles = (keys - (p.causal ? mean_nodes(p.a) / 2 : 0) + kTile - 1) / kTile;
  const long long rows = static_cast<long long>(mean_nodes(p.a)) * p.a.G, merge = 2 + (rows < kRows ? rows : kRows) / 32;
  int cs = 1;
  long long best = -1;
  for (int n = 1; n <= kMaxSplits; n = n == 8 ? kMaxSplits : n + 1) {
    if (n > 1 && tiles < n) break;
    const int slots = clusters_at_once(kernel, n, C::kThreads, C::kSmem, dev, &state);
    if (slots < 1) continue;
    const long long waves = (units + slots - 1) / slots;
    const long long cost = waves * (2 * ((tiles + n - 1) / n) + 8 + (n > 1 ? merge : 0));
    if (best < 0 || cost < best) {
      best = cost;
      cs = n;
    }
  }
  if (blocks * cs > 0x7FFFFFFFll) return SPEC_ERR_SHAPE;
  using S = PagedCfg<D, true>;
  auto small_kernel = tree_attn_paged_kernel<D, true>;
  static KernelState small_state;
  const long long small_waves = (units + S::kCtas * sm_count() - 1) / (S::kCtas * sm_count());
  const bool small = small_waves * (D == 128 ? 9 * mean_tiles + 8 : 6 * mean_tiles + 14) < 2 * best;
  if (small) {
    if (!allow_dynamic_smem(small_kernel, S::kSmem, small_state.granted)) return SPEC_ERR_CUDA;
    cs = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cluster_config(cfg, attr, cs, small ? S::kThreads : C::kThreads, small ? S::kSmem : C::kSmem);
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * cs), static_cast<unsigned>(p.a.Hkv), 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, small ? small_kernel : kernel, p, tmk, tmv, cs) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

}  // namespace spec

extern "C" int spec_tree_attn_paged(const void *q, const void *k_pages, const void *v_pages, void *o, int dtype, int B,
                                    int T, int Hq, int Hkv, int D, int num_pages, int page_size,
                                    const int32_t *block_table, int max_pages, int max_prefix,
                                    const int32_t *prefix_lens, const int32_t *offsets, const uint32_t *mask,
                                    const int32_t *parents, int causal, float softmax_scale, int32_t *status,
                                    void *stream) {
  using namespace spec;
  if (((!q || !o) && T != 0) || !k_pages || !v_pages || !block_table || !prefix_lens || !offsets || !status ||
      (!causal && !mask && !parents))
    return SPEC_ERR_NULL;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  PagedAttnArgs p = {};
  const int rc = check_pages(num_pages, page_size, max_pages, &p.pages.shift);
  if (rc != SPEC_OK) return rc;
  if (causal && (mask || parents)) return SPEC_ERR_SHAPE;
  if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hkv > 65535 || Hq % Hkv || Hq / Hkv > SPEC_MAX_TREE_NODES ||
      (D != 64 && D != 128) || max_prefix < 0 || static_cast<long long>(T) * Hq > 0x7FFFFFFFll)
    return SPEC_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages) |
       reinterpret_cast<uintptr_t>(o) | reinterpret_cast<uintptr_t>(mask)) & 15)
    return SPEC_ERR_ALIGNMENT;
  if (T == 0) return SPEC_OK;
  AttnArgs &a = p.a;
  a.q = q;
  a.k = k_pages;
  a.v = v_pages;
  a.o = o;
  a.prefix_lens = prefix_lens;
  a.offsets = offsets;
  a.mask = reinterpret_cast<const uint4 *>(mask);
  a.parents = mask ? nullptr : parents;
  a.status = status;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.D = D;
  p.pages.table = block_table;
  p.pages.max_pages = max_pages;
  p.pages.pages = num_pages;
  p.pages.status = status;
  p.causal = causal != 0;
  const long long slots = static_cast<long long>(max_pages) << p.pages.shift;
  a.S_cap = static_cast<int>(slots < 0x7FFFFFFFll - 4096 ? slots : 0x7FFFFFFFll - 4096);
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf(static_cast<float>(D));
  a.scale_log2 = scale * 1.4426950408889634f;
  if (dtype == SPEC_F32) return launch_attn_paged_f32(p, max_prefix, stream);
  return D == 128 ? launch_bf16<128>(p, max_prefix, stream) : launch_bf16<64>(p, max_prefix, stream);
}
