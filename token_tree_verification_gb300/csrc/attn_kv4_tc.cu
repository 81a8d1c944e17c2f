// Tree attention over the 4-bit KV cache on the 5th-generation tensor cores,
// bf16 queries.
//
// Both products are taken transposed, so that the tile of 128 keys (or the D
// dims) fills the MMA's M = 128 whatever the number of rows, and the rows are
// its N:
//   S^T[keys][rows] = K Q^T    A = K   (keys x dims, in TMEM),        B = Q   (rows x dims)
//   O^T[dims][rows] = V^T P^T  A = V^T (dims x keys, shared memory),  B = P^T (rows x keys)
// With rows along M, a tree of 6 nodes would cost as much tensor time as one
// of 128; and a thread of the softmax now holds one key's weights of several
// rows, which lie next to one another in P^T.  The decoded keys and values
// are exact halves (kv4.cuh), so half-precision products lose nothing, and
// weights take 11 bits in one product.
//
// One CTA = one split of the keys x one block of N rows x one (request, KV
// head).  Warp roles:
//   warp 0      brings tiles of 128 records, one bulk copy each
//   warp 1      allocates TMEM and issues S^T_i as soon as tile i's keys
//               are decoded and the parity's S^T has been read
//   warp 2      issues O^T += V_i^T P_i^T
//   then        softmax: a key per TMEM lane, so four warps for the keys of a
//               tile; for more than 16 rows two such groups (half of the
//               rows each) for even tiles and two for odd ones, else one each.
//               The sums of weights stay in registers, one per row, until the end
//   then        decoders, four warps per operand (two such sets, which take
//               turns, for up to 16 rows): keys into TMEM, values into shared
//               memory (128-byte swizzle), one key per lane, so that a warp's
//               16-byte loads (records 36 words apart) and stores (rows 128
//               bytes apart, swizzled) are both free of bank conflicts.  Keys in
//               TMEM spare shared memory the decoded K twice, written and read
// A chain of eight MMAs takes about 850 cycles from issue to its barrier, a
// tile's two chains and its softmax about 3000, so what counts is how many
// tiles are under way: three decoded, two in the softmax.
//
// What bounds it, 32 rows, D = 128: about 1140 cycles a tile, of them 970 of
// shared-memory traffic (records in and out, V's operand in and out, P), issue
// slots 61% busy, the tensor pipe 15%.  8 requests x 32 heads behind 8192 keys:
// 32 rows 101 us, 16 rows 81 us (302 MB, 3.7 TB/s); with a window of 4096 behind
// 32768 61 us, in two waves of CTAs of which each spends about 10 us on its
// set-up, first tile and output.
#include <type_traits>

#include "attn_kv4_tc.cuh"

namespace spec {

namespace {

constexpr int kSoftFirst = 4;         // warps: four issuers, then the softmax, then the decoders
constexpr int kDecodeWarps = 4;       // of one set, for keys, and as many for values
constexpr int kTcThreads = 32 * 28;
// Registers: 28 warps launch with 72 a thread; sixteen softmax warps take 88
// (eight: 120), the decoders keep 56 and the issuers 40.
constexpr int kLaunchRegs = 72, kDecodeRegs = 56, kIssueRegs = 40;
constexpr int kOps = 3;               // decoded K tiles (TMEM), decoded V tiles (shared memory)

template <int D, int N>
struct Kv4Tc {
  // 32 rows: the softmax bounds, so two groups share a tile's rows; 16: the
  // decoding does, and two sets of decoders take turns.  (32 heads x 8 requests
  // behind 6759 to 8192: 16 rows 84 -> 76 us with two sets; 32 rows 92 us with two
  // softmax groups, 100 us with two sets.)
  static constexpr int kHalves = N == 16 ? 1 : 2;
  static constexpr int kSets = N == 16 ? 2 : 1;
  static constexpr int kSoftWarps = 8 * kHalves, kSoftThreads = 32 * kSoftWarps;
  static constexpr int kDecodeFirst = kSoftFirst + kSoftWarps;
  static constexpr int kSoftRegs = kHalves == 2 ? 88 : 120;
  static_assert(kDecodeFirst + 2 * kSets * kDecodeWarps == kTcThreads / 32, "warps");
  static_assert(kSoftWarps * kSoftRegs + 2 * kSets * kDecodeWarps * kDecodeRegs + kSoftFirst * kIssueRegs <=
                    kTcThreads / 32 * kLaunchRegs,
                "register split");
  static constexpr int R = kv4_record_bytes(D);
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTile * 128;             // 128 rows of 64 halves
  static constexpr int kOpBytes = kBoxes * kBoxBytes;       // a decoded V tile
  static constexpr int kQBoxBytes = N * 128;
  static constexpr int kQBytes = (kBoxes * kQBoxBytes + 1023) / 1024 * 1024;
  static constexpr int kPPitch = N * 2;                     // a key's weights: their own swizzle width
  static constexpr int kPBytes = kTile * kPPitch;
  static constexpr int kRawBytes = kTile * R;
  // Stages of records (32 rows: 4 take 61.0 us for the window below, 5 61.9; 16
  // rows: 75.4 and 73.5 us).  A set of decoders that skips the other's tiles must
  // not meet a stage whose last copy it cannot know to be over, or the phase that
  // it waits for would be taken for the one before the last: either the stage's
  // last tile was its own, or it was consumed when the set's last tile was written.
  static constexpr int kRaw = N == 16 ? 5 : 4;
  static_assert(kSets == 1 || kRaw % kSets == 0 || kRaw >= kOps + kSets, "stages of records");
  static constexpr int kOffV = 0;
  static constexpr int kOffP = kOffV + kOps * kOpBytes;
  static constexpr int kOffQ = kOffP + 2 * kPBytes;
  static constexpr int kOffRaw = kOffQ + kQBytes;
  static constexpr int kSmem = kOffRaw + kRaw * kRawBytes + 1024;
  static constexpr int kRowsPer = N / kHalves;              // rows of one softmax thread
  // TMEM: S^T and O^T of even and odd tiles, K tiles (a pair of dims per column)
  static constexpr uint32_t kColO = 2 * N;
  static constexpr uint32_t kColK = 4 * N;
  static constexpr uint32_t kColsUsed = kColK + kOps * (D / 2);
  static constexpr uint32_t kTmemCols = kColsUsed <= 128 ? 128 : kColsUsed <= 256 ? 256 : 512;
  // after the loop: the rows of both parities, then the ones received
  static constexpr int kOffRecv = 2 * N * (D + 4) * 4;
  static_assert(kOffRecv + (N * D + 4 * kMaxSplits) * 4 <= kSmem - 1024, "staged and received rows fit");
  static_assert(kColsUsed <= 512, "TMEM columns");
  static_assert(kSmem <= 227 * 1024 - 8192, "shared memory budget");
};

template <int D, int N>
__global__ void __launch_bounds__(kTcThreads, 1)
tree_attn_kv4_tc_kernel(const Kv4AttnArgs p) {
  using C = Kv4Tc<D, N>;
  constexpr int R = C::R, RP = C::kRowsPer, kRaw = C::kRaw, kSets = C::kSets;
  constexpr int kSoftWarps = C::kSoftWarps, kSoftThreads = C::kSoftThreads, kDecodeFirst = C::kDecodeFirst;
  const AttnArgs &a = p.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ struct {
    uint64_t raw_full[kRaw], raw_empty[kRaw];
    uint64_t k_full[kOps], k_empty[kOps], v_full[kOps], v_empty[kOps];
    uint64_t s_full[2], s_empty[2], p_full[2], o_done[2], q_full, drained[2];
  } bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_timeout;
  __shared__ int s_par[SPEC_MAX_TREE_NODES];
  __shared__ long long s_row[N];                       // a row's first element of o
  __shared__ uint4 s_tree[N];
  __shared__ uint32_t s_sees[SPEC_MAX_TREE_NODES];     // the rows that see a tree node, as bits
  __shared__ int s_first[N];
  __shared__ __align__(16) float s_c[N];               // a row's score factor
  // per parity of the tiles: 8 - the row's reference, the last move of it
  // (factor of the old sums, shift of the scores: infinite when the row starts
  // again), the reference, the sum of weights, and the parts of maxima and sums
  // that the four lane quarters hold
  __shared__ __align__(16) float s_n[2][N];
  __shared__ __align__(16) float2 s_move[2][N];
  __shared__ float s_ref[2][N], s_sum[2][N];
  __shared__ float s_part[2][4][N];
  __shared__ float2 s_ml[kMaxSplits][N];

  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
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
    for (int s = 0; s < kOps; ++s) {
      mbar_init(&bars.k_full[s], kDecodeWarps);
      mbar_init(&bars.v_full[s], kDecodeWarps);
      mbar_init(&bars.k_empty[s], 1);
      mbar_init(&bars.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
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

  const ReqGeom G = kv4_geometry(a, b);
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
    for (int row0 = static_cast<int>(blockIdx.y) * N; row0 < rows_total; row0 += static_cast<int>(gridDim.y) * N) {
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

  // (each group of four warps has one register budget)
  if (warp < kSoftFirst) {
    give_registers<kIssueRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- records
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
      // ---------------------------------------------------------- S^T = K Q^T
      constexpr uint32_t id = tc::idesc_f16_f32(128, N, 0, 0);
      const uint64_t qd0 = tc::smem_desc_sw128(sb + C::kOffQ, 16, 1024);
      const uint32_t k_full = smem_addr(bars.k_full);
      Ring<2> sr;
      Ring<kOps> kr;
      sr.phase = 1;
      const bool leader = tc::elect_one();
      uint32_t q_phase = 0;
      turns([&](int) {
        if (ntiles == 0) return;
        ok = mbar_sleep(smem_addr(&bars.q_full), q_phase);
        q_phase ^= 1;
        for (int i = 0; i < ntiles; ++i, sr.next(), kr.next()) {
          ok = ok && mbar_sleep(s_empty + 8 * sr.at, sr.phase) && mbar_sleep(k_full + 8 * kr.at, kr.phase);
          tc::fence_after_sync();
          const uint32_t kt = tmem + C::kColK + kr.at * (D / 2);
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t qa = ((ks >> 2) * C::kQBoxBytes + (ks & 3) * 32) >> 4;
              tc::mma_bf16_ts(tmem + sr.at * N, kt + ks * 8, qd0 + qa, id, ks > 0);
            }
            tc::commit(&bars.s_full[sr.at]);
            tc::commit(&bars.k_empty[kr.at]);
          }
          __syncwarp();
        }
      }, wait_merge);
    } else if (warp == 2) {
      // ---------------------------------------------------------- O^T += V^T P^T
      constexpr uint32_t id = tc::idesc_f16_f32(128, N, 1, 1);
      // D = 64: both halves of M read the same 64 dims
      const uint64_t vd0 = tc::smem_desc_sw128(sb + C::kOffV, D == 128 ? C::kBoxBytes : 0, 1024);
      const uint64_t pd0 = tc::smem_desc_mn<N>(sb + C::kOffP);
      const uint32_t v_full = smem_addr(bars.v_full);
      Ring<2> pr;
      Ring<kOps> vr;
      const bool leader = tc::elect_one();
      turns([&](int) {
        for (int i = 0; i < ntiles; ++i, pr.next(), vr.next()) {
          ok = ok && mbar_sleep(v_full + 8 * vr.at, vr.phase) && mbar_sleep(p_full + 8 * pr.at, pr.phase);
          tc::fence_after_sync();
          const uint64_t vd = vd0 + static_cast<uint64_t>(vr.at * C::kOpBytes >> 4);
          const uint64_t pd = pd0 + static_cast<uint64_t>(pr.at * C::kPBytes >> 4);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              tc::mma_bf16(tmem + C::kColO + pr.at * N, vd + (kk * 16 * 128 >> 4), pd + (kk * 16 * C::kPPitch >> 4),
                           id, i > 1 || kk != 0);
            tc::commit(&bars.o_done[pr.at]);
            tc::commit(&bars.v_empty[vr.at]);
          }
          __syncwarp();
        }
      }, wait_merge);
    } else {
      turns([](int) {}, wait_merge);
    }
  } else if (warp >= kDecodeFirst) {
    // ------------------------------------------------------------ decode
    give_registers<kDecodeRegs>();
    const int set = ((warp - kDecodeFirst) / kDecodeWarps) % kSets;
    auto decode = [&](auto of_v) {
      constexpr bool kV = decltype(of_v)::value;
      const int key = (warp & 3) * 32 + lane;               // and the warp's TMEM lanes
      const uint32_t full = smem_addr(kV ? bars.v_full : bars.k_full);
      const uint32_t empty = smem_addr(kV ? bars.v_empty : bars.k_empty);
      const uint8_t *rec0 = smem + C::kOffRaw + key * R;
      // V: 16-byte pieces of the key's row, piece j of a box at j ^ (key % 8);
      // K: the key's TMEM lane, 8 columns per 16 dims
      const uint32_t row = sb + C::kOffV + key * 128 + ((key & 7) << 4);
      const uint32_t col = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kColK;
      const LiveKeys live(G.L, G.keys, p.window, p.sinks);
      Ring<kRaw> raw;
      Ring<kOps> op;
      op.phase = 1;
      int turn_of = 0;           // the set whose tile the rings are at
      turns([&](int) {
        for (int i = 0; i < ntiles; ++i, raw.next(), op.next(), turn_of ^= kSets - 1) {
          if (turn_of != set) continue;
          ok = ok && mbar_sleep(raw_full + 8 * raw.at, raw.phase);
          const KeyCodes<D> key_codes(rec0 + raw.at * C::kRawBytes, kV, live(tiles.key0(t0 + i) + key));
          ok = ok && mbar_sleep(empty + 8 * op.at, op.phase);
          if constexpr (!kV) {
            __syncwarp();
            tc::fence_after_sync();
          }
          const uint32_t dst = row + op.at * C::kOpBytes, dcol = col + op.at * (D / 2);
          key_codes.decode([&](int g, const uint32_t(&h)[8]) {
            if constexpr (kV) put_swizzled<C::kBoxBytes>(dst, g, h);
            else tc::st8(dcol + 8 * g, h);
          });
          if constexpr (kV) {
            fence_proxy_async_smem();
          } else {
            tc::wait_st();
            tc::fence_before_sync();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_at(full + 8 * op.at);
            mbar_arrive_at(raw_empty + 8 * raw.at);
          }
        }
      }, wait_merge);
    };
    if (warp >= kDecodeFirst + kSets * kDecodeWarps) decode(std::true_type{});
    else decode(std::false_type{});
  } else {
    // ------------------------------------------------------------ softmax
    // Groups of four warps: one or two (each with half of the rows) for even
    // tiles and as many for odd ones, so that the chain S^T, weights, product of
    // one tile runs beside that of the next.  The parities keep references,
    // sums and O^T of their own, merged at the end like splits of the keys.
    take_registers<C::kSoftRegs>();
    const int w = warp - kSoftFirst, quad = warp & 3, half = (w >> 2) % C::kHalves, par = w / (4 * C::kHalves);
    const int soft = tid - 32 * kSoftFirst;            // 0 .. kSoftThreads - 1
    const int r0 = half * RP, group = 2 + (w >> 2);    // first row; named barrier of the group
    const int key_lane = quad * 32 + lane;             // key of a tile, and TMEM lane
    // this key's row of P, swizzled over its 64 or 32 bytes
    const int swz = N == 32 ? (key_lane >> 1) & 3 : (key_lane >> 2) & 1;
    const uint32_t prow =
        sb + C::kOffP + par * C::kPBytes + key_lane * C::kPPitch + (((half * (RP / 8)) ^ swz) << 4);
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_col = trow + par * N + r0, o_col = trow + C::kColO + par * N + r0;
    uint32_t phase = 0;        // of this parity's S^T; flips with every tile of it
    int numbered = 0;          // tiles of earlier turns
    turns([&](int row0) {
      const int rows_here = min(N, rows_total - row0);
      // ---- Q as halves: 8 dims of a row per thread and round; every load of
      //      the set-up is under way before the first is used
      constexpr int kPieces = D / 8, kRounds = (N * kPieces + kSoftThreads - 1) / kSoftThreads;
      uint4 x4[kRounds], m = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int rr = 0; rr < kRounds; ++rr) {
        const int idx = rr * kSoftThreads + soft, r = idx / kPieces, c = idx % kPieces;
        x4[rr] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows_here && in_bounds(G.lo + (row0 + r) / a.G, a.T, a.status, b))
          x4[rr] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                         (static_cast<size_t>(G.lo + (row0 + r) / a.G) * a.Hq +
                                                          g_kv * a.G + (row0 + r) % a.G) *
                                                             D) +
                         c);
      }
      const int node = (row0 + soft) / a.G;
      if (a.mask) {
        if (soft < rows_here && in_bounds(G.lo + node, a.T, a.status, b)) m = __ldg(a.mask + G.lo + node);
      } else if (row0 == static_cast<int>(blockIdx.y) * N) {
        for (int i = soft; i < G.n; i += kSoftThreads)
          s_par[i] = in_bounds(G.lo + i, a.T, a.status, b) ? __ldg(a.parents + G.lo + i) : -2;
      }
#pragma unroll
      for (int rr = 0; rr < kRounds; ++rr) {
        const int idx = rr * kSoftThreads + soft, r = idx / kPieces, c = idx % kPieces;
        if (r >= N) break;       // whole warps
        const uint32_t u[4] = {x4[rr].x, x4[rr].y, x4[rr].z, x4[rr].w};
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xFFFF0000u))));
#pragma unroll
        for (int k = 1; k < kPieces; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const int up = row_exponent(top);
        const float grow = power_of_two(up);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = pack_half2(__uint_as_float(u[e] << 16) * grow, __uint_as_float(u[e] & 0xFFFF0000u) * grow);
        st_shared_v4(sb + C::kOffQ + (c >> 3) * C::kQBoxBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4), h[0], h[1], h[2],
                     h[3]);
        if (c == 0) {
          const int node_r = (row0 + r) / a.G;
          s_c[r] = a.scale_log2 * power_of_two(-up);
          s_row[r] = r < rows_here && in_bounds(G.lo + node_r, a.T, a.status, b)
                         ? (static_cast<long long>(G.lo + node_r) * a.Hq + g_kv * a.G + (row0 + r) - node_r * a.G) * D
                         : -1;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(smem_addr(&bars.q_full));
      // ---- what each row sees
      if (!a.mask) named_bar_sync(1, kSoftThreads);      // the parents
      if (soft < N) {
        if (a.mask) {
          m = clip_mask(m, G.n);
        } else if (soft < rows_here) {
          bool bad = false;
          m = ancestor_mask([&](int i) { return s_par[i]; }, node, &bad);
          if (bad) report(a.status, b, SPEC_ERR_BAD_PARENT);
        }
        const RowKeys see = row_keys(m, G.L, p.window, p.sinks);
        s_tree[soft] = see.tree;
        s_first[soft] = see.first;
        for (int q = 0; q < 2; ++q) {
          s_n[q][soft] = kWeightLog2;
          s_ref[q][soft] = soft < rows_here ? -INFINITY : 0.f;    // rows of no node need no reference
        }
      }
      named_bar_sync(1, kSoftThreads);
      // the rows' sets turned round, a word of rows for every node
      for (int u = w; u < G.n; u += kSoftWarps) {
        const uint32_t *tree = reinterpret_cast<const uint32_t *>(&s_tree[lane % N]);
        const bool sees = lane < N && ((tree[u >> 5] >> (u & 31)) & 1u);
        const uint32_t rows = __ballot_sync(0xffffffffu, sees);
        if (lane == 0) s_sees[u] = rows;
      }
      named_bar_sync(1, kSoftThreads);

      float sum[RP];
#pragma unroll
      for (int j = 0; j < RP; ++j) sum[j] = 0.f;
      bool unset = true;        // a row of this group has no reference yet
      const int first = (par ^ numbered) & 1;
      for (int i = first; i < ntiles; i += 2, phase ^= 1) {
        const int key0 = tiles.key0(t0 + i);
        ok = ok && mbar_sleep(s_full + 8 * par, phase);
        __syncwarp();
        tc::fence_after_sync();
        float x[RP];
        tc::ld16(s_col, x);
        tc::wait_ld();
        // x = score - reference + 8, in powers of two
#pragma unroll
        for (int j = 0; j < RP; j += 4) {
          const float4 c = *reinterpret_cast<const float4 *>(&s_c[r0 + j]);
          const float4 m = *reinterpret_cast<const float4 *>(&s_n[par][r0 + j]);
          fma2(x[j], x[j + 1], c.x, c.y, m.x, m.y);
          fma2(x[j + 2], x[j + 3], c.z, c.w, m.z, m.w);
        }
        const bool whole = key0 + kTile <= G.L &&
                           (p.window == 0 || key0 + kTile <= p.sinks || key0 >= G.L + G.n - p.window);
        if (!whole) {
          const int key = key0 + key_lane, up = key - G.L;       // node of a tree key
          uint32_t sees = 0u;                                    // rows of this thread that see the key
          if (up >= 0) {
            if (key < G.keys) sees = s_sees[up] >> r0;
          } else if (p.window == 0 || key < p.sinks) {
            sees = ~0u;
          } else {
#pragma unroll
            for (int j = 0; j < RP; ++j) sees |= key >= s_first[r0 + j] ? 1u << j : 0u;
          }
#pragma unroll
          for (int j = 0; j < RP; ++j)
            if (!((sees >> j) & 1u)) x[j] = -INFINITY;
        }
        const float most = max_of(x);
        if (named_bar_or(group, 128, unset || most > kWeightLog2 + kMoveLog2)) {
          // some reference moves (or is not there yet): the rows' maxima over
          // the tile's keys, new references, and what has been summed so far
          // brought to them
          const float mx = reduce_scatter(x, lane, [](float u, float v) { return fmaxf(u, v); });
          if (lane < RP) s_part[par][quad][r0 + lane] = mx;
          named_bar_sync(group, 128);
          bool still = false;
          if (key_lane < RP) {                 // a thread of the group for each of its rows
            const int r = r0 + key_lane;
            const float m = fmaxf(fmaxf(s_part[par][0][r], s_part[par][1][r]),
                                  fmaxf(s_part[par][2][r], s_part[par][3][r]));
            const float ref = s_ref[par][r];
            const bool fresh = ref == -INFINITY;
            float2 move = make_float2(1.f, 0.f);
            if (far_above(m, s_n[par][r], fresh)) {
              move = make_float2(0.f, INFINITY);
              s_ref[par][r] = -INFINITY;
              s_n[par][r] = kWeightLog2;
            } else if (m > (fresh ? -INFINITY : kWeightLog2 + kMoveLog2)) {
              const float by = reference_step(m);
              move = make_float2(fresh ? 0.f : exp2f(-by), -by);
              s_n[par][r] -= by;
              s_ref[par][r] = kWeightLog2 - s_n[par][r];
            }
            still = s_ref[par][r] == -INFINITY;
            s_move[par][r] = move;
          }
          unset = named_bar_or(group, 128, still);
          if (i > 1) {
            // O^T holds the products of this turn's earlier tiles of the parity
            ok = ok && mbar_sleep(o_done + 8 * par, phase ^ 1);
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll
            for (int j = 0; j < RP; j += 8) {
              float o[8];
              tc::ld8(o_col + j, o);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] *= s_move[par][r0 + j + e].x;
              tmem_st(o_col + j, o);
            }
            tc::wait_st();
          }
          bool again = false;
#pragma unroll
          for (int j = 0; j < RP; ++j) {
            const float2 move = s_move[par][r0 + j];
            sum[j] *= move.x;
            x[j] += move.y;
            again |= move.y == INFINITY;
          }
          if (again) {           // (the same in the whole group)
            i -= 2;
            phase ^= 1;
            continue;
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(s_empty + 8 * par);
        // ---- weights; P's buffer is free once the parity's last product is done
        const bool room = mbar_over(o_done + 8 * par, phase ^ 1);
#pragma unroll
        for (int j = 0; j < RP; ++j) x[j] = fast_exp2(x[j]);
#pragma unroll
        for (int j = 0; j < RP; j += 2) add2(sum[j], sum[j + 1], x[j], x[j + 1]);
        ok = ok && (room || mbar_sleep(o_done + 8 * par, phase ^ 1));
#pragma unroll
        for (int c = 0; c < RP / 8; ++c)
          st_shared_v4(prow ^ (c << 4), pack_half2(x[8 * c], x[8 * c + 1]), pack_half2(x[8 * c + 2], x[8 * c + 3]),
                       pack_half2(x[8 * c + 4], x[8 * c + 5]), pack_half2(x[8 * c + 6], x[8 * c + 7]));
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(p_full + 8 * par);
      }
      numbered += ntiles;
      // ---- the block's rows out of TMEM.  Their place in shared memory is free
      //      once the last products of both parities are done; a thread whose
      //      waits ran out writes nothing.
      ok = ok && mbar_sleep(o_done + 8 * par, phase ^ 1);
      if (CS > 1) cluster_arrive_relaxed();
      __syncwarp();
      tc::fence_after_sync();
      const float l = reduce_scatter(sum, lane, [](float u, float v) { return u + v; });
      if (lane < RP) s_part[par][quad][r0 + lane] = l;
      if (!ok) s_timeout = 1;
      named_bar_sync(1, kSoftThreads);
      if (s_timeout == 0) {
        const bool any = first < ntiles;
        if (key_lane < RP) {
          const int r = r0 + key_lane;
          s_sum[par][r] = (s_part[par][0][r] + s_part[par][1][r]) + (s_part[par][2][r] + s_part[par][3][r]);
          if (!any) s_ref[par][r] = -INFINITY;
        }
        float *so = reinterpret_cast<float *>(smem) + (par * N + r0) * (D + 4) + key_lane;
#pragma unroll
        for (int j = 0; j < RP; j += 8) {
          float o[8] = {};
          if (any) {
            tc::ld8(o_col + j, o);
            tc::wait_ld();
          }
          if (D == 128 || key_lane < D) {
#pragma unroll
            for (int e = 0; e < 8; ++e) so[(j + e) * (D + 4)] = o[e];
          }
        }
      }
    }, [&](int row0) {
      const bool timed_out = s_timeout != 0;
      if (timed_out && soft == 0) report(a.status, b, SPEC_ERR_TIMEOUT);
      auto out_row = [&](int r) { return s_row[r] < 0 ? nullptr : static_cast<__nv_bfloat16 *>(a.o) + s_row[r]; };
      return merge_rows<D, 2, N, kSoftThreads, __nv_bfloat16>(
          soft, CS, split, min(N, rows_total - row0), timed_out, reinterpret_cast<float *>(smem), s_ref, s_sum, s_ml,
          reinterpret_cast<float4 *>(smem + C::kOffRecv), [] { cluster_wait(); }, out_row);
    });
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

template <int D, int N>
int launch_tc(const Kv4AttnArgs &p, int max_prefix, void *stream) {
  static KernelState state;
  const int blocks = (mean_nodes(p.a) * p.a.G + N - 1) / N;
  return launch_kv4_tiles(tree_attn_kv4_tc_kernel<D, N>, p, kTcThreads, kLaunchRegs, Kv4Tc<D, N>::kSmem, blocks,
                          max_prefix, &state, stream);
}

template <int D>
int by_rows(const Kv4AttnArgs &p, int max_prefix, void *stream) {
  const int rows = mean_nodes(p.a) * p.a.G;
  return rows <= 16 ? launch_tc<D, 16>(p, max_prefix, stream) : launch_tc<D, 32>(p, max_prefix, stream);
}

}  // namespace

int launch_kv4_tc(const Kv4AttnArgs &p, int max_prefix, void *stream) {
  return p.a.D == 128 ? by_rows<128>(p, max_prefix, stream) : by_rows<64>(p, max_prefix, stream);
}

}  // namespace spec
