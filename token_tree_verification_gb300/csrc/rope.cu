// Rotary positions, on dense rows and on the way into a paged cache.
//
// Pair i of a head's first r dims, (i, i + r/2) or (2i, 2i + 1), is turned by the
// angle p theta_i of the row's position p:
//   y_a = s (x_a cos - x_b sin),  y_b = s (x_a sin + x_b cos)
// theta_i = base^(-2i/r), scaled for contexts longer than the model's (see
// spec_rope_table); the other D - r dims stay as they are.
//
// Angles.  At position 2^20 an fp32 product p theta is off by up to 2^-5
// radians, and fp64 arithmetic is slow here.  The table holds theta / 2 pi, the
// turns a position, as a 64-bit fraction rounded to its last place: p times it,
// modulo 2^64, is the angle's fraction of a turn, off by at most p 2^-65 turns.
// Its upper 32 bits (the others, 2^-32 turns, are cut) go to sincospif as a
// number of half turns in [-1, 1), which rounds to 2^-25.
//
// A thread has one item of a row, two vectors of 16 bytes (fewer where alignment or the
// pairs' ends ask for it): both ends of eight (four, fp32) pairs, or two vectors of dims
// that are copied; it keeps it along a run of
// rows, so that what an item is (head, place, source, destination) is worked out
// once, and rows differ by a stride, a slot and the angles, which one CTA computes
// once for all heads.  (With an item worked out for every row and head the
// instructions bound it: 112 us where this takes 102.)  The first rows' loads need
// no look-up and are issued in front of them: offsets, start and depth, page are a
// chain of three loads.
//
// Memory bounds long runs: 51200 rows of 40 heads, D = 128, 1.05 GB in 162 us, 6.5
// TB/s, 0.95 of a copy's rate; 14237 rows of 80 heads into pages of 64 slots, 583 MB
// in 103 us, 5.7 TB/s; single tokens of 4096 requests, 48 heads, 101 MB in 24 us, 4.1
// TB/s.  fp32: 25600 rows of 40 heads, 1.05 GB in 160 us; 14237 of 80 into pages, 1.17
// GB in 184.  A few tokens (2.9 us) and a 64-node tree of 96 heads (3.6 us) are the chain
// of loads.
#include <cuda_bf16.h>

#include <cmath>

#include "paged.cuh"

namespace spec {

namespace {

constexpr int kMaxThreads = 192;
constexpr int kMaxRows = 32;                 // of a CTA
constexpr int kLong = 2;                     // rows of a thread whose loads are under way, along a run
constexpr int kRun = 8;                      // rows of a run
constexpr int kAngleBytes = 32 * 1024;

struct Rows {
  const void *x;
  long long st, sh;       // element strides of a row and of a head
};

struct RopeArgs {
  Rows q, k, v;                      // v.x: null without a cache
  void *y;                           // rotated q
  long long y_st, y_sh;
  void *k_pages, *v_pages;
  PageTable pages;
  const unsigned long long *freqs;   // [r / 2] turns a position, times 2^64
  float scale;
  const int32_t *slots, *start, *depth, *offsets;   // slots: prefix lengths (cache)
  int32_t *status;
  int B, T, Hq, Hkv, D, r;
  int turn_items, copy_items;        // of a rotated and of a copied head
  int row_items, span;               // of a row, and of a row in one CTA
  int rows, side;                    // of a CTA, and how many side by side
};

// V elements as one load, of 16, 8 or 4 bytes; V = 1: a single element.
template <typename E, int V>
struct Vec {
  using Load = E;
};
template <int V>
struct Words {
  uint32_t w[V];
};
template <int V>
struct BfVec {
  using Load = typename std::conditional<V == 8, uint4, typename std::conditional<V == 4, uint2, uint32_t>::type>::type;
  static __device__ __forceinline__ void unpack(Load v, float (&f)[V]) {
    const Words<V / 2> u = *reinterpret_cast<const Words<V / 2> *>(&v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(u.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(u.w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ Load pack(const float (&f)[V]) {
    Words<V / 2> u;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u.w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return *reinterpret_cast<const Load *>(&u);
  }
};
template <>
struct Vec<__nv_bfloat16, 8> : BfVec<8> {};
template <>
struct Vec<__nv_bfloat16, 4> : BfVec<4> {};
template <>
struct Vec<__nv_bfloat16, 2> : BfVec<2> {};
template <int V>
struct FloatVec {
  using Load = typename std::conditional<V == 4, uint4, uint2>::type;
  static __device__ __forceinline__ void unpack(Load v, float (&f)[V]) {
    const Words<V> u = *reinterpret_cast<const Words<V> *>(&v);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __uint_as_float(u.w[i]);
  }
  static __device__ __forceinline__ Load pack(const float (&f)[V]) {
    Words<V> u;
#pragma unroll
    for (int i = 0; i < V; ++i) u.w[i] = __float_as_uint(f[i]);
    return *reinterpret_cast<const Load *>(&u);
  }
};
template <>
struct Vec<float, 4> : FloatVec<4> {};
template <>
struct Vec<float, 2> : FloatVec<2> {};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float x, float *y) { *y = x; }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16 *y) { *y = __float2bfloat16_rn(x); }

// (x_a, x_b) turned, in fp32; which product is rounded is said, so that every form
// gives the same bits.
__device__ __forceinline__ void turn(float &xa, float &xb, float2 cs) {
  const float a = __fmaf_rn(xa, cs.x, -__fmul_rn(xb, cs.y)), b = __fmaf_rn(xa, cs.y, __fmul_rn(xb, cs.x));
  xa = a;
  xb = b;
}

// One unit of a thread's work: where its elements lie in a head, and whether
// they are turned.  Vectors (V > 1): two of them at pa and pb (pb < 0: one).  Else
// single elements: the two of a pair, or one that is copied.
struct Item {
  int head, pa, pb;           // head: q's, then k's, then v's
  bool turn_a, turn_b;
  int pair;                   // first pair of pa's cosines
};

template <int V, bool kInter>
__device__ __forceinline__ Item item_at(const RopeArgs &a, int i) {
  Item it;
  constexpr bool kVec = V > 1;
  const int turned = (a.Hq + a.Hkv) * a.turn_items;
  it.turn_a = it.turn_b = false;
  it.pair = 0;
  it.pb = -1;
  if (i >= turned) {
    i -= turned;
    const int h = i / a.copy_items, j = i - h * a.copy_items;
    it.head = a.Hq + a.Hkv + h;
    it.pa = j * V;
    if (kVec && j + a.copy_items < a.D / V) it.pb = (j + a.copy_items) * V;
    return it;
  }
  it.head = i / a.turn_items;
  const int j = i - it.head * a.turn_items;
  if constexpr (kVec && kInter) {
    it.pa = j * V;
    it.turn_a = it.pa < a.r;
    it.pair = it.pa / 2;
    if (j + a.turn_items < a.D / V) it.pb = (j + a.turn_items) * V;
    it.turn_b = it.pb >= 0 && it.pb < a.r;
  } else {
    const int half = a.r / 2 / V;
    if (j < half) {
      it.turn_a = it.turn_b = true;
      it.pair = j * V;
      it.pa = kInter ? 2 * j : j * V;
      it.pb = kInter ? 2 * j + 1 : a.r / 2 + j * V;
    } else if (kVec) {
      it.pa = a.r + 2 * (j - half) * V;
      if (it.pa + V < a.D) it.pb = it.pa + V;
    } else {
      it.pa = a.r + j - half;
    }
  }
  return it;
}

template <typename E, int V, bool kInter, int kAhead>
__global__ void __launch_bounds__(kMaxThreads, kAhead == 1 ? 1 : 6)
rope_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) float s_angle[];     // [rows][cosines, sines][r / 2]
  __shared__ int s_ok[kMaxRows], s_pos[kMaxRows];      // request + 1 (0: not to be written), position
  __shared__ long long s_slot[kMaxRows];               // first element of the slot's head 0 in the pools
  const int tid = threadIdx.x, threads = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = static_cast<int>(blockIdx.x) * a.rows;
  const int rows = min(a.rows, a.T - t0), pairs = a.r / 2;
  using Load = typename Vec<E, V>::Load;
  pdl_trigger();
  pdl_wait();

  // ---- this thread's item, and the first of its rows
  const int sub = tid / a.span, i = static_cast<int>(blockIdx.y) * a.span + tid - sub * a.span;
  const bool busy = sub < a.side && i < a.row_items;
  const Item it = item_at<V, kInter>(a, busy ? i : 0);
  const bool is_q = it.head < a.Hq, is_k = !is_q && it.head < a.Hq + a.Hkv;
  const int head = is_q ? it.head : it.head - a.Hq - (is_k ? 0 : a.Hkv);
  const long long x_st = is_q ? a.q.st : is_k ? a.k.st : a.v.st;
  const E *x = static_cast<const E *>(is_q ? a.q.x : is_k ? a.k.x : a.v.x) +
               head * (is_q ? a.q.sh : is_k ? a.k.sh : a.v.sh) + it.pa + t0 * x_st;
  const int to_b = it.pb - it.pa;
  const bool two = it.pb >= 0;
  Load la[kAhead], lb[kAhead];
  auto load = [&](int u, int row) {
    if (!busy || row >= rows) return;
    la[u] = *reinterpret_cast<const Load *>(x + row * x_st);
    if (two) lb[u] = *reinterpret_cast<const Load *>(x + row * x_st + to_b);
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, sub + u * a.side);

  // ---- each row's request, position and slot, by a warp
  bool none = false;      // no row is to be written
  for (int row = warp; row < rows; row += threads / 32) {
    const int t = t0 + row;
    const int b = warp_find_request(a.offsets, a.B, t, lane);
    bool ok = b >= 0 && in_bounds(b, a.B, a.status, 0);
    long long slot_at = 0;
    int position = 0, depth = 0;
    if (ok) {
      const RowRange R = row_range(a.offsets, b, a.T);
      const int start = __ldg(a.start + b);
      depth = a.depth ? __ldg(a.depth + t) : t - R.lo;
      ok = !R.err && t >= R.lo && start >= 0;
      position = static_cast<int>(static_cast<unsigned>(start) + static_cast<unsigned>(depth));
      if (ok && a.v.x) {
        const int L = __ldg(a.slots + b);
        ok = L >= 0 && static_cast<long long>(L) + R.n <= a.pages.capacity();
        if (ok) {
          const int slot = L + t - R.lo;
          const int page = a.pages.page(b, slot >> a.pages.shift);
          // rows that are all of one request share its pages out (65536 rows of 12 heads
          // into pages of 8: 147 us; with all of them looked at for every row 247)
          const bool alone = R.lo <= t0 && R.lo + R.n >= t0 + rows;
          if (warp_finds_bad_page(a.pages, b, L, L + R.n, lane, alone ? row : 0, alone ? rows : 1) || page < 0) {
            if (lane == 0) report(a.status, b, SPEC_ERR_PAGE);
            ok = false;
            none |= alone;
          }
          const int size = 1 << a.pages.shift;
          slot_at = ((static_cast<long long>(page) * a.Hkv << a.pages.shift) + (slot & (size - 1))) * a.D;
        }
      }
    }
    if (ok && depth < 0) {
      if (lane == 0) report(a.status, b, SPEC_ERR_PREFIX_RANGE);
      ok = false;
    }
    if (lane == 0) {
      s_ok[row] = ok ? b + 1 : 0;
      s_pos[row] = position;
      s_slot[row] = slot_at;
    }
  }
  // (whole batches are checked once, so that a request without rows here reports too)
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int b = tid; b < a.B; b += threads) {
      const RowRange R = row_range(a.offsets, b, a.T);
      int err = R.err;
      if (!err && __ldg(a.start + b) < 0) err = SPEC_ERR_PREFIX_RANGE;
      if (!err && a.v.x) {
        const int L = __ldg(a.slots + b);
        if (L < 0 || static_cast<long long>(L) + R.n > a.pages.capacity()) err = SPEC_ERR_PREFIX_RANGE;
      }
      if (err) report(a.status, b, err);
    }
  }
  if (__syncthreads_or(none)) return;
  for (int p = tid; p < rows * pairs; p += threads) {
    const int row = p / pairs, at = p - row * pairs;
    const unsigned long long turns =
        static_cast<unsigned long long>(static_cast<unsigned>(s_pos[row])) * __ldg(a.freqs + at);
    const float half_turns = static_cast<float>(static_cast<int>(turns >> 32)) * 4.656612873077393e-10f;   // 2^-31
    float s, c;
    sincospif(half_turns, &s, &c);
    s_angle[row * a.r + at] = c * a.scale;
    s_angle[row * a.r + pairs + at] = s * a.scale;
  }
  __syncthreads();
  if (!busy) return;

  E *y = static_cast<E *>(is_q ? a.y : is_k ? a.k_pages : a.v_pages) + it.pa +
         (is_q ? head * a.y_sh + t0 * a.y_st : (static_cast<long long>(head) << a.pages.shift) * a.D);
  auto store = [&](int u, int row) {
    if (!s_ok[row]) return;
    const float *cosine = s_angle + row * a.r + it.pair, *sine = cosine + pairs;
    if constexpr (V > 1) {
      if constexpr (kInter) {
        auto turn_vec = [&](Load &x, int from) {
          float f[V];
          Vec<E, V>::unpack(x, f);
#pragma unroll
          for (int e = 0; e < V; e += 2) turn(f[e], f[e + 1], make_float2(cosine[from + e / 2], sine[from + e / 2]));
          x = Vec<E, V>::pack(f);
        };
        if (it.turn_a) turn_vec(la[u], 0);
        if (it.turn_b) turn_vec(lb[u], to_b / 2);
      } else if (it.turn_a) {
        float fa[V], fb[V];
        Vec<E, V>::unpack(la[u], fa);
        Vec<E, V>::unpack(lb[u], fb);
        // (pairs in multiples of V: whole vectors of angles)
        using Angles = typename std::conditional<V == 2, float2, float4>::type;
        constexpr int kStep = V == 2 ? 2 : 4;
        float c[V], s[V];
#pragma unroll
        for (int e = 0; e < V; e += kStep) {
          *reinterpret_cast<Angles *>(c + e) = *reinterpret_cast<const Angles *>(cosine + e);
          *reinterpret_cast<Angles *>(s + e) = *reinterpret_cast<const Angles *>(sine + e);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) turn(fa[e], fb[e], make_float2(c[e], s[e]));
        la[u] = Vec<E, V>::pack(fa);
        lb[u] = Vec<E, V>::pack(fb);
      }
    } else if (it.turn_a) {
      float fa = to_float(la[u]), fb = to_float(lb[u]);
      turn(fa, fb, make_float2(*cosine, *sine));
      from_float(fa, &la[u]);
      from_float(fb, &lb[u]);
    }
    if (kChecked && !is_q &&
        !a.pages.holds((s_slot[row] + (static_cast<long long>(head) << a.pages.shift) * a.D) / a.D, 1, a.Hkv, s_ok[row] - 1))
      return;
    E *dst = y + (is_q ? row * a.y_st : s_slot[row]);
    *reinterpret_cast<Load *>(dst) = la[u];
    if (two) *reinterpret_cast<Load *>(dst + to_b) = lb[u];
  };
  for (int row0 = sub; row0 < rows; row0 += kAhead * a.side) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int row = row0 + u * a.side;
      if (row >= rows) break;
      store(u, row);
      load(u, row + kAhead * a.side);
    }
  }
}

// An item a thread, a row's items in as few CTAs as take them in kMaxThreads, or
// several rows side by side where a row has few; and rows in a run up to kRun (32 in
// all) while that leaves sixteen CTAs an SM.  Device us for the 51200 rows, the 14237,
// the 4096 above (in L2 here) and a run of 8192 rows of 48 heads:
//   192 threads, 2 rows ahead of the stores, runs of 8 and 6: 162, 102, 21, 36
//   runs of 16 and 4: 169, 111, 21, 36 and 164, 103, 21, 38
//   192 threads, 3 rows ahead: 165, 105, 22, 38
//   256 threads, 2 ahead: 168, 106, 22, 37; 320 threads, 2 ahead: 167, 100, 22, 37
//   384 threads, 4 ahead: 165, 101, 50, 43 (its registers spill, or do not, at a touch)
// A single row a thread takes no registers for a run: 3.6 in place of 4.4 us for the
// tree.
template <typename E, int V, bool kInter>
int launch(RopeArgs &a, void *stream) {
  constexpr bool kVec = V > 1;
  const int vecs = a.D / V;
  a.copy_items = kVec ? (vecs + 1) / 2 : vecs;
  a.turn_items = kVec ? (kInter ? (vecs + 1) / 2 : a.r / 2 / V + ((a.D - a.r) / V + 1) / 2) : a.r / 2 + a.D - a.r;
  const long long items = static_cast<long long>(a.Hq + a.Hkv) * a.turn_items +
                          (a.v.x ? static_cast<long long>(a.Hkv) * a.copy_items : 0);
  if (items > 0xFFFFll * kMaxThreads) return SPEC_ERR_SHAPE;      // (the grid's second dimension)
  a.row_items = static_cast<int>(items);
  const int parts = (a.row_items + kMaxThreads - 1) / kMaxThreads;
  a.span = (a.row_items + parts - 1) / parts;
  a.side = 1;
  if (a.span > 32) a.span = (a.span + 31) / 32 * 32;
  const long long runs = static_cast<long long>(a.T) * parts / (16ll * sm_count());
  int most = kRun;
  if (a.span < 128) {
    a.side = 128 / a.span < a.T ? 128 / a.span : a.T;
    if (a.side > 16) a.side = 16;
    most = kRun * a.side < kMaxRows ? kRun * a.side : kMaxRows;
  }
  a.rows = runs < a.side ? a.side : runs < most ? static_cast<int>(runs) : most;
  if (a.rows > a.side) a.rows -= a.rows % a.side;
  while (a.rows > 1 && a.rows * a.r * 4 > kAngleBytes) a.rows = a.rows / 2;
  if (a.side > a.rows) a.side = a.rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.T + a.rows - 1) / a.rows),
                     static_cast<unsigned>((a.row_items + a.span - 1) / a.span), 1);
  cfg.blockDim = dim3((a.span * a.side + 31) / 32 * 32, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.rows) * a.r * sizeof(float);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = a.rows > a.side ? rope_kernel<E, V, kInter, kLong> : rope_kernel<E, V, kInter, 1>;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// The widest vectors that every pointer, stride and the pairs' ends allow, of 16 bytes
// and less; single elements otherwise.  (12000 rows of 80 heads into pages, D = 128, the
// first 128, 24 and 20 dims turned, bf16, 16, 8 and 4 bytes: 85, 110 and 177 us; by
// single elements 470 and 475.)
template <typename E, int V>
bool fits(const RopeArgs &a, bool interleaved) {
  auto whole = [](const void *p, long long st, long long sh) {
    return reinterpret_cast<uintptr_t>(p) % (V * sizeof(E)) == 0 && st % V == 0 && sh % V == 0;
  };
  return a.D % V == 0 && (interleaved ? a.r % V == 0 : a.r / 2 % V == 0) &&
         (!a.Hq || (whole(a.q.x, a.q.st, a.q.sh) && whole(a.y, a.y_st, a.y_sh))) &&
         (!a.v.x || (whole(a.k.x, a.k.st, a.k.sh) && whole(a.v.x, a.v.st, a.v.sh)));
}
template <typename E, int V>
int launch_by_form(RopeArgs &a, bool interleaved, void *stream) {
  if constexpr (V > 1)
    if (!fits<E, V>(a, interleaved)) return launch_by_form<E, V / 2>(a, interleaved, stream);
  return interleaved ? launch<E, V, true>(a, stream) : launch<E, V, false>(a, stream);
}

// What both calls ask of the rotation and of the rows.
int check(int dtype, int B, int T, int D, const void *freqs, int r, float scale) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  if (B < 1 || T < 0 || T > 0x7FFFFFFF - kMaxRows || D < 8 || D > 512 || D % 8 || r < 0 || r > D || r % 2 || !(fabsf(scale) < INFINITY))
    return SPEC_ERR_SHAPE;
  if (r > 0 && !freqs) return SPEC_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(freqs) & 7) return SPEC_ERR_ALIGNMENT;
  return SPEC_OK;
}

// Sums of two doubles, about 105 bits: the table's fractions have 64, and the error of
// one is multiplied by the position.  (Frequencies in double were off by 2^-55 of a turn,
// at position 2^31 the angle by 3e-7.)  The sums of Knuth (1969) and Dekker (1971); a
// product is kept from being fused with what follows, which its error term presumes.
struct Two {
  double hi, lo;
};
Two sum_of(double a, double b) {
  const double s = a + b, x = s - a;
  return {s, (a - (s - x)) + (b - x)};
}
Two sum(Two a, Two b) {
  const Two s = sum_of(a.hi, b.hi), t = sum_of(a.lo, b.lo), u = sum_of(s.hi, s.lo + t.hi);
  return sum_of(u.hi, u.lo + t.lo);
}
Two mul(Two a, Two b) {
  const volatile double p = a.hi * b.hi;
  return sum_of(p, std::fma(a.lo, b.hi, std::fma(a.hi, b.lo, std::fma(a.hi, b.hi, -p))));
}
Two div(Two a, Two b) {
  const double q = a.hi / b.hi;
  const Two rest = mul(b, {-q, 0.0});
  return sum_of(q, sum(a, rest).hi / b.hi);
}
// x^(1/n): one step of Newton's method squares the double's error.
Two root(double x, int n) {
  const Two g = {std::pow(x, 1.0 / n), 0.0};
  Two power = {1.0, 0.0};
  for (int i = 0; i < n; ++i) power = mul(power, g);
  const Two off = sum(div({x, 0.0}, power), {-1.0, 0.0});
  return sum(g, mul(g, div(off, {static_cast<double>(n), 0.0})));
}
// 2^64 x to the nearest whole number, x in [0, 1/4).
uint64_t turns_of(Two x) {
  const double hi = std::ldexp(x.hi, 64), whole = std::floor(hi);
  return static_cast<uint64_t>(whole) +
         static_cast<uint64_t>(static_cast<int64_t>(std::floor((hi - whole) + std::ldexp(x.lo, 64) + 0.5)));
}

// A stride between rows or heads of which there is only one is never taken.
bool bad_strides(int T, int H, int64_t &st, int64_t &sh) {
  if (T <= 1) st = 0;
  if (H <= 1) sh = 0;
  return st < 0 || sh < 0;
}

}  // namespace

}  // namespace spec

extern "C" int spec_rope_table(int rotary_dim, double base, int scaling, double factor, double original, double low,
                               double high, uint64_t *freqs, float *scale) {
  using namespace spec;
  const double kPi = 3.14159265358979323846;
  const int r = rotary_dim;
  if (!freqs || !scale) return SPEC_ERR_NULL;
  if (r < 2 || r > 512 || r % 2 || !(base > 1.0 && base < 1e30) || scaling < SPEC_ROPE_NONE ||
      scaling > SPEC_ROPE_BANDS)
    return SPEC_ERR_SHAPE;
  if (scaling == SPEC_ROPE_NONE) factor = 1.0;
  if (!(factor >= 1.0 && factor < 1e9)) return SPEC_ERR_SHAPE;
  if (scaling == SPEC_ROPE_NTK && r < 4) return SPEC_ERR_SHAPE;
  const bool ranged = scaling == SPEC_ROPE_YARN || scaling == SPEC_ROPE_BANDS;
  if (ranged && !(original > 0.0 && original < 1e12 && low > 0.0 && high > low && high < 1e12)) return SPEC_ERR_SHAPE;
  // the pair whose wavelength makes `turns` turns in the original context
  auto pair_of = [&](double turns) { return r * std::log(original / (2.0 * kPi * turns)) / (2.0 * std::log(base)); };
  double from = 0.0, width = 1.0;
  if (scaling == SPEC_ROPE_YARN) {
    from = std::fmax(0.0, std::floor(pair_of(high)));
    const double to = std::fmin(r - 1.0, std::ceil(pair_of(low)));
    width = std::fmax(to - from, 0.001);
  }
  const Two one = {1.0, 0.0}, per_turn = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};      // 1 / 2 pi
  Two step = div(one, root(base, r / 2)), theta = one;
  // (base factor^(r / (r - 2)))^(-2 / r) = base^(-2 / r) factor^(-2 / (r - 2))
  if (scaling == SPEC_ROPE_NTK) step = div(step, root(factor, r / 2 - 1));
  for (int i = 0; i < r / 2; ++i, theta = mul(theta, step)) {
    Two keep = one;      // how much of the unscaled frequency stays
    if (scaling == SPEC_ROPE_LINEAR) keep = {0.0, 0.0};
    if (scaling == SPEC_ROPE_YARN && i > from)
      keep = i - from < width ? sum(one, div({from - i, 0.0}, {width, 0.0})) : Two{0.0, 0.0};
    if (scaling == SPEC_ROPE_BANDS) {
      const Two over = sum(mul(mul(theta, per_turn), {original, 0.0}), {-low, 0.0}), all = sum_of(high, -low);
      if (over.hi <= 0.0) keep = {0.0, 0.0};
      else if (sum(over, {-all.hi, -all.lo}).hi < 0.0) keep = div(over, all);
    }
    const Two less = mul(div(theta, {factor, 0.0}), sum(one, {-keep.hi, -keep.lo}));
    freqs[i] = turns_of(mul(sum(mul(theta, keep), less), per_turn));
  }
  *scale = scaling == SPEC_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  return SPEC_OK;
}

extern "C" int spec_rope(const void *x, void *y, int dtype, int B, int T, int H, int D, int64_t x_row_stride,
                         int64_t x_head_stride, int64_t y_row_stride, int64_t y_head_stride, const uint64_t *freqs,
                         int rotary_dim, float scale, int interleaved, const int32_t *start, const int32_t *depth,
                         const int32_t *offsets, int32_t *status, void *stream) {
  using namespace spec;
  if (((!x || !y) && T != 0) || !start || !offsets || !status) return SPEC_ERR_NULL;
  const int rc = check(dtype, B, T, D, freqs, rotary_dim, scale);
  if (rc != SPEC_OK) return rc;
  if (H < 1 || bad_strides(T, H, x_row_stride, x_head_stride) || bad_strides(T, H, y_row_stride, y_head_stride))
    return SPEC_ERR_SHAPE;
  if ((T > 1 && y_row_stride == 0) || (H > 1 && y_head_stride == 0)) return SPEC_ERR_SHAPE;
  const uintptr_t es = dtype == SPEC_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % es) return SPEC_ERR_ALIGNMENT;
  if (T == 0) return SPEC_OK;
  RopeArgs a = {};
  a.q = {x, x_row_stride, x_head_stride};
  a.y = y;
  a.y_st = y_row_stride;
  a.y_sh = y_head_stride;
  a.freqs = reinterpret_cast<const unsigned long long *>(freqs);
  a.scale = scale;
  a.start = start;
  a.depth = depth;
  a.offsets = offsets;
  a.status = status;
  a.B = B;
  a.T = T;
  a.Hq = H;
  a.D = D;
  a.r = rotary_dim;
  return dtype == SPEC_BF16 ? launch_by_form<__nv_bfloat16, 8>(a, interleaved != 0, stream)
                            : launch_by_form<float, 4>(a, interleaved != 0, stream);
}

extern "C" int spec_rope_write_paged(const void *q, void *q_out, const void *k, const void *v, int dtype, int B, int T,
                                     int Hq, int Hkv, int D, int64_t q_row_stride, int64_t q_head_stride,
                                     int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride,
                                     int64_t v_head_stride, const uint64_t *freqs, int rotary_dim, float scale,
                                     int interleaved, void *k_pages, void *v_pages, int num_pages, int page_size,
                                     const int32_t *block_table, int max_pages, const int32_t *prefix_lens,
                                     const int32_t *start, const int32_t *depth, const int32_t *offsets,
                                     int32_t *status, void *stream) {
  using namespace spec;
  if (((!k || !v || (Hq && (!q || !q_out))) && T != 0) || !k_pages || !v_pages || !block_table || !prefix_lens ||
      !offsets || !status)
    return SPEC_ERR_NULL;
  RopeArgs a = {};
  int rc = check(dtype, B, T, D, freqs, rotary_dim, scale);
  if (rc == SPEC_OK) rc = check_pages(num_pages, page_size, max_pages, &a.pages.shift);
  if (rc != SPEC_OK) return rc;
  if (Hq < 0 || Hkv < 1 || bad_strides(T, Hq, q_row_stride, q_head_stride) ||
      bad_strides(T, Hkv, k_row_stride, k_head_stride) || bad_strides(T, Hkv, v_row_stride, v_head_stride))
    return SPEC_ERR_SHAPE;
  const uintptr_t es = dtype == SPEC_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out) | reinterpret_cast<uintptr_t>(k) |
       reinterpret_cast<uintptr_t>(v)) % es ||
      ((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15))
    return SPEC_ERR_ALIGNMENT;
  if (T == 0) return SPEC_OK;
  a.q = {q, q_row_stride, q_head_stride};
  a.k = {k, k_row_stride, k_head_stride};
  a.v = {v, v_row_stride, v_head_stride};
  a.y = q_out;
  a.y_st = static_cast<long long>(Hq) * D;
  a.y_sh = D;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.pages.table = block_table;
  a.pages.max_pages = max_pages;
  a.pages.pages = num_pages;
  a.pages.status = status;
  a.freqs = reinterpret_cast<const unsigned long long *>(freqs);
  a.scale = scale;
  a.slots = prefix_lens;
  a.start = start ? start : prefix_lens;
  a.depth = depth;
  a.offsets = offsets;
  a.status = status;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.r = rotary_dim;
  return dtype == SPEC_BF16 ? launch_by_form<__nv_bfloat16, 8>(a, interleaved != 0, stream)
                            : launch_by_form<float, 4>(a, interleaved != 0, stream);
}
