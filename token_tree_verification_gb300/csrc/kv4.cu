// Writing dense key and value rows into the 4-bit cache, and reading them back.
#include "kv4.cuh"

namespace spec {

namespace {

constexpr int kRowThreads = 128;

struct Kv4Args {
  void *k, *v;                              // dense rows [T][Hkv][D]
  long long k_st, k_sh, v_st, v_sh;         // element strides of a row and of a head
  uint8_t *kv;
  const int32_t *start, *offsets;
  int32_t *status;
  int B, T, H, S_cap;
};

// A magnitude's scale byte: amax / 6 rounded to the nearest scale, ties to
// even, in exact arithmetic.  Every boundary between two scales is 6 x (a
// number of at most 5 significant bits), which has at most 7, so amax may
// first be cut to 12 significant bits with everything below folded into the
// last one (that moves it across no boundary and onto none; a bf16 has 8 to
// begin with).  What is then no tie stays 2^-12 away from one, far more than
// the product with 1/6 can err, and rounding that product to 16 bits makes a
// true tie exact again.
template <typename E>
__device__ __forceinline__ uint32_t round_sticky(uint32_t bits) {
  if constexpr (sizeof(E) == 2) return bits;
  return (bits & 0xFFFFF000u) | ((bits & 0xFFFu) ? 0x1000u : 0u);
}

template <typename E>
__device__ __forceinline__ uint32_t scale_of(uint32_t amax_bits) {
  const float x = __uint_as_float(round_sticky<E>(amax_bits)) * (1.0f / 6.0f);
  const uint32_t q = (__float_as_uint(x) + 0x80u) & 0xFFFFFF00u;
  const uint32_t normal = ((q + 0x7FFFFu + ((q >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
  const uint32_t small = static_cast<uint32_t>(__float2int_rn(__uint_as_float(q) * 131072.f));
  return min(q < 0x38800000u ? small : normal, kKv4MaxScale);   // 2^-14 parts the two
}

// The codes of eight elements, x / scale rounded to the nearest with ties to
// even, exactly.  The boundaries are multiples of 1/4; an element (12
// significant bits) that is on none stays 2^-14 away from it, so its quotient
// may be rounded to multiples of 2^-14 first: adding and taking away 768 does
// that, and removes the 2^-21 by which the product with 1 / scale can err.  (A
// zero keeps the element's sign.)
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float inv) {
  constexpr float kGrid = 768.f;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    y[i] = x[i];
    y[i + 1] = x[i + 1];
    fma2(y[i], y[i + 1], inv, inv, kGrid, kGrid);
    add2(y[i], y[i + 1], -kGrid, -kGrid);
    y[i] = copysignf(y[i], x[i]);
    y[i + 1] = copysignf(y[i + 1], x[i + 1]);
  }
  uint32_t c;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(c)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return c;
}

// Eight elements of a row, 16-byte loads and stores.
template <typename E>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldg(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void clear() { v = make_uint4(0u, 0u, 0u, 0u); }
  // the largest magnitude, as the bits of a float
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Eight<float> {
  uint4 v, w;
  __device__ __forceinline__ void load(const float *p) {
    v = __ldg(reinterpret_cast<const uint4 *>(p));
    w = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
  }
  __device__ __forceinline__ void clear() { v = w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = max(max(max(v.x & 0x7FFFFFFFu, v.y & 0x7FFFFFFFu), max(v.z & 0x7FFFFFFFu, v.w & 0x7FFFFFFFu)),
                           max(max(w.x & 0x7FFFFFFFu, w.y & 0x7FFFFFFFu), max(w.z & 0x7FFFFFFFu, w.w & 0x7FFFFFFFu)));
    return m;
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    const uint32_t u[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
  }
};

// A walk along consecutive flattened rows t * H + h: the dense row's offset and
// the record move on by strides within a token's heads; the request is looked
// up again only when t leaves the present one's rows.
template <int R>
struct RowWalk {
  const Kv4Args &a;
  long long st, sh, dense;       // element strides, and offset of the present row
  uint8_t *rec;
  int h, b;
  uint32_t t;                     // (the last warps' walks may end behind 2^31)
  bool ok;                        // the row belongs to a request without error
  Kv4Rows r;

  __device__ __forceinline__ RowWalk(const Kv4Args &args, long long row_stride, long long head_stride, uint32_t row)
      : a(args), st(row_stride), sh(head_stride) {
    t = row / static_cast<uint32_t>(a.H);
    h = static_cast<int>(row - t * static_cast<uint32_t>(a.H));
    look_up();
  }
  __device__ __forceinline__ void look_up() {
    b = t < static_cast<uint32_t>(a.T) ? find_request(a.offsets, a.B, static_cast<int>(t)) : -1;
    r = {0, 0, 0, 1};
    if (b >= 0) r = kv4_rows(a.offsets, a.start, b, a.T, a.S_cap);
    place();
  }
  __device__ __forceinline__ void place() {
    const int i = static_cast<int>(t) - r.lo;        // of the request's rows
    dense = t * st + h * sh;
    ok = b >= 0 && !r.err && i < r.n && in_bounds(r.start + i, a.S_cap, a.status, b);
    rec = a.kv + ((static_cast<size_t>(max(b, 0)) * a.H + h) * a.S_cap + r.start + i) * R;
  }
  __device__ __forceinline__ void advance(int rows) {
    h += rows;
    dense += rows * sh;
    rec += static_cast<size_t>(rows) * a.S_cap * R;
    if (h < a.H) return;
    do {
      h -= a.H;
      ++t;
    } while (h >= a.H);
    if (b < 0 || static_cast<int>(t) - r.lo >= r.n) look_up();
    else place();
  }
};

__device__ __forceinline__ void report_bad_rows(const Kv4Args &a) {
  if (blockIdx.x != 0) return;
  for (int b = threadIdx.x; b < a.B; b += kRowThreads) {
    const Kv4Rows r = kv4_rows(a.offsets, a.start, b, a.T, a.S_cap);
    if (r.err) report(a.status, b, r.err);
  }
}

// One row (key and value of one request, head and slot) is D / 8 lanes when
// written, a group of 16 dimensions each, and D / 4 when read, eight dimensions
// each.  A warp walks `rounds` x U x (32 / lanes of a row) consecutive rows, U
// rounds of loads under way at once; reading requests the next ones too.
//
// A short run (64 rows of 32 heads: 2.5 us) is bound by the chain of look-ups in
// front of its first load.  A long one: 269 MB of bf16 rows and records (51200
// rows of 8 heads, D = 128) are written in 46 us, 5.8 TB/s, 0.86 of what a copy
// reaches; with eight dimensions a lane, and a group's scale found by both of its
// lanes, 59 us, the conversions' instructions then filling the issue slots.
// Reading writes twice what it computes: 153 MB in 27.8 us, 5.5 TB/s, 0.81 of a
// copy.
template <int D, int U, typename E>
__global__ void __launch_bounds__(kRowThreads)
kv4_write_kernel(const Kv4Args a, int rounds) {
  constexpr int kLanes = D / 8;                 // lanes of a row: a group of 16 each
  constexpr int kSide = 32 / kLanes;            // rows of a warp side by side
  constexpr int R = kv4_record_bytes(D);
  const int tid = threadIdx.x, lane = tid & 31;
  const int sub = lane % kLanes;                // place within the row
  const bool is_v = sub >= kLanes / 2;
  const E *base = static_cast<const E *>(is_v ? a.v : a.k) + sub % (kLanes / 2) * 16;
  pdl_trigger();
  pdl_wait();
  const uint32_t warp = (blockIdx.x * kRowThreads + tid) / 32;
  RowWalk<R> w(a, is_v ? a.v_st : a.k_st, is_v ? a.v_sh : a.k_sh,
               warp * static_cast<uint32_t>(rounds * U * kSide) + lane / kLanes);
  for (int round = 0; round < rounds; ++round) {
    Eight<E> in[U][2];
    uint32_t *rec[U];
    int req[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rec[u] = w.ok ? reinterpret_cast<uint32_t *>(w.rec) : nullptr;
      req[u] = w.b;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (w.ok) in[u][e].load(base + w.dense + 8 * e);
        else in[u][e].clear();
      }
      w.advance(kSide);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t top = max(in[u][0].top(), in[u][1].top());
      if (top >= 0x7F800000u) {                 // NaN or infinity: the group becomes zeros
        report(a.status, req[u], SPEC_ERR_NONFINITE);
        top = 0;
        in[u][0].clear();
        in[u][1].clear();
      }
      uint32_t byte = scale_of<E>(top);
      float inv = 0.f;
      if (byte) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(__half2float(__ushort_as_half(byte << 7))));
      uint32_t codes[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x[8];
        in[u][e].floats(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(round_sticky<E>(__float_as_uint(x[i])));
        codes[e] = codes_of(x, inv);
      }
      // scale bytes of four neighbouring groups to one word
      byte |= __shfl_down_sync(0xffffffffu, byte, 1) << 8;
      byte |= __shfl_down_sync(0xffffffffu, byte, 2) << 16;
      if (rec[u]) {
        *reinterpret_cast<uint2 *>(rec[u] + 2 * sub) = make_uint2(codes[0], codes[1]);
        if (sub % 4 == 0) rec[u][D / 4 + sub / 4] = byte;
        if (D == 64 && sub % 4 == 2) rec[u][D / 4 + 2 + sub / 4] = 0u;
      }
    }
  }
  report_bad_rows(a);
}

template <int D, int U, typename E>
__global__ void __launch_bounds__(kRowThreads)
kv4_read_kernel(const Kv4Args a, int rounds) {
  constexpr int kLanes = D / 4;
  constexpr int kSide = 32 / kLanes;
  constexpr int R = kv4_record_bytes(D);
  const int tid = threadIdx.x, lane = tid & 31;
  const int sub = lane % kLanes;
  const bool is_v = sub >= kLanes / 2;
  E *base = static_cast<E *>(is_v ? a.v : a.k) + sub % (kLanes / 2) * 8;
  pdl_trigger();
  pdl_wait();
  const uint32_t warp = (blockIdx.x * kRowThreads + tid) / 32;
  RowWalk<R> w(a, is_v ? a.v_st : a.k_st, is_v ? a.v_sh : a.k_sh,
               warp * static_cast<uint32_t>(rounds * U * kSide) + lane / kLanes);
  uint32_t next_code[U], next_scale[U];
  E *next_dst[U];
  auto load = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      next_dst[u] = w.ok ? base + w.dense : nullptr;
      next_code[u] = next_scale[u] = 0u;
      if (w.ok) {
        next_code[u] = __ldg(reinterpret_cast<const uint32_t *>(w.rec) + sub);
        next_scale[u] = __ldg(w.rec + D + sub / 2);
      }
      w.advance(kSide);
    }
  };
  load();
  for (int round = 0; round < rounds; ++round) {
    uint32_t code[U], scale[U];
    E *dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      dst[u] = next_dst[u];
      code[u] = next_code[u];
      scale[u] = next_scale[u];
    }
    if (round + 1 < rounds) load();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!dst[u]) continue;
      uint32_t p[4];
      kv4_codes_to_half2(code[u], p);
      const uint32_t s = kv4_scale_half2(scale[u]);
      float2 f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t y = mul_half2(p[i], s);
        f[i] = __half22float2(*reinterpret_cast<const __half2 *>(&y));
      }
      if constexpr (sizeof(E) == 4) {
        reinterpret_cast<float4 *>(dst[u])[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        reinterpret_cast<float4 *>(dst[u])[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
      } else {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(f[i].x, f[i].y);
          o[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        *reinterpret_cast<uint4 *>(dst[u]) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  report_bad_rows(a);
}

// Checks that both calls share.  Dense rows: 16-byte vectors, so every row
// and head starts on a 16-byte boundary.  A stride between rows or heads of which
// there is only one is never taken, whatever it is: it becomes 0.
int check_rows(const void *k, const void *v, int dtype, int B, int T, int Hkv, int D,
               int64_t &k_st, int64_t &k_sh, int64_t &v_st, int64_t &v_sh, const void *kv, int S_cap,
               const int32_t *start, const int32_t *offsets, const int32_t *status) {
  if (((!k || !v) && T != 0) || !kv || !start || !offsets || !status) return SPEC_ERR_NULL;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  if (B < 1 || T < 0 || Hkv < 1 || S_cap < 1 || (D != 64 && D != 128)) return SPEC_ERR_SHAPE;
  if (T <= 1) k_st = v_st = 0;
  if (Hkv == 1) k_sh = v_sh = 0;
  const int es = dtype == SPEC_F32 ? 4 : 2;
  if (k_st < 0 || k_sh < 0 || v_st < 0 || v_sh < 0) return SPEC_ERR_SHAPE;
  if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(kv)) & 15) ||
      ((k_st * es | k_sh * es | v_st * es | v_sh * es) & 15))
    return SPEC_ERR_ALIGNMENT;
  return SPEC_OK;
}

template <typename Kernel>
int launch_rows(Kernel kernel, const Kv4Args &args, long long warps, int rounds, void *stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps * 32 + kRowThreads - 1) / kRowThreads), 1, 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args, rounds) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// One round of rows per warp while that leaves every SM at most 32 warps, so
// that a tree's few rows spread over the GPU; beyond, U rounds at once, and as
// many turns of them as make kWaves waves of 32 warps on every SM.  U by
// registers: reading 29081 rows of 8 heads, D = 128, takes 27.7 us with 4 and 30.5
// with 2 for bf16, 64.3 and 59.7 for fp32 (272 MB, 4.6 TB/s); writing 51200 rows of
// 8 heads 45.9 with 2 and 51.7 with 1 for bf16, 75.7 and 77.4 for fp32 (478 MB, 6.3
// TB/s).
template <bool kWrite, int D, typename E>
int rows_by_size(const Kv4Args &args, void *stream) {
  constexpr int U = !kWrite && sizeof(E) == 2 ? 4 : 2, kWaves = 4;
  const long long rows = static_cast<long long>(args.T) * args.H, side = 32 / (kWrite ? D / 8 : D / 4);
  if (rows == 0) return SPEC_OK;
  if (rows > 0x7FFFFFFFll) return SPEC_ERR_SHAPE;      // rows are counted in 32 bits
  const long long one = (rows + side - 1) / side, wave = 32ll * sm_count();
  if (one <= wave) {
    if constexpr (kWrite) return launch_rows(kv4_write_kernel<D, 1, E>, args, one, 1, stream);
    else return launch_rows(kv4_read_kernel<D, 1, E>, args, one, 1, stream);
  }
  const long long rounds = (one + U * kWaves * wave - 1) / (U * kWaves * wave);
  const long long warps = (one + U * rounds - 1) / (U * rounds);
  if constexpr (kWrite) return launch_rows(kv4_write_kernel<D, U, E>, args, warps, static_cast<int>(rounds), stream);
  else return launch_rows(kv4_read_kernel<D, U, E>, args, warps, static_cast<int>(rounds), stream);
}

template <bool kWrite>
int launch_by_type(const Kv4Args &args, int dtype, int D, void *stream) {
  if (dtype == SPEC_BF16)
    return D == 128 ? rows_by_size<kWrite, 128, __nv_bfloat16>(args, stream)
                    : rows_by_size<kWrite, 64, __nv_bfloat16>(args, stream);
  return D == 128 ? rows_by_size<kWrite, 128, float>(args, stream) : rows_by_size<kWrite, 64, float>(args, stream);
}

}  // namespace

}  // namespace spec

extern "C" size_t spec_kv4_record_bytes(int D) {
  return D == 64 || D == 128 ? static_cast<size_t>(spec::kv4_record_bytes(D)) : 0;
}

extern "C" int spec_kv4_write(const void *k, const void *v, int dtype, int B, int T, int Hkv, int D,
                              int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride,
                              int64_t v_head_stride, void *kv_cache, int S_cap, const int32_t *start,
                              const int32_t *offsets, int32_t *status, void *stream) {
  using namespace spec;
  const int rc = check_rows(k, v, dtype, B, T, Hkv, D, k_row_stride, k_head_stride, v_row_stride, v_head_stride,
                            kv_cache, S_cap, start, offsets, status);
  if (rc != SPEC_OK) return rc;
  const Kv4Args args = {const_cast<void *>(k), const_cast<void *>(v), k_row_stride, k_head_stride, v_row_stride,
                        v_head_stride, static_cast<uint8_t *>(kv_cache), start, offsets, status, B, T, Hkv, S_cap};
  return launch_by_type<true>(args, dtype, D, stream);
}

extern "C" int spec_kv4_read(void *k, void *v, int dtype, int B, int T, int Hkv, int D, int64_t k_row_stride,
                             int64_t k_head_stride, int64_t v_row_stride, int64_t v_head_stride,
                             const void *kv_cache, int S_cap, const int32_t *start, const int32_t *offsets,
                             int32_t *status, void *stream) {
  using namespace spec;
  const int rc = check_rows(k, v, dtype, B, T, Hkv, D, k_row_stride, k_head_stride, v_row_stride, v_head_stride,
                            kv_cache, S_cap, start, offsets, status);
  if (rc != SPEC_OK) return rc;
  if ((T > 1 && (!k_row_stride || !v_row_stride)) || (Hkv > 1 && (!k_head_stride || !v_head_stride)))
    return SPEC_ERR_SHAPE;
  const Kv4Args args = {k, v, k_row_stride, k_head_stride, v_row_stride, v_head_stride,
                        static_cast<uint8_t *>(const_cast<void *>(kv_cache)), start, offsets, status, B, T, Hkv, S_cap};
  return launch_by_type<false>(args, dtype, D, stream);
}
