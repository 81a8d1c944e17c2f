// Writing dense key and value rows into the 4-bit cache, and reading them back.
#include "kv4.cuh"

namespace spec {

namespace {

constexpr int kRowThreads = 256;

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
// last one (that moves it across no boundary and onto none).  What is then no
// tie stays 2^-12 away from one, far more than the product with 1/6 can err,
// and rounding that product to 16 bits makes a true tie exact again.
__device__ __forceinline__ uint32_t round_sticky(uint32_t bits) {
  return (bits & 0xFFFFF000u) | ((bits & 0xFFFu) ? 0x1000u : 0u);
}
__device__ __forceinline__ uint32_t snap16(uint32_t bits) { return (bits + 0x80u) & 0xFFFFFF00u; }

__device__ __forceinline__ uint32_t scale_of(uint32_t amax_bits) {
  const float x = __uint_as_float(round_sticky(amax_bits));
  const uint32_t q = snap16(__float_as_uint(x * (1.0f / 6.0f)));
  const uint32_t normal = ((q + 0x7FFFFu + ((q >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
  const uint32_t small = static_cast<uint32_t>(__float2int_rn(__uint_as_float(q) * 131072.f));
  return min(q < 0x38800000u ? small : normal, kKv4MaxScale);   // 2^-14 parts the two
}

// One row (key and value of one request, head and slot) is 2 x D / 8 lanes of
// eight dimensions each: a whole warp for D = 128, half of one for D = 64.
template <int D, typename E>
__global__ void __launch_bounds__(kRowThreads)
kv4_write_kernel(const Kv4Args a) {
  constexpr int kLanes = D / 4;                 // lanes of a row
  constexpr int R = kv4_record_bytes(D);
  const int tid = threadIdx.x, lane = tid & 31;
  const int sub = lane % kLanes;                // place within the row
  const bool is_v = sub >= kLanes / 2;
  const int chunk = sub % (kLanes / 2);
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0)
    for (int b = tid; b < a.B; b += kRowThreads) {
      const Kv4Rows r = kv4_rows(a.offsets, a.start, b, a.T, a.S_cap);
      if (r.err) report(a.status, b, r.err);
    }
  const long long rows = static_cast<long long>(a.T) * a.H;
  const long long step = static_cast<long long>(gridDim.x) * (kRowThreads / kLanes);
  for (long long w = (static_cast<long long>(blockIdx.x) * kRowThreads + tid - lane) / kLanes; w < rows; w += step) {
    const long long row = w + lane / kLanes;
    const int t = static_cast<int>(min(row, rows - 1) / a.H), h = static_cast<int>(min(row, rows - 1) % a.H);
    const int b = find_request(a.offsets, a.B, t);
    Kv4Rows r = {0, 0, 0, 1};
    if (b >= 0) r = kv4_rows(a.offsets, a.start, b, a.T, a.S_cap);
    // lanes without a row still take part in the shuffles below
    const bool ok = row < rows && b >= 0 && !r.err && t >= r.lo && t < r.lo + r.n;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (ok) {
      const E *src = static_cast<const E *>(is_v ? a.v : a.k) +
                     t * (is_v ? a.v_st : a.k_st) + h * (is_v ? a.v_sh : a.k_sh) + chunk * 8;
      for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(src[i]);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const bool finite = top < 0x7F800000u;
    if (!finite) report(a.status, b, SPEC_ERR_NONFINITE);
    uint32_t byte = finite ? scale_of(top) : 0u;
    const float inv = byte ? 1.0f / __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7))) : 0.f;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float z = finite ? __uint_as_float(round_sticky(__float_as_uint(x[2 * i + e]))) * inv : 0.f;
        y[e] = __uint_as_float(snap16(__float_as_uint(z)));
      }
      uint32_t c;
      asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
          : "=r"(c)
          : "f"(y[0]), "f"(y[1]));
      codes |= c << (8 * i);
    }
    // scale bytes of four neighbouring groups to one word
    byte |= __shfl_down_sync(0xffffffffu, byte, 2) << 8;
    byte |= __shfl_down_sync(0xffffffffu, byte, 4) << 16;
    if (ok && in_bounds(r.start + (t - r.lo), a.S_cap, a.status, b)) {
      uint32_t *rec = reinterpret_cast<uint32_t *>(
          a.kv + ((static_cast<size_t>(b) * a.H + h) * a.S_cap + r.start + (t - r.lo)) * R);
      rec[sub] = codes;
      if (sub % 8 == 0) rec[D / 4 + sub / 8] = byte;
      if (D == 64 && sub % 8 == 4) rec[D / 4 + 2 + sub / 8] = 0u;
    }
  }
}

template <int D, typename E>
__global__ void __launch_bounds__(kRowThreads)
kv4_read_kernel(const Kv4Args a) {
  constexpr int kLanes = D / 4;
  constexpr int R = kv4_record_bytes(D);
  const int tid = threadIdx.x, lane = tid & 31;
  const int sub = lane % kLanes;
  const bool is_v = sub >= kLanes / 2;
  const int chunk = sub % (kLanes / 2);
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0)
    for (int b = tid; b < a.B; b += kRowThreads) {
      const Kv4Rows r = kv4_rows(a.offsets, a.start, b, a.T, a.S_cap);
      if (r.err) report(a.status, b, r.err);
    }
  const long long rows = static_cast<long long>(a.T) * a.H;
  const long long step = static_cast<long long>(gridDim.x) * (kRowThreads / kLanes);
  for (long long row = (static_cast<long long>(blockIdx.x) * kRowThreads + tid) / kLanes; row < rows; row += step) {
    const int t = static_cast<int>(row / a.H), h = static_cast<int>(row % a.H);
    const int b = find_request(a.offsets, a.B, t);
    if (b < 0) continue;
    const Kv4Rows r = kv4_rows(a.offsets, a.start, b, a.T, a.S_cap);
    if (r.err || t < r.lo || t >= r.lo + r.n || !in_bounds(r.start + (t - r.lo), a.S_cap, a.status, b)) continue;
    const uint8_t *rec = a.kv + ((static_cast<size_t>(b) * a.H + h) * a.S_cap + r.start + (t - r.lo)) * R;
    uint32_t p[4];
    kv4_codes_to_half2(__ldg(reinterpret_cast<const uint32_t *>(rec) + sub), p);
    const uint32_t s = kv4_scale_half2(__ldg(rec + D + sub / 2));
    E *dst = static_cast<E *>(is_v ? a.v : a.k) + t * (is_v ? a.v_st : a.k_st) +
             h * (is_v ? a.v_sh : a.k_sh) + chunk * 8;
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = mul_half2(p[i], s);
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y));
      dst[2 * i] = static_cast<E>(f.x);
      dst[2 * i + 1] = static_cast<E>(f.y);
    }
  }
}

// Checks that both calls share.  Dense rows: 16-byte vectors, so every row
// and head starts on a 16-byte boundary.
int check_rows(const void *k, const void *v, int dtype, int B, int T, int Hkv, int D,
               long long k_st, long long k_sh, long long v_st, long long v_sh, const void *kv, int S_cap,
               const int32_t *start, const int32_t *offsets, const int32_t *status) {
  if (!k || !v || !kv || !start || !offsets || !status) return SPEC_ERR_NULL;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  if (B < 1 || T < 0 || Hkv < 1 || S_cap < 1 || (D != 64 && D != 128)) return SPEC_ERR_SHAPE;
  const int es = dtype == SPEC_F32 ? 4 : 2;
  if (k_st < 0 || k_sh < 0 || v_st < 0 || v_sh < 0) return SPEC_ERR_SHAPE;
  if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(kv)) & 15) ||
      ((k_st * es | k_sh * es | v_st * es | v_sh * es) & 15))
    return SPEC_ERR_ALIGNMENT;
  return SPEC_OK;
}

template <typename Kernel>
int launch_rows(Kernel kernel, const Kv4Args &args, int D, void *stream) {
  const long long lanes = static_cast<long long>(args.T) * args.H * (D / 4);
  if (lanes == 0) return SPEC_OK;
  cudaLaunchConfig_t cfg = {};
  const long long blocks = (lanes + kRowThreads - 1) / kRowThreads;
  const long long most = static_cast<long long>(sm_count()) * 8;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most), 1, 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  pdl_attribute(attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
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
  if (dtype == SPEC_BF16)
    return D == 128 ? launch_rows(kv4_write_kernel<128, __nv_bfloat16>, args, D, stream)
                    : launch_rows(kv4_write_kernel<64, __nv_bfloat16>, args, D, stream);
  return D == 128 ? launch_rows(kv4_write_kernel<128, float>, args, D, stream)
                  : launch_rows(kv4_write_kernel<64, float>, args, D, stream);
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
  if (dtype == SPEC_BF16)
    return D == 128 ? launch_rows(kv4_read_kernel<128, __nv_bfloat16>, args, D, stream)
                    : launch_rows(kv4_read_kernel<64, __nv_bfloat16>, args, D, stream);
  return D == 128 ? launch_rows(kv4_read_kernel<128, float>, args, D, stream)
                  : launch_rows(kv4_read_kernel<64, float>, args, D, stream);
}
