// The 4-bit KV cache's slot record and its decoding.
//
// One record per (request, KV head, slot):
//   K codes  D/2 bytes   e2m1, two per byte, the even dimension in the low half
//   V codes  D/2 bytes
//   K scales D/16 bytes  one per 16 dimensions
//   V scales D/16 bytes
//   zero padding to a multiple of 16 bytes
// (144 bytes for D = 128, 80 for D = 64).  Key and value share a record so
// that a tile of slots is one contiguous run of bytes: one bulk copy brings
// it, and every record starts on the 16-byte boundary such copies need.  Read
// from shared memory, the record's stride of 36 (or 20) words spreads eight
// consecutive records' 16-byte pieces over all 32 banks, without padding.
//
// An e2m1 code is sign, two exponent bits and one mantissa bit: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6 and their negatives.  A scale has five exponent bits (bias
// 15) and three mantissa bits and no sign: bits 14 .. 7 of a half.  The value
// code x scale has at most 2 + 4 significant bits and lies between 2^-18 and
// 61440, so it is exact in half precision and in bfloat16: nothing that reads
// the cache rounds.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace spec {

__host__ __device__ constexpr int kv4_record_bytes(int D) { return (D + D / 8 + 15) / 16 * 16; }

constexpr uint32_t kKv4MaxScale = 0xE2;    // 10240: 6 x 10240 is the largest value, a finite half

// Eight codes (one word, dimension 0 in the lowest nibble) as four half pairs.
__device__ __forceinline__ void kv4_codes_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// A scale byte as a pair of equal halves.
__device__ __forceinline__ uint32_t kv4_scale_half2(uint32_t byte) { return byte * 0x00800080u; }

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// Two fp32 at once.
__device__ __forceinline__ void fma2(float &x0, float &x1, float c0, float c1, float n0, float n1) {
  asm("{\n\t.reg .b64 x, c, n;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 c, {%2, %3};\n\tmov.b64 n, {%4, %5};\n\t"
      "fma.rn.f32x2 x, x, c, n;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(c0), "f"(c1), "f"(n0), "f"(n1));
}
__device__ __forceinline__ void add2(float &x0, float &x1, float y0, float y1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(y0), "f"(y1));
}

// Rows of a ragged batch against the cache: request b's rows are
// [offsets[b], offsets[b+1]) and its row i belongs to slot start[b] + i.
struct Kv4Rows {
  int lo, n, start, err;
};

__device__ __forceinline__ Kv4Rows kv4_rows(const int32_t *offsets, const int32_t *start, int b,
                                            int T, int S_cap) {
  Kv4Rows r;
  r.lo = __ldg(offsets + b);
  const int hi = __ldg(offsets + b + 1);
  r.n = hi - r.lo;
  r.start = __ldg(start + b);
  r.err = 0;
  if (r.lo < 0 || hi > T || hi < r.lo) r.err = SPEC_ERR_TREE_TOO_LARGE;
  else if (r.start < 0 || static_cast<long long>(r.start) + r.n > S_cap) r.err = SPEC_ERR_PREFIX_RANGE;
  return r;
}

}  // namespace spec
