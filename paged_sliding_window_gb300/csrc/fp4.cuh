// fp4.cuh -- the 4-bit page format and device pieces shared by its kernels.
// Library-internal.
//
// A page of one KV head of one tensor (16 tokens of HD values) is one run of
// 9 HD bytes, so that one plain bulk copy brings it to shared memory:
//   codes   HD / 256 parts of 2048 bytes, 16 rows of 128 bytes each. Part p of
//           token r holds values 256 p .. 256 p + 255 in eight 16-byte units of
//           32 values; unit u stands at place u ^ (r & 7). Byte b of a unit is
//           the E2M1 codes of its values 2 b (low four bits) and 2 b + 1.
//   scales  16 rows of HD / 16 E4M3 bytes, one for every 16 values (block k);
//           with k = 8 c + 2 t + e it stands at byte t HD / 64 + 2 c' + e, c' = c
//           (HD 256) or 2 (c mod 2) + c / 2 (HD 512).
// The decode's two products read a page along its tokens and along its values:
// the places make both free of bank conflicts and keep a lane's scales together.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "psw_internal.h"
#include "ptx.cuh"

namespace psw {
namespace fp4 {

template <int HD>
struct Page {
  static constexpr int kCodeBytes = kBlockSize * HD / 2;
  static constexpr int kBytes = 9 * HD;
  static constexpr int kScaleRow = HD / 16;
  static constexpr int kLaneScales = HD / 64;  // scale bytes of lane t of a product over keys
  static_assert(HD == 256 || HD == 512, "head_dim");

  // place of 16-byte unit u (0 .. HD / 32 - 1) of token r
  __host__ __device__ static constexpr int unit(int r, int u) {
    return (u >> 3) * 2048 + r * 128 + (((u & 7) ^ (r & 7)) << 4);
  }
  // place of the scale of block k (0 .. HD / 16 - 1) of token r
  __host__ __device__ static constexpr int scale(int r, int k) {
    const int c = k >> 3, t = (k >> 1) & 3, e = k & 1;
    const int cc = HD == 256 ? c : 2 * (c & 1) + (c >> 1);
    return kCodeBytes + r * kScaleRow + t * kLaneScales + 2 * cc + e;
  }
};

// The two codes of byte I of w as f16 values (low code in the low half).
template <int I>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
  uint32_t d;
  if constexpr (I == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(d) : "r"(w));
  else if constexpr (I == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(d) : "r"(w));
  else if constexpr (I == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(d) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(d) : "r"(w));
  return d;
}

// Two E4M3 bytes (the low half of w) as f16 values.
__device__ __forceinline__ uint32_t scales_f16(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(d) : "r"(w));
  return d;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

__device__ __forceinline__ float e4m3_float(uint32_t byte) {
  return f16x2_to_float2(scales_f16(byte)).x;
}

// Eight floats as E2M1 codes, the first in the lowest bits (nearest, ties to even, saturating).
__device__ __forceinline__ uint32_t e2m1_codes(const float2 (&x)[4]) {
  uint32_t d;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(d)
      : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y),
        "f"(x[3].x), "f"(x[3].y));
  return d;
}

// The E4M3 scale of a block whose largest |y| is amax.
__device__ __forceinline__ uint32_t block_scale(float amax) {
  return __nv_cvt_float_to_fp8(__fmul_rn(amax, 1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
}

// Markstein's division (IBM RS/6000, 1990): a quotient from the reciprocal rounded to nearest,
// corrected by its exact remainder, is the correctly rounded one (but for divisors whose bits are all
// ones, which four bits are not).
//
// 1 / s of a block's scale, rounded to nearest (0 where s is 0). s has four significant bits, so
// 1 - s r is exact for an approximation r off by up to two units in the last place, and one
// correction by it gives the nearest number for each of the eight significands.
__device__ __forceinline__ float scale_reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r = __fmaf_rn(r, __fmaf_rn(-s, r, 1.f), r);
  return s > 0.f ? r : 0.f;
}

// Two y / s rounded as a division is, given -s and r = 1 / s (rounded to nearest, which the
// method asks for) twice. Where s is 0, r is 0 and so is the result.
__device__ __forceinline__ float2 quotients(uint64_t y, uint64_t minus_s, uint64_t r) {
  const uint64_t q = f2_mul(y, r);
  return f2_unpack(f2_fma(f2_fma(q, minus_s, y), r, q));
}

// ---- the visible pages of a batch, in sequence order
struct SeqPages {
  int len, lo, p0, np;  // valid length, first position wanted, its page, pages
};
__device__ __forceinline__ SeqPages seq_pages(int len, int lo) {
  SeqPages s{len, lo, lo / kBlockSize, 0};
  if (len > lo) s.np = (len - 1) / kBlockSize - s.p0 + 1;
  return s;
}

}  // namespace fp4
}  // namespace psw
