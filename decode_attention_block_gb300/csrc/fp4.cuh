// fp4.cuh -- 4-bit pages (SPARK_FP4, include/spark_paged.h): where a row's
// codes and scales lie in its block, and conversions from and to them.
#pragma once

#include <cuda_fp16.h>

#include "../../include/spark_paged.h"

#include "common.cuh"
#include "paged.h"

namespace spark {
namespace fp4 {

constexpr int kRows = 16;                      // positions of a block
constexpr int kCodes = kHeadDim / 2;           // bytes of a row's codes
constexpr int kScales = kHeadDim / 16;         // bytes of a row's scales
constexpr int kScalesAt = kRows * kCodes;
constexpr int kBlock = kRows * (kCodes + kScales);
static_assert(kBlock == SPARK_FP4_BLOCK_BYTES, "a block as the header says");

// Chunk c (32 dims, 16 bytes) of row r lies at c ^ turn(r).  An attention warp
// reads a block's codes 16 bytes a lane: of K the lanes 4 g + t of a quarter
// warp rows g and g + 1 (g even), chunks 2 t; of V rows 4 t + j, chunks g and
// g + 1.  Either way the eight lie in eight different places mod 128 bytes.
SPARK_HD int turn(int row) { return (row & 1) | (((row >> 2) & 3) << 1); }
SPARK_HD int code_at(int row, int dim) { return row * kCodes + ((((dim >> 5) ^ turn(row)) << 4) | ((dim & 31) >> 1)); }
SPARK_HD int scale_at(int row, int dim) { return kScalesAt + row * kScales + (dim >> 4); }

// byte offset of the block that holds row `row` of a page, of a KV head
SPARK_HD int64_t block_at(int page, int row, int head, int page_size, int n_kv) {
  return (((int64_t)page * (page_size / kRows) + row / kRows) * n_kv + head) * kBlock;
}

#if defined(__CUDACC__)

// a scale byte as fp32 (0xF8 and above: infinity, NaN)
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __half2float(__ushort_as_half((unsigned short)(b << 7)));
}
constexpr uint32_t kScaleNan = 0xFF, kScaleMost = 0xE2;  // 10240

// The scale of 16 elements of largest magnitude m (finite): m / 6 to 3 mantissa
// bits, ties to even; below 2^-14 to steps of 2^-17.
__device__ __forceinline__ uint32_t scale_of(float m) {
  const float top = __fdiv_rn(m, 6.0f);
  const uint32_t bits = __float_as_uint(top);
  const uint32_t normal = ((bits + 0x7FFFFu + ((bits >> 20) & 1u)) >> 20) - (112u << 3);
  const uint32_t b = top < 6.103515625e-05f ? (uint32_t)__float2int_rn(top * 131072.0f) : normal;
  return b < kScaleMost ? b : kScaleMost;
}

// eight quotients x / scale as codes, the first in the lowest bits
__device__ __forceinline__ uint32_t codes8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// eight codes as four fp16 pairs
__device__ __forceinline__ void halves8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// two fp32 as an fp16 pair, the first in the low half
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// x, or what its fp16 leaves of it
__device__ __forceinline__ float split_part(float x, bool lo) { return lo ? x - __half2float(__float2half_rn(x)) : x; }

// Where a row's probabilities lie in fp16's range: e^(s - ref) with the largest
// score kBelow above ref (base 2) when ref is set, and ref raised once a score
// passes it by kMost, so that none passes 2^15.  Half of fp16's smallest step then
// is 2^-36 of the row's largest or less.  (With ref the maximum itself, a dominant
// key and 131071 others 17.4 nats below it: all of their weight was lost, 3.6e-3
// of the row's.)
constexpr float kBelow = 11.f, kMost = 15.f;
// (rounded so that no score lies further above, whatever fp32's steps of them)
__device__ __forceinline__ float below(float top) { return __fsub_ru(top, kBelow); }
__device__ __forceinline__ bool past(float top, float ref) { return top > __fadd_rd(ref, kMost); }

// The power of two that takes values of largest magnitude m into [1, 2), and
// its inverse: 1 where m is infinite, NaN or below the smallest normal number.
__device__ __forceinline__ float2 unit_of(float m) {
  int e = (int)(__float_as_uint(m) >> 23);  // m >= 0
  if (e == 0 || e == 255) return make_float2(1.f, 1.f);
  e = e < 253 ? e : 253;
  return make_float2(__uint_as_float((uint32_t)(254 - e) << 23), __uint_as_float((uint32_t)e << 23));
}

#endif  // __CUDACC__

}  // namespace fp4
}  // namespace spark
