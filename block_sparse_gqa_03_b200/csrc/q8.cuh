// Device helpers of the 8-bit KV cache: e4m3 codes with one fp32 scale per (block of
// tokens, KV head), value = code * scale.
//
// The scales that the cache write makes are powers of two.  e4m3 is a floating
// format, so above 2^-6 of the scale a power of two costs no precision against a free
// scale (below, on e4m3's fixed grid, up to one bit against max |x| / 448); x / scale is
// exact in fp32 (no rounding next to a code border depends on how the division is
// done); a larger scale keeps every code that stays normal exact; and code * scale
// is a bf16 number (but for codes of 256 and more at a scale of 2^120, which rows above
// 3.3e38 have: they read back as infinity).
//
// The tensor-core products of the decode kernels run on f16 operands: every e4m3 value
// is an f16 value, and the hardware widens two codes per instruction.  (The e4m3 product
// with a query in two e4m3 terms needs no widening of K, but keeps two sums per score:
// the 128K decode attention at batch 32 took 93.7 us with it, 90.7 us without.)  Queries are bf16, so a row is
// scaled by a power of two that puts its largest magnitude into [2^14, 2^15): all
// elements within 2^-31 of the largest stay exact, smaller ones are off by at most
// 2^-39 of it, far below the fp32 accumulation error.
#pragma once

#include <cuda_fp16.h>
#include <limits.h>

#include "common.cuh"

namespace msa {
namespace q8 {

constexpr int kMinExp = -100;  // smallest scale 2^-100 (also that of an all-zero block)
constexpr int kMaxExp = 120;   // largest scale a bf16 row can need

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of the smallest power-of-two scale s with amax <= 448 s, amax given as
// the bits of a non-negative finite bf16: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u ? 1 : 0);
  return max(e, kMinExp);  // zero and subnormal maxima included
}

// Exponent of a stored scale, or INT_MIN when it is not a power of two in range.
__device__ __forceinline__ int stored_exp(float s) {
  const uint32_t b = __float_as_uint(s);
  const int e = (int)(b >> 23) - 127;  // a set sign bit gives e >= 129
  return (b & 0x7fffffu) == 0 && e >= kMinExp && e <= kMaxExp ? e : INT_MIN;
}

// Four floats to four codes (round to nearest even, saturating at +-448; NaN stays
// NaN), x in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x4(float x, float y, float z, float w) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y), "f"(x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(w), "f"(z));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Two codes (the low or high half of a register) to f16x2, exactly.
__device__ __forceinline__ uint32_t to_f16x2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
__device__ __forceinline__ uint32_t lo_f16x2(uint32_t codes) { return to_f16x2((uint16_t)codes); }
__device__ __forceinline__ uint32_t hi_f16x2(uint32_t codes) {
  return to_f16x2((uint16_t)(codes >> 16));
}

__device__ __forceinline__ float2 f16x2_floats(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// D += A * B for one 16x8x16 tile, f16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk `chunk` of row `row` in a tile of RB-byte rows stored
// with the RB-byte TMA swizzle (128, 64 or 32; tile base 1024-aligned).
template <int RB>
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t chunk) {
  static_assert(RB == 128 || RB == 64 || RB == 32, "row bytes");
  if constexpr (RB == 128) return row * 128u + ((chunk ^ (row & 7u)) << 4);
  if constexpr (RB == 64) return row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
  return row * 32u + ((chunk ^ ((row >> 2) & 1u)) << 4);
}

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t x) {
  return __vmaxu2(m, x & 0x7fff7fffu);
}

// The fragments of one bf16 row of NC * 16 elements for products with e4m3 rows: the
// four lanes of a quad hold elements 16c + 4j .. 16c + 4j + 3 (j = lane % 4) of each
// 16-element step c, which is where the four codes of one ldmatrix register lie.
// `p` points at element 4j of the row.  The row is scaled by a power of two (above);
// returns the factor that undoes it.  An invalid row gives zeros.
template <int NC>
__device__ __forceinline__ float load_row_f16(const uint16_t* p, bool valid, uint32_t (&lo)[NC],
                                              uint32_t (&hi)[NC]) {
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const uint2 u = valid ? *reinterpret_cast<const uint2*>(p + 16 * c) : make_uint2(0u, 0u);
    lo[c] = u.x;
    hi[c] = u.y;
    m = abs_max2(abs_max2(m, u.x), u.y);
  }
  m = max(m & 0xffffu, m >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const int e = max((int)(m >> 7), 15);  // biased exponent of the largest magnitude
  const float f = __int_as_float((268 - e) << 23);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    lo[c] = pack_f16(__uint_as_float(lo[c] << 16) * f, __uint_as_float(lo[c] & 0xffff0000u) * f);
    hi[c] = pack_f16(__uint_as_float(hi[c] << 16) * f, __uint_as_float(hi[c] & 0xffff0000u) * f);
  }
  return __int_as_float((e - 14) << 23);
}

}  // namespace q8
}  // namespace msa
