// 4-bit rows: two e2m1 values a byte (the even column in the low half) and one
// scale byte b, for 2^(b - 127), a group of 32 columns.  e2m1 stands for 0,
// 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives.  Every value is exact in bf16, where
// it is subnormal too (b of 0 and 1: multiples of 2^-128), but for magnitudes past
// its range, which become infinities (from 4 on under b = 253, from 2 under 254).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace itl {

constexpr int kFp4Group = 32;

// The scale as fp32: 2^-127 for 0, NaN for 255.
__device__ __forceinline__ float fp4_scale(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
}

// The value of a 4-bit code (its low four bits): for magnitudes from 1 on the
// code's exponent and mantissa bits are those of an fp32 shifted.
__device__ __forceinline__ float fp4_value(uint32_t q) {
  const uint32_t m = q & 7u;
  const uint32_t big = ((m >> 1) + 126u) << 23 | (m & 1u) << 22;
  return __uint_as_float((m >= 2 ? big : m == 1 ? 0x3f000000u : 0u) | (q & 8u) << 28);
}

// data [n, ld_d] bytes and scales [n, ld_s] bytes of x [n, ld_x]: b the
// smallest scale that brings the group within 6 (1 to 252; 255 for a group
// with an infinity or a NaN), values rounded to the nearest, ties to an even
// code.
void launch_fp4_quantize(int dtype, const void* x, int64_t ld_x, int64_t n, int64_t h,
                         uint8_t* data, int64_t ld_d, uint8_t* scales, int64_t ld_s,
                         hipStream_t s);

}  // namespace itl
