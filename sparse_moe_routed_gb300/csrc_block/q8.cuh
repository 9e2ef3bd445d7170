// Activations in 8 bits: 32 adjacent columns share a power of two.
//
// q = round(x / 2^e) with the smallest 2^e (-126 <= e <= 121) that keeps the
// group's largest |x| at or below 127 * 2^e.  Dividing by a power of two is
// exact, so q needs no care beyond one rounding, and |q| <= 127 times a power of
// two has at most seven significant bits: a bf16 number, which the tensor cores
// take as it is.  A scale of amax / 127 would halve the worst error and need a
// second rounding there.
#pragma once

#include <stdint.h>

namespace moe {
namespace blk {

constexpr int kGroup = 32;

// Exponent byte (e + 127) of a group from the bits of its largest |x|: amax =
// m * 2^p with 1 <= m < 2 is at or below 127 * 2^(p-6) up to m = 127/64, whose
// mantissa bits are 0x7e0000; adding 0x1ffff carries into the exponent for any
// larger mantissa.  255 for a NaN or an infinity.
__device__ __forceinline__ uint32_t exp_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int b = static_cast<int>((amax_bits + 0x1ffffu) >> 23) - 6;
  return static_cast<uint32_t>(min(max(b, 1), 248));
}

// 2^-e for an exponent byte that exp_byte gave (255: any finite number, the
// group reads back as NaN whatever its q are).
__device__ __forceinline__ float inv_scale(uint32_t b) { return __uint_as_float((254u - min(b, 253u)) << 23); }

// Four values to four bytes.  Adding 1.5 * 2^23 rounds the (exact) product to a
// whole number, ties to even, and leaves its two's complement in the low byte.
// Only exponent byte 248 can hold values past 127.
__device__ __forceinline__ uint32_t q8x4(float a, float b, float c, float d, float inv, bool top) {
  if (top) {
    const float most = 127.f / inv;
    a = fminf(fmaxf(a, -most), most);
    b = fminf(fmaxf(b, -most), most);
    c = fminf(fmaxf(c, -most), most);
    d = fminf(fmaxf(d, -most), most);
  }
  constexpr float kRound = 12582912.f;
  const uint32_t ra = __float_as_uint(fmaf(a, inv, kRound)), rb = __float_as_uint(fmaf(b, inv, kRound)),
                 rc = __float_as_uint(fmaf(c, inv, kRound)), rd = __float_as_uint(fmaf(d, inv, kRound));
  return __byte_perm(__byte_perm(ra, rb, 0x0040), __byte_perm(rc, rd, 0x0040), 0x5410);
}

// Byte i of four as a value: 2^23 + 128 + q is a float whose low byte is q + 128.
__device__ __forceinline__ float q8_value(uint32_t four, int i, float scale) {
  const uint32_t f = __byte_perm(four ^ 0x80808080u, 0x4b000000u, 0x7440u | i);
  return (__uint_as_float(f) - 8388736.f) * scale;
}

// 2^(b-127) for any byte: 2^-127 is below the normal range, 255 is NaN.
__device__ __forceinline__ float scale_of(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255u ? 0x7fffffffu : b << 23);
}

}  // namespace blk
}  // namespace moe
