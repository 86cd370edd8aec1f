// act8.cuh -- activations held in 8 bits: the arithmetic of one thread's eight consecutive
// values and of the four neighbouring lanes that share a block of 32 (include/act8_train.h has
// the format).
//
// Scales are powers of two: scaling is then exact, so a value's 8-bit number depends on nothing
// but the value and its block's greatest magnitude, and what is unpacked again has 7 significant
// bits: exact in BF16, its products with BF16 values exact in FP32.  (A scale of amax / 127 would
// hold half a bit more on average.)
#pragma once

#include "types.cuh"

namespace rmsn {

constexpr int kAct8Block = 32;

// Bytes of a packed row: the numbers, then a byte a block, each padded to 16.
__host__ __device__ inline int64_t act8_scale_offset(int64_t H) {
  return (H + 15) & ~static_cast<int64_t>(15);
}
__host__ __device__ inline int64_t act8_row_size(int64_t H) {
  return act8_scale_offset(H) + (((H + kAct8Block - 1) / kAct8Block + 15) & ~static_cast<int64_t>(15));
}

// The bits of the greatest magnitude of 8 values in FP32 (NaN above infinity).
__device__ __forceinline__ uint32_t act8_max8(const f2 (&v)[4]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = max(m, __float_as_uint(f2_lo(v[i])) & 0x7fffffffu);
    m = max(m, __float_as_uint(f2_hi(v[i])) & 0x7fffffffu);
  }
  return m;
}

// Over the four lanes of a block.
__device__ __forceinline__ uint32_t act8_max_block(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// The block's scale byte from the bits of its greatest magnitude: 127 + e, e the smallest
// exponent >= -120 with amax 2^(6-e) < 127.5.  amax = 1.m 2^k takes e = k unless its top seven
// fraction bits are all ones (1.m >= 127.5 / 64), where the addition carries into the exponent.
__device__ __forceinline__ uint32_t act8_scale_byte(uint32_t amax) {
  const uint32_t e = min(max((amax + 0x10000u) >> 23, 7u), 254u);
  return amax >= 0x7f800000u ? 255u : e;
}

// Eight values as numbers of one byte, the first in the lowest byte of .x.
__device__ __forceinline__ uint2 act8_pack8(const f2 (&v)[4], uint32_t amax, uint32_t scale) {
  // amax 2^(6-e) >= 127.5 although e has reached its end (the last 0.4 % of FP32's range)
  const bool clamp = amax >= 0x7f7f0000u;
  const f2 inv = f2_splat(__uint_as_float((260u - min(scale, 254u)) << 23));
  // adding 1.5 * 2^23 leaves the rounded whole number in the low bits, in two's complement
  const f2 magic = f2_splat(12582912.f);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f2 a = v[i];
    if (clamp) {
      const float c = __uint_as_float(0x7f7e0000u);  // 127 * 2^121
      a = f2_make(fminf(fmaxf(f2_lo(a), -c), c), fminf(fmaxf(f2_hi(a), -c), c));
    }
    const f2 t = f2_fma(a, inv, magic);
    w[i] = __byte_perm(__float_as_uint(f2_lo(t)), __float_as_uint(f2_hi(t)), 0x0040);
  }
  const uint2 q = make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
  return scale == 255u ? make_uint2(0u, 0u) : q;
}

// The factor of a scale byte's numbers, 2^(e-6); NaN for a block that held one or an infinity.
__device__ __forceinline__ float act8_unit(uint32_t scale) {
  return __uint_as_float(scale == 255u ? 0x7fc00000u : (max(scale, 6u) - 6u) << 23);
}

// Eight numbers of one byte as FP32 values, exactly.
__device__ __forceinline__ void act8_unpack8(const uint2& q, float unit, f2 (&v)[4]) {
  const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};  // number + 128
  const f2 off = f2_splat(-8388736.f), u2 = f2_splat(unit);      // -(2^23 + 128)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t s = w[i >> 1];
    const uint32_t at = (i & 1) * 2;
    const f2 t = f2_make(__uint_as_float(__byte_perm(s, 0x4b000000u, 0x7650u + at)),
                         __uint_as_float(__byte_perm(s, 0x4b000000u, 0x7651u + at)));
    v[i] = f2_mul(f2_add(t, off), u2);
  }
}

}  // namespace rmsn
