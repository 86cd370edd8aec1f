// act8.cuh -- activations held in 8 bits: the arithmetic of one thread's eight consecutive
// values and of the four neighbouring lanes that share a block of 32 (include/act8_train.h has
// the format).
//
// Scales are powers of two: scaling is then exact, so a value's 8-bit number depends on nothing
// but the value and its block's greatest magnitude, and what is unpacked again has 7 significant
// bits: exact in BF16.  (A scale of amax / 127 would hold half a bit more on average.)
#pragma once

#include <type_traits>

#include "types.cuh"

namespace rmsn {

constexpr int kAct8Block = 32;

// Bytes of a packed row: the numbers, then a byte a block, each padded to 16.
__host__ __device__ inline int64_t act8_scale_offset(int64_t H) {
  return (H + 15) & ~static_cast<int64_t>(15);
}
__host__ __device__ inline int64_t act8_row_size(int64_t H) {
  const int64_t blocks = (H + kAct8Block - 1) / kAct8Block;
  return act8_scale_offset(H) + ((blocks + 15) & ~static_cast<int64_t>(15));
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The FP32 bits of the greatest magnitude of the eight values of one (two: FP32) 16-byte vector
// (NaN above infinity).  Magnitudes of one type compare as whole numbers.
template <typename T>
__device__ __forceinline__ uint32_t act8_max8(const uint4 (&u)[sizeof(T) / 2]) {
  if constexpr (sizeof(T) == 2) {
    constexpr uint32_t mag = 0x7fff7fffu;
    const uint32_t m = max_u16x2(max_u16x2(u[0].x & mag, u[0].y & mag),
                                 max_u16x2(u[0].z & mag, u[0].w & mag));
    const uint32_t k = max(m & 0xffffu, m >> 16);
    if constexpr (std::is_same_v<T, __nv_bfloat16>)
      return k << 16;
    else  // (the sign cleared: a NaN keeps its own)
      return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(k)))) &
             0x7fffffffu;
  } else {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, u4_get(u[i >> 2], i & 3) & 0x7fffffffu);
    return m;
  }
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

// The numbers of eight values as the low bytes of four pairs of words, put together.
__device__ __forceinline__ uint2 act8_bytes(const f2 (&t)[4], uint32_t scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __byte_perm(__float_as_uint(f2_lo(t[i])), __float_as_uint(f2_hi(t[i])), 0x0040);
  const uint2 q = make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
  return scale == 255u ? make_uint2(0u, 0u) : q;
}

// Eight values as numbers of one byte, the first in the lowest byte of .x.
__device__ __forceinline__ uint2 act8_pack8(const f2 (&v)[4], uint32_t amax, uint32_t scale) {
  // amax 2^(6-e) >= 127.5 although e has reached its end (the last 0.4 % of FP32's range)
  const bool clamp = amax >= 0x7f7f0000u;
  const f2 inv = f2_splat(__uint_as_float((260u - min(scale, 254u)) << 23));
  // adding 1.5 * 2^23 leaves the rounded whole number in the low bits, in two's complement
  const f2 magic = f2_splat(12582912.f);
  f2 t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = f2_fma(v[i], inv, magic);
  if (clamp) {
    const float c = __uint_as_float(0x7f7e0000u);  // 127 * 2^121
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t[i] = f2_fma(f2_make(fminf(fmaxf(f2_lo(v[i]), -c), c), fminf(fmaxf(f2_hi(v[i]), -c), c)),
                    inv, magic);
  }
  return act8_bytes(t, scale);
}

// The same from a 16-byte vector of a 16-bit type.
template <typename T>
__device__ __forceinline__ uint2 act8_pack8(const uint4& u, uint32_t amax, uint32_t scale) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    if (amax < 0x7f7f0000u) {  // (infinities and NaN, and where act8_pack8 clamps: below)
      // the mixed-precision fma reads the BF16 halves as they are; 2^(6-e) is a BF16 value
      const uint32_t inv = (260u - scale) << 7;
      f2 t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 a0, a1, s, z;\n\t.reg .f32 p0, p1;\n\t"
            "mov.b32 {a0, a1}, %1;\n\tmov.b32 {s, z}, %2;\n\t"
            "fma.rn.f32.bf16 p0, a0, s, 0f4B400000;\n\t"
            "fma.rn.f32.bf16 p1, a1, s, 0f4B400000;\n\t"
            "mov.b64 %0, {p0, p1};\n\t}"
            : "=l"(t[i].v)
            : "r"(u4_get(u, i)), "r"(inv));
      return act8_bytes(t, scale);
    }
  }
  f2 v[4];
  VecOf<T>::unpack(u, v);
  return act8_pack8(v, amax, scale);
}

// The zeros behind a row's `blocks` scale bytes at p (16-byte aligned) up to a multiple of 16, by three
// threads (k = 0 to 2): up to a multiple of four a byte each, then a word each.
__device__ __forceinline__ void act8_pad_scales(unsigned char* p, int blocks, int k) {
  if (blocks + k < ((blocks + 3) & ~3)) p[blocks + k] = 0;
  const int word = ((blocks + 3) & ~3) + 4 * k;
  if (word < ((blocks + 15) & ~15)) *reinterpret_cast<uint32_t*>(p + word) = 0u;
}

// The factor of a scale byte's numbers, 2^(e-6); NaN for a block that held one or an infinity.
__device__ __forceinline__ float act8_unit(uint32_t scale) {
  return __uint_as_float(scale == 255u ? 0x7fc00000u : (max(scale, 6u) - 6u) << 23);
}

// Eight numbers of one byte in FP32.
__device__ __forceinline__ void act8_numbers8(const uint2& q, f2 (&v)[4]) {
  const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};  // number + 128
  const f2 off = f2_splat(-8388736.f);                           // -(2^23 + 128)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t s = w[i >> 1];
    const uint32_t at = (i & 1) * 2;
    v[i] = f2_add(f2_make(__uint_as_float(__byte_perm(s, 0x4b000000u, 0x7650u + at)),
                          __uint_as_float(__byte_perm(s, 0x4b000000u, 0x7651u + at))),
                  off);
  }
}

// Their values, exactly.
__device__ __forceinline__ void act8_unpack8(const uint2& q, float unit, f2 (&v)[4]) {
  act8_numbers8(q, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2_mul(v[i], f2_splat(unit));
}

}  // namespace rmsn
