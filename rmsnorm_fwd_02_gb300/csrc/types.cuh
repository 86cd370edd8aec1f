// types.cuh -- activation element types of the kernels that take BF16, FP16 and FP32: loads
// and stores of 16-byte vectors as FP32 pairs.
#pragma once

#include <cuda_fp16.h>

#include "rmsn_common.cuh"

namespace rmsn {

// FP32 pairs (f2) of a 16-byte vector: four for the 16-bit types, two for FP32.
template <typename T>
struct VecOf;

template <>
struct VecOf<__nv_bfloat16> {
  static constexpr int kPairs = 4;
  __device__ static __forceinline__ void unpack(const uint4& u, f2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = bf2_to_f2(u4_get(u, i));
  }
  __device__ static __forceinline__ f2 pair(const uint4& u, int i) {
    return bf2_to_f2(u4_get(u, i));
  }
  // pair i of u plus nk, each rounded once: a mixed-precision fma x * 1 + nk per element reads
  // the 16-bit halves without a conversion
  __device__ static __forceinline__ f2 plus(const uint4& u, int i, f2 nk) {
    f2 r;
    asm("{\n\t.reg .b16 a0, a1, one;\n\t.reg .f32 c0, c1, p0, p1;\n\t"
        "mov.b32 {a0, a1}, %1;\n\tmov.b16 one, 0x3F80;\n\tmov.b64 {c0, c1}, %2;\n\t"
        "fma.rn.f32.bf16 p0, a0, one, c0;\n\t"
        "fma.rn.f32.bf16 p1, a1, one, c1;\n\t"
        "mov.b64 %0, {p0, p1};\n\t}"
        : "=l"(r.v)
        : "r"(u4_get(u, i)), "l"(nk.v));
    return r;
  }
  __device__ static __forceinline__ uint4 pack(const f2 (&f)[4]) {
    return make_uint4(f2_to_bf2(f[0]), f2_to_bf2(f[1]), f2_to_bf2(f[2]), f2_to_bf2(f[3]));
  }
};

template <>
struct VecOf<__half> {
  static constexpr int kPairs = 4;
  __device__ static __forceinline__ f2 widen(uint32_t u) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u));
    return f2_make(v.x, v.y);
  }
  __device__ static __forceinline__ uint32_t narrow(f2 a) {
    const __half2 h = __floats2half2_rn(f2_lo(a), f2_hi(a));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ static __forceinline__ void unpack(const uint4& u, f2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = widen(u4_get(u, i));
  }
  __device__ static __forceinline__ f2 pair(const uint4& u, int i) { return widen(u4_get(u, i)); }
  __device__ static __forceinline__ f2 plus(const uint4& u, int i, f2 nk) {
    f2 r;
    asm("{\n\t.reg .b16 a0, a1, one;\n\t.reg .f32 c0, c1, p0, p1;\n\t"
        "mov.b32 {a0, a1}, %1;\n\tmov.b16 one, 0x3C00;\n\tmov.b64 {c0, c1}, %2;\n\t"
        "fma.rn.f32.f16 p0, a0, one, c0;\n\t"
        "fma.rn.f32.f16 p1, a1, one, c1;\n\t"
        "mov.b64 %0, {p0, p1};\n\t}"
        : "=l"(r.v)
        : "r"(u4_get(u, i)), "l"(nk.v));
    return r;
  }
  __device__ static __forceinline__ uint4 pack(const f2 (&f)[4]) {
    return make_uint4(narrow(f[0]), narrow(f[1]), narrow(f[2]), narrow(f[3]));
  }
};

template <>
struct VecOf<float> {
  static constexpr int kPairs = 2;
  __device__ static __forceinline__ void unpack(const uint4& u, f2 (&f)[2]) {
    f[0] = f2_make(__uint_as_float(u.x), __uint_as_float(u.y));
    f[1] = f2_make(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  __device__ static __forceinline__ f2 pair(const uint4& u, int i) {
    return i == 0 ? f2_make(__uint_as_float(u.x), __uint_as_float(u.y))
                  : f2_make(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  __device__ static __forceinline__ f2 plus(const uint4& u, int i, f2 nk) {
    return f2_add(pair(u, i), nk);
  }
  __device__ static __forceinline__ uint4 pack(const f2 (&f)[2]) {
    return make_uint4(__float_as_uint(f2_lo(f[0])), __float_as_uint(f2_hi(f[0])),
                      __float_as_uint(f2_lo(f[1])), __float_as_uint(f2_hi(f[1])));
  }
};

__device__ __forceinline__ float widen1(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen1(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen1(float v) { return v; }
__device__ __forceinline__ void narrow1(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void narrow1(float v, __half* p) { *p = __float2half_rn(v); }
__device__ __forceinline__ void narrow1(float v, float* p) { *p = v; }

}  // namespace rmsn
