// drop.cu -- dropout forward and backward for sm_103a, and their C ABI
// (include/dropout_train.h).
//
// y_i = [residual_i +] (keep_i ? x_i * scale : 0), keep_i drawn by drop_philox.cuh; the
// backward is the same kernel on dy.  HBM-bound: two (three with a residual) tensors of
// traffic against five integer and about three floating-point instructions an element.
// A thread takes kUnroll groups of eight elements, a block's groups side by side, all loads
// issued before the first is used.
// Measured: 65536 x 4096 fp16 153 us (7.0 TB/s, a plain copy's rate); 4099 x 2051 fp32 with a
// residual 17.3 us (15 of bandwidth, the rest the launch's ramp).
#include <cmath>
#include <cstdint>

#include "dropout_train.h"  // include/ (on the include path)
#include "drop_philox.cuh"
#include "types.cuh"

namespace rmsn {

namespace {

constexpr int kDropThreads = 256;
constexpr int kDropUnroll = 4;

// One group of eight elements held as FP32 pairs: kept ones scaled, dropped ones zero, the
// residual added (one rounding: fma).
template <bool kRes, bool kDrop>
__device__ __forceinline__ void drop_pairs(const DropParams& d, const uint4& bits, f2 (&v)[4],
                                           const f2 (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo = f2_lo(v[i]), hi = f2_hi(v[i]);
    const float rl = kRes ? f2_lo(r[i]) : 0.f, rh = kRes ? f2_hi(r[i]) : 0.f;
    if constexpr (kDrop) {
      const uint32_t w = u4_get(bits, i);
      lo = drop_keep_lo(d, w) ? (kRes ? __fmaf_rn(lo, d.scale, rl) : lo * d.scale) : rl;
      hi = drop_keep_hi(d, w) ? (kRes ? __fmaf_rn(hi, d.scale, rh) : hi * d.scale) : rh;
    } else if constexpr (kRes) {
      lo += rl;
      hi += rh;
    }
    v[i] = f2_make(lo, hi);
  }
}

template <typename T>
struct Group {  // eight elements: one 16-byte vector of a 16-bit type, two of FP32
  static constexpr int kVecs = static_cast<int>(sizeof(T) / 2);
  uint4 u[kVecs];
  __device__ __forceinline__ void load(const T* p, int64_t q) {
    const uint4* g = reinterpret_cast<const uint4*>(p) + q * kVecs;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) u[i] = g[i];
  }
  __device__ __forceinline__ void store(T* p, int64_t q) const {
    uint4* g = reinterpret_cast<uint4*>(p) + q * kVecs;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) g[i] = u[i];
  }
  __device__ __forceinline__ void get(f2 (&f)[4]) const {
    constexpr int n = VecOf<T>::kPairs;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      f2 t[n];
      VecOf<T>::unpack(u[i], t);
#pragma unroll
      for (int k = 0; k < n; ++k) f[i * n + k] = t[k];
    }
  }
  __device__ __forceinline__ void set(const f2 (&f)[4]) {
    constexpr int n = VecOf<T>::kPairs;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      f2 t[n];
#pragma unroll
      for (int k = 0; k < n; ++k) t[k] = f[i * n + k];
      u[i] = VecOf<T>::pack(t);
    }
  }
};

template <typename T, bool kRes, bool kDrop>
__global__ void __launch_bounds__(kDropThreads)
    dropout_kernel(const T* __restrict__ x, const T* __restrict__ res, T* __restrict__ y,
                   int64_t n, const DropParams d) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int64_t whole = n >> 3;  // whole groups
  const int64_t q0 = static_cast<int64_t>(blockIdx.x) * (kDropThreads * kDropUnroll) + threadIdx.x;
  Group<T> xv[kDropUnroll], rv[kRes ? kDropUnroll : 1];
#pragma unroll
  for (int i = 0; i < kDropUnroll; ++i) {
    const int64_t q = q0 + i * kDropThreads;
    if (q < whole) {
      xv[i].load(x, q);
      if constexpr (kRes) rv[i].load(res, q);
    }
  }
  const uint2 c = kDrop ? drop_counter(d) : make_uint2(0u, 0u);
#pragma unroll
  for (int i = 0; i < kDropUnroll; ++i) {
    const int64_t q = q0 + i * kDropThreads;
    if (q < whole) {
      f2 v[4], r[4];
      xv[i].get(v);
      if constexpr (kRes) rv[i].get(r);
      const uint4 bits = kDrop ? drop_block(d, c, static_cast<uint64_t>(q))
                               : make_uint4(0u, 0u, 0u, 0u);
      drop_pairs<kRes, kDrop>(d, bits, v, r);
      xv[i].set(v);
      xv[i].store(y, q);
    }
  }
  // the last n % 8 elements: one thread of the last block each
  const int tail = static_cast<int>(n & 7);
  if (blockIdx.x == gridDim.x - 1 && static_cast<int>(threadIdx.x) < tail) {
    const int64_t at = whole * 8 + threadIdx.x;
    float v = widen1(x[at]);
    const float r = kRes ? widen1(res[at]) : 0.f;
    if constexpr (kDrop) {  // as drop_pairs, an element at a time (no + 0: a kept -0 stays)
      const uint4 bits = drop_block(d, c, static_cast<uint64_t>(whole));
      const uint32_t w = u4_get(bits, threadIdx.x >> 1);
      const bool keep = (threadIdx.x & 1) ? drop_keep_hi(d, w) : drop_keep_lo(d, w);
      v = keep ? (kRes ? __fmaf_rn(v, d.scale, r) : v * d.scale) : r;
    } else if constexpr (kRes) {
      v += r;
    }
    narrow1(v, y + at);
  }
}

template <typename T>
const void* pick(bool res, bool drop) {
  if (res)
    return drop ? reinterpret_cast<const void*>(&dropout_kernel<T, true, true>)
                : reinterpret_cast<const void*>(&dropout_kernel<T, true, false>);
  return drop ? reinterpret_cast<const void*>(&dropout_kernel<T, false, true>)
              : reinterpret_cast<const void*>(&dropout_kernel<T, false, false>);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxElements = int64_t{1} << 40;

int dropout_any(const void* x, const void* residual, void* y, int dtype, int64_t n, double p,
                uint64_t seed, uint64_t offset, const uint64_t* step, void* stream) {
  if (dtype != DROPOUT_BF16 && dtype != DROPOUT_FP32 && dtype != DROPOUT_FP16)
    return RMSN_ERR_INVALID_ARG;
  if (n < 0) return RMSN_ERR_INVALID_ARG;
  if (n >= kMaxElements) return RMSN_ERR_UNSUPPORTED;
  if (n > 0 && (!x || !y)) return RMSN_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(y)) return RMSN_ERR_INVALID_ARG;
  DropParams d;
  if (!drop_params(p, seed, offset, step, &d)) return RMSN_ERR_INVALID_ARG;
  if (n == 0) return RMSN_OK;
  const int st = check_device();
  if (st != RMSN_OK) return st;
  return launch_dropout(x, residual, y, dtype, n, d, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? RMSN_OK
             : RMSN_ERR_CUDA;
}

}  // namespace

bool drop_params(double p, uint64_t seed, uint64_t offset, const void* step, DropParams* d) {
  if (!(p >= 0.0 && p <= 1.0)) return false;  // NaN too
  if (reinterpret_cast<uintptr_t>(step) & 7u) return false;
  const uint32_t t = static_cast<uint32_t>(65536.0 * p + 0.5);  // 0 .. 65536
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
  for (int r = 0; r < 10; ++r) {
    d->rk[2 * r] = k0;
    d->rk[2 * r + 1] = k1;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  d->offset = offset;
  d->step = static_cast<const unsigned long long*>(step);
  d->drop_below = (t << 16) - 1u;
  d->scale = t < 65536u ? static_cast<float>(65536.0 / (65536 - static_cast<int>(t))) : 0.f;
  d->active = t > 0u;
  return true;
}

cudaError_t launch_dropout(const void* x, const void* residual, void* y, int dtype, int64_t n,
                           const DropParams& d, cudaStream_t st) {
  const bool res = residual != nullptr, drop = d.active != 0;
  const void* fn = dtype == DROPOUT_BF16   ? pick<__nv_bfloat16>(res, drop)
                   : dtype == DROPOUT_FP32 ? pick<float>(res, drop)
                                           : pick<__half>(res, drop);
  constexpr int64_t per = static_cast<int64_t>(kDropThreads) * kDropUnroll * 8;
  const int64_t blocks = (n + per - 1) / per;  // below 2^27 for n below 2^40
  DropParams copy = d;
  void* args[] = {&x, &residual, &y, &n, &copy};
  return launch_pdl(fn, dim3(static_cast<unsigned>(blocks)), dim3(kDropThreads), 0, st, args);
}

}  // namespace rmsn

using namespace rmsn;

extern "C" {

int dropout_train_fwd(const void* x, const void* residual, void* y, int dtype, int64_t n,
                      double p, uint64_t seed, uint64_t offset, const uint64_t* step,
                      void* stream) {
  return dropout_any(x, residual, y, dtype, n, p, seed, offset, step, stream);
}

int dropout_train_bwd(const void* dy, void* dx, int dtype, int64_t n, double p, uint64_t seed,
                      uint64_t offset, const uint64_t* step, void* stream) {
  return dropout_any(dy, nullptr, dx, dtype, n, p, seed, offset, step, stream);
}

}  // extern "C"
