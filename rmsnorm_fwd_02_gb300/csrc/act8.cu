// act8.cu -- activations packed into 8 bits and unpacked for sm_103a, and their C ABI
// (include/act8_train.h).
//
// HBM-bound: 2 (4) + 1.03 bytes an element each way for about six instructions.  A thread takes
// eight consecutive elements of a row, the four lanes of a block agree on its greatest magnitude
// by two shuffles.  Warps take tiles of 32 such groups (256 elements) of a row, or, where a row
// has fewer groups, the groups of consecutive rows side by side (each row's padded to a multiple
// of four, so that no block straddles a warp).
#include <cstdint>
#include <type_traits>

#include "act8.cuh"
#include "act8_train.h"  // include/ (on the include path)

namespace rmsn {

namespace {

constexpr int kAct8Threads = 256;
constexpr int kAct8Unroll = 4;  // groups a thread has in flight

// Eight elements from p, of which n (1..8) exist; vec: 16-byte loads are allowed.
template <typename T>
__device__ __forceinline__ void load_group(const T* p, int n, bool vec, f2 (&f)[4]) {
  constexpr int kVecs = static_cast<int>(sizeof(T) / 2), kP = VecOf<T>::kPairs;
  if (vec && n == 8) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      f2 t[kP];
      VecOf<T>::unpack(reinterpret_cast<const uint4*>(p)[i], t);
#pragma unroll
      for (int k = 0; k < kP; ++k) f[i * kP + k] = t[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = f2_make(2 * i < n ? widen1(p[2 * i]) : 0.f, 2 * i + 1 < n ? widen1(p[2 * i + 1]) : 0.f);
  }
}

template <typename T>
__device__ __forceinline__ void store_group(T* p, int n, bool vec, const f2 (&f)[4]) {
  constexpr int kVecs = static_cast<int>(sizeof(T) / 2), kP = VecOf<T>::kPairs;
  if (vec && n == 8) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      f2 t[kP];
#pragma unroll
      for (int k = 0; k < kP; ++k) t[k] = f[i * kP + k];
      reinterpret_cast<uint4*>(p)[i] = VecOf<T>::pack(t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i < n) narrow1(f2_lo(f[i]), p + 2 * i);
      if (2 * i + 1 < n) narrow1(f2_hi(f[i]), p + 2 * i + 1);
    }
  }
}

// v, or FP16's largest value of its sign where it is finite and past it (NaN stays).
__device__ __forceinline__ float within_half(float v) {
  return fabsf(v) > 65504.f ? copysignf(65504.f, v) : v;
}

struct Act8Args {
  const void* in;
  void* out;
  int64_t R, H, s_row;  // s_row: elements between rows of the wide tensor
  int64_t groups;       // groups a row, a multiple of 4
  int64_t total;        // R * groups
  int32_t vec;
};

// Where group i lies: its row and its place there.
__device__ __forceinline__ void act8_place(const Act8Args& a, int64_t i, int64_t* row, int64_t* c) {
  if (a.total <= 0x7fffffff) {
    const uint32_t r = static_cast<uint32_t>(i) / static_cast<uint32_t>(a.groups);
    *row = r;
    *c = static_cast<uint32_t>(i) - r * static_cast<uint32_t>(a.groups);
  } else {
    *row = i / a.groups;
    *c = i - *row * a.groups;
  }
}

template <typename T>
__global__ void __launch_bounds__(kAct8Threads) act8_pack_kernel(const Act8Args a) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kAct8Threads * kAct8Unroll) + threadIdx.x;
  const T* x = static_cast<const T*>(a.in);
  f2 v[kAct8Unroll][4];
  int64_t row[kAct8Unroll], c[kAct8Unroll];
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    const int64_t i = first + u * kAct8Threads;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[u][k] = f2_splat(0.f);
    row[u] = -1;
    if (i < a.total) {
      act8_place(a, i, &row[u], &c[u]);
      const int64_t n = a.H - 8 * c[u];
      if (n > 0)
        load_group(x + row[u] * a.s_row + 8 * c[u], static_cast<int>(n < 8 ? n : 8), a.vec != 0, v[u]);
    }
  }
  const int64_t first_scale = act8_scale_offset(a.H), bytes = act8_row_size(a.H);
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    const uint32_t amax = act8_max_block(act8_max8(v[u]));
    const uint32_t s = act8_scale_byte(amax);
    if (row[u] >= 0) {
      uint8_t* p = static_cast<uint8_t*>(a.out) + row[u] * bytes;
      if (8 * c[u] < first_scale)
        *reinterpret_cast<uint2*>(p + 8 * c[u]) = act8_pack8(v[u], amax, s);
      if ((c[u] & 3) == 0) {
        p += first_scale + (c[u] >> 2);
        *p = static_cast<uint8_t>(s);
        if (c[u] + 4 == a.groups)  // the row's last block: the padding behind it
          for (uint8_t* q = p + 1; reinterpret_cast<uintptr_t>(q) & 15u; ++q) *q = 0;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kAct8Threads) act8_unpack_kernel(const Act8Args a) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kAct8Threads * kAct8Unroll) + threadIdx.x;
  const int64_t first_scale = act8_scale_offset(a.H), bytes = act8_row_size(a.H);
  T* y = static_cast<T*>(a.out);
  uint2 q[kAct8Unroll];
  uint32_t s[kAct8Unroll];
  int64_t row[kAct8Unroll], c[kAct8Unroll];
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    const int64_t i = first + u * kAct8Threads;
    row[u] = -1;
    if (i < a.total) {
      act8_place(a, i, &row[u], &c[u]);
      if (8 * c[u] < a.H) {
        const uint8_t* p = static_cast<const uint8_t*>(a.in) + row[u] * bytes;
        q[u] = *reinterpret_cast<const uint2*>(p + 8 * c[u]);
        s[u] = p[first_scale + (c[u] >> 2)];
      } else {
        row[u] = -1;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    if (row[u] < 0) continue;
    f2 v[4];
    act8_unpack8(q[u], act8_unit(s[u]), v);
    if constexpr (std::is_same_v<T, __half>) {  // FP16's last values round up to 2^16: no infinity
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = f2_make(within_half(f2_lo(v[k])), within_half(f2_hi(v[k])));
    }
    const int64_t n = a.H - 8 * c[u];
    store_group(y + row[u] * a.s_row + 8 * c[u], static_cast<int>(n < 8 ? n : 8), a.vec != 0, v);
  }
}

constexpr int64_t kAct8MaxBytes = int64_t{1} << 42;  // of a packed tensor

int act8_run(const void* wide, int dtype, const void* packed, int64_t R, int64_t H, int64_t s_row,
             bool pack, void* stream) {
  if (dtype != ACT8_BF16 && dtype != ACT8_FP32 && dtype != ACT8_FP16) return RMSN_ERR_INVALID_ARG;
  if (R < 0 || H < 1 || s_row < 0) return RMSN_ERR_INVALID_ARG;
  if (H > INT32_MAX || R > kAct8MaxBytes / act8_row_size(H)) return RMSN_ERR_UNSUPPORTED;
  if (R > 0 && (!wide || !packed)) return RMSN_ERR_INVALID_ARG;
  const uintptr_t elem = dtype == ACT8_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(wide) % elem || (reinterpret_cast<uintptr_t>(packed) & 15u))
    return RMSN_ERR_INVALID_ARG;
  if (R == 0) return RMSN_OK;
  const int st = check_device();
  if (st != RMSN_OK) return st;
  Act8Args a{};
  a.in = pack ? wide : packed;
  a.out = const_cast<void*>(pack ? packed : wide);
  a.R = R;
  a.H = H;
  a.s_row = R > 1 ? s_row : H;
  a.groups = (H + kAct8Block - 1) / kAct8Block * 4;
  a.total = R * a.groups;
  a.vec = reinterpret_cast<uintptr_t>(wide) % 16 == 0 && a.s_row * elem % 16 == 0;
  const void* fn;
#define ACT8_PICK(K)                                                                  \
  (dtype == ACT8_BF16   ? reinterpret_cast<const void*>(&K<__nv_bfloat16>)            \
   : dtype == ACT8_FP32 ? reinterpret_cast<const void*>(&K<float>)                    \
                        : reinterpret_cast<const void*>(&K<__half>))
  fn = pack ? ACT8_PICK(act8_pack_kernel) : ACT8_PICK(act8_unpack_kernel);
#undef ACT8_PICK
  constexpr int64_t per = static_cast<int64_t>(kAct8Threads) * kAct8Unroll;
  const int64_t blocks = (a.total + per - 1) / per;  // below 2^31: 2^42 / 8 / 1024
  void* args[] = {&a};
  return launch_pdl(fn, dim3(static_cast<unsigned>(blocks)), dim3(kAct8Threads), 0,
                    static_cast<cudaStream_t>(stream), args) == cudaSuccess
             ? RMSN_OK
             : RMSN_ERR_CUDA;
}

}  // namespace

}  // namespace rmsn

using namespace rmsn;

extern "C" {

int64_t act8_train_row_bytes(int64_t H) { return H < 1 || H > INT32_MAX ? 0 : act8_row_size(H); }

int act8_train_pack(const void* x, int dtype, void* packed, int64_t R, int64_t H, int64_t s_row,
                    void* stream) {
  return act8_run(x, dtype, packed, R, H, s_row, true, stream);
}

int act8_train_unpack(const void* packed, void* y, int dtype, int64_t R, int64_t H,
                      void* stream) {
  return act8_run(y, dtype, packed, R, H, H, false, stream);
}

}  // extern "C"
