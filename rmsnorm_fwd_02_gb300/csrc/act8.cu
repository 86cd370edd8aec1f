// act8.cu -- activations packed into 8 bits and unpacked for sm_103a, and their C ABI
// (include/act8_train.h).
//
// HBM-bound: 2 (4) + 1.03 bytes an element each way.  A thread takes groups of eight consecutive
// elements of a row, the four lanes of a block agree on its greatest magnitude by two shuffles.
// Groups are counted in multiples of four a row, so that no block straddles a warp.
#include <cstdint>
#include <type_traits>

#include "act8.cuh"
#include "act8_train.h"  // include/ (on the include path)

namespace rmsn {

namespace {

constexpr int kAct8Threads = 256;
constexpr int kAct8Unroll = 4;  // groups a thread has in flight

struct Act8Args {
  const void* in;
  void* out;
  int64_t R, H, s_row;   // s_row: elements between rows of the wide tensor
  uint32_t groups;       // groups a row, a multiple of 4
  uint32_t total;        // flat launches: R * groups, below 2^31,
  uint32_t mul, shift;   // and division by groups: (i * mul) >> (32 + shift)
  int32_t vec;           // 16-byte accesses are allowed
};

template <typename T>
using Words = uint4[sizeof(T) / 2];  // a group of eight elements

// Eight elements from p, of which n (1..8) exist.
template <typename T>
__device__ __forceinline__ void load_group(const T* p, int64_t n, bool vec, Words<T>& u) {
  if (vec && n >= 8) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      u[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    T* q = reinterpret_cast<T*>(u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = p[i];
  }
}

// v, or FP16's largest value of its sign where it is finite and past it (NaN stays).
__device__ __forceinline__ float within_half(float v) {
  return fabsf(v) > 65504.f ? copysignf(65504.f, v) : v;
}

template <typename T>
__device__ __forceinline__ void values_of(const uint2& q, uint32_t scale, Words<T>& u) {
  constexpr int kP = VecOf<T>::kPairs;
  f2 v[4];
  act8_unpack8(q, act8_unit(scale), v);
  if constexpr (std::is_same_v<T, __half>) {  // FP16's last values round up to 2^16: no infinity
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = f2_make(within_half(f2_lo(v[k])), within_half(f2_hi(v[k])));
  }
#pragma unroll
  for (int i = 0; i < 4 / kP; ++i) {
    f2 t[kP];
#pragma unroll
    for (int k = 0; k < kP; ++k) t[k] = v[i * kP + k];
    u[i] = VecOf<T>::pack(t);
  }
}

template <typename T>
__device__ __forceinline__ void store_group(T* p, int64_t n, bool vec, const Words<T>& u) {
  if (vec && n >= 8) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      reinterpret_cast<uint4*>(p)[i] = u[i];
  } else {
    const T* q = reinterpret_cast<const T*>(u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = q[i];
  }
}

// Group c of a packed row, from its values; the four lanes of a block call it together, `here`
// where the group is within the row's groups.
template <typename T>
__device__ __forceinline__ void pack_group(const Act8Args& a, unsigned char* row, uint32_t c, bool here,
                                           const Words<T>& u) {
  const uint32_t amax = act8_max_block(act8_max8<T>(u));
  const uint32_t s = act8_scale_byte(amax);
  if (!here) return;
  const uint32_t first_scale = static_cast<uint32_t>(act8_scale_offset(a.H));
  if (8 * c < first_scale) {
    uint2 q;
    if constexpr (sizeof(T) == 2) {
      q = act8_pack8<T>(u[0], amax, s);
    } else {
      f2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = VecOf<T>::pair(u[i >> 1], i & 1);
      q = act8_pack8(v, amax, s);
    }
    *reinterpret_cast<uint2*>(row + 8 * c) = q;
  }
  if ((c & 3) == 0) {
    unsigned char* p = row + first_scale + (c >> 2);
    *p = static_cast<unsigned char>(s);
    if (c + 4 == a.groups)  // the row's last block: the padding behind it
      for (++p; reinterpret_cast<uintptr_t>(p) & 15u; ++p) *p = 0;
  }
}

// ---- wide rows: a warp takes kAct8Unroll * 32 groups of one row -------------------------------
//
// kVec: rows start and end at 16-byte vectors.  Else a warp's 256 elements of each turn pass through
// shared memory, so that each access of memory takes 32 neighbouring elements (a place of padding
// in eight: lane l's eight elements from 9 l on, in as many banks as there are lanes).
template <typename T, bool kVec, bool kPack>
__global__ void __launch_bounds__(kAct8Threads) act8_wide_kernel(const Act8Args a) {
  __shared__ T turn[kVec ? 1 : kAct8Threads / 32][kVec ? 1 : 288];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kAct8Threads / 32) + warp;
  if (row >= a.R) return;
  const int64_t bytes = act8_row_size(a.H);
  T* wide = static_cast<T*>(const_cast<void*>(kPack ? a.in : a.out)) + row * a.s_row;
  unsigned char* packed =
      static_cast<unsigned char*>(const_cast<void*>(kPack ? a.out : a.in)) + row * bytes;
  const uint32_t first_scale = static_cast<uint32_t>(act8_scale_offset(a.H));
  for (uint32_t c0 = blockIdx.y * (32 * kAct8Unroll); c0 < a.groups;
       c0 += gridDim.y * (32 * kAct8Unroll)) {
    Words<T> u[kAct8Unroll];
    uint2 q[kAct8Unroll];
    uint32_t s[kAct8Unroll];
#pragma unroll
    for (int i = 0; i < kAct8Unroll; ++i) {  // every load in flight before the first is used
      const uint32_t c = c0 + i * 32 + lane;
      const int64_t n = a.H - 8 * static_cast<int64_t>(c);
      if constexpr (kPack) {
#pragma unroll
        for (uint4& w : u[i]) w = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (kVec) {
          if (n > 0) load_group(wide + 8 * static_cast<int64_t>(c), n, true, u[i]);
        } else {
          const int64_t at = 8 * static_cast<int64_t>(c0 + i * 32);
          T* own = reinterpret_cast<T*>(u[i]);  // for now, elements at + 32 k + lane
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (at + 32 * k + lane < a.H) own[k] = wide[at + 32 * k + lane];
        }
      } else if (n > 0) {
        q[i] = *reinterpret_cast<const uint2*>(packed + 8 * static_cast<int64_t>(c));
        s[i] = packed[first_scale + (c >> 2)];
      }
    }
#pragma unroll
    for (int i = 0; i < kAct8Unroll; ++i) {
      const uint32_t c = c0 + i * 32 + lane;
      const int64_t n = a.H - 8 * static_cast<int64_t>(c);
      T* own = reinterpret_cast<T*>(u[i]);
      const int64_t at = 8 * static_cast<int64_t>(c0 + i * 32);
      if constexpr (kPack) {
        if constexpr (!kVec) {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) turn[warp][32 * k + lane + (32 * k + lane) / 8] = own[k];
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) own[k] = turn[warp][9 * lane + k];
        }
        pack_group<T>(a, packed, c, c < a.groups, u[i]);
      } else {
        if (n > 0) values_of<T>(q[i], s[i], u[i]);
        if constexpr (kVec) {
          if (n > 0) store_group(wide + 8 * static_cast<int64_t>(c), n, true, u[i]);
        } else {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) turn[warp][9 * lane + k] = own[k];
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (at + 32 * k + lane < a.H)
              wide[at + 32 * k + lane] = turn[warp][32 * k + lane + (32 * k + lane) / 8];
        }
      }
    }
  }
}

// ---- narrow rows: the groups of all rows side by side -----------------------------------------

template <typename T, bool kPack>
__global__ void __launch_bounds__(kAct8Threads) act8_flat_kernel(const Act8Args a) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const uint32_t first = blockIdx.x * (kAct8Threads * kAct8Unroll) + threadIdx.x;
  const int64_t bytes = act8_row_size(a.H);
  const uint32_t first_scale = static_cast<uint32_t>(act8_scale_offset(a.H));
  Words<T> u[kAct8Unroll];
  uint2 q[kAct8Unroll];
  uint32_t s[kAct8Unroll], row[kAct8Unroll], c[kAct8Unroll];
#pragma unroll
  for (int i = 0; i < kAct8Unroll; ++i) {
    const uint32_t at = first + i * kAct8Threads;
    row[i] = __umulhi(at, a.mul) >> a.shift;
    c[i] = at - row[i] * a.groups;
    const int64_t n = at < a.total ? a.H - 8 * static_cast<int64_t>(c[i]) : 0;
    if constexpr (kPack) {
#pragma unroll
      for (uint4& w : u[i]) w = make_uint4(0u, 0u, 0u, 0u);
      if (n > 0)
        load_group(static_cast<const T*>(a.in) + row[i] * a.s_row + 8 * c[i], n, a.vec != 0, u[i]);
    } else if (n > 0) {
      const unsigned char* p = static_cast<const unsigned char*>(a.in) + row[i] * bytes;
      q[i] = *reinterpret_cast<const uint2*>(p + 8 * c[i]);
      s[i] = p[first_scale + (c[i] >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < kAct8Unroll; ++i) {
    const bool here = first + i * kAct8Threads < a.total;
    const int64_t n = here ? a.H - 8 * static_cast<int64_t>(c[i]) : 0;
    if constexpr (kPack) {
      pack_group<T>(a, static_cast<unsigned char*>(a.out) + row[i] * bytes, c[i], here, u[i]);
    } else if (n > 0) {
      values_of<T>(q[i], s[i], u[i]);
      store_group(static_cast<T*>(a.out) + row[i] * a.s_row + 8 * c[i], n, a.vec != 0, u[i]);
    }
  }
}

template <typename T, bool kPack>
const void* wide_fn(bool vec) {
  return vec ? reinterpret_cast<const void*>(&act8_wide_kernel<T, true, kPack>)
             : reinterpret_cast<const void*>(&act8_wide_kernel<T, false, kPack>);
}

template <bool kPack>
const void* pick(int dtype, bool flat, bool vec) {
  if (flat)
    return dtype == ACT8_BF16   ? reinterpret_cast<const void*>(&act8_flat_kernel<__nv_bfloat16, kPack>)
           : dtype == ACT8_FP32 ? reinterpret_cast<const void*>(&act8_flat_kernel<float, kPack>)
                                : reinterpret_cast<const void*>(&act8_flat_kernel<__half, kPack>);
  return dtype == ACT8_BF16   ? wide_fn<__nv_bfloat16, kPack>(vec)
         : dtype == ACT8_FP32 ? wide_fn<float, kPack>(vec)
                              : wide_fn<__half, kPack>(vec);
}

// Rows of at least this many groups are taken warp by warp: a warp's 128 are then three quarters
// there, and a row's place costs it no division.
constexpr uint32_t kAct8WideGroups = 96;
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
  a.groups = static_cast<uint32_t>((H + kAct8Block - 1) / kAct8Block * 4);
  a.vec = reinterpret_cast<uintptr_t>(wide) % 16 == 0 && a.s_row * elem % 16 == 0;
  const bool flat = a.groups < kAct8WideGroups;
  const void* fn = pack ? pick<true>(dtype, flat, a.vec) : pick<false>(dtype, flat, a.vec);
  const cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
  void* args[] = {&a};
  if (!flat) {
    constexpr int64_t warps = kAct8Threads / 32;
    const int64_t chunks = (a.groups + 32 * kAct8Unroll - 1) / (32 * kAct8Unroll);
    const dim3 grid(static_cast<unsigned>((R + warps - 1) / warps),  // below 2^42 / 776 / 8
                    static_cast<unsigned>(chunks < 65535 ? chunks : 65535));
    return launch_pdl(fn, grid, dim3(kAct8Threads), 0, stream_, args) == cudaSuccess
               ? RMSN_OK
               : RMSN_ERR_CUDA;
  }
  // groups counted in 31 bits: more rows take several launches.  Division by d = groups for i below
  // 2^31: with 2^(s-1) < d <= 2^s, (i * (floor(2^(31+s) / d) + 1)) >> (31 + s) is exact (Granlund
  // and Montgomery, "Division by invariant integers using multiplication", PLDI 1994).
  uint32_t s = 1;
  while ((uint64_t{1} << s) < a.groups) ++s;
  a.mul = static_cast<uint32_t>((uint64_t{1} << (31 + s)) / a.groups + 1);
  a.shift = s - 1;
  const int64_t most = 0x7fff0000 / a.groups;
  for (int64_t r = 0; r < R; r += most) {
    a.R = R - r < most ? R - r : most;
    a.total = static_cast<uint32_t>(a.R * a.groups);
    const int64_t at_wide = r * a.s_row * static_cast<int64_t>(elem), at_packed = r * act8_row_size(H);
    a.in = static_cast<const unsigned char*>(pack ? wide : packed) + (pack ? at_wide : at_packed);
    a.out = static_cast<unsigned char*>(const_cast<void*>(pack ? packed : wide)) +
            (pack ? at_packed : at_wide);
    constexpr uint32_t per = kAct8Threads * kAct8Unroll;
    const dim3 grid((a.total + per - 1) / per);
    if (launch_pdl(fn, grid, dim3(kAct8Threads), 0, stream_, args) != cudaSuccess)
      return RMSN_ERR_CUDA;
  }
  return RMSN_OK;
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
