// act8.cu -- activations packed into 8 bits and unpacked for sm_103a, and their C ABI
// (include/act8_train.h).
//
// HBM-bound: 2 (4) + 1.03 bytes an element each way.  A thread takes groups of eight consecutive
// elements of a row, the four lanes of a block agree on its greatest magnitude by two shuffles.
// Groups are counted in multiples of four a row, so that no block straddles a warp.  Rows of one
// block are a thread's each.
// Measured: 65536 x 4096 bf16 123 us packing, 122 unpacking, a plain copy's rate over its bytes;
// 3000000 x 5 bf16 21 and 19 (18.9 of bandwidth).  Rows that start between 16-byte vectors run at two
// thirds of that rate (65536 x 2051 bf16 96 and 92 us): in 16 bits they are bound by their instructions,
// 21 an element for 14 and 10 of rows of whole vectors, in 76 % of issue slots (each group's place is
// found and its words shifted); in FP32, whose groups are loaded as three vectors and shifted by
// selections, by those and L1 together (65 to 76 % of its throughput, 62 to 71 % of issue slots).
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
  uint32_t tiles;        // wide rows: tiles of 32 groups a row
  uint32_t total;        // narrow rows: R * groups, below 2^31,
  uint32_t mul, shift;   // and division by groups: (i * mul) >> (32 + shift)
  int32_t vec;           // rows start at 16-byte vectors and are whole groups
};

// Elements of group c that the row has: 8, fewer in its last one, 0 or less behind it (a row has at
// most 2^30).
__device__ __forceinline__ int group_size(const Act8Args& a, int c) {
  return min(static_cast<int>(a.H) - 8 * c, 8);
}

template <typename T>
using Words = uint4[sizeof(T) / 2];  // a group of eight elements

// N words from `bytes` bytes on of w (bytes a multiple of the elements' size, below 16).
template <int N, int kFrom, bool kHalves>
__device__ __forceinline__ void words_from(const uint32_t (&w)[N + 4], uint32_t bytes,
                                           uint32_t (&o)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = w[i + kFrom];
  if constexpr (kHalves) {
    if (bytes & 2u) {
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = __funnelshift_r(w[i + kFrom], w[i + kFrom + 1], 16);
    }
  }
}
// kSame: bytes is the same for the whole warp (a branch instead of selections).
template <int N, bool kHalves, bool kSame>
__device__ __forceinline__ void shift_words(const uint32_t (&w)[N + 4], uint32_t bytes,
                                            uint32_t (&o)[N]) {
  if constexpr (!kSame) {
    uint32_t a[N + 2], b[N + 1];
#pragma unroll
    for (int i = 0; i < N + 2; ++i) a[i] = (bytes & 8u) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < N + 1; ++i) b[i] = (bytes & 4u) ? a[i + 1] : a[i];
#pragma unroll
    for (int i = 0; i < N; ++i)
      o[i] = kHalves ? __funnelshift_r(b[i], b[i + 1], (bytes & 2u) * 8u) : b[i];
    return;
  }
  switch (bytes >> 2) {
    case 0: words_from<N, 0, kHalves>(w, bytes, o); break;
    case 1: words_from<N, 1, kHalves>(w, bytes, o); break;
    case 2: words_from<N, 2, kHalves>(w, bytes, o); break;
    default: words_from<N, 3, kHalves>(w, bytes, o); break;
  }
}

// What memory holds of eight elements from p, of which n exist (1 to 8; none: zeros): the 16-byte
// vectors from p on, or, unless kVec, those that the elements lie in, from p's own on.
template <typename T, bool kVec>
struct Raw {
  static constexpr int kVecs = static_cast<int>(sizeof(T) / 2) + (kVec ? 0 : 1);
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        v[i] = n > 0 ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      const uint4* q = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
      const int last = n <= 0 ? 0 : static_cast<int>(at & 15u) + n * static_cast<int>(sizeof(T));
#pragma unroll
      for (int i = 0; i < kVecs; ++i) v[i] = 16 * i < last ? q[i] : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // the elements in place, zeros from element n on
  template <bool kSame>
  __device__ __forceinline__ void get(const T* p, int n, Words<T>& u) const {
    constexpr int kOut = static_cast<int>(sizeof(T) / 2);
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < kOut; ++i) u[i] = v[i];
    } else {
      uint32_t w[4 * kVecs], o[4 * kOut];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        w[4 * i] = v[i].x;
        w[4 * i + 1] = v[i].y;
        w[4 * i + 2] = v[i].z;
        w[4 * i + 3] = v[i].w;
      }
      const uint32_t bytes = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
      shift_words<4 * kOut, sizeof(T) == 2, kSame>(w, bytes, o);
#pragma unroll
      for (int i = 0; i < kOut; ++i)
        u[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    }
    if (!kVec && n < 8) {
      T* e = reinterpret_cast<T*>(u);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= n) e[i] = T(0.f);
    }
  }
};

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
__device__ __forceinline__ void store_group(T* p, int n, bool vec, const Words<T>& u) {
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

// A group's numbers.
template <typename T>
__device__ __forceinline__ uint2 numbers_of(const Words<T>& u, uint32_t amax, uint32_t scale) {
  if constexpr (sizeof(T) == 2) {
    return act8_pack8<T>(u[0], amax, scale);
  } else {
    f2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = VecOf<T>::pair(u[i >> 1], i & 1);
    return act8_pack8(v, amax, scale);
  }
}

// Group c of a packed row, from its values; the four lanes of a block call it together, `here`
// where the group is within the row's groups.
template <typename T>
__device__ __forceinline__ void pack_group(const Act8Args& a, unsigned char* row, int c, bool here,
                                           const Words<T>& u) {
  const uint32_t amax = act8_max_block(act8_max8<T>(u));
  const uint32_t s = act8_scale_byte(amax);
  if (!here) return;
  const int first_scale = static_cast<int>(act8_scale_offset(a.H));
  if (8 * c < first_scale) *reinterpret_cast<uint2*>(row + 8 * c) = numbers_of<T>(u, amax, s);
  if ((c & 3) == 0)
    row[first_scale + (c >> 2)] = static_cast<unsigned char>(s);
  else if (c + 4 > static_cast<int>(a.groups))  // the row's last block: the padding behind it
    act8_pad_scales(row + first_scale, static_cast<int>(a.groups >> 2), (c & 3) - 1);
}

// ---- wide rows: a warp takes kAct8Unroll tiles of 32 groups, rows after one another -----------
//
// kVec: rows are whole 16-byte vectors.  Else memory is read as Raw does, and written in whole vectors
// too: a lane's vector of memory holds the last elements of the lane before and its own
// first ones; what is left at the ends of rows and of the warp's tiles goes element by element.
template <typename T, bool kVec, bool kPack>
__global__ void __launch_bounds__(kAct8Threads, std::is_same_v<T, __nv_bfloat16> && kVec ? 6 : 4)
    act8_wide_kernel(const Act8Args a) {
  constexpr int kVecs = static_cast<int>(sizeof(T) / 2);
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kAct8Threads / 32) + warp) * kAct8Unroll;
  const int64_t row0 = (t0 >> 32) == 0 ? static_cast<uint32_t>(t0) / a.tiles : t0 / a.tiles;
  if (row0 >= a.R) return;
  const int c_end = static_cast<int>(a.tiles) * 32 + static_cast<int>(lane);  // behind a row
  const int c0 = static_cast<int>(t0 - row0 * a.tiles) * 32 + static_cast<int>(lane);
  const int64_t bytes = act8_row_size(a.H);
  const int first_scale = static_cast<int>(act8_scale_offset(a.H));
  unsigned char* const packed0 =
      static_cast<unsigned char*>(const_cast<void*>(kPack ? a.out : a.in)) + row0 * bytes;
  T* const wide0 = static_cast<T*>(const_cast<void*>(kPack ? a.in : a.out)) + row0 * a.s_row;
  const int rows = static_cast<int>(min(a.R - row0, static_cast<int64_t>(kAct8Unroll)));
  Raw<T, kVec> raw[kAct8Unroll];
  uint2 q[kAct8Unroll];
  uint32_t s[kAct8Unroll];
  {
    const T* wide = wide0;
    const unsigned char* packed = packed0;
    int c = c0, row = 0;
#pragma unroll
    for (int i = 0; i < kAct8Unroll; ++i) {  // every load in flight before the first is used
      const int n = row < rows ? group_size(a, c) : 0;
      if constexpr (kPack) {
        raw[i].load(wide + 8 * static_cast<int64_t>(c), n);
      } else if (n > 0) {
        q[i] = *reinterpret_cast<const uint2*>(packed + 8 * static_cast<int64_t>(c));
        s[i] = packed[first_scale + (c >> 2)];
      }
      c += 32;
      if (c == c_end) {
        c = static_cast<int>(lane);
        ++row;
        wide += a.s_row;
        packed += bytes;
      }
    }
  }
  T* wide = wide0;
  unsigned char* packed = packed0;
  int c = c0, row = 0;
  uint32_t before[4];  // lane 31's last vector of the tile before
#pragma unroll
  for (int i = 0; i < kAct8Unroll; ++i) {
    if (row == rows) return;
    const int n = group_size(a, c);
    T* p = wide + 8 * static_cast<int64_t>(c);
    Words<T> u;
    if constexpr (kPack) {
      raw[i].template get<true>(p, n, u);
      pack_group<T>(a, packed, c, c < static_cast<int>(a.groups), u);
    } else {
      if (n > 0) values_of<T>(q[i], s[i], u);
      if constexpr (kVec) {
        if (n > 0) store_group(p, n, true, u);
      } else {
        // the lane before's last vector, then own ones; from them the vectors of memory that own
        // elements begin in: their elements are `shift` places before own ones
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
        const int shift = static_cast<int>(off / sizeof(T));
        uint32_t w[4 * kVecs + 4], o[4 * kVecs];
#pragma unroll
        for (int k = 0; k < 4 * kVecs; ++k) w[4 + k] = u4_get(u[k >> 2], k & 3);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t v = __shfl_sync(0xffffffffu, w[4 * kVecs + k], (lane + 31) & 31);
          w[k] = lane == 0 && i > 0 ? before[k] : v;
          before[k] = v;
        }
        if (off != 0) {
          shift_words<4 * kVecs, sizeof(T) == 2, true>(w, 16u - off, o);
        } else {
#pragma unroll
          for (int k = 0; k < 4 * kVecs; ++k) o[k] = w[4 + k];
        }
        constexpr int kIn = static_cast<int>(16 / sizeof(T));  // elements of a vector
        // of the eight elements from p - shift on, [lo, hi) are this warp's and the row's
        const int lo = lane == 0 && (i == 0 || c == 0) ? shift : 0;
        const int hi = min(n + shift, 8);
        const T* e = reinterpret_cast<const T*>(o);
        T* d = p - shift;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          if (lo <= k * kIn && (k + 1) * kIn <= hi) {
            reinterpret_cast<uint4*>(d)[k] =
                make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          } else if (hi > k * kIn) {
#pragma unroll
            for (int x = k * kIn; x < (k + 1) * kIn; ++x)
              if (lo <= x && x < hi) d[x] = e[x];
          }
        }
        // what the next tile's first lane would write, were it the same row's and this warp's
        if (lane == 31 && (i == kAct8Unroll - 1 || c + 32 == c_end)) {
          const T* own = reinterpret_cast<const T*>(u);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (x >= 8 - shift && x < n) p[x] = own[x];
        }
      }
    }
    c += 32;
    if (c == c_end) {
      c = static_cast<int>(lane);
      ++row;
      wide += a.s_row;
      packed += bytes;
    }
  }
}

// Elements before p in its 16-byte vector.
template <typename T>
__device__ __forceinline__ int in_vector(const T* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}
// A CTA's n elements for out, staged from stage + in_vector(out) on, so that the vectors of both
// coincide.
template <typename T>
__device__ __forceinline__ void copy_out(const T* stage, T* out, int n) {
  constexpr int kIn = static_cast<int>(16 / sizeof(T));
  const int shift = in_vector(out);
  T* const base = out - shift;  // elements [shift, shift + n) of it are the CTA's
  const int end = shift + n;
  for (int i = static_cast<int>(threadIdx.x); i * kIn < end; i += kAct8Threads) {
    const int lo = i * kIn;
    if (lo >= shift && lo + kIn <= end) {
      reinterpret_cast<uint4*>(base)[i] = reinterpret_cast<const uint4*>(stage)[i];
    } else {
#pragma unroll
      for (int x = 0; x < kIn; ++x)
        if (lo + x >= shift && lo + x < end) base[lo + x] = stage[lo + x];
    }
  }
}

// ---- narrow rows: the groups of all rows side by side -----------------------------------------

template <typename T, bool kVec, bool kPack>
__global__ void __launch_bounds__(kAct8Threads) act8_flat_kernel(const Act8Args a) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const uint32_t first = blockIdx.x * (kAct8Threads * kAct8Unroll) + threadIdx.x;
  const int64_t bytes = act8_row_size(a.H);
  const uint32_t first_scale = static_cast<uint32_t>(act8_scale_offset(a.H));
  // unpacked rows between vectors: the CTA's groups, whose elements are back to back, pass through
  // shared memory
  constexpr bool kStaged = !kPack && !kVec;
  __shared__ __align__(16) T stage[kStaged ? kAct8Threads * kAct8Unroll * 8 + 8 : 1];
  auto element = [&](uint32_t group) {  // the first element of a group, or of the next row
    const int64_t r = __umulhi(group, a.mul) >> a.shift;
    return r * a.H + min(static_cast<int64_t>(8) * (group - static_cast<uint32_t>(r) * a.groups), a.H);
  };
  const int64_t at0 = kStaged ? element(blockIdx.x * (kAct8Threads * kAct8Unroll)) : 0;
  T* const out = kStaged ? static_cast<T*>(a.out) + at0 : nullptr;
  Raw<T, kVec> raw[kAct8Unroll];
  uint2 q[kAct8Unroll];
  uint32_t s[kAct8Unroll], row[kAct8Unroll];
  int c[kAct8Unroll];
#pragma unroll
  for (int i = 0; i < kAct8Unroll; ++i) {
    const uint32_t at = first + i * kAct8Threads;
    row[i] = __umulhi(at, a.mul) >> a.shift;
    c[i] = static_cast<int>(at - row[i] * a.groups);
    const int n = at < a.total ? group_size(a, c[i]) : 0;
    if constexpr (kPack) {
      raw[i].load(static_cast<const T*>(a.in) + row[i] * a.s_row + 8 * c[i], n);
    } else if (n > 0) {
      const unsigned char* p = static_cast<const unsigned char*>(a.in) + row[i] * bytes;
      q[i] = *reinterpret_cast<const uint2*>(p + 8 * c[i]);
      s[i] = p[first_scale + (c[i] >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < kAct8Unroll; ++i) {
    const bool here = first + i * kAct8Threads < a.total;
    const int n = here ? group_size(a, c[i]) : 0;
    Words<T> u;
    if constexpr (kPack) {
      raw[i].template get<false>(static_cast<const T*>(a.in) + row[i] * a.s_row + 8 * c[i], n, u);
      pack_group<T>(a, static_cast<unsigned char*>(a.out) + row[i] * bytes, c[i], here, u);
    } else if (n > 0) {
      values_of<T>(q[i], s[i], u);
      const int64_t at = row[i] * a.H + 8 * c[i];
      if constexpr (kStaged) {
        const T* e = reinterpret_cast<const T*>(u);
        T* const own = stage + in_vector(out) + static_cast<int>(at - at0);
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (x < n) own[x] = e[x];
      } else {
        store_group(static_cast<T*>(a.out) + at, n, true, u);
      }
    }
  }
  if constexpr (kStaged) {
    __syncthreads();
    const uint32_t end = min(a.total, blockIdx.x * (kAct8Threads * kAct8Unroll) +
                                          kAct8Threads * kAct8Unroll);
    copy_out(stage, out, static_cast<int>(element(end) - at0));
  }
}

// ---- rows of one block: a thread a row (of kG groups; up to 16 elements in 32 bytes, then 48) ----

template <typename T, int kG, bool kVec, bool kPack>
__global__ void __launch_bounds__(kAct8Threads) act8_block_kernel(const Act8Args a) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  // unpacked rows between vectors: the CTA's, which are back to back, pass through shared memory
  constexpr bool kStaged = !kPack && !kVec && kG > 1;
  __shared__ __align__(16) T stage[kStaged ? kAct8Threads * 8 * kG + 8 : 1];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kAct8Threads, row = row0 + threadIdx.x;
  if (!kStaged && row >= a.R) return;
  constexpr int kNumbers = kG > 2 ? 2 : 1;  // 16-byte vectors of numbers
  uint4* const packed = static_cast<uint4*>(const_cast<void*>(kPack ? a.out : a.in)) +
                        row * (kNumbers + 1);
  T* const wide = static_cast<T*>(const_cast<void*>(kPack ? a.in : a.out)) + row * a.s_row;
  uint2 q[2 * kNumbers];
  if constexpr (kStaged) {
    const int H = static_cast<int>(a.H);
    T* const own = stage + in_vector(static_cast<const T*>(a.out) + row0 * H) +
                   static_cast<int>(threadIdx.x) * H;
    if (row < a.R) {
      uint32_t words[4 * kNumbers];
#pragma unroll
      for (int i = 0; i < kNumbers; ++i) {
        const uint4 v = packed[i];
        words[4 * i] = v.x;
        words[4 * i + 1] = v.y;
        words[4 * i + 2] = v.z;
        words[4 * i + 3] = v.w;
      }
      const uint32_t s = *reinterpret_cast<const unsigned char*>(packed + kNumbers);
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        Words<T> u;
        values_of<T>(make_uint2(words[2 * g], words[2 * g + 1]), s, u);
        const T* e = reinterpret_cast<const T*>(u);
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (8 * g + x < H) own[8 * g + x] = e[x];
      }
    }
    __syncthreads();
    const int n = static_cast<int>(min(a.R - row0, static_cast<int64_t>(kAct8Threads))) * H;
    copy_out(stage, static_cast<T*>(a.out) + row0 * H, n);
  } else if constexpr (kPack) {
    Raw<T, kVec> raw[kG];
#pragma unroll
    for (int g = 0; g < kG; ++g) raw[g].load(wide + 8 * g, group_size(a, g));
    Words<T> u[kG];
    uint32_t amax = 0u;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      raw[g].template get<false>(wide + 8 * g, group_size(a, g), u[g]);
      amax = max(amax, act8_max8<T>(u[g]));
    }
    const uint32_t s = act8_scale_byte(amax);
#pragma unroll
    for (int g = 0; g < 2 * kNumbers; ++g)
      q[g] = g < kG ? numbers_of<T>(u[g < kG ? g : 0], amax, s) : make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < kNumbers; ++i)
      packed[i] = make_uint4(q[2 * i].x, q[2 * i].y, q[2 * i + 1].x, q[2 * i + 1].y);
    packed[kNumbers] = make_uint4(s, 0u, 0u, 0u);
  } else {
#pragma unroll
    for (int i = 0; i < kNumbers; ++i) {
      const uint4 v = packed[i];
      q[2 * i] = make_uint2(v.x, v.y);
      q[2 * i + 1] = make_uint2(v.z, v.w);
    }
    const uint32_t s = *reinterpret_cast<const unsigned char*>(packed + kNumbers);
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int n = group_size(a, g);
      Words<T> u;
      values_of<T>(q[g], s, u);
      if (n > 0) store_group(wide + 8 * g, n, kVec, u);
    }
  }
}

template <typename T, bool kPack>
const void* pick_block(int64_t H, bool vec) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
#define ACT8_PICK(G)                                           \
  (vec ? fn(&act8_block_kernel<T, G, true, kPack>)             \
       : fn(&act8_block_kernel<T, G, false, kPack>))
  return H <= 8 ? ACT8_PICK(1) : H <= 16 ? ACT8_PICK(2) : ACT8_PICK(4);
#undef ACT8_PICK
}

// Whether rows are taken by a thread each: those of one block, but for unpacked rows of whole vectors
// past 16 elements, which lanes side by side write better.
bool one_block(int64_t H, bool vec, bool pack) {
  return H <= (vec && !pack ? kAct8Block / 2 : kAct8Block);
}

template <typename T, bool kPack>
const void* pick_of(int64_t H, bool flat, bool vec) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
  if (one_block(H, vec, kPack)) return pick_block<T, kPack>(H, vec);
  if (flat)
    return vec ? fn(&act8_flat_kernel<T, true, kPack>) : fn(&act8_flat_kernel<T, false, kPack>);
  return vec ? fn(&act8_wide_kernel<T, true, kPack>) : fn(&act8_wide_kernel<T, false, kPack>);
}

template <bool kPack>
const void* pick(int dtype, int64_t H, bool flat, bool vec) {
  return dtype == ACT8_BF16   ? pick_of<__nv_bfloat16, kPack>(H, flat, vec)
         : dtype == ACT8_FP32 ? pick_of<float, kPack>(H, flat, vec)
                              : pick_of<__half, kPack>(H, flat, vec);
}

// Rows of at least this many groups (six blocks) are taken in tiles of 32, which are the same row's for a
// whole warp.  Three quarters of a row's one tile are then there; just past a multiple of 32 fewer,
// 36 of 64 at the least (65536 x 264 bf16 17 us packing, 14 unpacking, 8 of bandwidth; x 384, where
// three quarters are there again, 17.5 and 15.5 of 11.5).
constexpr uint32_t kAct8WideGroups = 24;
constexpr int64_t kAct8MaxH = int64_t{1} << 30;
constexpr int64_t kAct8MaxBytes = int64_t{1} << 42;  // of a packed tensor

int act8_run(const void* wide, int dtype, const void* packed, int64_t R, int64_t H, int64_t s_row,
             bool pack, void* stream) {
  if (dtype != ACT8_BF16 && dtype != ACT8_FP32 && dtype != ACT8_FP16) return RMSN_ERR_INVALID_ARG;
  if (R < 0 || H < 1 || s_row < 0) return RMSN_ERR_INVALID_ARG;
  if (H > kAct8MaxH || R > kAct8MaxBytes / act8_row_size(H)) return RMSN_ERR_UNSUPPORTED;
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
  a.vec = reinterpret_cast<uintptr_t>(wide) % 16 == 0 && a.s_row * elem % 16 == 0 && H % 8 == 0;
  const bool flat = a.groups < kAct8WideGroups;
  const void* fn = pack ? pick<true>(dtype, H, flat, a.vec) : pick<false>(dtype, H, flat, a.vec);
  const cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
  void* args[] = {&a};
  if (one_block(H, a.vec, pack)) {
    const dim3 grid(static_cast<unsigned>((R + kAct8Threads - 1) / kAct8Threads));  // 2^42 / 32 / 256
    return launch_pdl(fn, grid, dim3(kAct8Threads), 0, stream_, args) == cudaSuccess
               ? RMSN_OK
               : RMSN_ERR_CUDA;
  }
  if (!flat) {
    a.tiles = (a.groups + 31) / 32;
    constexpr int64_t per = kAct8Threads / 32 * kAct8Unroll;  // tiles a CTA
    // (a tile has 144 packed bytes at least, at H = 257: below 2^42 / 144 / 32)
    const dim3 grid(static_cast<unsigned>((R * a.tiles + per - 1) / per));
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

int64_t act8_train_row_bytes(int64_t H) { return H < 1 || H > kAct8MaxH ? 0 : act8_row_size(H); }

int act8_train_pack(const void* x, int dtype, void* packed, int64_t R, int64_t H, int64_t s_row,
                    void* stream) {
  return act8_run(x, dtype, packed, R, H, s_row, true, stream);
}

int act8_train_unpack(const void* packed, void* y, int dtype, int64_t R, int64_t H,
                      void* stream) {
  return act8_run(y, dtype, packed, R, H, H, false, stream);
}

}  // extern "C"
