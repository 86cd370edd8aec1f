// gn_common.cuh -- device helpers of the group norm kernels: activations, parameters, staging,
// and the sums over a CTA and a cluster.
#pragma once

#include <type_traits>

#include "gn_launch.h"
#include "groupnorm_train.h"
#include "ln_common.cuh"
#include "types.cuh"

namespace gnorm {

using namespace rmsn;
using lnorm::cluster_cta_rank;
using lnorm::peer_addr;

__device__ __forceinline__ float ex2_approx(float a) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ float rcp_approx(float a) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}

// 1 / (1 + exp(-z)) of a pair, to a few FP32 roundings (z below -87: 0).
__device__ __forceinline__ f2 sigmoid2(f2 z) {
  const f2 t = f2_mul(z, f2_splat(-1.44269504088896340736f));
  const f2 d = f2_add(f2_make(ex2_approx(f2_lo(t)), ex2_approx(f2_hi(t))), f2_splat(1.f));
  return f2_make(rcp_approx(f2_lo(d)), rcp_approx(f2_hi(d)));
}

__device__ __forceinline__ float normal_cdf(float z) {
  return 0.5f * (1.f + erff(z * 0.70710678118654752440f));
}
__device__ __forceinline__ float gelu_slope(float z) {
  // Phi(z) + z * phi(z)
  return __fmaf_rn(z * 0.39894228040143267794f, ex2_approx(z * z * -0.72134752044448170368f),
                   normal_cdf(z));
}

template <int kAct>
__device__ __forceinline__ f2 act2(f2 z) {
  if constexpr (kAct == GROUPNORM_ACT_SILU) return f2_mul(z, sigmoid2(z));
  if constexpr (kAct == GROUPNORM_ACT_GELU)
    return f2_make(f2_lo(z) * normal_cdf(f2_lo(z)), f2_hi(z) * normal_cdf(f2_hi(z)));
  return z;
}

// dy * act'(z)
template <int kAct>
__device__ __forceinline__ f2 act_grad2(f2 z, f2 dy) {
  if constexpr (kAct == GROUPNORM_ACT_SILU) {  // s + z s (1 - s)
    const f2 s = sigmoid2(z);
    return f2_mul(dy, f2_fma(f2_mul(z, s), f2_sub(f2_splat(1.f), s), s));
  }
  if constexpr (kAct == GROUPNORM_ACT_GELU)
    return f2_mul(dy, f2_make(gelu_slope(f2_lo(z)), gelu_slope(f2_hi(z))));
  return dy;
}

// Element i of a parameter array of dtype GROUPNORM_*.
__device__ __forceinline__ float load_param(const void* p, int dtype, int i) {
  if (dtype == GROUPNORM_FP32) return static_cast<const float*>(p)[i];
  if (dtype == GROUPNORM_BF16) return widen1(static_cast<const __nv_bfloat16*>(p)[i]);
  return widen1(static_cast<const __half*>(p)[i]);
}

// 2 kPairs consecutive floats of shared memory (16-byte aligned) as pairs.
template <int kPairs>
__device__ __forceinline__ void lds_pairs(const float* p, f2* out) {
#pragma unroll
  for (int i = 0; i < kPairs; i += 2) {
    const float4 v = *reinterpret_cast<const float4*>(p + 2 * i);
    out[i] = f2_make(v.x, v.y);
    out[i + 1] = f2_make(v.z, v.w);
  }
}

__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most `left` (0 .. 3) of this thread's latest groups are in flight.
__device__ __forceinline__ void cp_async_wait(int left) {
  if (left >= 3)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (left == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (left == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float2 ld_peer_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr)
               : "memory");
  return v;
}

// Four neighbouring floats of shared memory (16-byte aligned) as two pairs, and back.
__device__ __forceinline__ void lds_quad(const float* p, f2 (&v)[2]) { lds_pairs<2>(p, v); }
__device__ __forceinline__ void sts_quad(float* p, const f2 (&v)[2]) {
  *reinterpret_cast<float4*>(p) = make_float4(f2_lo(v[0]), f2_hi(v[0]), f2_lo(v[1]), f2_hi(v[1]));
}

// A thread's 2 kPairs column values to its place in a plane of red.
template <int kPairs>
__device__ __forceinline__ void sts_pairs(float* p, const f2* v) {
#pragma unroll
  for (int i = 0; i < kPairs; i += 2) {
    const f2 q[2] = {v[i], v[i + 1]};
    sts_quad(p + 2 * i, q);
  }
}

// Sum over the eight lanes of an aligned octet; every lane gets the same bits.
__device__ __forceinline__ float octet_sum(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the four octets of a warp, lane by lane.
__device__ __forceinline__ float across_octets(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

__device__ __forceinline__ f2 across_octets(f2 v) {
  return f2_make(across_octets(f2_lo(v)), across_octets(f2_hi(v)));
}

// f(i, vector) for i in [from, to), vectors `stride` 16-byte units apart, four loads ahead.
template <typename F>
__device__ __forceinline__ void for_staged(const uint4* p, int from, int to, int stride, F f) {
  int i = from;
  p += from * stride;
  for (; i + 4 <= to; i += 4, p += 4 * stride) {
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = p[j * stride];
#pragma unroll
    for (int j = 0; j < 4; ++j) f(i + j, u[j]);
  }
  for (; i < to; ++i, p += stride) f(i, *p);
}

// First of `places` places that rank k of a cluster takes.
__device__ __forceinline__ int rank_start(int places, int k, const GnShape& s) {
  return static_cast<int>((static_cast<int64_t>(places) * k) >> s.ctas_log2);
}

struct Smem {
  float* red;   // [2][lanes][red_stride]
  float* gm;    // [gs][2]
  float* w;     // [cs]
  float* b;     // [cs]
  float* c0;    // [cs]
  float* c1;    // [cs]
  float* col;   // [2][cs]
  float* run;   // [2][cs][2]
};
__device__ __forceinline__ Smem carve(unsigned char* base, const GnShape& s, bool bwd) {
  Smem m;
  float* p = reinterpret_cast<float*>(base + gn_stage_bytes(s, bwd) * (s.on_chip ? s.stages : 1));
  m.w = p;  // 16-byte aligned: cs is a multiple of 4
  m.b = m.w + s.cs;
  m.c0 = m.b + s.cs;
  m.c1 = m.c0 + s.cs;
  m.red = m.c1 + s.cs;
  m.col = m.red + 2 * s.lanes * red_stride(s);
  m.run = m.col + 2 * s.cs;
  m.gm = m.run + (bwd && s.on_chip ? 4 * s.cs : 0);
  return m;
}
// The slab's parameters to shared memory (no synchronization).
__device__ __forceinline__ void load_params(const GnArgs& a, float* w, float* b, int slab) {
  for (int i = threadIdx.x; i < a.s.cs; i += a.s.threads) {
    w[i] = load_param(a.w, a.wb_dtype, slab * a.s.cs + i);
    b[i] = load_param(a.b, a.wb_dtype, slab * a.s.cs + i);
  }
}

// What a thread of the statistics kernels owns.
struct Owner {
  int lane, rank, slab, rest, chunk;
  int c;            // its first channel in the slab
  int len;          // places of the chunk
  int64_t r0;       // first place of the CTA
  int rows;         // places of the CTA
  int cnt;          // places of the thread
};
template <bool kOnChip>
__device__ __forceinline__ Owner owner(const GnArgs& a) {
  const GnShape& s = a.s;
  Owner o;
  o.lane = threadIdx.x / s.vecs;
  o.c = (threadIdx.x - o.lane * s.vecs) * s.ev;
  o.rank = s.ctas > 1 ? static_cast<int>(cluster_cta_rank()) : 0;
  const int unit = blockIdx.x >> s.ctas_log2;
  o.rest = unit / s.slabs;
  o.slab = unit - o.rest * s.slabs;
  o.chunk = 0;
  o.len = static_cast<int>(a.S);
  o.r0 = 0;
  if constexpr (!kOnChip) {
    o.chunk = o.rest % s.chunks;
    o.len = s.chunk_base + (o.chunk < s.chunk_more ? 1 : 0);
    o.r0 = static_cast<int64_t>(o.chunk) * s.chunk_base + min(o.chunk, s.chunk_more);
  }
  const int start = rank_start(o.len, o.rank, s);
  o.r0 += start;
  o.rows = rank_start(o.len, o.rank + 1, s) - start;
  o.cnt = o.lane < s.lanes && o.lane < o.rows ? (o.rows - o.lane + s.lanes - 1) / s.lanes : 0;
  return o;
}

// What a thread of the second launch's kernels owns (no cluster).
__device__ __forceinline__ Owner out_owner(const GnArgs& a, int64_t* n) {
  const GnShape& s = a.s;
  Owner o;
  o.lane = threadIdx.x / s.vecs;
  o.c = (threadIdx.x - o.lane * s.vecs) * s.ev;
  o.rank = 0;
  const int unit = gridDim.x - 1 - blockIdx.x;  // backwards
  o.rest = unit / s.slabs;
  o.slab = unit - o.rest * s.slabs;
  const int sample = o.rest / s.parts;
  o.chunk = o.rest - sample * s.parts;
  *n = a.n0 + sample;
  o.len = o.rows = s.part_base + (o.chunk < s.part_more ? 1 : 0);
  o.r0 = static_cast<int64_t>(o.chunk) * s.part_base + min(o.chunk, s.part_more);
  o.cnt = o.lane < s.lanes && o.lane < o.rows ? (o.rows - o.lane + s.lanes - 1) / s.lanes : 0;
  return o;
}

// A thread's own copies through its ring: kTensors 16-byte vectors a place (tensor t's slots
// kRingGroups * kRingPlaces * threads behind tensor t - 1's), kRingPlaces places a copy group,
// kRingGroups - 1 groups on their way while one is used.
template <int kTensors>
struct Ring {
  uint4* slot;
  const unsigned char* p[kTensors];
  int64_t step[kTensors];  // bytes
  int cnt, threads, next;
  __device__ __forceinline__ void issue() {
#pragma unroll
    for (int j = 0; j < kRingPlaces; ++j, ++next) {
      if (next < cnt) {
        uint4* d = slot + (next & (kRingGroups * kRingPlaces - 1)) * threads;
#pragma unroll
        for (int t = 0; t < kTensors; ++t) {
          cp_async_16(d + t * kRingGroups * kRingPlaces * threads, p[t]);
          p[t] += step[t];
        }
      }
    }
    cp_async_commit();
  }
  __device__ __forceinline__ void start() {
    next = 0;
#pragma unroll
    for (int g = 0; g + 1 < kRingGroups; ++g) issue();
  }
  // f(place, its slots' base) for every place of the thread, in order
  template <typename F>
  __device__ __forceinline__ void run(F f) {
    for (int i = 0; i < cnt; i += kRingPlaces) {
      issue();
      cp_async_wait(kRingGroups - 1);
#pragma unroll
      for (int j = 0; j < kRingPlaces; ++j)
        if (i + j < cnt)
          f(i + j, slot + ((i + j) & (kRingGroups * kRingPlaces - 1)) * threads);
    }
  }
};
constexpr int kRingSlots = kRingGroups * kRingPlaces;

}  // namespace gnorm
