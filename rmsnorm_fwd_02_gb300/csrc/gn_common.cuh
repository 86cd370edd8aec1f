// gn_common.cuh -- device helpers of the group norm kernels: activations, parameters, and the
// sums over a CTA and a cluster.
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

// 1 / (1 + exp(-z)) of a pair, to a few FP32 roundings.  16-bit activations share one
// reciprocal between the two (1/a = b * 1/(ab)); exp(-z) is held to 2^62 so that ab stays
// finite, which leaves sigmoid below 2^-62 at 2^-62 -- and the smaller (the clamp) of a NaN
// and 62 is 62, so neither element's NaN reaches the other through the product (it stays in z).
template <typename T>
__device__ __forceinline__ f2 sigmoid2(f2 z) {
  const f2 t = f2_mul(z, f2_splat(-1.44269504088896340736f));
  if constexpr (sizeof(T) == 2) {
    const float a = 1.f + ex2_approx(fminf(f2_lo(t), 62.f));
    const float b = 1.f + ex2_approx(fminf(f2_hi(t), 62.f));
    const float r = rcp_approx(a * b);
    return f2_make(r * b, r * a);
  } else {
    return f2_make(rcp_approx(1.f + ex2_approx(f2_lo(t))), rcp_approx(1.f + ex2_approx(f2_hi(t))));
  }
}

__device__ __forceinline__ float normal_cdf(float z) {
  return 0.5f * (1.f + erff(z * 0.70710678118654752440f));
}
__device__ __forceinline__ float gelu_slope(float z) {
  // Phi(z) + z * phi(z)
  return __fmaf_rn(z * 0.39894228040143267794f, ex2_approx(z * z * -0.72134752044448170368f),
                   normal_cdf(z));
}

template <typename T, int kAct>
__device__ __forceinline__ f2 act2(f2 z) {
  if constexpr (kAct == GROUPNORM_ACT_SILU) return f2_mul(z, sigmoid2<T>(z));
  if constexpr (kAct == GROUPNORM_ACT_GELU)
    return f2_make(f2_lo(z) * normal_cdf(f2_lo(z)), f2_hi(z) * normal_cdf(f2_hi(z)));
  return z;
}

// dy * act'(z)
template <typename T, int kAct>
__device__ __forceinline__ f2 act_grad2(f2 z, f2 dy) {
  if constexpr (kAct == GROUPNORM_ACT_SILU) {  // s + z s (1 - s)
    const f2 s = sigmoid2<T>(z);
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

// First place of piece k of `pieces` of `places` places.
__device__ __forceinline__ int64_t piece_start(int64_t places, int64_t k, int64_t pieces) {
  return places * k / pieces;
}

struct Smem {
  float* red;
  float* parts;
  float* gm;      // [gs][2]
  float2* all;    // [gs][ctas]
  float* gf;      // [gs][2]
  float* col;     // [2][cs]
  float* run;     // [2][cs][2]
};
__device__ __forceinline__ Smem carve(unsigned char* base, const GnShape& s, bool bwd) {
  Smem m;
  float* p = reinterpret_cast<float*>(base + gn_stage_bytes(s, bwd));
  m.red = p;
  p += (bwd ? 2 : 1) * s.threads * s.ev;
  // pairs of floats from here on, but for `parts`, which goes last
  m.gm = p;
  p += 2 * s.gs;
  m.all = reinterpret_cast<float2*>(p);
  p += 2 * s.gs * s.ctas;
  m.gf = p;
  p += 2 * s.gs;
  m.col = p;
  p += bwd ? 2 * s.cs : 0;
  m.run = p;
  p += bwd && s.on_chip ? 4 * s.cs : 0;
  m.parts = p;
  return m;
}

// Sums of red [lanes][cs] over the lanes and channels of each group, in a fixed order, to
// out[2 g] (stride 2).  Warps share a group's values evenly, then one thread a group adds the
// warps' parts.  Starts and ends with the CTA synchronized.
__device__ __forceinline__ void group_sums(const Smem& m, const GnShape& s, float* out) {
  __syncthreads();
  const int nw = s.threads >> 5, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = s.gs < nw ? nw / s.gs : 1;  // warps a group
  const int n = s.lanes * s.cg;
  for (int t = w; t < s.gs * per; t += nw) {
    const int g = t / per, k = t - g * per;
    const float* src = m.red + g * s.cg;
    float acc = 0.f;
    for (int i = k * 32 + lane; i < n; i += per * 32) {
      const int l = i / s.cg;
      acc += src[l * s.cs + (i - l * s.cg)];
    }
    acc = warp_allsum(acc);
    if (lane == 0) m.parts[t] = acc;
  }
  __syncthreads();
  for (int g = threadIdx.x; g < s.gs; g += s.threads) {
    float acc = 0.f;
    for (int k = 0; k < per; ++k) acc += m.parts[g * per + k];
    out[2 * g] = acc;
  }
  __syncthreads();
}

// Gathers every cluster CTA's group values m.gm into m.all[g][k].  Starts and ends with the
// CTA synchronized; the caller pairs the arrival made here, after its reads, with a
// cluster_wait() before gm changes or the CTA exits.
__device__ __forceinline__ void gather_cluster(const Smem& m, const GnShape& s) {
  if (s.ctas > 1) {
    cluster_arrive();
    cluster_wait();
    for (int i = threadIdx.x; i < s.gs * s.ctas; i += s.threads) {
      const int g = i / s.ctas, k = i - g * s.ctas;
      m.all[i] = ld_peer_f2(peer_addr(m.gm + 2 * g, static_cast<uint32_t>(k)));
    }
    cluster_arrive();
  } else {
    for (int g = threadIdx.x; g < s.gs; g += s.threads)
      m.all[g] = make_float2(m.gm[2 * g], m.gm[2 * g + 1]);
  }
  __syncthreads();
}
__device__ __forceinline__ void release_cluster(const GnShape& s) {
  if (s.ctas > 1) cluster_wait();
}

// The group of channel c of a slab.
__device__ __forceinline__ int group_of(const GnShape& s, int c) { return c / s.cg; }

}  // namespace gnorm
