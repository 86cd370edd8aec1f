// gn_common.cuh -- device helpers of the group norm kernels: activations, parameters, staging,
// and the sums over a CTA and a cluster.
#pragma once

#include <cooperative_groups.h>

#include <utility>

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

// s = 1 / (1 + exp(-z)) of pairs, within 2^-21 of itself and, below zero, 1.25 |z| FP32 roundings
// more (the exponential's argument's); far below zero exp(-z) is infinite and s is 0.  (Two values
// can share a reciprocal, 1/a = b * 1/(ab), if exp(-z) is held to 2^62 so that ab stays finite: the
// clamp costs what the reciprocal saves, 2 % either way, and leaves z * 2^-62 where the product
// should vanish.)
template <int kPairs>
__device__ __forceinline__ void sigmoid_vec(const f2 (&z)[kPairs], f2 (&s)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const f2 t = f2_mul(z[i], f2_splat(-1.44269504088896340736f));
    const f2 d = f2_add(f2_make(ex2_approx(f2_lo(t)), ex2_approx(f2_hi(t))), f2_splat(1.f));
    s[i] = f2_make(rcp_approx(f2_lo(d)), rcp_approx(f2_hi(d)));
  }
}

// GELU, pairs, by the normal distribution's tail: a = |z|, e = exp(-z^2/2) and q = Phi(-a) =
// e t R(t) with t = 1 / (1 + 0.35 a), R a polynomial fitted to erfcx(a / sqrt 2) / (2 t) for this
// (least squares, weights raised where the error is largest).  The derivative's phi takes e again.
// (1 + erf loses the tail: all of it at z = -6 in FP32.)
struct NormalTail {
  f2 a, e, q;
};
// For 16-bit outputs: R keeps the largest (1 + a) e times its error small.  q is within 2.7e-8, and
// 1.5e-7 with the FP32 roundings, and relative to its own size within 2e-5 up to a = 5 -- far below
// a 16-bit rounding.  (erff instead: 1 x 232341 x 96 bf16, backward, 75.8 against 58.4 us;
// 38 x 979 x 480 bf16, forward, 34.9 against 28.0.)
__device__ __forceinline__ NormalTail normal_tail(f2 z) {
  NormalTail n;
  n.a = f2_make(fabsf(f2_lo(z)), fabsf(f2_hi(z)));
  const f2 d = f2_fma(n.a, f2_splat(0.35f), f2_splat(1.f));
  const f2 t = f2_make(rcp_approx(f2_lo(d)), rcp_approx(f2_hi(d)));
  const f2 x = f2_mul(f2_mul(z, z), f2_splat(-0.72134752044448170368f));
  n.e = f2_make(ex2_approx(f2_lo(x)), ex2_approx(f2_hi(x)));
  f2 r = f2_fma(t, f2_splat(0.040748097002506256f), f2_splat(-0.16716481745243073f));
  r = f2_fma(r, t, f2_splat(0.17960256338119507f));
  r = f2_fma(r, t, f2_splat(0.03882385790348053f));
  r = f2_fma(r, t, f2_splat(0.12764227390289307f));
  r = f2_fma(r, t, f2_splat(0.14100906252861023f));
  r = f2_fma(r, t, f2_splat(0.13933898508548737f));
  n.q = f2_mul(f2_mul(r, t), n.e);
  return n;
}
// For FP32 outputs: R's relative error is 1.4e-8, and exp's argument is formed to twice FP32's
// length (a rounded one costs z^2 / 2 roundings of e): q within 2^-20.5 of itself at every a.
// a ends at 32, where e is 0: a * a stays finite.
__device__ __forceinline__ NormalTail normal_tail_fp32(f2 z) {
  constexpr float kLog2e2 = 0.72134752044448170368f;  // log2(e) / 2
  constexpr float kRest = static_cast<float>(0.72134752044448170368 - double{kLog2e2});
  NormalTail n;
  n.a = f2_make(fminf(fabsf(f2_lo(z)), 32.f), fminf(fabsf(f2_hi(z)), 32.f));
  const f2 d = f2_fma(n.a, f2_splat(0.35f), f2_splat(1.f));
  const f2 t = f2_make(rcp_approx(f2_lo(d)), rcp_approx(f2_hi(d)));
  const f2 minus = f2_splat(-1.f);
  const f2 s = f2_mul(n.a, n.a), s_low = f2_fma(n.a, n.a, f2_mul(s, minus));
  const f2 x = f2_mul(s, f2_splat(-kLog2e2));
  f2 low = f2_fma(s, f2_splat(-kLog2e2), f2_mul(x, minus));
  low = f2_fma(s_low, f2_splat(-kLog2e2), low);
  low = f2_fma(s, f2_splat(-kRest), low);
  n.e = f2_make(ex2_approx(f2_lo(x)), ex2_approx(f2_hi(x)));
  n.e = f2_fma(f2_mul(low, f2_splat(0.69314718055994530942f)), n.e, n.e);
  f2 r = f2_fma(t, f2_splat(0.019322199746966362f), f2_splat(-0.10849655419588089f));
  r = f2_fma(r, t, f2_splat(0.235971599817276f));
  r = f2_fma(r, t, f2_splat(-0.22601933777332306f));
  r = f2_fma(r, t, f2_splat(0.06964033335447311f));
  r = f2_fma(r, t, f2_splat(-0.02842709608376026f));
  r = f2_fma(r, t, f2_splat(0.04841167479753494f));
  r = f2_fma(r, t, f2_splat(0.08778508752584457f));
  r = f2_fma(r, t, f2_splat(0.1225530356168747f));
  r = f2_fma(r, t, f2_splat(0.13962922990322113f));
  r = f2_fma(r, t, f2_splat(0.1396297961473465f));
  n.q = f2_mul(f2_mul(r, t), n.e);
  return n;
}
// z Phi(z) = max(z, 0) - a q (a q is 0 long before the bound on a, which an infinite z needs)
template <typename T>
__device__ __forceinline__ f2 gelu_pair(f2 z) {
  if constexpr (sizeof(T) == 2) {
    const NormalTail n = normal_tail(z);
    const f2 a = f2_make(fminf(f2_lo(n.a), 1024.f), fminf(f2_hi(n.a), 1024.f));
    return f2_sub(f2_make(fmaxf(f2_lo(z), 0.f), fmaxf(f2_hi(z), 0.f)), f2_mul(a, n.q));
  } else {
    const NormalTail n = normal_tail_fp32(z);
    // (a NaN is not below 0 and stays)
    const f2 up = f2_make(f2_lo(z) < 0.f ? 0.f : f2_lo(z), f2_hi(z) < 0.f ? 0.f : f2_hi(z));
    return f2_fma(f2_mul(n.a, f2_splat(-1.f)), n.q, up);
  }
}
// Phi(z) + z phi(z)
template <typename T>
__device__ __forceinline__ f2 gelu_slope_pair(f2 z) {
  const NormalTail n = sizeof(T) == 2 ? normal_tail(z) : normal_tail_fp32(z);
  const f2 u = f2_sub(f2_splat(1.f), n.q);
  const f2 cdf = f2_make(f2_lo(z) < 0.f ? f2_lo(n.q) : f2_lo(u),
                         f2_hi(z) < 0.f ? f2_hi(n.q) : f2_hi(u));
  return f2_fma(f2_mul(z, f2_splat(0.39894228040143267794f)), n.e, cdf);
}

// z becomes act(z); T is the output's type.
template <typename T, int kAct, int kPairs>
__device__ __forceinline__ void act_vec(f2 (&z)[kPairs]) {
  if constexpr (kAct == GROUPNORM_ACT_SILU) {
    f2 s[kPairs];
    sigmoid_vec(z, s);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) z[i] = f2_mul(z[i], s[i]);
  } else if constexpr (kAct == GROUPNORM_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) z[i] = gelu_pair<T>(z[i]);
  }
}

// dy becomes dy * act'(z).
template <typename T, int kAct, int kPairs>
__device__ __forceinline__ void act_grad_vec(const f2 (&z)[kPairs], f2 (&dy)[kPairs]) {
  if constexpr (kAct == GROUPNORM_ACT_SILU) {  // s + z (s - s^2)
    f2 s[kPairs];
    sigmoid_vec(z, s);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const f2 v = f2_fma(f2_mul(s[i], f2_splat(-1.f)), s[i], s[i]);
      dy[i] = f2_mul(dy[i], f2_fma(z[i], v, s[i]));
    }
  } else if constexpr (kAct == GROUPNORM_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      dy[i] = f2_mul(dy[i], gelu_slope_pair<T>(z[i]));
  }
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

// (staged vectors are addressed in the 32-bit shared window)
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void cp_async_wait_n() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
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

// Streamed: the lanes of a warp that join the chunks of a group: 32, fewer where the slab has more
// groups than the CTA has warps, so that a warp waits for several groups' loads at once.
__device__ __forceinline__ int join_lanes_log2(const GnShape& s) {
  const int warps = s.threads >> 5;
  return s.gs <= warps ? 5 : (s.gs <= 2 * warps ? 4 : 3);
}
// The slab's groups, up to whole warps of joining lanes.
__device__ __forceinline__ int join_groups(const GnShape& s, int lanes_log2) {
  const int a_warp = 32 >> lanes_log2;
  return (s.gs + a_warp - 1) & ~(a_warp - 1);
}
__device__ __forceinline__ float join_sum(float v, int lanes_log2) {
  for (int o = 1 << (lanes_log2 - 1); o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ f2 across_octets(f2 v) {
  return f2_make(across_octets(f2_lo(v)), across_octets(f2_hi(v)));
}

// f(vector) for i in [from, to), vectors `stride` bytes apart from p on, four loads ahead.
template <typename F>
__device__ __forceinline__ void for_staged(uint32_t p, int from, int to, uint32_t stride, F f) {
  int i = from;
  p += from * stride;
  for (; i + 4 <= to; i += 4, p += 4 * stride) {
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = lds128_at(p + j * stride);
#pragma unroll
    for (int j = 0; j < 4; ++j) f(u[j]);
  }
  for (; i < to; ++i, p += stride) f(lds128_at(p));
}
// The same over pairs of vectors, the second `off` bytes behind the first, two pairs ahead.
template <typename F>
__device__ __forceinline__ void for_staged2(uint32_t p, uint32_t off, int from, int to,
                                            uint32_t stride, F f) {
  int i = from;
  p += from * stride;
  for (; i + 2 <= to; i += 2, p += 2 * stride) {
    uint4 u[2], v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u[j] = lds128_at(p + j * stride);
      v[j] = lds128_at(p + j * stride + off);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) f(u[j], v[j]);
  }
  if (i < to) f(lds128_at(p), lds128_at(p + off));
}

// First of `places` places that rank k of a cluster takes.
__device__ __forceinline__ int rank_start(int places, int k, const GnShape& s) {
  return static_cast<int>((static_cast<int64_t>(places) * k) >> s.ctas_log2);
}

struct Smem {
  float* red;   // [2][lanes][red_stride]
  float* gm;    // [gs][2]
  float* ms;    // [gs][2]
  float* w;     // [cs]
  float* b;     // [cs]
  float* c0;    // [cs]
  float* c1;    // [cs]
  float* col;   // [2][cs]
  float* run;   // [2][cs][2]
};
__device__ __forceinline__ Smem carve(unsigned char* base, const GnShape& s, bool bwd) {
  Smem m;
  float* p = reinterpret_cast<float*>(base + gn_front_bytes(s, bwd));
  m.w = p;  // 16-byte aligned: cs is a multiple of 4
  m.b = m.w + s.cs;
  m.c0 = m.b + s.cs;
  m.c1 = m.c0 + s.cs;
  m.col = m.c1 + s.cs;
  m.run = m.col + 2 * s.cs;
  m.gm = m.run + (bwd && s.on_chip ? 4 * s.cs : 0);
  m.ms = m.gm + 2 * s.gs;
  m.red = s.on_chip ? m.gm + 4 * s.gs : reinterpret_cast<float*>(base);
  return m;
}
// The slab's parameters to shared memory (no synchronization).
__device__ __forceinline__ void load_params(const GnArgs& a, float* w, float* b, int slab) {
  for (int i = threadIdx.x; i < a.s.cs; i += a.s.threads) {
    w[i] = load_param(a.w, a.wb_dtype, slab * a.s.cs + i);
    b[i] = load_param(a.b, a.wb_dtype, slab * a.s.cs + i);
  }
}

// What a thread owns of its kernel's work.
struct Owner {
  int lane, rank, slab, chunk;
  int64_t n;        // (first) sample
  int c;            // its first channel in the slab
  int len;          // places of the chunk
  int64_t r0;       // first place of the CTA
  int rows;         // places of the CTA
  int cnt;          // places of the thread
};
__device__ __forceinline__ void set_lane(Owner& o, const GnShape& s) {
  o.lane = threadIdx.x / s.vecs;
  o.c = (threadIdx.x - o.lane * s.vecs) * s.ev;
}
__device__ __forceinline__ void set_count(Owner& o, const GnShape& s) {
  o.cnt = o.lane < s.lanes && o.lane < o.rows ? (o.rows - o.lane + s.lanes - 1) / s.lanes : 0;
}
__device__ __forceinline__ Owner on_chip_owner(const GnArgs& a) {
  const GnShape& s = a.s;
  Owner o;
  set_lane(o, s);
  o.rank = s.ctas > 1 ? static_cast<int>(cluster_cta_rank()) : 0;
  const int cluster = blockIdx.x >> s.ctas_log2, first = cluster / s.slabs;
  o.n = first;
  o.slab = cluster - first * s.slabs;
  o.chunk = 0;
  o.len = static_cast<int>(a.S);
  const int start = rank_start(o.len, o.rank, s);
  o.r0 = start;
  o.rows = rank_start(o.len, o.rank + 1, s) - start;
  set_count(o, s);
  return o;
}
// Piece v of a turn that starts at unit u0 and takes nu: neighbouring pieces are neighbouring
// slabs of the same places.
__device__ __forceinline__ void set_piece(Owner& o, const GnArgs& a, int u0, int nu, int v) {
  const GnShape& s = a.s;
  o.rank = 0;
  o.chunk = v / nu;
  const int u = u0 + (v - o.chunk * nu), n = u / s.slabs;
  o.n = n;
  o.slab = u - n * s.slabs;
  o.len = o.rows = s.chunk_base + (o.chunk < s.chunk_more ? 1 : 0);
  o.r0 = static_cast<int64_t>(o.chunk) * s.chunk_base + min(o.chunk, s.chunk_more);
  set_count(o, s);
}

// A thread's own copies through its ring: kTensors 16-byte vectors a place (tensor t's slots
// kSlots strides behind tensor t - 1's), kRingPlaces places a copy group, kGroups - 1 groups on
// their way while one is used.
template <int kTensors>
struct Ring {
  static constexpr int kGroups = ring_groups(kTensors), kSlots = ring_slots(kTensors);
  uint32_t slot;           // this thread's first slot (shared window)
  uint32_t stride;         // bytes from slot to slot
  const unsigned char* p[kTensors];
  int64_t step[kTensors];  // bytes from place to place
  int left;                // places not issued yet

  __device__ __forceinline__ void copy(uint32_t d) {
#pragma unroll
    for (int t = 0; t < kTensors; ++t) {
      cp_async_16(d + t * kSlots * stride, p[t]);
      p[t] += step[t];
    }
  }
  __device__ __forceinline__ void issue(uint32_t d) {  // a group that may pass the end
#pragma unroll
    for (int j = 0; j < kRingPlaces; ++j)
      if (left > j) copy(d + j * stride);
    left -= kRingPlaces;
    cp_async_commit();
  }
  __device__ __forceinline__ void start() {
#pragma unroll
    for (int g = 0; g + 1 < kGroups; ++g) issue(slot + g * kRingPlaces * stride);
  }
  // f(its slot) for each of the thread's cnt places in order
  template <typename F>
  __device__ __forceinline__ void run(int cnt, F f) {
    const uint32_t group = kRingPlaces * stride, end = slot + kSlots * stride;
    uint32_t rd = slot, wr = end - group;
    int i = 0;
    for (; left >= kRingPlaces; left -= kRingPlaces, i += kRingPlaces) {  // whole groups
#pragma unroll
      for (int j = 0; j < kRingPlaces; ++j) copy(wr + j * stride);
      cp_async_commit();
      wr = wr + group == end ? slot : wr + group;
      cp_async_wait_n<kGroups - 1>();
#pragma unroll
      for (int j = 0; j < kRingPlaces; ++j) f(rd + j * stride);
      rd = rd + group == end ? slot : rd + group;
    }
    for (; i < cnt; i += kRingPlaces) {
      issue(wr);
      wr = wr + group == end ? slot : wr + group;
      cp_async_wait_n<kGroups - 1>();
#pragma unroll
      for (int j = 0; j < kRingPlaces; ++j)
        if (i + j < cnt) f(rd + j * stride);
      rd = rd + group == end ? slot : rd + group;
    }
  }
};

}  // namespace gnorm
