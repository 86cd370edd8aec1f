// blk_common.cuh -- device code shared by the forward and backward kernels of a block's boundary.
//
// Staging: a CTA is a number of teams, each with a contiguous run of rows and a ring of its own
// in shared memory that bulk asynchronous copies fill; the team's first thread starts a slot's
// next copies as soon as the team is known to be done with it: one-warp teams after a __syncwarp
// behind the slot, others behind the next slot's first reduction, whose barrier every warp reaches
// only after its last read.  There is no producer warp, and
// a slot is held for one row's work only: the rest of the ring is on its way.
#pragma once

#include "act8.cuh"
#include "blk_launch.h"
#include "rmsn_tmem.cuh"
#include "types.cuh"

namespace blk {

using namespace rmsn;  // f2, the barriers and copies of rmsn_common.cuh, VecOf

// The 8 values from element 8 * c on of a vector of dtype code 0 (BF16), 1 (FP32) or 2 (FP16).
__device__ __forceinline__ void load8(const void* p, int code, int64_t c, f2 (&f)[4]) {
  if (code == 1) {
    const float4* q = static_cast<const float4*>(p) + 2 * c;
    const float4 a = __ldg(q), b = __ldg(q + 1);
    f[0] = f2_make(a.x, a.y);
    f[1] = f2_make(a.z, a.w);
    f[2] = f2_make(b.x, b.y);
    f[3] = f2_make(b.z, b.w);
  } else {
    const uint4 u = __ldg(static_cast<const uint4*>(p) + c);
    if (code == 0)
      VecOf<__nv_bfloat16>::unpack(u, f);
    else
      VecOf<__half>::unpack(u, f);
  }
}
__device__ __forceinline__ float load1(const void* p, int code, int64_t i) {
  if (code == 1) return static_cast<const float*>(p)[i];
  return code == 0 ? widen1(static_cast<const __nv_bfloat16*>(p)[i])
                   : widen1(static_cast<const __half*>(p)[i]);
}

// s + err == a + b exactly (Knuth).
__device__ __forceinline__ float add_exact(float a, float b, float& err) {
  const float s = __fadd_rn(a, b);
  const float bp = __fsub_rn(s, a);
  const float ap = __fsub_rn(s, bp);
  err = __fadd_rn(__fsub_rn(a, ap), __fsub_rn(b, bp));
  return s;
}

// The elementwise products of two words of two 16-bit values each, as an FP32 pair: exact (in BF16 16
// bits, in FP16 22), by mixed-precision fma that reads the halves without a conversion.
template <typename T>
__device__ __forceinline__ f2 mul_exact(uint32_t a, uint32_t b) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    return bf2_mul_exact(a, b);
  } else {
    f2 r;
    asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\t.reg .f32 p0, p1;\n\t"
        "mov.b32 {a0, a1}, %1;\n\tmov.b32 {b0, b1}, %2;\n\t"
        "fma.rn.f32.f16 p0, a0, b0, 0f80000000;\n\t"
        "fma.rn.f32.f16 p1, a1, b1, 0f80000000;\n\t"
        "mov.b64 %0, {p0, p1};\n\t}"
        : "=l"(r.v)
        : "r"(a), "r"(b));
    return r;
  }
}
// acc + a * a, likewise (the square is exact).
template <typename T>
__device__ __forceinline__ f2 square_onto(uint32_t a, f2 acc) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    return bf2_sq_acc(a, acc);
  } else {
    f2 r;
    asm("{\n\t.reg .b16 a0, a1;\n\t.reg .f32 c0, c1, p0, p1;\n\t"
        "mov.b32 {a0, a1}, %1;\n\tmov.b64 {c0, c1}, %2;\n\t"
        "fma.rn.f32.f16 p0, a0, a0, c0;\n\t"
        "fma.rn.f32.f16 p1, a1, a1, c1;\n\t"
        "mov.b64 %0, {p0, p1};\n\t}"
        : "=l"(r.v)
        : "r"(a), "l"(acc.v));
    return r;
  }
}

// scale * gate * w_post of a thread's columns (each factor where it is there), sample n's gate.
template <int VPT, bool kPostW>
__device__ __forceinline__ void load_factor(const Args& a, int32_t n, int lt, f2 (&k1)[VPT][4]) {
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = lt + v * a.ntg;
#pragma unroll
    for (int q = 0; q < 4; ++q) k1[v][q] = f2_splat(a.scale);
    if (8 * c < a.H) {
      f2 t[4];
      if (a.gate != nullptr) {
        load8(a.gate, a.gate_dtype, static_cast<int64_t>(n) * (a.H >> 3) + c, t);
#pragma unroll
        for (int q = 0; q < 4; ++q) k1[v][q] = f2_mul(k1[v][q], t[q]);
      }
      if constexpr (kPostW) {
        load8(a.w_post, a.w_dtype, c, t);
#pragma unroll
        for (int q = 0; q < 4; ++q) k1[v][q] = f2_mul(k1[v][q], t[q]);
      }
    }
  }
}

__device__ __forceinline__ float sum8(const f2 (&f)[4]) {
  const f2 s = f2_add(f2_add(f[0], f[1]), f2_add(f[2], f[3]));
  return f2_lo(s) + f2_hi(s);
}

// A thread's place in its CTA, its team's rows, ring and reductions.
struct Team {
  uint32_t ring;        // shared address of the team's slots
  uint32_t zero;        // shared address of 16 bytes of zeros, what vectors that are not there read
  uint64_t* full;       // its barriers
  float* red;           // [2][16]: warp sums, taken in turns
  volatile int* abort_flag;
  uint32_t* tmem;       // shared word: the tensor memory's address
  int32_t r0, r1;       // first row; end of the rows
  int32_t stride;       // rows between two of its slots' first
  int32_t nslots;
  int64_t k;            // among all teams (taking turns: the CTA)
  int lt;               // thread of the row
  int sub;              // row of the warp (teams of a part of a warp)
  int team;             // of the CTA
  int warps;            // of the team
  int turn;             // of red
  int32_t issued;       // slots (the leader's)
  bool leader;
};

// bulk_g2s with the shared address as such.
__device__ __forceinline__ void bulk_g2s_at(uint32_t dst, const void* src, uint32_t bytes,
                                            uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint2 lds64_at(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8_at(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// The copies of slot j of the team's rows (its leader; nothing once a wait has given up).
template <int kTensors>
__device__ __forceinline__ void issue(const Args& a, Team& t, int32_t j, uint64_t pol) {
  if (*t.abort_flag) return;
  t.issued = j + 1;
  const int s = j % a.stages;
  const int32_t ra = t.r0 + j * t.stride;
  const int32_t n = min(a.rows, t.r1 - ra);
  uint32_t row = 0;
#pragma unroll
  for (int i = 0; i < kTensors; ++i)
    if (a.in[i].p != nullptr) row += a.in[i].bytes;
  mbar_arrive_expect_tx(&t.full[s], row * static_cast<uint32_t>(n));
  const uint32_t dst = t.ring + static_cast<uint32_t>(s) * a.slot;
#pragma unroll
  for (int i = 0; i < kTensors; ++i) {
    const Staged& in = a.in[i];
    if (in.p == nullptr) continue;
    const unsigned char* src = in.p + static_cast<int64_t>(ra) * in.stride;
    if (in.stride == in.bytes) {
      bulk_g2s_at(dst + in.off, src, in.bytes * static_cast<uint32_t>(n), &t.full[s], pol);
    } else {
      for (int32_t r = 0; r < n; ++r)
        bulk_g2s_at(dst + in.off + static_cast<uint32_t>(r) * in.bytes, src + r * in.stride, in.bytes,
                    &t.full[s], pol);
    }
  }
}

// Sets the CTA up; returns with the team's first slots on their way.
// turns: a CTA's teams take the slots of its rows in turns (neighbouring rows at one time are
// fewer streams of memory: 65536 x 1536 forward 151 us against 157); else each has a run of its
// own.
// kTmem: columns of tensor memory that the CTA takes (0: none).
template <int kTensors, int kTmem = 0>
__device__ __forceinline__ Team team_begin(const Args& a, unsigned char* smem, uint64_t pol,
                                           bool turns) {
  Team t;
  const int tid = static_cast<int>(threadIdx.x);
  const int per = a.ntg < 32 ? 32 : a.ntg;  // threads of a team
  t.team = tid / per;
  const int in_team = tid - t.team * per;
  t.lt = a.ntg < 32 ? in_team % a.ntg : in_team;
  t.sub = a.ntg < 32 ? in_team / a.ntg : 0;
  t.warps = per >> 5;
  t.turn = 0;
  t.issued = 0;
  t.leader = in_team == 0;
  const size_t ring = static_cast<size_t>(a.stages) * a.slot;
  unsigned char* behind = smem + ring * a.teams;
  t.ring = smem_u32(smem + ring * t.team);
  uint64_t* full = reinterpret_cast<uint64_t*>(behind);
  t.full = full + t.team * a.stages;
  float* red = reinterpret_cast<float*>(behind + ((8 * a.teams * a.stages + 15) & ~15));
  t.red = red + 2 * kMaxWarps * t.team;
  uint4* zero = reinterpret_cast<uint4*>(red + 2 * kMaxWarps * a.teams);
  t.zero = smem_u32(zero);
  t.abort_flag = reinterpret_cast<volatile int*>(zero + 1);
  if (tid == 0) *zero = make_uint4(0u, 0u, 0u, 0u);
  for (int i = tid; i < 2 * kMaxWarps * a.teams; i += static_cast<int>(blockDim.x)) red[i] = 0.f;
  for (int i = tid; i < a.teams * a.stages; i += static_cast<int>(blockDim.x)) mbar_init(&full[i], 1u);
  t.tmem = reinterpret_cast<uint32_t*>(zero + 1) + 2;
  if (tid == 0) *t.abort_flag = 0;
  fence_barrier_init();
  if constexpr (kTmem > 0) {
    if (tid < 32) {
      __syncwarp();
      tmem_alloc_warp(t.tmem, kTmem);
      tmem_fence_before_sync();
    }
  }
  __syncthreads();
  if constexpr (kTmem > 0) tmem_fence_after_sync();
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  if (turns) {
    t.k = blockIdx.x;
    t.stride = a.teams * a.rows;
    t.r0 = team_row(t.k, a.R, gridDim.x) + t.team * a.rows;
    t.r1 = team_row(t.k + 1, a.R, gridDim.x);
  } else {
    const int64_t all = static_cast<int64_t>(gridDim.x) * a.teams;
    t.k = static_cast<int64_t>(blockIdx.x) * a.teams + t.team;
    t.stride = a.rows;
    t.r0 = team_row(t.k, a.R, all);
    t.r1 = team_row(t.k + 1, a.R, all);
  }
  t.nslots = t.r1 > t.r0 ? (t.r1 - t.r0 + t.stride - 1) / t.stride : 0;
  if (t.leader)
    for (int32_t j = 0; j < a.stages && j < t.nslots; ++j) issue<kTensors>(a, t, j, pol);
  return t;
}

__device__ __forceinline__ void wait_slot(const Args& a, const Team& t, int s, uint32_t parity) {
  mbar_wait_bounded(&t.full[s], parity, t.abort_flag, a.err, kErrConsumerWait);
}

// After a wait that gave up: no copy may still write this CTA's shared memory when it exits.
__device__ __forceinline__ void drain(const Args& a, const Team& t) {
  if (*t.abort_flag && t.leader) mbar_drain(t.full, a.stages, t.issued);
}

// Eight consecutive columns of this thread's lane of tensor memory <-> r.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const f2 (&r)[4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "f"(f2_lo(r[0])), "f"(f2_hi(r[0])), "f"(f2_lo(r[1])), "f"(f2_hi(r[1])), "f"(f2_lo(r[2])),
      "f"(f2_hi(r[2])), "f"(f2_lo(r[3])), "f"(f2_hi(r[3]))
      : "memory");
}

// Sum over the threads of a row; every one of them gets the same bits.
__device__ __forceinline__ float row_sum(const Args& a, Team& t, float v) {
  if (a.ntg <= 32) return subwarp_allsum(v, a.ntg);
  v = warp_allsum(v);
  float* red = t.red + kMaxWarps * t.turn;
  t.turn ^= 1;
  if ((threadIdx.x & 31) == 0) red[t.lt >> 5] = v;
  named_bar_sync(static_cast<uint32_t>(t.team) + 1u, static_cast<uint32_t>(a.ntg));
  // places behind the team's warps hold zeros
  const float4* q = reinterpret_cast<const float4*>(red);
  float4 s = q[0];
  v = (s.x + s.y) + (s.z + s.w);
  if (t.warps > 4) {
    s = q[1];
    v += (s.x + s.y) + (s.z + s.w);
    if (t.warps > 8) {
      s = q[2];
      v += (s.x + s.y) + (s.z + s.w);
      if (t.warps > 12) {
        s = q[3];
        v += (s.x + s.y) + (s.z + s.w);
      }
    }
  }
  return v;
}

// 1 / sqrt(sum / H + eps): the hardware's estimate and one Newton step, within two units of the
// last place (the correctly rounded root takes some twenty instructions a row and thread more).
// A mean of 0 (with eps 0), infinity or NaN keeps the estimate: infinity, 0, NaN.
__device__ __forceinline__ float row_rstd(float sum, float inv_h, float eps) {
  const float m = __fmaf_rn(sum, inv_h, eps);
  const float y = rsqrtf(m);
  const float e = __fmaf_rn(-m * y, y, 1.f);
  return e == e && fabsf(e) < 1.f ? __fmaf_rn(0.5f * y, e, y) : y;
}

}  // namespace blk
