// gn_fwd.cu -- group norm training forward with an activation, channels last, for sm_103a
// (include/groupnorm_train.h gives the formulas).
//
// HBM-bound: one read and one write of the activation.  Where a cluster's shared memory holds
// a sample's slab (gn_launch.h), x is read once: asynchronous 16-byte copies stage each
// thread's own vectors (the next samples' on their way meanwhile), the cluster's CTAs exchange
// a few floats a group, and the staged vectors are normalized and written.  Larger samples are
// streamed: a cooperative grid takes some tens of megabytes of their slabs at a time, sums them,
// meets at a barrier, and reads x again, as far as it goes from L2, for the output.  (Two launches
// instead, with their ramps, cost 5 us each more.)
//
// Measured (SiLU): on chip 8 x 4096 x 320 bf16 14.6 us, of which about 5 are the launch's ramp
// and 6 the bandwidth's; streamed 1 x 262144 x 128 fp32 66 us, where L2 gives back 58 MB of the
// 134 and the rest of x is read twice (60 us at a copy's rate).
//
// Statistics: each thread sums its channels' values less K, the middle one of its first three (of
// kFewPlaces and fewer, the first): sum d and sum d^2 of d = x - K, so neither sum cancels when the
// mean is far from zero.  A column's mean is K + sum d / n and its M2 = sum d^2 - (sum d)^2 / n.
// (With the first value as K everywhere, one value a thousand times the others' spread there, as
// an activation at place 0 can be, leaves n (x - K)^2 to cancel: 2.7e-5 of rstd lost at
// 1 x 262144 x 128 fp32.)  Means combine weighted by their counts, and M2 about the combined mean:
// M2 = sum of M2_i + n_i (mean_i - mean)^2 -- from threads to columns, groups, the cluster or the
// chunks.
#include "gn_common.cuh"

namespace gnorm {

// The middle one of three values, for both of a pair (a NaN is passed over).
__device__ __forceinline__ float middle(float a, float b, float c) {
  return fmaxf(fminf(a, b), fminf(fmaxf(a, b), c));
}
__device__ __forceinline__ f2 middle(f2 a, f2 b, f2 c) {
  return f2_make(middle(f2_lo(a), f2_lo(b), f2_lo(c)), middle(f2_hi(a), f2_hi(b), f2_hi(c)));
}

// Places a thread up to which K is its first value: n (x - K)^2 of so few costs 1e-6 of rstd at
// most, and small samples feel two loads more (3 % at 1024 x 49 x 512).
constexpr int kFewPlaces = 8;

template <typename T>
struct ColumnStats {
  static constexpr int kPairs = VecOf<T>::kPairs;
  f2 nk[kPairs], s[kPairs], q[kPairs];  // -K, sum d, sum d^2
  // K from the thread's first place, or its first three, `stride` bytes apart
  __device__ __forceinline__ void start(uint32_t slot, uint32_t stride, bool three) {
    f2 k[kPairs];
    VecOf<T>::unpack(lds128_at(slot), k);
    if (three) {
      f2 x1[kPairs], x2[kPairs];
      VecOf<T>::unpack(lds128_at(slot + stride), x1);
      VecOf<T>::unpack(lds128_at(slot + 2u * stride), x2);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) k[i] = middle(k[i], x1[i], x2[i]);
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      nk[i] = f2_mul(k[i], f2_splat(-1.f));
      s[i] = q[i] = f2_splat(0.f);
    }
  }
  __device__ __forceinline__ void add(const uint4& u) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const f2 d = VecOf<T>::plus(u, i, nk[i]);
      s[i] = f2_add(s[i], d);
      q[i] = f2_fma(d, d, q[i]);
    }
  }
};

__device__ __forceinline__ float clamp_below(float v) { return v < 0.f ? 0.f : v; }  // NaN stays

// A thread's constants for its channels: z = (x - mean) * scale + bias, scale = rstd * w.
template <typename T>
struct Consts {
  static constexpr int kPairs = VecOf<T>::kPairs;
  f2 nm[kPairs], scale[kPairs], bias[kPairs];
  __device__ __forceinline__ void load(const float* c0, const float* c1, const float* b, int c) {
    lds_pairs<kPairs>(c0 + c, nm);
    lds_pairs<kPairs>(c1 + c, scale);
    lds_pairs<kPairs>(b + c, bias);
  }
  template <int kAct>
  __device__ __forceinline__ uint4 norm(const uint4& u) const {
    f2 z[kPairs];
#pragma unroll
    for (int h = 0; h < kPairs; h += 2) {  // four values at a time
      f2 v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = f2_fma(VecOf<T>::plus(u, h + i, nm[h + i]), scale[h + i], bias[h + i]);
      act_vec<T, kAct>(v);
      z[h] = v[0];
      z[h + 1] = v[1];
    }
    return VecOf<T>::pack(z);
  }
};

// Channel constants of group g of the slab, lane k of `lanes` threads.
__device__ __forceinline__ void set_group(const Smem& m, const GnShape& s, int g, int k, int lanes,
                                          float mean, float rstd) {
  for (int i = g * s.cg + k; i < (g + 1) * s.cg; i += lanes) {
    m.c0[i] = -mean;
    m.c1[i] = rstd * m.w[i];
  }
}

// The CTA's group values (mean, M2) to m.gm from its threads' statistics: columns over the
// lanes, then groups over their columns (an octet of threads a group).  A warp takes eight
// quads of columns, four lanes of each at a time: wide loads, and the other warps' issue slots
// stay free.  A column's lanes combine about r, the mean of one of them in the middle (not that with
// place 0): with d = mean_l - r, mean = r + sum n_l d / n and
// M2 = sum (M2_l + n_l d^2) - (sum n_l d)^2 / n; what that can cancel is at most the lanes over a
// lane's places times the rest.
template <typename T>
__device__ __forceinline__ void cta_stats(const Smem& m, const GnShape& s, const Owner& o,
                                          const ColumnStats<T>& st) {
  constexpr int NP = VecOf<T>::kPairs;
  const int rs = red_stride(s), plane = s.lanes * rs;
  if (o.lane < s.lanes) {
    const f2 ic = f2_splat(o.cnt > 0 ? 1.f / static_cast<float>(o.cnt) : 0.f);
    f2 mean[NP], m2[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const f2 sm = f2_mul(st.s[i], ic);  // mean of d
      mean[i] = o.cnt > 0 ? f2_sub(sm, st.nk[i]) : f2_splat(0.f);
      m2[i] = o.cnt > 0 ? f2_sub(st.q[i], f2_mul(sm, st.s[i])) : f2_splat(0.f);
    }
    sts_pairs<NP>(m.red + o.lane * rs + o.c, mean);
    sts_pairs<NP>(m.red + plane + o.lane * rs + o.c, m2);
  }
  __syncthreads();
  const int nw = s.threads >> 5, w = threadIdx.x >> 5, l8 = threadIdx.x & 7;
  const int oct = (threadIdx.x & 31) >> 3;
  const float rows = static_cast<float>(o.rows);
  // lane l of the threads has base places, one more below `more`
  const int base = o.rows / s.lanes, more = o.rows - base * s.lanes;
  for (int t = w; 32 * t < s.cs; t += nw) {
    const int c = 4 * (8 * t + l8);
    const float* p = m.red + (c < s.cs ? c : 0);
    f2 ref[2], sum[2], q[2];
    lds_quad(p + (min(s.lanes, o.rows) >> 1) * rs, ref);
    sum[0] = sum[1] = q[0] = q[1] = f2_splat(0.f);
#pragma unroll 2
    for (int l = oct; l < s.lanes; l += 4) {
      f2 mean[2], m2[2];
      lds_quad(p + l * rs, mean);
      lds_quad(p + plane + l * rs, m2);
      const f2 n = f2_splat(static_cast<float>(base + (l < more)));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f2 d = f2_sub(mean[i], ref[i]), nd = f2_mul(n, d);
        sum[i] = f2_add(sum[i], nd);
        q[i] = f2_add(q[i], f2_fma(nd, d, m2[i]));
      }
    }
    const f2 inv = f2_splat(o.rows > 0 ? 1.f / rows : 0.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] = across_octets(sum[i]);
      q[i] = across_octets(q[i]);
      const f2 d = f2_mul(sum[i], inv);
      ref[i] = f2_add(ref[i], d);
      q[i] = f2_sub(q[i], f2_mul(d, sum[i]));
    }
    if (oct == 0 && c < s.cs) {
      sts_quad(m.col + c, ref);
      sts_quad(m.col + s.cs + c, q);
    }
  }
  __syncthreads();
  const float icg = 1.f / static_cast<float>(s.cg);
  for (int g0 = 4 * w; g0 < s.gs; g0 += 4 * nw) {  // whole warps: the shuffles need them
    const int g = g0 + oct;
    const float* p = m.col + g * s.cg;
    float sum = 0.f;
    if (g < s.gs)
      for (int i = l8; i < s.cg; i += 8) sum += p[i];
    const float mean = octet_sum(sum) * icg;
    float m2 = 0.f;
    if (g < s.gs)
      for (int i = l8; i < s.cg; i += 8) {
        const float d = p[i] - mean;
        m2 += __fmaf_rn(d * d, rows, p[s.cs + i]);
      }
    m2 = octet_sum(m2);
    if (l8 == 0 && g < s.gs) {
      m.gm[2 * g] = mean;
      m.gm[2 * g + 1] = m2;
    }
  }
}

template <typename T, int kAct, bool kWide>
__global__ void __launch_bounds__(max_threads(kWide), min_ctas(kWide))
    gn_fwd_kernel(const GnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  const GnShape& s = a.s;
  const Smem m = carve(smem, s, false);
  const Owner o = on_chip_owner(a);
  const int tid = threadIdx.x;
  const int ch = o.slab * s.cs + o.c;
  const int64_t step = s.lanes * a.s_s;
  const T* const px = static_cast<const T*>(a.x) + (o.r0 + o.lane) * a.s_s + ch;
  const float total = static_cast<float>(o.len) * static_cast<float>(s.cg);
  const int l8 = tid & 7;
  // values a group of cluster rank l8
  const float nk = l8 < s.ctas ? static_cast<float>(rank_start(o.len, l8 + 1, s) -
                                                    rank_start(o.len, l8, s)) *
                                     static_cast<float>(s.cg)
                               : 0.f;

  pdl_wait_prior_grid();
  pdl_allow_next_grid();

  // this thread's slot of place i of stage k is stage + (k * iters + i) * stride
  const uint32_t stride = 16u * s.threads, stage = smem_u32(smem) + 16u * tid;
  auto stage_places = [&](int64_t n, int k, int from, int to) {
    if (n < a.N) {
      const T* p = px + n * a.s_n + from * step;
      uint32_t d = stage + (k * s.iters + from) * stride;
      for (int i = from; i < min(to, o.cnt); ++i, p += step, d += stride) cp_async_16(d, p);
    }
    cp_async_commit();
  };
  constexpr int kBatches = 4;  // of a single-stage sample
  const int per = (s.iters + kBatches - 1) / kBatches;
  const bool three = o.cnt > kFewPlaces;
  int64_t n = o.n;
  if (s.stages == 1)
    for (int b = 0; b < kBatches; ++b) stage_places(n, 0, b * per, (b + 1) * per);
  for (int k = 0; k + 1 < s.stages; ++k) stage_places(n + k * s.lanes_n, k, 0, s.iters);
  load_params(a, m.w, m.b, o.slab);

  for (int k = 0; n < a.N; n += s.lanes_n) {
    ColumnStats<T> st;
    const uint32_t mine = stage + k * s.iters * stride;
    if (s.stages == 1) {  // the sums follow the copies, batch by batch
      for (int b = 0; b < kBatches; ++b) {
        cp_async_wait(kBatches - 1 - b);
        if (b == 0 && o.cnt > 0) st.start(mine, stride, three);  // (then per is three at least)
        for_staged(mine, b * per, min(o.cnt, (b + 1) * per), stride,
                   [&](const uint4& u) { st.add(u); });
      }
    } else {
      const int ahead = s.stages - 1;
      stage_places(n + ahead * s.lanes_n, k + ahead < s.stages ? k + ahead : k + ahead - s.stages,
                   0, s.iters);
      cp_async_wait(ahead);
      if (o.cnt > 0) st.start(mine, stride, three);
      for_staged(mine, 0, o.cnt, stride, [&](const uint4& u) { st.add(u); });
    }
    cta_stats(m, s, o, st);

    // the cluster's group values: an octet of threads a group, a CTA a thread
    if (s.ctas > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    for (int g0 = 4 * (tid >> 5); g0 < s.gs; g0 += s.threads >> 3) {
      const int g = g0 + ((tid & 31) >> 3);
      float2 v = make_float2(0.f, 0.f);
      if (g < s.gs && l8 < s.ctas)
        v = s.ctas > 1 ? ld_peer_f2(peer_addr(m.gm + 2 * g, static_cast<uint32_t>(l8)))
                       : make_float2(m.gm[2 * g], m.gm[2 * g + 1]);
      const float mean = octet_sum(nk * v.x) / total;
      const float d = nk > 0.f ? v.x - mean : 0.f;
      const float m2 = octet_sum(__fmaf_rn(d * d, nk, v.y));
      const float rstd = __frsqrt_rn(__fadd_rn(clamp_below(m2 / total), a.eps));
      if (g < s.gs) {
        set_group(m, s, g, l8, 8, mean, rstd);
        if (l8 == 0 && o.rank == 0) {
          a.mean[n * a.G + o.slab * s.gs + g] = mean;
          a.rstd[n * a.G + o.slab * s.gs + g] = rstd;
        }
      }
    }
    if (s.ctas > 1) cluster_arrive();  // this CTA's reads of the others are done
    __syncthreads();
    if (o.cnt > 0) {
      Consts<T> q;
      q.load(m.c0, m.c1, m.b, o.c);
      T* py = static_cast<T*>(a.out) + (n * a.S + o.r0 + o.lane) * a.C + ch;
      const int64_t ystep = static_cast<int64_t>(s.lanes) * a.C;
      for_staged(mine, 0, o.cnt, stride, [&](const uint4& u) {
        stg128(py, q.template norm<kAct>(u));
        py += ystep;
      });
    }
    if (s.stages == 1) {
      for (int b = 0; b < kBatches; ++b) stage_places(n + s.lanes_n, 0, b * per, (b + 1) * per);
    } else if (++k == s.stages) {
      k = 0;
    }
    if (s.ctas > 1) cluster_wait();
  }
}

// Streamed.  Each turn's pieces (a unit's chunk each) are dealt out to the grid.  A CTA sums its
// pieces of turn t + 1 before it waits for every CTA's sums of turn t and writes its pieces of
// that one, so the grid's barrier and the CTAs' unevenness hide behind a turn's sums (L2 holds
// part of the two turns that are live).  Before the output a unit's chunks combine (some lanes of
// a warp a group, the chunks over them).  A piece is written from its last place back, so that the
// part L2 still holds is read first.  Every unit has its own place in part.
template <typename T, int kAct, bool kWide>
__global__ void __launch_bounds__(max_threads(kWide), min_ctas(kWide))
    gn_fwd_stream_kernel(const GnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  const GnShape& s = a.s;
  const Smem m = carve(smem, s, false);
  const int tid = threadIdx.x;
  const int join_log2 = join_lanes_log2(s), jl = tid & ((1 << join_log2) - 1);
  const int gs_up = join_groups(s, join_log2);
  const int64_t step = s.lanes * a.s_s, ystep = static_cast<int64_t>(s.lanes) * a.C;
  const float total = static_cast<float>(a.S) * static_cast<float>(s.cg);
  const float cg = static_cast<float>(s.cg);
  Owner o;
  set_lane(o, s);
  const int all = static_cast<int>(a.N) * s.slabs;
  auto units_at = [&](int u0) { return min(s.units, all - u0); };
  auto ring_of = [&](bool back) {  // piece o's, from its last place if back
    const T* p = static_cast<const T*>(a.x) + o.n * a.s_n + (o.r0 + o.lane) * a.s_s +
                 o.slab * s.cs + o.c + (back ? (o.cnt - 1) * step : 0);
    return Ring<1>{smem_u32(smem) + 16u * tid, 16u * s.threads,
                   {reinterpret_cast<const unsigned char*>(p)},
                   {(back ? -step : step) * static_cast<int64_t>(sizeof(T))}, o.cnt};
  };
  auto sum_turn = [&](int u0) {
    const int nu = units_at(u0);
    for (int v = blockIdx.x; v < nu * s.chunks; v += gridDim.x) {
      set_piece(o, a, u0, nu, v);
      Ring<1> ring = ring_of(false);
      ring.start();
      ColumnStats<T> st;
      if (o.cnt > 0) {
        static_assert(2 * kRingPlaces >= 3 && Ring<1>::kGroups >= 3, "three places have arrived");
        cp_async_wait_n<Ring<1>::kGroups - 3>();
        st.start(ring.slot, ring.stride, o.cnt > kFewPlaces);
      }
      ring.run(o.cnt, [&](uint32_t slot) { st.add(lds128_at(slot)); });
      __syncthreads();  // red takes the rings' place
      cta_stats(m, s, o, st);
      __syncthreads();
      float2* part = a.part + (o.n * s.chunks + o.chunk) * a.G + o.slab * s.gs;
      for (int g = tid; g < s.gs; g += s.threads)
        part[g] = make_float2(m.gm[2 * g], m.gm[2 * g + 1]);
    }
  };

  auto grid = cooperative_groups::this_grid();
  sum_turn(0);
  auto token = grid.barrier_arrive();
  for (int u0 = 0; u0 < all; u0 += s.units) {
    const bool more = u0 + s.units < all;
    if (more) sum_turn(u0 + s.units);
    grid.barrier_wait(std::move(token));
    if (more) token = grid.barrier_arrive();
    const int nu = units_at(u0);
    for (int v = blockIdx.x; v < nu * s.chunks; v += gridDim.x) {
      set_piece(o, a, u0, nu, v);
      Ring<1> ring = ring_of(true);
      ring.start();
      __syncthreads();  // the piece before is done with w, b, c0, c1
      // one round trip to memory: the parameters and the chunks' statistics
      load_params(a, m.w, m.b, o.slab);
      for (int g0 = tid >> join_log2; g0 < gs_up; g0 += s.threads >> join_log2) {
        const int g = min(g0, s.gs - 1);  // whole warps: the shuffles need them
        const float2* p = a.part + o.n * s.chunks * a.G + o.slab * s.gs + g;
        // about the first chunk's mean, as in cta_stats; not through L1, which may hold an
        // earlier turn's line
        const float ref = __ldcg(p).x;
        float sum = 0.f, m2 = 0.f;
#pragma unroll 8
        for (int k = jl; k < s.chunks; k += 1 << join_log2) {
          const float2 x = __ldcg(p + static_cast<int64_t>(k) * a.G);
          const float d = x.x - ref;
          const float nd = static_cast<float>(s.chunk_base + (k < s.chunk_more ? 1 : 0)) * cg * d;
          sum += nd;
          m2 += __fmaf_rn(nd, d, x.y);
        }
        sum = join_sum(sum, join_log2);
        m2 = join_sum(m2, join_log2);
        if (jl == 0 && g0 < s.gs) {
          const float off = sum / total, mean = ref + off;
          m2 = __fmaf_rn(-off, sum, m2);
          const float rstd = __frsqrt_rn(__fadd_rn(clamp_below(m2 / total), a.eps));
          m.gm[2 * g] = mean;
          m.gm[2 * g + 1] = rstd;
          if (o.chunk == 0) {
            a.mean[o.n * a.G + o.slab * s.gs + g] = mean;
            a.rstd[o.n * a.G + o.slab * s.gs + g] = rstd;
          }
        }
      }
      __syncthreads();
      for (int c = tid; c < s.cs; c += s.threads) {
        const int g = c / s.cg;
        m.c0[c] = -m.gm[2 * g];
        m.c1[c] = m.gm[2 * g + 1] * m.w[c];
      }
      __syncthreads();
      if (o.cnt > 0) {
        Consts<T> q;
        q.load(m.c0, m.c1, m.b, o.c);
        T* py = static_cast<T*>(a.out) + (o.n * a.S + o.r0 + o.lane) * a.C + o.slab * s.cs + o.c +
                (o.cnt - 1) * ystep;
        ring.run(o.cnt, [&](uint32_t slot) {  // y is not read here again: it leaves L2 first
          __stcs(reinterpret_cast<uint4*>(py), q.template norm<kAct>(lds128_at(slot)));
          py -= ystep;
        });
      }
    }
    __syncthreads();  // the sums reuse the shared memory
  }
}

namespace {

// The kernel builds for a dtype T, activation and width.
template <typename T, bool kWide>
const void* pick_act(const GnShape& s, int act) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
  if (s.on_chip)
    return act == GROUPNORM_ACT_NONE   ? fn(&gn_fwd_kernel<T, GROUPNORM_ACT_NONE, kWide>)
           : act == GROUPNORM_ACT_SILU ? fn(&gn_fwd_kernel<T, GROUPNORM_ACT_SILU, kWide>)
                                       : fn(&gn_fwd_kernel<T, GROUPNORM_ACT_GELU, kWide>);
  return act == GROUPNORM_ACT_NONE   ? fn(&gn_fwd_stream_kernel<T, GROUPNORM_ACT_NONE, kWide>)
         : act == GROUPNORM_ACT_SILU ? fn(&gn_fwd_stream_kernel<T, GROUPNORM_ACT_SILU, kWide>)
                                     : fn(&gn_fwd_stream_kernel<T, GROUPNORM_ACT_GELU, kWide>);
}
template <typename T>
const void* pick_fwd(const GnShape& s, int act) {
  return s.vecs > kThreads ? pick_act<T, true>(s, act) : pick_act<T, false>(s, act);
}

}  // namespace

cudaError_t launch_gn_fwd(const GnArgs& a, int dtype, int act, cudaStream_t st) {
  const void* fn = dtype == GROUPNORM_BF16   ? pick_fwd<__nv_bfloat16>(a.s, act)
                   : dtype == GROUPNORM_FP32 ? pick_fwd<float>(a.s, act)
                                             : pick_fwd<__half>(a.s, act);
  return launch_gn(fn, a, st);
}

}  // namespace gnorm
