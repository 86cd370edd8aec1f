// gn_bwd.cu -- group norm training backward with an activation, channels last, for sm_103a
// (include/groupnorm_train.h gives the formulas).
//
// Per channel of a sample, A_c = sum over places of dz * xhat and B_c = sum of dz; a group's
// mean(g * xhat) and mean(g) are w-weighted sums of them, and dw_c, db_c their sums over the
// samples -- one set of sums serves all.  As the forward (gn_fwd.cu): x and dy stay on chip
// between the sums and dx where a cluster's shared memory holds them, and are streamed by a
// cooperative grid, twice, where not.  dz is formed twice from x and dy rather than
// kept (keeping it in FP32 would double the staged bytes).  The column sums of each CTA (on
// chip, and for pieces of a few places: over all that it takes, compensated; else of each piece)
// go to the workspace, and a finishing kernel adds them in a fixed order.
//
// Measured (SiLU): on chip 5 x 1023 x 640 fp16 15.5 us, two launches; streamed
// 2 x 262144 x 128 bf16 117 us: x and dy of a sample, 134 MB, are more than L2 gives back, so
// both passes read memory, 98.7 us at a copy's rate.
#include "gn_common.cuh"

namespace gnorm {

// Whether rstd^2 stays well inside FP32's range (false for NaN).  Past it, groups of values around
// 1e-20 or 1e20, the factor rstd^2 of dx's last term is applied in two steps.
__device__ __forceinline__ bool rstd_is_near(float rstd) {
  return rstd >= 0x1p-40f && rstd <= 0x1p40f;
}

// A thread's constants for its channels: d = x - mean, z = d * scale + bias, scale = rstd * w.
template <typename T>
struct Consts {
  static constexpr int kPairs = VecOf<T>::kPairs;
  f2 nm[kPairs], scale[kPairs], bias[kPairs];
  bool far;  // some group's rstd is not near
  // w, b: the slab's parameters in shared memory; mean, rstd: the sample's group values, `gap`
  // floats apart, from the slab's first group on; c: the thread's first channel, place r of
  // group g
  __device__ __forceinline__ void load(const float* w, const float* b, const float* mean,
                                       const float* rstd, int gap, int cg, int c, int g, int r) {
    lds_pairs<kPairs>(w + c, scale);
    lds_pairs<kPairs>(b + c, bias);
    float m = mean[gap * g], q = rstd[gap * g];
    float v[2 * kPairs], u[2 * kPairs];
    far = !rstd_is_near(q);
#pragma unroll
    for (int j = 0; j < 2 * kPairs; ++j) {
      v[j] = -m;
      u[j] = q;
      if (j + 1 < 2 * kPairs && ++r == cg) {
        r = 0;
        ++g;
        m = mean[gap * g];
        q = rstd[gap * g];
        far = far || !rstd_is_near(q);
      }
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      nm[i] = f2_make(v[2 * i], v[2 * i + 1]);
      scale[i] = f2_mul(scale[i], f2_make(u[2 * i], u[2 * i + 1]));
    }
  }
  // d, and dz = dy * act'(z), of pairs h and h + 1 of a vector
  template <int kAct>
  __device__ __forceinline__ void dz(const uint4& xu, const uint4& du, int h, f2 (&d)[2],
                                     f2 (&out)[2]) const {
    f2 z[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      d[i] = VecOf<T>::plus(xu, h + i, nm[h + i]);
      z[i] = f2_fma(d[i], scale[h + i], bias[h + i]);
      out[i] = VecOf<T>::pair(du, h + i);
    }
    act_grad_vec<T, kAct>(z, out);
  }
};

// The group terms of dx = scale * dz + nc1 + d * nc2, with nc1 = -rstd * mean(g) and
// nc2 = -rstd^2 * mean(g * xhat); of a far group, dx = scale * dz + nc1 + (d * rstd) * nc2 with
// nc2 = -rstd * mean(g * xhat).
__device__ __forceinline__ float group_nc2(float rstd, float mean) {
  return (rstd_is_near(rstd) ? -rstd * rstd : -rstd) * mean;
}
template <typename T>
struct GroupTerms {
  static constexpr int kPairs = VecOf<T>::kPairs;
  f2 nc1[kPairs], nc2[kPairs];
  __device__ __forceinline__ void load(const float* c0, const float* c1, int c) {
    lds_pairs<kPairs>(c0 + c, nc1);
    lds_pairs<kPairs>(c1 + c, nc2);
  }
};

// d of two pairs from channel c of the slab on, times rstd where the group is far; rstd: the groups'
// values, `gap` floats apart.
__device__ __forceinline__ void scale_far(const float* rstd, int gap, int cg, int c, f2 (&d)[2]) {
  int g = c / cg, r = c - g * cg;
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float q = rstd[gap * g];
    v[j] = rstd_is_near(q) ? 1.f : q;
    if (j < 3 && ++r == cg) {
      r = 0;
      ++g;
    }
  }
  d[0] = f2_mul(d[0], f2_make(v[0], v[1]));
  d[1] = f2_mul(d[1], f2_make(v[2], v[3]));
}

// far(pair, d): what is done to d of two pairs before the group's term
template <typename T, int kAct, typename F>
__device__ __forceinline__ uint4 dx_vec(const Consts<T>& k, const GroupTerms<T>& t,
                                        const uint4& xu, const uint4& du, F far) {
  constexpr int NP = VecOf<T>::kPairs;
  f2 v[NP];
#pragma unroll
  for (int h = 0; h < NP; h += 2) {
    f2 d[2], dz[2];
    k.template dz<kAct>(xu, du, h, d, dz);
    far(h, d);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[h + i] = f2_fma(dz[i], k.scale[h + i], f2_fma(d[i], t.nc2[h + i], t.nc1[h + i]));
  }
  return VecOf<T>::pack(v);
}

// A thread's column sums over its places: A = sum of dz * d, B = sum of dz.
template <typename T, int kAct>
struct ColumnSums {
  static constexpr int kPairs = VecOf<T>::kPairs;
  f2 A[kPairs], B[kPairs];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) A[i] = B[i] = f2_splat(0.f);
  }
  __device__ __forceinline__ void add(const Consts<T>& k, const uint4& xu, const uint4& du) {
#pragma unroll
    for (int h = 0; h < kPairs; h += 2) {
      f2 d[2], dz[2];
      k.template dz<kAct>(xu, du, h, d, dz);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        A[h + i] = f2_fma(dz[i], d[i], A[h + i]);
        B[h + i] = f2_add(B[h + i], dz[i]);
      }
    }
  }
};

// Column sums over the CTA's places from its threads': A * rstd (= sum of dz * xhat) to
// m.col[0, cs), B to [cs, 2 cs).  A warp takes eight quads of columns, four lanes of each at a
// time; each value also goes to sink(half, column of the slab, value); rstd: the groups' values,
// `gap` floats apart.  Then the CTA's group sums
// of w * A and w * B to m.gm, an octet of threads a group.
template <typename T, int kAct, typename F>
__device__ __forceinline__ void cta_sums(const Smem& m, const GnShape& s, const Owner& o,
                                         const ColumnSums<T, kAct>& sum, const float* rstd,
                                         int gap, F sink) {
  constexpr int NP = VecOf<T>::kPairs;
  const int w = threadIdx.x >> 5, nw = s.threads >> 5, l8 = threadIdx.x & 7;
  const int oct = (threadIdx.x & 31) >> 3;
  const int rs = red_stride(s), plane = s.lanes * rs;
  if (o.lane < s.lanes) {
    sts_pairs<NP>(m.red + o.lane * rs + o.c, sum.A);
    sts_pairs<NP>(m.red + plane + o.lane * rs + o.c, sum.B);
  }
  __syncthreads();
  const int tasks = (s.cs + 31) >> 5;
  for (int t = w; t < 2 * tasks; t += nw) {
    const int half = t >= tasks ? 1 : 0;
    const int c = 4 * (8 * (t - half * tasks) + l8);
    const float* p = m.red + half * plane + (c < s.cs ? c : 0);
    f2 v[2] = {f2_splat(0.f), f2_splat(0.f)};
#pragma unroll 4
    for (int l = oct; l < s.lanes; l += 4) {
      f2 u[2];
      lds_quad(p + l * rs, u);
      v[0] = f2_add(v[0], u[0]);
      v[1] = f2_add(v[1], u[1]);
    }
    v[0] = across_octets(v[0]);
    v[1] = across_octets(v[1]);
    // lane `oct` of the four keeps column c + oct
    const float mine = oct == 0 ? f2_lo(v[0])
                       : oct == 1 ? f2_hi(v[0]) : (oct == 2 ? f2_lo(v[1]) : f2_hi(v[1]));
    if (c < s.cs) {
      const int cc = c + oct;
      const float val = half == 0 ? mine * rstd[gap * (cc / s.cg)] : mine;
      m.col[half * s.cs + cc] = val;
      sink(half, cc, val);
    }
  }
  __syncthreads();
  for (int b = 4 * w; b < s.gs; b += 4 * nw) {  // whole warps: the shuffles need them
    const int g = b + oct;
    float sa = 0.f, sb = 0.f;
    if (g < s.gs)
      for (int i = g * s.cg + l8; i < (g + 1) * s.cg; i += 8) {
        sa = __fmaf_rn(m.w[i], m.col[i], sa);
        sb = __fmaf_rn(m.w[i], m.col[s.cs + i], sb);
      }
    sa = octet_sum(sa);
    sb = octet_sum(sb);
    if (l8 == 0 && g < s.gs) {
      m.gm[2 * g] = sa;
      m.gm[2 * g + 1] = sb;
    }
  }
}

// Channel constants of group g of the slab from its sums sa = sum g * xhat and sb = sum g, lane k
// of `lanes` threads.
__device__ __forceinline__ void set_group(const Smem& m, const GnShape& s, int g, int k, int lanes,
                                          float rstd, float sa, float sb, float total) {
  const float nc1 = -rstd * (sb / total), nc2 = group_nc2(rstd, sa / total);
  for (int i = g * s.cg + k; i < (g + 1) * s.cg; i += lanes) {
    m.c0[i] = nc1;
    m.c1[i] = nc2;
  }
}

// Kahan's running sum; an infinite one stays infinite.
__device__ __forceinline__ void running_add(float* sum, float* comp, float v) {
  const float s = *sum, y = __fsub_rn(v, *comp);
  const float r = __fadd_rn(s, y);
  *comp = isinf(r) ? 0.f : __fsub_rn(__fsub_rn(r, s), y);
  *sum = r;
}

// The piece's column sums col [2][cs] into a row of running ones, their compensations `gap` floats
// behind them: four columns a thread, all of a round's loads on their way together.
__device__ __forceinline__ void add_to_row(const float* col, float* row, int64_t gap, int C,
                                           const GnShape& s) {
#pragma unroll 4
  for (int i = 4 * threadIdx.x; i < 2 * s.cs; i += 4 * s.threads) {
    float* p = row + (i < s.cs ? i : C + i - s.cs);
    float4 sum = *reinterpret_cast<float4*>(p), comp = *reinterpret_cast<float4*>(p + gap);
    const float4 v = *reinterpret_cast<const float4*>(col + i);
    running_add(&sum.x, &comp.x, v.x);
    running_add(&sum.y, &comp.y, v.y);
    running_add(&sum.z, &comp.z, v.z);
    running_add(&sum.w, &comp.w, v.w);
    *reinterpret_cast<float4*>(p) = sum;
    *reinterpret_cast<float4*>(p + gap) = comp;
  }
}

template <typename T, int kAct, bool kWide>
__global__ void __launch_bounds__(max_threads(kWide), min_ctas(kWide))
    gn_bwd_kernel(const GnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  const GnShape& s = a.s;
  const Smem m = carve(smem, s, true);
  const Owner o = on_chip_owner(a);
  const int tid = threadIdx.x;
  const int ch = o.slab * s.cs + o.c, group0 = o.slab * s.gs;
  const int og = o.c / s.cg, orr = o.c - og * s.cg;
  const int64_t step = s.lanes * a.s_s, dstep = static_cast<int64_t>(s.lanes) * a.C;
  const T* const px = static_cast<const T*>(a.x) + (o.r0 + o.lane) * a.s_s + ch;
  const int64_t at0 = (o.r0 + o.lane) * a.C + ch;  // in sample 0 of dy and dx
  const T* const pd = static_cast<const T*>(a.dy) + at0;
  const float total = static_cast<float>(a.S) * static_cast<float>(s.cg);

  pdl_wait_prior_grid();
  pdl_allow_next_grid();

  // this thread's slot of place i of stage k is stage + (2 * k * iters + i) * stride for x, and
  // dy_off behind it for dy
  const uint32_t stride = 16u * s.threads, stage = smem_u32(smem) + 16u * tid;
  const uint32_t dy_off = s.iters * stride;
  auto stage_places = [&](int64_t n, int k, int from, int to) {
    if (n < a.N) {
      const T* p = px + n * a.s_n + from * step;
      const T* q = pd + n * a.S * a.C + from * dstep;
      uint32_t d = stage + (2 * k * s.iters + from) * stride;
      for (int i = from; i < min(to, o.cnt); ++i, p += step, q += dstep, d += stride) {
        cp_async_16(d, p);
        cp_async_16(d + dy_off, q);
      }
    }
    cp_async_commit();
  };
  constexpr int kBatches = 4;  // of a single-stage sample
  const int per = (s.iters + kBatches - 1) / kBatches;
  int64_t n = o.n;
  if (s.stages == 1)
    for (int b = 0; b < kBatches; ++b) stage_places(n, 0, b * per, (b + 1) * per);
  for (int k = 0; k + 1 < s.stages; ++k) stage_places(n + k * s.lanes_n, k, 0, s.iters);
  // running column totals (sum, compensation)
  for (int i = tid; i < 4 * s.cs; i += s.threads) m.run[i] = 0.f;
  load_params(a, m.w, m.b, o.slab);
  __syncthreads();

  const int l8 = tid & 7, oct = (tid & 31) >> 3;
  for (int k = 0; n < a.N; n += s.lanes_n) {
    const float* const mean = a.mean + n * a.G + group0;
    const float* const rstd = a.rstd + n * a.G + group0;
    Consts<T> q;
    ColumnSums<T, kAct> sum;
    sum.clear();
    const uint32_t mine = stage + 2 * k * s.iters * stride;
    auto add = [&](const uint4& xu, const uint4& du) { sum.add(q, xu, du); };
    if (s.stages == 1) {  // the sums follow the copies, batch by batch
      if (o.cnt > 0) q.load(m.w, m.b, mean, rstd, 1, s.cg, o.c, og, orr);
      for (int b = 0; b < kBatches; ++b) {
        cp_async_wait(kBatches - 1 - b);
        for_staged2(mine, dy_off, b * per, min(o.cnt, (b + 1) * per), stride, add);
      }
    } else {
      const int ahead = s.stages - 1;
      stage_places(n + ahead * s.lanes_n, k + ahead < s.stages ? k + ahead : k + ahead - s.stages,
                   0, s.iters);
      if (o.cnt > 0) q.load(m.w, m.b, mean, rstd, 1, s.cg, o.c, og, orr);
      cp_async_wait(ahead);
      for_staged2(mine, dy_off, 0, o.cnt, stride, add);
    }
    cta_sums(m, s, o, sum, rstd, 1, [&](int half, int c, float v) {
      float* run = m.run + 2 * (half * s.cs + c);  // over the samples
      running_add(run, run + 1, v);
    });
    // the cluster's: an octet of threads a group, a CTA a thread
    if (s.ctas > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    for (int b = 4 * (tid >> 5); b < s.gs; b += s.threads >> 3) {
      const int g = b + oct;
      float2 v = make_float2(0.f, 0.f);
      if (g < s.gs && l8 < s.ctas)
        v = s.ctas > 1 ? ld_peer_f2(peer_addr(m.gm + 2 * g, static_cast<uint32_t>(l8)))
                       : make_float2(m.gm[2 * g], m.gm[2 * g + 1]);
      const float sa = octet_sum(v.x), sb = octet_sum(v.y);
      if (g < s.gs) set_group(m, s, g, l8, 8, rstd[g], sa, sb, total);
    }
    if (s.ctas > 1) cluster_arrive();  // this CTA's reads of the others are done
    __syncthreads();
    if (o.cnt > 0) {
      GroupTerms<T> t;
      t.load(m.c0, m.c1, o.c);
      T* po = static_cast<T*>(a.out) + n * a.S * a.C + at0;
      if (!q.far) {
        for_staged2(mine, dy_off, 0, o.cnt, stride, [&](const uint4& xu, const uint4& du) {
          stg128(po, dx_vec<T, kAct>(q, t, xu, du, [](int, f2 (&)[2]) {}));
          po += dstep;
        });
      } else {  // (a branch inside the loop costs up to 5 % of small samples)
        for (int i = 0; i < o.cnt; ++i, po += dstep) {
          const uint32_t p = mine + i * stride;
          stg128(po, dx_vec<T, kAct>(q, t, lds128_at(p), lds128_at(p + dy_off),
                                     [&](int h, f2 (&d)[2]) {
                                       scale_far(rstd, 1, s.cg, o.c + 2 * h, d);
                                     }));
        }
      }
    }
    if (s.stages == 1) {
      for (int b = 0; b < kBatches; ++b) stage_places(n + s.lanes_n, 0, b * per, (b + 1) * per);
    } else if (++k == s.stages) {
      k = 0;
    }
    if (s.ctas > 1) cluster_wait();
  }
  __syncthreads();
  // this CTA's totals over its samples
  float* out = a.cols + (o.n * s.ctas + o.rank) * 2 * a.C + o.slab * s.cs;
  for (int t = tid; t < 2 * s.cs; t += s.threads)
    out[t < s.cs ? t : a.C + t - s.cs] = m.run[2 * t];
}

// Streamed, as the forward's (gn_fwd.cu): the sums of turn t + 1, the barrier, dx of turn t.
template <typename T, int kAct, bool kWide>
__global__ void __launch_bounds__(max_threads(kWide), min_ctas(kWide))
    gn_bwd_stream_kernel(const GnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  const GnShape& s = a.s;
  const Smem m = carve(smem, s, true);
  const int tid = threadIdx.x;
  const int join_log2 = join_lanes_log2(s), jl = tid & ((1 << join_log2) - 1);
  const int gs_up = join_groups(s, join_log2);
  const int64_t step = s.lanes * a.s_s, dstep = static_cast<int64_t>(s.lanes) * a.C;
  const float total = static_cast<float>(a.S) * static_cast<float>(s.cg);
  const uint32_t stride = 16u * s.threads;
  Owner o;
  set_lane(o, s);
  const int og = o.c / s.cg, orr = o.c - og * s.cg;
  const int all = static_cast<int>(a.N) * s.slabs;
  auto units_at = [&](int u0) { return min(s.units, all - u0); };
  auto place = [&] { return (o.n * a.S + o.r0 + o.lane) * a.C + o.slab * s.cs + o.c; };
  auto ring_of = [&](bool back) {  // piece o's, from its last place if back
    const int64_t last = back ? o.cnt - 1 : 0, es = back ? -int64_t{sizeof(T)} : int64_t{sizeof(T)};
    const T* p = static_cast<const T*>(a.x) + o.n * a.s_n + (o.r0 + o.lane) * a.s_s +
                 o.slab * s.cs + o.c + last * step;
    const T* d = static_cast<const T*>(a.dy) + place() + last * dstep;
    return Ring<2>{smem_u32(smem) + 16u * tid, stride,
                   {reinterpret_cast<const unsigned char*>(p),
                    reinterpret_cast<const unsigned char*>(d)}, {step * es, dstep * es}, o.cnt};
  };
  // piece o's parameters and statistics to shared memory (its copies have started)
  auto load_piece = [&] {
    __syncthreads();  // the piece before is done with them
    load_params(a, m.w, m.b, o.slab);
    for (int g = tid; g < s.gs; g += s.threads) {
      m.ms[2 * g] = a.mean[o.n * a.G + o.slab * s.gs + g];
      m.ms[2 * g + 1] = a.rstd[o.n * a.G + o.slab * s.gs + g];
    }
  };
  // (a sequence a CTA, unless a smaller grid runs them)
  const int ways = s.seqs > 0 ? s.seqs : static_cast<int>(gridDim.x);
  auto sum_turn = [&](int u0) {
    const int nu = units_at(u0);
    for (int w = blockIdx.x; w < ways; w += gridDim.x)
      for (int v = w; v < nu * s.chunks; v += ways) {
        set_piece(o, a, u0, nu, v);
        Ring<2> ring = ring_of(false);
        ring.start();
        load_piece();
        __syncthreads();
        Consts<T> q;
        if (o.cnt > 0) q.load(m.w, m.b, m.ms, m.ms + 1, 2, s.cg, o.c, og, orr);
        ColumnSums<T, kAct> sum;
        sum.clear();
        ring.run(o.cnt, [&](uint32_t slot) {
          sum.add(q, lds128_at(slot), lds128_at(slot + Ring<2>::kSlots * stride));
        });
        __syncthreads();  // red takes the rings' place
        const int64_t row = s.seqs > 0 ? w : o.n * s.chunks + o.chunk;
        float* cols = a.cols + row * 2 * a.C + o.slab * s.cs;
        cta_sums(m, s, o, sum, m.ms + 1, 2, [&](int half, int c, float val) {
          if (s.seqs == 0) cols[half * a.C + c] = val;
        });
        __syncthreads();
        if (s.seqs > 0) add_to_row(m.col, cols, static_cast<int64_t>(s.seqs) * 2 * a.C, a.C, s);
        float2* part = a.part + (o.n * s.chunks + o.chunk) * a.G + o.slab * s.gs;
        for (int g = tid; g < s.gs; g += s.threads)
          part[g] = make_float2(m.gm[2 * g], m.gm[2 * g + 1]);
      }
  };
  // this CTA's sequences: sums and compensations
  for (int w = blockIdx.x; w < s.seqs; w += gridDim.x)
    for (int t = tid; t < 2 * a.C; t += s.threads) {
      float* p = a.cols + static_cast<int64_t>(w) * 2 * a.C + t;
      p[0] = p[static_cast<int64_t>(s.seqs) * 2 * a.C] = 0.f;
    }

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
      Ring<2> ring = ring_of(true);
      ring.start();
      load_piece();
      for (int g0 = tid >> join_log2; g0 < gs_up; g0 += s.threads >> join_log2) {
        const int g = min(g0, s.gs - 1);  // whole warps: the shuffles need them
        const float2* p = a.part + o.n * s.chunks * a.G + o.slab * s.gs + g;
        float sa = 0.f, sb = 0.f;
#pragma unroll 8
        for (int k = jl; k < s.chunks; k += 1 << join_log2) {  // not through L1 (gn_fwd.cu)
          const float2 x = __ldcg(p + static_cast<int64_t>(k) * a.G);
          sa += x.x;
          sb += x.y;
        }
        sa = join_sum(sa, join_log2);
        sb = join_sum(sb, join_log2);
        if (jl == 0 && g0 < s.gs) {
          m.gm[2 * g] = sa / total;
          m.gm[2 * g + 1] = sb / total;
        }
      }
      __syncthreads();
      for (int c = tid; c < s.cs; c += s.threads) {
        const int g = c / s.cg;
        const float r = m.ms[2 * g + 1];
        m.c0[c] = -r * m.gm[2 * g + 1];
        m.c1[c] = group_nc2(r, m.gm[2 * g]);
      }
      Consts<T> q;
      if (o.cnt > 0) q.load(m.w, m.b, m.ms, m.ms + 1, 2, s.cg, o.c, og, orr);
      __syncthreads();
      if (o.cnt > 0) {
        GroupTerms<T> t;
        t.load(m.c0, m.c1, o.c);
        T* po = static_cast<T*>(a.out) + place() + (o.cnt - 1) * dstep;
        ring.run(o.cnt, [&](uint32_t slot) {  // dx is not read here again: it leaves L2 first
          const uint4 xu = lds128_at(slot), du = lds128_at(slot + Ring<2>::kSlots * stride);
          uint4 v;
          if (__builtin_expect(!q.far, 1)) {
            v = dx_vec<T, kAct>(q, t, xu, du, [](int, f2 (&)[2]) {});
          } else {
            v = dx_vec<T, kAct>(q, t, xu, du, [&](int h, f2 (&d)[2]) {
              scale_far(m.ms + 1, 2, s.cg, o.c + 2 * h, d);
            });
          }
          __stcs(reinterpret_cast<uint4*>(po), v);
          po -= dstep;
        });
      }
    }
    __syncthreads();  // the sums reuse the shared memory
  }
}

constexpr int kFinishCols = 32;

// dw_c and db_c: column t of the [rows][2 C] sums.  kSlices slices of rows a column, each added
// in row order (loads a few rows ahead), then joined pairwise in slice order; TwoSum keeps the
// additions' errors beside.  Few rows take eight slices: the joins are what such a call waits on.
template <int kSlices>
__global__ void __launch_bounds__(kFinishCols* kSlices)
    gn_finish_kernel(const float* __restrict__ cols, float* __restrict__ dw,
                     float* __restrict__ db, int64_t rows, int C) {
  __shared__ float sh[kSlices][kFinishCols], se[kSlices][kFinishCols];
  const int x = threadIdx.x % kFinishCols, y = threadIdx.x / kFinishCols;
  const int t = blockIdx.x * kFinishCols + x;
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  float sum = 0.f, err = 0.f;
  auto add = [&](float v) {
    const float r = __fadd_rn(sum, v), b = __fsub_rn(r, sum);
    err += __fadd_rn(__fsub_rn(sum, __fsub_rn(r, b)), __fsub_rn(v, b));
    sum = r;
  };
  if (t < 2 * C) {
    const int64_t end = rows * (y + 1) / kSlices;
    int64_t r = rows * y / kSlices;
    const float* p = cols + r * 2 * C + t;
    constexpr int kU = 8;
    for (; r + kU <= end; r += kU, p += static_cast<int64_t>(kU) * 2 * C) {
      float v[kU];
#pragma unroll
      for (int j = 0; j < kU; ++j) v[j] = p[static_cast<int64_t>(j) * 2 * C];
#pragma unroll
      for (int j = 0; j < kU; ++j) add(v[j]);
    }
    for (; r < end; ++r, p += 2 * static_cast<int64_t>(C)) add(*p);
  }
  sh[y][x] = sum;
  se[y][x] = err;
#pragma unroll
  for (int stride = kSlices / 2; stride > 0; stride >>= 1) {
    __syncthreads();
    if (y < stride) {
      err += se[y + stride][x];
      add(sh[y + stride][x]);
      sh[y][x] = sum;
      se[y][x] = err;
    }
  }
  if (y == 0 && t < 2 * C) (t < C ? dw : db)[t < C ? t : t - C] = isinf(sum) ? sum : sum + err;
}

namespace {

// The kernel builds for a dtype T, activation and width.
template <typename T, bool kWide>
const void* pick_act(const GnShape& s, int act) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
  if (s.on_chip)
    return act == GROUPNORM_ACT_NONE   ? fn(&gn_bwd_kernel<T, GROUPNORM_ACT_NONE, kWide>)
           : act == GROUPNORM_ACT_SILU ? fn(&gn_bwd_kernel<T, GROUPNORM_ACT_SILU, kWide>)
                                       : fn(&gn_bwd_kernel<T, GROUPNORM_ACT_GELU, kWide>);
  return act == GROUPNORM_ACT_NONE   ? fn(&gn_bwd_stream_kernel<T, GROUPNORM_ACT_NONE, kWide>)
         : act == GROUPNORM_ACT_SILU ? fn(&gn_bwd_stream_kernel<T, GROUPNORM_ACT_SILU, kWide>)
                                     : fn(&gn_bwd_stream_kernel<T, GROUPNORM_ACT_GELU, kWide>);
}
template <typename T>
const void* pick_bwd(const GnShape& s, int act) {
  return s.vecs > kThreads ? pick_act<T, true>(s, act) : pick_act<T, false>(s, act);
}

}  // namespace

cudaError_t launch_gn_bwd(const GnArgs& a, int dtype, int act, cudaStream_t st) {
  const void* fn = dtype == GROUPNORM_BF16   ? pick_bwd<__nv_bfloat16>(a.s, act)
                   : dtype == GROUPNORM_FP32 ? pick_bwd<float>(a.s, act)
                                             : pick_bwd<__half>(a.s, act);
  return launch_gn(fn, a, st);
}

cudaError_t launch_gn_finish(const float* cols, float* dw, float* db, int64_t rows, int C,
                             cudaStream_t st) {
  void* args[] = {&cols, &dw, &db, &rows, &C};
  const bool few = rows <= 64;
  const void* fn = few ? reinterpret_cast<const void*>(&gn_finish_kernel<8>)
                       : reinterpret_cast<const void*>(&gn_finish_kernel<32>);
  return launch_pdl(fn, dim3(static_cast<unsigned>((2 * C + kFinishCols - 1) / kFinishCols)),
                    dim3(static_cast<unsigned>(kFinishCols * (few ? 8 : 32))), 0, st, args);
}

}  // namespace gnorm
