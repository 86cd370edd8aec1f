// gn_bwd.cu -- group norm training backward with an activation, channels last, for sm_103a
// (include/groupnorm_train.h gives the formulas).
//
// Per channel of a sample, A_c = sum over places of dz * xhat and B_c = sum of dz; a group's
// mean(g * xhat) and mean(g) are w-weighted sums of them, and dw_c, db_c their sums over the
// samples -- one set of sums serves all.  As the forward (gn_fwd.cu): one launch that keeps x
// and dy on chip between the sums and dx where a cluster's shared memory holds them, else two
// launches over as many samples as L2 holds.  dz is formed twice from x and dy rather than kept
// (keeping it in FP32 would double the staged bytes).  The column sums of each CTA (on chip:
// over all the samples it takes, compensated) go to the workspace, and a finishing kernel adds
// them in a fixed order.
#include "gn_common.cuh"

namespace gnorm {

// A thread's constants for its channels: xhat = (x - mean) * rstd, z = xhat * w + b.
template <typename T>
struct Consts {
  static constexpr int kPairs = VecOf<T>::kPairs;
  f2 mean[kPairs], rstd[kPairs], w[kPairs], b[kPairs];
  __device__ __forceinline__ void load_params(const GnArgs& a, int ch) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      w[i] = f2_make(load_param(a.w, a.wb_dtype, ch + 2 * i),
                     load_param(a.w, a.wb_dtype, ch + 2 * i + 1));
      b[i] = f2_make(load_param(a.b, a.wb_dtype, ch + 2 * i),
                     load_param(a.b, a.wb_dtype, ch + 2 * i + 1));
    }
  }
  // group values of sample n, the slab's first group g0 and this thread's first channel c
  __device__ __forceinline__ void load_stats(const GnArgs& a, int64_t n, int g0, int c) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int64_t p = n * a.G + g0 + group_of(a.s, c + 2 * i);
      const int64_t q = n * a.G + g0 + group_of(a.s, c + 2 * i + 1);
      mean[i] = f2_make(a.mean[p], a.mean[q]);
      rstd[i] = f2_make(a.rstd[p], a.rstd[q]);
    }
  }
};

template <typename T, int kAct>
__device__ __forceinline__ void xhat_dz(const Consts<T>& k, const uint4& xu, const uint4& du,
                                        f2* xhat, f2* dz) {
  constexpr int NP = VecOf<T>::kPairs;
  f2 x[NP], dy[NP];
  VecOf<T>::unpack(xu, x);
  VecOf<T>::unpack(du, dy);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    xhat[i] = f2_mul(f2_sub(x[i], k.mean[i]), k.rstd[i]);
    dz[i] = act_grad2<T, kAct>(f2_fma(xhat[i], k.w[i], k.b[i]), dy[i]);
  }
}

// The group terms of dx: dx = rw * dz - (rc1 + xhat * rc2), with rw = rstd * w and
// rc1 = rstd * mean(g), rc2 = rstd * mean(g * xhat).
template <typename T>
struct GroupTerms {
  static constexpr int kPairs = VecOf<T>::kPairs;
  f2 rw[kPairs], nc1[kPairs], nc2[kPairs];  // negated
  // gf[2 g] = mean(g * xhat), gf[2 g + 1] = mean(g)
  __device__ __forceinline__ void load(const GnShape& s, const Consts<T>& k, const float* gf,
                                       int c) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int g = group_of(s, c + 2 * i), h = group_of(s, c + 2 * i + 1);
      const f2 nr = f2_mul(k.rstd[i], f2_splat(-1.f));
      rw[i] = f2_mul(k.rstd[i], k.w[i]);
      nc2[i] = f2_mul(nr, f2_make(gf[2 * g], gf[2 * h]));
      nc1[i] = f2_mul(nr, f2_make(gf[2 * g + 1], gf[2 * h + 1]));
    }
  }
};

template <typename T, int kAct>
__device__ __forceinline__ uint4 dx_vec(const Consts<T>& k, const GroupTerms<T>& t,
                                        const uint4& xu, const uint4& du) {
  constexpr int NP = VecOf<T>::kPairs;
  f2 xhat[NP], dz[NP];
  xhat_dz<T, kAct>(k, xu, du, xhat, dz);
#pragma unroll
  for (int i = 0; i < NP; ++i)
    dz[i] = f2_fma(dz[i], t.rw[i], f2_fma(xhat[i], t.nc2[i], t.nc1[i]));
  return VecOf<T>::pack(dz);
}

template <typename T, int kAct, bool kOnChip>
__global__ void __launch_bounds__(kMaxThreads, 1) gn_bwd_kernel(const GnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int NP = VecOf<T>::kPairs;
  const GnShape& s = a.s;
  const Smem m = carve(smem, s, true);
  uint4* stage_x = reinterpret_cast<uint4*>(smem);
  uint4* stage_d = stage_x + static_cast<size_t>(s.iters) * s.threads;

  const int tid = threadIdx.x;
  const int lane = tid / s.vecs, vec = tid - lane * s.vecs;
  const bool active = lane < s.lanes;
  const int rank = s.ctas > 1 ? static_cast<int>(cluster_cta_rank()) : 0;
  const int unit = blockIdx.x / s.ctas;
  const int slab = unit % s.slabs, rest = unit / s.slabs;
  const int c = vec * s.ev, ch = slab * s.cs + c;
  const int chunk = kOnChip ? 0 : rest % s.chunks;
  const int64_t lo = kOnChip ? 0 : piece_start(a.S, chunk, s.chunks);
  const int64_t hi = kOnChip ? a.S : piece_start(a.S, chunk + 1, s.chunks);
  const int64_t r0 = lo + piece_start(hi - lo, rank, s.ctas);
  const int64_t r1 = lo + piece_start(hi - lo, rank + 1, s.ctas);
  const int rows = static_cast<int>(r1 - r0);
  const int cnt = active && lane < rows ? (rows - lane + s.lanes - 1) / s.lanes : 0;

  pdl_wait_prior_grid();
  pdl_allow_next_grid();

  Consts<T> k;
  if (active) k.load_params(a, ch);
  if constexpr (kOnChip)  // running column totals (sum, compensation)
    for (int i = tid; i < 4 * s.cs; i += s.threads) m.run[i] = 0.f;

  for (int64_t n = a.n0 + (kOnChip ? rest : rest / s.chunks); n < a.n1;
       n += kOnChip ? s.lanes_n : a.n1) {
    const T* px = static_cast<const T*>(a.x) + n * a.s_n + (r0 + lane) * a.s_s + ch;
    const T* pd = static_cast<const T*>(a.dy) + (n * a.S + r0 + lane) * a.C + ch;
    const int64_t step = s.lanes * a.s_s, dstep = static_cast<int64_t>(s.lanes) * a.C;
    f2 A[NP], B[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) A[i] = B[i] = f2_splat(0.f);
    auto add = [&](const uint4& xu, const uint4& du) {
      f2 xhat[NP], dz[NP];
      xhat_dz<T, kAct>(k, xu, du, xhat, dz);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        A[i] = f2_fma(dz[i], xhat[i], A[i]);
        B[i] = f2_add(B[i], dz[i]);
      }
    };
    if constexpr (kOnChip) {
      constexpr int kBatches = 4;
      const int per = (s.iters + kBatches - 1) / kBatches;
#pragma unroll 1
      for (int b = 0; b < kBatches; ++b) {
        const int end = min(cnt, (b + 1) * per);
        for (int i = b * per; i < end; ++i) {
          cp_async_16(stage_x + i * s.threads + tid, px + i * step);
          cp_async_16(stage_d + i * s.threads + tid, pd + i * dstep);
        }
        cp_async_commit();
      }
      if (active) k.load_stats(a, n, slab * s.gs, c);
#pragma unroll 1
      for (int b = 0; b < kBatches; ++b) {
        cp_async_wait(kBatches - 1 - b);
        const int end = min(cnt, (b + 1) * per);
        for (int i = b * per; i < end; ++i)
          add(stage_x[i * s.threads + tid], stage_d[i * s.threads + tid]);
      }
    } else {
      if (active) k.load_stats(a, n, slab * s.gs, c);
      constexpr int kU = 4;
      for (int i = 0; i < cnt; i += kU) {
        uint4 xu[kU], du[kU];
#pragma unroll
        for (int j = 0; j < kU; ++j)
          if (i + j < cnt) {
            xu[j] = *reinterpret_cast<const uint4*>(px + (i + j) * step);
            du[j] = *reinterpret_cast<const uint4*>(pd + (i + j) * dstep);
          }
#pragma unroll
        for (int j = 0; j < kU; ++j)
          if (i + j < cnt) add(xu[j], du[j]);
      }
    }

    // column sums over the CTA's places: A in [0, cs), B in [cs, 2 cs)
    const int plane = s.lanes * s.cs;
    if (active) {
      f2* ra = reinterpret_cast<f2*>(m.red) + tid * NP;
      f2* rb = reinterpret_cast<f2*>(m.red + plane) + tid * NP;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        ra[i] = A[i];
        rb[i] = B[i];
      }
    }
    __syncthreads();
    for (int t = tid; t < 2 * s.cs; t += s.threads) {
      const float* src = t < s.cs ? m.red + t : m.red + plane + (t - s.cs);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      int l = 0;
      for (; l + 4 <= s.lanes; l += 4)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += src[(l + j) * s.cs];
      for (; l < s.lanes; ++l) acc[0] += src[l * s.cs];
      const float v = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      m.col[t] = v;
      if constexpr (kOnChip) {  // Kahan's running sum over the samples
        const float y = __fsub_rn(v, m.run[2 * t + 1]);
        const float sum = __fadd_rn(m.run[2 * t], y);
        m.run[2 * t + 1] = __fsub_rn(__fsub_rn(sum, m.run[2 * t]), y);
        m.run[2 * t] = sum;
      }
    }
    __syncthreads();
    // the CTA's group sums of w * A and w * B: a warp a group
    for (int g = tid >> 5; g < s.gs; g += s.threads >> 5) {
      float sa = 0.f, sb = 0.f;
      for (int i = tid & 31; i < s.cg; i += 32) {
        const float w = load_param(a.w, a.wb_dtype, slab * s.cs + g * s.cg + i);
        sa = __fmaf_rn(w, m.col[g * s.cg + i], sa);
        sb = __fmaf_rn(w, m.col[s.cs + g * s.cg + i], sb);
      }
      sa = warp_allsum(sa);
      sb = warp_allsum(sb);
      if ((tid & 31) == 0) {
        m.gm[2 * g] = sa;
        m.gm[2 * g + 1] = sb;
      }
    }
    if constexpr (!kOnChip) {  // this CTA's column sums, for dw and db
      float* out = a.cols + ((n * s.chunks + chunk) * s.ctas + rank) * 2 * a.C + slab * s.cs;
      for (int t = tid; t < 2 * s.cs; t += s.threads)
        out[t < s.cs ? t : a.C + t - s.cs] = m.col[t];
    }
    __syncthreads();
    gather_cluster(m, s);
    for (int g = tid; g < s.gs; g += s.threads) {
      float sa = 0.f, sb = 0.f;
      for (int q = 0; q < s.ctas; ++q) {
        sa += m.all[g * s.ctas + q].x;
        sb += m.all[g * s.ctas + q].y;
      }
      if constexpr (kOnChip) {
        const float total = static_cast<float>(a.S) * static_cast<float>(s.cg);
        m.gf[2 * g] = sa / total;
        m.gf[2 * g + 1] = sb / total;
      } else if (rank == 0) {
        a.part[(n * s.chunks + chunk) * a.G + slab * s.gs + g] = make_float2(sa, sb);
      }
    }
    if constexpr (kOnChip) {
      __syncthreads();
      if (cnt > 0) {
        GroupTerms<T> t;
        t.load(s, k, m.gf, c);
        T* po = static_cast<T*>(a.out) + (n * a.S + r0 + lane) * a.C + ch;
#pragma unroll 2
        for (int i = 0; i < cnt; ++i)
          stg128(po + i * dstep, dx_vec<T, kAct>(k, t, stage_x[i * s.threads + tid],
                                                 stage_d[i * s.threads + tid]));
      }
    }
    release_cluster(s);
  }
  if constexpr (kOnChip) {  // this CTA's totals over its samples
    // (each thread reads the running sums it wrote itself)
    float* out = a.cols + (static_cast<int64_t>(rest) * s.ctas + rank) * 2 * a.C + slab * s.cs;
    for (int t = tid; t < 2 * s.cs; t += s.threads)
      out[t < s.cs ? t : a.C + t - s.cs] = m.run[2 * t];
  }
}

// The second launch: the chunks' group sums add up (in a fixed order), and dx is formed from x
// and dy, read again backwards.
template <typename T, int kAct>
__global__ void __launch_bounds__(kMaxThreads, 1) gn_bwd_out_kernel(const GnArgs a) {
  extern __shared__ __align__(128) float gf[];  // [gs][2]
  const GnShape& s = a.s;
  const int tid = threadIdx.x;
  const int lane = tid / s.vecs, vec = tid - lane * s.vecs;
  const int unit = gridDim.x - 1 - blockIdx.x;
  const int slab = unit % s.slabs, rest = unit / s.slabs;
  const int part = rest % s.parts;
  const int64_t n = a.n0 + rest / s.parts;
  const int64_t r0 = piece_start(a.S, part, s.parts);
  const int rows = static_cast<int>(piece_start(a.S, part + 1, s.parts) - r0);
  const int c = vec * s.ev, ch = slab * s.cs + c;

  pdl_wait_prior_grid();
  pdl_allow_next_grid();

  const float total = static_cast<float>(a.S) * static_cast<float>(s.cg);
  for (int g = tid >> 5; g < s.gs; g += s.threads >> 5) {
    const float2* p = a.part + n * s.chunks * a.G + slab * s.gs + g;
    float sa = 0.f, sb = 0.f;
    for (int q = tid & 31; q < s.chunks; q += 32) {
      const float2 v = p[static_cast<int64_t>(q) * a.G];
      sa += v.x;
      sb += v.y;
    }
    sa = warp_allsum(sa);
    sb = warp_allsum(sb);
    if ((tid & 31) == 0) {
      gf[2 * g] = sa / total;
      gf[2 * g + 1] = sb / total;
    }
  }
  __syncthreads();
  if (lane >= s.lanes || lane >= rows) return;

  Consts<T> k;
  k.load_params(a, ch);
  k.load_stats(a, n, slab * s.gs, c);
  GroupTerms<T> t;
  t.load(s, k, gf, c);
  const T* px = static_cast<const T*>(a.x) + n * a.s_n + (r0 + lane) * a.s_s + ch;
  const int64_t at = (n * a.S + r0 + lane) * a.C + ch;
  const T* pd = static_cast<const T*>(a.dy) + at;
  T* po = static_cast<T*>(a.out) + at;
  const int64_t step = s.lanes * a.s_s, dstep = static_cast<int64_t>(s.lanes) * a.C;
  const int cnt = (rows - lane + s.lanes - 1) / s.lanes;
  constexpr int kU = 4;
  for (int i = 0; i < cnt; i += kU) {
    uint4 xu[kU], du[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (i + j < cnt) {
        xu[j] = *reinterpret_cast<const uint4*>(px + (i + j) * step);
        du[j] = *reinterpret_cast<const uint4*>(pd + (i + j) * dstep);
      }
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (i + j < cnt)  // dx is not read here again: it leaves L2 first
        __stcs(reinterpret_cast<uint4*>(po + (i + j) * dstep), dx_vec<T, kAct>(k, t, xu[j], du[j]));
  }
}

constexpr int kFinishCols = 32, kFinishSlices = 32;

// dw_c and db_c: column t of the [rows][2 C] sums, 32 slices of rows a column, each added in
// row order in FP64 and then in slice order.
__global__ void __launch_bounds__(kFinishCols* kFinishSlices)
    gn_finish_kernel(const float* __restrict__ cols, float* __restrict__ dw,
                     float* __restrict__ db, int64_t rows, int C) {
  __shared__ double sh[kFinishSlices][kFinishCols + 1];
  const int x = threadIdx.x % kFinishCols, y = threadIdx.x / kFinishCols;
  const int t = blockIdx.x * kFinishCols + x;
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  double acc = 0.0;
  if (t < 2 * C) {
    const int64_t end = rows * (y + 1) / kFinishSlices;
    for (int64_t r = rows * y / kFinishSlices; r < end; ++r) acc += cols[r * 2 * C + t];
  }
  sh[y][x] = acc;
  __syncthreads();
  if (y == 0 && t < 2 * C) {
    for (int i = 1; i < kFinishSlices; ++i) acc += sh[i][x];
    (t < C ? dw : db)[t < C ? t : t - C] = static_cast<float>(acc);
  }
}

namespace {

template <typename T, bool kOnChip>
const void* pick_sums(int act) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
  return act == GROUPNORM_ACT_NONE   ? fn(&gn_bwd_kernel<T, GROUPNORM_ACT_NONE, kOnChip>)
         : act == GROUPNORM_ACT_SILU ? fn(&gn_bwd_kernel<T, GROUPNORM_ACT_SILU, kOnChip>)
                                     : fn(&gn_bwd_kernel<T, GROUPNORM_ACT_GELU, kOnChip>);
}
template <typename T>
const void* pick_out(int act) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
  return act == GROUPNORM_ACT_NONE   ? fn(&gn_bwd_out_kernel<T, GROUPNORM_ACT_NONE>)
         : act == GROUPNORM_ACT_SILU ? fn(&gn_bwd_out_kernel<T, GROUPNORM_ACT_SILU>)
                                     : fn(&gn_bwd_out_kernel<T, GROUPNORM_ACT_GELU>);
}

}  // namespace

cudaError_t launch_gn_bwd(const GnArgs& a, int dtype, int act, cudaStream_t st) {
  const bool chip = a.s.on_chip != 0;
  const void* fn =
      dtype == GROUPNORM_BF16
          ? (chip ? pick_sums<__nv_bfloat16, true>(act) : pick_sums<__nv_bfloat16, false>(act))
      : dtype == GROUPNORM_FP32
          ? (chip ? pick_sums<float, true>(act) : pick_sums<float, false>(act))
          : (chip ? pick_sums<__half, true>(act) : pick_sums<__half, false>(act));
  return launch_cluster(fn, gn_stats_ctas(a.s, a.n1 - a.n0), a.s, a, st);
}

cudaError_t launch_gn_bwd_out(const GnArgs& a, int dtype, int act, cudaStream_t st) {
  const void* fn = dtype == GROUPNORM_BF16   ? pick_out<__nv_bfloat16>(act)
                   : dtype == GROUPNORM_FP32 ? pick_out<float>(act)
                                             : pick_out<__half>(act);
  GnArgs copy = a;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(static_cast<unsigned>(gn_out_ctas(a.s, a.n1 - a.n0))),
                    dim3(static_cast<unsigned>(a.s.threads)), 8 * static_cast<size_t>(a.s.gs), st,
                    args);
}

cudaError_t launch_gn_finish(const float* cols, float* dw, float* db, int64_t rows, int C,
                             cudaStream_t st) {
  void* args[] = {&cols, &dw, &db, &rows, &C};
  return launch_pdl(reinterpret_cast<const void*>(&gn_finish_kernel),
                    dim3(static_cast<unsigned>((2 * C + kFinishCols - 1) / kFinishCols)),
                    dim3(kFinishCols * kFinishSlices), 0, st, args);
}

}  // namespace gnorm
