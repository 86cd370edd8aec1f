// gn_fwd.cu -- group norm training forward with an activation, channels last, for sm_103a
// (include/groupnorm_train.h gives the formulas).
//
// HBM-bound: one read and one write of the activation.  Where a cluster's shared memory holds
// a sample's slab (gn_launch.h), one launch reads it once: asynchronous 16-byte copies stage
// each thread's own vectors, the statistics follow them batch by batch as they land, the
// cluster's CTAs exchange a few floats a group, and the staged vectors are normalized and
// written.  Larger samples take two launches, the second reading x again -- from L2 where the
// samples of one pair of launches fit it, which is how many a pair takes.
//
// Statistics: each thread sums its channels' values less the first of them, K (sum d and
// sum d^2 of d = x - K), so neither sum cancels when the mean is far from zero; a column's
// mean is K + sum d / n and its M2 = sum d^2 - (sum d)^2 / n.  Means combine weighted by their
// counts, and M2 about the combined mean: M2 = sum of M2_i + n_i (mean_i - mean)^2, from
// threads to the CTA, the cluster and (two launches) the sample.
#include "gn_common.cuh"

namespace gnorm {

template <typename T>
struct ColumnStats {
  static constexpr int kPairs = VecOf<T>::kPairs;
  f2 k[kPairs], s[kPairs], q[kPairs];
  __device__ __forceinline__ void add(const uint4& u, bool first) {
    f2 x[kPairs];
    VecOf<T>::unpack(u, x);
    if (first) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        k[i] = x[i];
        s[i] = q[i] = f2_splat(0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const f2 d = f2_sub(x[i], k[i]);
      s[i] = f2_add(s[i], d);
      q[i] = f2_fma(d, d, q[i]);
    }
  }
};

__device__ __forceinline__ float clamp_below(float v) { return v < 0.f ? 0.f : v; }  // NaN stays

// y of one vector: act((x - mean) * a + b), a = rstd * w.
template <typename T, int kAct>
__device__ __forceinline__ uint4 norm_vec(const uint4& u, const f2* mean, const f2* a,
                                          const f2* b) {
  constexpr int NP = VecOf<T>::kPairs;
  f2 x[NP];
  VecOf<T>::unpack(u, x);
#pragma unroll
  for (int i = 0; i < NP; ++i) x[i] = act2<T, kAct>(f2_fma(f2_sub(x[i], mean[i]), a[i], b[i]));
  return VecOf<T>::pack(x);
}

// A thread's constants for its channels [c, c + ev) of the slab at channel c0 of x.
template <typename T>
__device__ __forceinline__ void load_consts(const GnArgs& a, const float* gf, int c, int ch,
                                            f2* mean, f2* scale, f2* bias) {
#pragma unroll
  for (int i = 0; i < VecOf<T>::kPairs; ++i) {
    const int g0 = group_of(a.s, c + 2 * i), g1 = group_of(a.s, c + 2 * i + 1);
    mean[i] = f2_make(gf[2 * g0], gf[2 * g1]);
    scale[i] = f2_make(gf[2 * g0 + 1] * load_param(a.w, a.wb_dtype, ch + 2 * i),
                       gf[2 * g1 + 1] * load_param(a.w, a.wb_dtype, ch + 2 * i + 1));
    bias[i] = f2_make(load_param(a.b, a.wb_dtype, ch + 2 * i),
                      load_param(a.b, a.wb_dtype, ch + 2 * i + 1));
  }
}

template <typename T, int kAct, bool kOnChip>
__global__ void __launch_bounds__(kMaxThreads, 1) gn_fwd_kernel(const GnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int NP = VecOf<T>::kPairs;
  const GnShape& s = a.s;
  const Smem m = carve(smem, s, false);
  uint4* stage = reinterpret_cast<uint4*>(smem);

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

  for (int64_t n = a.n0 + (kOnChip ? rest : rest / s.chunks); n < a.n1;
       n += kOnChip ? s.lanes_n : a.n1) {
    const T* px = static_cast<const T*>(a.x) + n * a.s_n + (r0 + lane) * a.s_s + ch;
    const int64_t step = s.lanes * a.s_s;
    ColumnStats<T> st;
    if constexpr (kOnChip) {
      constexpr int kBatches = 4;
      const int per = (s.iters + kBatches - 1) / kBatches;
#pragma unroll 1
      for (int b = 0; b < kBatches; ++b) {
        const int end = min(cnt, (b + 1) * per);
        for (int i = b * per; i < end; ++i)
          cp_async_16(stage + i * s.threads + tid, px + i * step);
        cp_async_commit();
      }
#pragma unroll 1
      for (int b = 0; b < kBatches; ++b) {
        cp_async_wait(kBatches - 1 - b);
        const int end = min(cnt, (b + 1) * per);
        for (int i = b * per; i < end; ++i) st.add(stage[i * s.threads + tid], i == 0);
      }
    } else {
      constexpr int kU = 8;
      for (int i = 0; i < cnt; i += kU) {
        uint4 u[kU];
#pragma unroll
        for (int j = 0; j < kU; ++j)
          if (i + j < cnt) u[j] = *reinterpret_cast<const uint4*>(px + (i + j) * step);
#pragma unroll
        for (int j = 0; j < kU; ++j)
          if (i + j < cnt) st.add(u[j], i + j == 0);
      }
    }

    // the CTA's sums and, about their means, its M2
    const float fc = static_cast<float>(cnt), ic = cnt > 0 ? 1.f / fc : 0.f;
    f2* red = reinterpret_cast<f2*>(m.red) + tid * NP;
    if (active) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        red[i] = cnt > 0 ? f2_fma(f2_splat(fc), st.k[i], st.s[i]) : f2_splat(0.f);
    }
    group_sums(m, s, m.gm);
    const float cta_n = static_cast<float>(rows) * static_cast<float>(s.cg);
    if (active) {
      const float inv = rows > 0 ? 1.f / cta_n : 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const f2 gm = f2_make(m.gm[2 * group_of(s, c + 2 * i)] * inv,
                              m.gm[2 * group_of(s, c + 2 * i + 1)] * inv);
        const f2 sm = f2_mul(st.s[i], f2_splat(ic));           // mean of d
        const f2 m2 = f2_sub(st.q[i], f2_mul(sm, st.s[i]));
        const f2 d = f2_add(f2_sub(st.k[i], gm), sm);
        red[i] = cnt > 0 ? f2_fma(f2_mul(d, d), f2_splat(fc), m2) : f2_splat(0.f);
      }
    }
    group_sums(m, s, m.gm + 1);

    // the cluster's
    gather_cluster(m, s);
    for (int g = tid; g < s.gs; g += s.threads) {
      const float total = static_cast<float>(hi - lo) * static_cast<float>(s.cg);
      float sum = 0.f;
      for (int k = 0; k < s.ctas; ++k) sum += m.all[g * s.ctas + k].x;
      const float mean = sum / total;
      float m2 = 0.f;
      for (int k = 0; k < s.ctas; ++k) {
        const float2 v = m.all[g * s.ctas + k];
        const float nk = static_cast<float>(piece_start(hi - lo, k + 1, s.ctas) -
                                            piece_start(hi - lo, k, s.ctas)) *
                         static_cast<float>(s.cg);
        const float d = nk > 0.f ? v.x / nk - mean : 0.f;
        m2 += __fmaf_rn(d * d, nk, v.y);
      }
      const int64_t at = n * a.G + slab * s.gs + g;
      if constexpr (kOnChip) {
        const float rstd = __frsqrt_rn(__fadd_rn(clamp_below(m2 / total), a.eps));
        m.gf[2 * g] = mean;
        m.gf[2 * g + 1] = rstd;
        if (rank == 0) {
          a.mean[at] = mean;
          a.rstd[at] = rstd;
        }
      } else if (rank == 0) {
        a.part[(n * s.chunks + chunk) * a.G + slab * s.gs + g] = make_float2(mean, m2);
      }
    }
    if constexpr (kOnChip) {
      __syncthreads();
      if (cnt > 0) {
        f2 mean[NP], scale[NP], bias[NP];
        load_consts<T>(a, m.gf, c, ch, mean, scale, bias);
        T* py = static_cast<T*>(a.out) + (n * a.S + r0 + lane) * a.C + ch;
        const int64_t ystep = static_cast<int64_t>(s.lanes) * a.C;
#pragma unroll 2
        for (int i = 0; i < cnt; ++i)
          stg128(py + i * ystep, norm_vec<T, kAct>(stage[i * s.threads + tid], mean, scale, bias));
      }
    }
    release_cluster(s);
  }
}

// The second launch: the chunks' statistics combine into the sample's (lanes of a warp take
// the chunks of a group), and the CTA's places are read again, normalized and written.  CTAs
// run through the places backwards, so that the last ones the statistics read come first, while
// L2 still holds them.
template <typename T, int kAct>
__global__ void __launch_bounds__(kMaxThreads, 1) gn_fwd_out_kernel(const GnArgs a) {
  extern __shared__ __align__(128) float gf[];  // [gs][2]
  constexpr int NP = VecOf<T>::kPairs;
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
    auto count = [&](int k) {
      return static_cast<float>(piece_start(a.S, k + 1, s.chunks) - piece_start(a.S, k, s.chunks)) *
             static_cast<float>(s.cg);
    };
    float sum = 0.f, m2 = 0.f;
    for (int k = tid & 31; k < s.chunks; k += 32)
      sum = __fmaf_rn(p[static_cast<int64_t>(k) * a.G].x, count(k), sum);
    const float mean = warp_allsum(sum) / total;
    for (int k = tid & 31; k < s.chunks; k += 32) {
      const float2 v = p[static_cast<int64_t>(k) * a.G];
      const float d = v.x - mean;
      m2 += __fmaf_rn(d * d, count(k), v.y);
    }
    m2 = warp_allsum(m2);
    if ((tid & 31) == 0) {
      const float rstd = __frsqrt_rn(__fadd_rn(clamp_below(m2 / total), a.eps));
      gf[2 * g] = mean;
      gf[2 * g + 1] = rstd;
      if (part == 0) {
        a.mean[n * a.G + slab * s.gs + g] = mean;
        a.rstd[n * a.G + slab * s.gs + g] = rstd;
      }
    }
  }
  __syncthreads();
  if (lane >= s.lanes || lane >= rows) return;

  f2 mean[NP], scale[NP], bias[NP];
  load_consts<T>(a, gf, c, ch, mean, scale, bias);
  const T* px = static_cast<const T*>(a.x) + n * a.s_n + (r0 + lane) * a.s_s + ch;
  T* py = static_cast<T*>(a.out) + (n * a.S + r0 + lane) * a.C + ch;
  const int64_t step = s.lanes * a.s_s, ystep = static_cast<int64_t>(s.lanes) * a.C;
  const int cnt = (rows - lane + s.lanes - 1) / s.lanes;
  constexpr int kU = 4;
  for (int i = 0; i < cnt; i += kU) {
    uint4 u[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (i + j < cnt) u[j] = *reinterpret_cast<const uint4*>(px + (i + j) * step);
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (i + j < cnt)  // y is not read here again: it leaves L2 first
        __stcs(reinterpret_cast<uint4*>(py + (i + j) * ystep),
               norm_vec<T, kAct>(u[j], mean, scale, bias));
  }
}

namespace {

// The build of kernel F<T, act> for a dtype and activation.
template <typename T, bool kOnChip>
const void* pick_stats(int act) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
  if constexpr (!kOnChip) {
    return fn(&gn_fwd_kernel<T, GROUPNORM_ACT_NONE, false>);  // statistics only
  } else {
    return act == GROUPNORM_ACT_NONE   ? fn(&gn_fwd_kernel<T, GROUPNORM_ACT_NONE, true>)
           : act == GROUPNORM_ACT_SILU ? fn(&gn_fwd_kernel<T, GROUPNORM_ACT_SILU, true>)
                                       : fn(&gn_fwd_kernel<T, GROUPNORM_ACT_GELU, true>);
  }
}
template <typename T>
const void* pick_out(int act) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
  return act == GROUPNORM_ACT_NONE   ? fn(&gn_fwd_out_kernel<T, GROUPNORM_ACT_NONE>)
         : act == GROUPNORM_ACT_SILU ? fn(&gn_fwd_out_kernel<T, GROUPNORM_ACT_SILU>)
                                     : fn(&gn_fwd_out_kernel<T, GROUPNORM_ACT_GELU>);
}

}  // namespace

cudaError_t launch_gn_fwd(const GnArgs& a, int dtype, int act, cudaStream_t st) {
  const bool chip = a.s.on_chip != 0;
  const void* fn =
      dtype == GROUPNORM_BF16
          ? (chip ? pick_stats<__nv_bfloat16, true>(act) : pick_stats<__nv_bfloat16, false>(act))
      : dtype == GROUPNORM_FP32
          ? (chip ? pick_stats<float, true>(act) : pick_stats<float, false>(act))
          : (chip ? pick_stats<__half, true>(act) : pick_stats<__half, false>(act));
  return launch_cluster(fn, gn_stats_ctas(a.s, a.n1 - a.n0), a.s, a, st);
}

cudaError_t launch_gn_fwd_out(const GnArgs& a, int dtype, int act, cudaStream_t st) {
  const void* fn = dtype == GROUPNORM_BF16   ? pick_out<__nv_bfloat16>(act)
                   : dtype == GROUPNORM_FP32 ? pick_out<float>(act)
                                             : pick_out<__half>(act);
  GnArgs copy = a;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(static_cast<unsigned>(gn_out_ctas(a.s, a.n1 - a.n0))),
                    dim3(static_cast<unsigned>(a.s.threads)), 8 * static_cast<size_t>(a.s.gs), st,
                    args);
}

}  // namespace gnorm
