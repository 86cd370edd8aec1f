// blk_finish.cu -- the last step of the column sums of a block's boundary: the rows that the teams
// wrote are added in a fixed order, and dw_pre, dw_post and the gate's gradient formed of them.
#include "blk_common.cuh"

namespace blk {

namespace {

constexpr int kLanes = kFinishCols / 4;  // threads of four columns each side by side

// Sums of n vectors f(0), f(1), ... of four columns over kSlices threads: each takes a contiguous
// share, five loads at a time (the rows of 152 CTAs: one turn), the shares are then joined
// pairwise.  The errors of the additions are carried along.  Every thread of the block calls it; the
// result is that of the threads with sl == 0.
template <int kSlices, typename F>
__device__ __forceinline__ float4 column_sums(int64_t n, int sl, int cl, bool live, F f) {
  __shared__ float4 sh[kSlices * kLanes], se[kSlices * kLanes];
  float s[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    const int64_t i1 = (sl + 1) * n / kSlices;
    for (int64_t i = sl * n / kSlices; i < i1; i += 5) {
      float4 v[5];
#pragma unroll
      for (int u = 0; u < 5; ++u) v[u] = i + u < i1 ? f(i + u) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        const float w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float err;
          s[k] = add_exact(s[k], w[k], err);
          e[k] = __fadd_rn(e[k], err);
        }
      }
    }
  }
  const int p = sl * kLanes + cl;
  sh[p] = make_float4(s[0], s[1], s[2], s[3]);
  se[p] = make_float4(e[0], e[1], e[2], e[3]);
  __syncthreads();
#pragma unroll
  for (int stride = kSlices / 2; stride > 0; stride >>= 1) {
    if (sl < stride) {
      const float4 a = sh[p + stride * kLanes], b = se[p + stride * kLanes];
      const float ss[4] = {a.x, a.y, a.z, a.w}, ee[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float err;
        s[k] = add_exact(s[k], ss[k], err);
        e[k] = __fadd_rn(__fadd_rn(e[k], ee[k]), err);
      }
      sh[p] = make_float4(s[0], s[1], s[2], s[3]);
      se[p] = make_float4(e[0], e[1], e[2], e[3]);
    }
    __syncthreads();
  }
  // (a sum that passed FP32's range, or met an infinity: its errors are no numbers)
#pragma unroll
  for (int k = 0; k < 4; ++k) s[k] = isfinite(s[k]) ? __fadd_rn(s[k], e[k]) : s[k];
  return make_float4(s[0], s[1], s[2], s[3]);
}

__device__ __forceinline__ float4 at4(const float* p, int64_t i) {
  return *reinterpret_cast<const float4*>(p + i);
}
// a * (four values of p from i on), or a where there is no p.
__device__ __forceinline__ float4 times(const float4& a, const void* p, int code, int64_t i) {
  if (p == nullptr) return a;
  return make_float4(a.x * load1(p, code, i), a.y * load1(p, code, i + 1),
                     a.z * load1(p, code, i + 2), a.w * load1(p, code, i + 3));
}
__device__ __forceinline__ float4 times(const float4& a, float b) {
  return make_float4(a.x * b, a.y * b, a.z * b, a.w * b);
}
// (outputs start at any element)
__device__ __forceinline__ void put4(float* p, int64_t i, const float4& v) {
  p[i] = v.x;
  p[i + 1] = v.y;
  p[i + 2] = v.z;
  p[i + 3] = v.w;
}

// Several samples: a sample's rows of S become one, scaled, in the first one's place, and its
// gradient of the gate.
template <int kSlices>
__global__ void __launch_bounds__(kLanes* kSlices) blk_samples_kernel(const FinishArgs a) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int cl = threadIdx.x % kLanes, sl = threadIdx.x / kLanes;
  const int col = blockIdx.y * kFinishCols + 4 * cl;
  const int64_t n = blockIdx.x;
  const int64_t rows = a.R / a.samples;
  const int64_t k0 = row_team(n * rows, a.R, a.teams), k1 = row_team((n + 1) * rows - 1, a.R, a.teams);
  float* p = a.part_s + (k0 + n) * a.H + col;
  const float4 s = times(column_sums<kSlices>(k1 - k0 + 1, sl, cl, col < a.H,
                                              [&](int64_t i) { return at4(p, i * a.H); }),
                         a.scale);
  if (sl == 0 && col < a.H) {
    *reinterpret_cast<float4*>(p) = s;
    if (a.dgate != nullptr) put4(a.dgate, n * a.H + col, times(s, a.w_post, a.w_dtype, col));
  }
}

__global__ void __launch_bounds__(kLanes* kFinishSlices) blk_finish_kernel(const FinishArgs a) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int cl = threadIdx.x % kLanes, sl = threadIdx.x / kLanes;
  const int col = blockIdx.x * kFinishCols + 4 * cl;
  const bool live = col < a.H;
  const bool pre = a.part_pre != nullptr && blockIdx.y == 0;
  const float* p = (pre ? a.part_pre : a.part_s) + col;
  if (pre || a.samples == 1) {
    const float4 s = column_sums<kFinishSlices>(a.ctas, sl, cl, live,
                                                [&](int64_t i) { return at4(p, i * a.H); });
    if (sl != 0 || !live) return;
    if (pre) {
      put4(a.dw_pre, col, s);
    } else {
      const float4 t = times(s, a.scale);
      if (a.dw_post != nullptr) put4(a.dw_post, col, times(t, a.gate, a.gate_dtype, col));
      if (a.dgate != nullptr) put4(a.dgate, col, times(t, a.w_post, a.w_dtype, col));
    }
  } else {  // the samples' sums, each times its gate
    const int64_t rows = a.R / a.samples;
    const float4 s = column_sums<kFinishSlices>(a.samples, sl, cl, live, [&](int64_t n) {
      return times(at4(p, (row_team(n * rows, a.R, a.teams) + n) * a.H), a.gate, a.gate_dtype,
                   n * a.H + col);
    });
    if (sl == 0 && live) put4(a.dw_post, col, s);
  }
}

}  // namespace

cudaError_t launch_finish(const FinishArgs& a, cudaStream_t st) {
  FinishArgs copy = a;
  void* args[] = {&copy};
  const unsigned cols = static_cast<unsigned>((a.H + kFinishCols - 1) / kFinishCols);
  const bool several = a.part_s != nullptr && a.samples > 1;
  if (several) {
    // few teams a sample: few threads a column
    const bool few = a.teams / a.samples <= 16;
    const void* fn = few ? reinterpret_cast<const void*>(&blk_samples_kernel<4>)
                         : reinterpret_cast<const void*>(&blk_samples_kernel<kFinishSlices>);
    const cudaError_t e =
        launch_pdl(fn, dim3(static_cast<unsigned>(a.samples), cols),
                   dim3(kLanes * (few ? 4 : kFinishSlices)), 0, st, args);
    if (e != cudaSuccess) return e;
  }
  const bool pre = a.part_pre != nullptr;
  const bool s = a.part_s != nullptr && (!several || a.dw_post != nullptr);
  if (!pre && !s) return cudaSuccess;
  return launch_pdl(reinterpret_cast<const void*>(&blk_finish_kernel),
                    dim3(cols, static_cast<unsigned>(pre) + static_cast<unsigned>(s)),
                    dim3(kLanes * kFinishSlices), 0, st, args);
}

}  // namespace blk
