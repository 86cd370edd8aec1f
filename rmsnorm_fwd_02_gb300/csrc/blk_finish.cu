// blk_finish.cu -- the last step of the column sums of a block's boundary: the rows that the teams
// wrote are added in a fixed order, and dw_pre, dw_post and the gate's gradient formed of them.
#include "blk_common.cuh"

namespace blk {

namespace {

// Sum of n values f(0), f(1), ... over kSlices threads a column: each takes a contiguous share,
// five loads at a time (the rows of 152 CTAs: two turns), the shares are then joined pairwise.  The errors of the additions are
// carried along.  Every thread of the block calls it; the result is thread 0's of the column.
template <int kSlices, typename F>
__device__ __forceinline__ float column_sum(int64_t n, int sl, int cl, bool live, float* sh, float* se,
                                            F f) {
  float s = 0.f, e = 0.f;
  if (live) {
    const int64_t i1 = (sl + 1) * n / kSlices;
    for (int64_t i = sl * n / kSlices; i < i1; i += 5) {
      float v[5];
#pragma unroll
      for (int u = 0; u < 5; ++u) v[u] = i + u < i1 ? f(i + u) : 0.f;
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        float err;
        s = add_exact(s, v[u], err);
        e = __fadd_rn(e, err);
      }
    }
  }
  sh[sl * kFinishCols + cl] = s;
  se[sl * kFinishCols + cl] = e;
  __syncthreads();
#pragma unroll
  for (int stride = kSlices / 2; stride > 0; stride >>= 1) {
    if (sl < stride) {
      const int p = sl * kFinishCols + cl, q = p + stride * kFinishCols;
      float err;
      const float t = add_exact(sh[p], sh[q], err);
      se[p] = __fadd_rn(__fadd_rn(se[p], se[q]), err);
      sh[p] = t;
    }
    __syncthreads();
  }
  // a sum that passed FP32's range, or met one: its errors are no numbers
  const float t = sh[cl];
  return isfinite(t) ? __fadd_rn(t, se[cl]) : t;
}

// Several samples: a sample's rows of S become one, scaled, in the first one's place, and its
// gradient of the gate.
template <int kSlices>
__global__ void __launch_bounds__(kFinishCols* kSlices) blk_samples_kernel(const FinishArgs a) {
  __shared__ float sh[kSlices * kFinishCols], se[kSlices * kFinishCols];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int cl = threadIdx.x % kFinishCols, sl = threadIdx.x / kFinishCols;
  const int col = blockIdx.y * kFinishCols + cl;
  const int64_t n = blockIdx.x;
  const int64_t rows = a.R / a.samples;
  const int64_t k0 = row_team(n * rows, a.R, a.teams), k1 = row_team((n + 1) * rows - 1, a.R, a.teams);
  float* p = a.part_s + (k0 + n) * a.H + col;
  const float s = column_sum<kSlices>(k1 - k0 + 1, sl, cl, col < a.H, sh, se,
                                      [&](int64_t i) { return p[i * a.H]; });
  if (sl == 0 && col < a.H) {
    const float t = a.scale * s;
    *p = t;
    if (a.dgate != nullptr)
      a.dgate[n * a.H + col] = a.w_post != nullptr ? load1(a.w_post, a.w_dtype, col) * t : t;
  }
}

__global__ void __launch_bounds__(kFinishCols* kFinishSlices) blk_finish_kernel(const FinishArgs a) {
  __shared__ float sh[kFinishSlices * kFinishCols], se[kFinishSlices * kFinishCols];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int cl = threadIdx.x % kFinishCols, sl = threadIdx.x / kFinishCols;
  const int col = blockIdx.x * kFinishCols + cl;
  const bool live = col < a.H;
  if (a.part_pre != nullptr && blockIdx.y == 0) {
    const float* p = a.part_pre + col;
    const float s = column_sum<kFinishSlices>(a.ctas, sl, cl, live, sh, se,
                                              [&](int64_t i) { return p[i * a.H]; });
    if (sl == 0 && live) a.dw_pre[col] = s;
    return;
  }
  const float* p = a.part_s + col;
  if (a.samples == 1) {
    const float s = a.scale * column_sum<kFinishSlices>(a.ctas, sl, cl, live, sh, se,
                                                        [&](int64_t i) { return p[i * a.H]; });
    if (sl == 0 && live) {
      if (a.dw_post != nullptr)
        a.dw_post[col] = a.gate != nullptr ? load1(a.gate, a.gate_dtype, col) * s : s;
      if (a.dgate != nullptr)
        a.dgate[col] = a.w_post != nullptr ? load1(a.w_post, a.w_dtype, col) * s : s;
    }
  } else {  // the samples' sums, each times its gate
    const int64_t rows = a.R / a.samples;
    const float s = column_sum<kFinishSlices>(a.samples, sl, cl, live, sh, se, [&](int64_t n) {
      return p[(row_team(n * rows, a.R, a.teams) + n) * a.H] *
             load1(a.gate, a.gate_dtype, n * a.H + col);
    });
    if (sl == 0 && live) a.dw_post[col] = s;
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
    const bool few = a.teams / a.samples < 40;
    const void* fn = few ? reinterpret_cast<const void*>(&blk_samples_kernel<4>)
                         : reinterpret_cast<const void*>(&blk_samples_kernel<kFinishSlices>);
    const cudaError_t e =
        launch_pdl(fn, dim3(static_cast<unsigned>(a.samples), cols),
                   dim3(kFinishCols * (few ? 4 : kFinishSlices)), 0, st, args);
    if (e != cudaSuccess) return e;
  }
  const bool pre = a.part_pre != nullptr;
  const bool s = a.part_s != nullptr && (!several || a.dw_post != nullptr);
  if (!pre && !s) return cudaSuccess;
  return launch_pdl(reinterpret_cast<const void*>(&blk_finish_kernel),
                    dim3(cols, static_cast<unsigned>(pre) + static_cast<unsigned>(s)),
                    dim3(kFinishCols * kFinishSlices), 0, st, args);
}

}  // namespace blk
