// blk_finish.cu -- the last step of the column sums of a block's boundary: the rows that the teams
// wrote are added in a fixed order, and dw_pre, dw_post and the gate's gradient formed of them.
#include "blk_common.cuh"

namespace blk {

namespace {

constexpr int kLanes = kFinishCols / 4;  // threads of four columns each side by side

// Sums of four columns over kFinishSlices threads each (sh: two vectors a thread): `each(add)` adds a
// thread's vectors, the threads' sums are then joined pairwise.  The errors of the additions are
// carried along.  Every thread of the block calls it; the result is that of the threads with sl == 0.
template <typename Each>
__device__ __forceinline__ float4 joined_sums(float4* sh, int sl, int cl, Each each) {
  float4* const se = sh + kFinishSlices * kLanes;
  float s[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
  each([&](const float4& v) {
    const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float err;
      s[k] = add_exact(s[k], w[k], err);
      e[k] = __fadd_rn(e[k], err);
    }
  });
  const int p = sl * kLanes + cl;
  sh[p] = make_float4(s[0], s[1], s[2], s[3]);
  se[p] = make_float4(e[0], e[1], e[2], e[3]);
  __syncthreads();
#pragma unroll
  for (int stride = kFinishSlices / 2; stride > 0; stride >>= 1) {
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

// Of n vectors f(0), f(1), ...: each thread takes a contiguous share, five loads at a time (the rows of
// 152 CTAs: one turn).
template <typename F>
__device__ __forceinline__ float4 column_sums(float4* sh, int64_t n, int sl, int cl, bool live, F f) {
  return joined_sums(sh, sl, cl, [&](auto add) {
    if (!live) return;
    const int64_t i1 = (sl + 1) * n / kFinishSlices;
    for (int64_t i = sl * n / kFinishSlices; i < i1; i += 5) {
      float4 v[5];
#pragma unroll
      for (int u = 0; u < 5; ++u) v[u] = i + u < i1 ? f(i + u) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 5; ++u) add(v[u]);
    }
  });
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

// Blocks: blockIdx.x 0 for dw_pre (with a norm before), then one for S's results with one sample;
// with several, one for dw_post (with a norm behind) and one for each sample's gate.
__global__ void __launch_bounds__(kLanes* kFinishSlices, 4) blk_finish_kernel(const FinishArgs a) {
  __shared__ float4 sh[2 * kFinishSlices * kLanes];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int cl = threadIdx.x % kLanes, sl = threadIdx.x / kLanes;
  const int col = blockIdx.y * kFinishCols + 4 * cl;
  const bool live = col < a.H, write = live && sl == 0;
  int64_t block = blockIdx.x;
  if (a.part_pre != nullptr && block-- == 0) {
    const float* p = a.part_pre + col;
    const float4 s = column_sums(sh, a.ctas, sl, cl, live,
                                                [&](int64_t i) { return at4(p, i * a.H); });
    if (write) put4(a.dw_pre, col, s);
    return;
  }
  const float* p = a.part_s + col;
  if (a.samples == 1) {
    const float4 s = times(column_sums(sh, a.ctas, sl, cl, live,
                                                      [&](int64_t i) { return at4(p, i * a.H); }),
                           a.scale);
    if (write && a.dw_post != nullptr) put4(a.dw_post, col, times(s, a.gate, a.gate_dtype, col));
    if (write && a.dgate != nullptr) put4(a.dgate, col, times(s, a.w_post, a.w_dtype, col));
    return;
  }
  if (a.dw_post != nullptr && block-- == 0) {  // every row of S times its sample's gate
    // a sample's rows by several threads a column, or several samples' by one
    const int64_t N = a.samples, L = a.R / N;
    const int parts = N < kFinishSlices ? kFinishSlices / static_cast<int>(N) : 1;
    const float4 s = joined_sums(sh, sl, cl, [&](auto add) {
      if (!live) return;
      for (int64_t n = sl / parts; n < N; n += kFinishSlices) {
        const int64_t k0 = row_team(n * L, a.R, a.teams);
        const int64_t rows = row_team((n + 1) * L - 1, a.R, a.teams) - k0 + 1;
        const int64_t i1 = (sl % parts + 1) * rows / parts;
        const float4 g =
            times(make_float4(1.f, 1.f, 1.f, 1.f), a.gate, a.gate_dtype, n * a.H + col);
        for (int64_t i = sl % parts * rows / parts; i < i1; i += 5) {
          float4 v[5];
#pragma unroll
          for (int u = 0; u < 5; ++u)
            v[u] = i + u < i1 ? at4(p, (k0 + n + i + u) * a.H) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int u = 0; u < 5; ++u)
            if (i + u < i1)
              add(make_float4(v[u].x * g.x, v[u].y * g.y, v[u].z * g.z, v[u].w * g.w));
        }
      }
    });
    if (write) put4(a.dw_post, col, times(s, a.scale));
    return;
  }
  const int64_t n = block, rows = a.R / a.samples;
  const int64_t k0 = row_team(n * rows, a.R, a.teams), k1 = row_team((n + 1) * rows - 1, a.R, a.teams);
  const float* q = p + (k0 + n) * a.H;
  const float4 s = column_sums(sh, k1 - k0 + 1, sl, cl, live,
                                              [&](int64_t i) { return at4(q, i * a.H); });
  if (write) put4(a.dgate, n * a.H + col, times(times(s, a.scale), a.w_post, a.w_dtype, col));
}

}  // namespace

cudaError_t launch_finish(const FinishArgs& a, cudaStream_t st) {
  FinishArgs copy = a;
  void* args[] = {&copy};
  int64_t blocks = a.part_pre != nullptr ? 1 : 0;
  if (a.part_s != nullptr)
    blocks += a.samples == 1 ? 1 : (a.dw_post != nullptr ? 1 : 0) + static_cast<int64_t>(a.samples);
  return launch_pdl(reinterpret_cast<const void*>(&blk_finish_kernel),
                    dim3(static_cast<unsigned>(blocks),
                         static_cast<unsigned>((a.H + kFinishCols - 1) / kFinishCols)),
                    dim3(kLanes * kFinishSlices), 0, st, args);
}

}  // namespace blk
