// blk_finish.cu -- the last step of the column sums of a block's boundary: the rows that the teams
// wrote are added in a fixed order, and dw_pre, dw_post and the gate's gradient formed of them.
#include "blk_common.cuh"

namespace blk {

namespace {

// A block is kL threads of four columns each side by side and kThreads / kL slices of the rows.  How
// many decides how long the loads of a thread follow one another, which is what the step's time is:
// 8 x 32 for the rows of 152 CTAs; 2 x 128 (whole 32-byte sectors) for those of every team; 64 x 4
// for the few of a sample's where there are many samples.  With 8 x 32 for all of them the backward of
// 131072 x 128 from 8 bits, eight samples, took 53.0 us against 50.6, of 4096 x 1536 with 64 samples
// 40 against 27, with 512 samples 124 against 43.
constexpr int kThreads = 256;

// Sums of four columns over the slices (sh: two vectors a thread): `each(add)` adds a thread's
// vectors, the threads' sums are then joined pairwise.  The errors of the additions are carried
// along.  Every thread of the block calls it; the result is that of the threads of slice 0.
template <int kL, typename Each>
__device__ __forceinline__ float4 joined_sums(float4* sh, Each each) {
  const int cl = threadIdx.x % kL, sl = threadIdx.x / kL;
  float4* const se = sh + kThreads;
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
  const int p = sl * kL + cl;
  sh[p] = make_float4(s[0], s[1], s[2], s[3]);
  se[p] = make_float4(e[0], e[1], e[2], e[3]);
  __syncthreads();
#pragma unroll
  for (int stride = kThreads / kL / 2; stride > 0; stride >>= 1) {
    if (sl < stride) {
      const float4 a = sh[p + stride * kL], b = se[p + stride * kL];
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

// Of n vectors f(0), f(1), ...: each thread takes a contiguous share, five loads at a time (the rows
// of 152 CTAs: one turn).
template <int kL, typename F>
__device__ __forceinline__ float4 column_sums(float4* sh, int64_t n, bool live, F f) {
  return joined_sums<kL>(sh, [&](auto add) {
    if (!live) return;
    constexpr int kSlices = kThreads / kL;
    const int sl = threadIdx.x / kL;
    const int64_t i1 = (sl + 1) * n / kSlices;
    for (int64_t i = sl * n / kSlices; i < i1; i += 5) {
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

// The gate's gradient of sample n, four columns a thread from `col` on.
template <int kL>
__device__ __forceinline__ void gate_grad(const FinishArgs& a, float4* sh, int64_t n, int col) {
  const bool live = col < a.H;
  const int64_t rows = a.R / a.samples, k0 = row_team(n * rows, a.R, a.teams);
  const int64_t k1 = row_team((n + 1) * rows - 1, a.R, a.teams);
  const float* q = a.part_s + (k0 + n) * a.H + col;
  const float4 s =
      column_sums<kL>(sh, k1 - k0 + 1, live, [&](int64_t i) { return at4(q, i * a.H); });
  if (live && threadIdx.x < kL)
    put4(a.dgate, n * a.H + col, times(times(s, a.scale), a.w_post, a.w_dtype, col));
}

// Whether a sample has so few rows of sums that a block takes eight times the columns of them, and
// with its neighbours along blockIdx.y that many samples.
constexpr int kWideSamples = 8;
__host__ __device__ inline bool wide_samples(const FinishArgs& a) {
  return a.samples > 1 && a.teams / a.samples + 2 <= 20;  // (a turn of loads)
}

// Blocks: blockIdx.x 0 for dw_pre (with a norm before), then one for S's results with one sample;
// with several, four for dw_post (with a norm behind) and one for each sample's gate, or for
// kWideSamples' of them.  blockIdx.y: kFinishCols columns (a quarter of them for each of the four).
__global__ void __launch_bounds__(kThreads, 4) blk_finish_kernel(const FinishArgs a) {
  __shared__ float4 sh[2 * kThreads];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int first = blockIdx.y * kFinishCols, tid = threadIdx.x;
  constexpr int kL = kFinishCols / 4;
  const int col = first + 4 * (tid % kL);
  const bool live = col < a.H, write = live && tid < kL;
  int64_t block = blockIdx.x;
  if (a.part_pre != nullptr && block-- == 0) {
    const float* p = a.part_pre + col;
    const float4 s =
        column_sums<kL>(sh, a.ctas, live, [&](int64_t i) { return at4(p, i * a.H); });
    if (write) put4(a.dw_pre, col, s);
    return;
  }
  if (a.samples == 1) {
    const float* p = a.part_s + col;
    const float4 s = times(
        column_sums<kL>(sh, a.ctas, live, [&](int64_t i) { return at4(p, i * a.H); }), a.scale);
    if (write && a.dw_post != nullptr) put4(a.dw_post, col, times(s, a.gate, a.gate_dtype, col));
    if (write && a.dgate != nullptr) put4(a.dgate, col, times(s, a.w_post, a.w_dtype, col));
    return;
  }
  if (a.dw_post != nullptr && (block -= 4) < 0) {  // every row of S times its sample's gate
    // a sample's rows by several threads a column, or several samples' by one
    constexpr int kPostL = kL / 4, kSlices = kThreads / kPostL;
    const int c = first + 4 * kPostL * static_cast<int>(block + 4) + 4 * (tid % kPostL);
    const int sl = tid / kPostL;
    const float* p = a.part_s + c;
    const int64_t N = a.samples, L = a.R / N;
    const int parts = N < kSlices ? kSlices / static_cast<int>(N) : 1;
    const float4 s = joined_sums<kPostL>(sh, [&](auto add) {
      if (c >= a.H) return;
      for (int64_t n = sl / parts; n < N; n += kSlices) {
        const int64_t k0 = row_team(n * L, a.R, a.teams);
        const int64_t rows = row_team((n + 1) * L - 1, a.R, a.teams) - k0 + 1;
        const int64_t i1 = (sl % parts + 1) * rows / parts;
        const float4 g =
            times(make_float4(1.f, 1.f, 1.f, 1.f), a.gate, a.gate_dtype, n * a.H + c);
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
    if (c < a.H && tid < kPostL) put4(a.dw_post, c, times(s, a.scale));
    return;
  }
  if (!wide_samples(a)) return gate_grad<kL>(a, sh, block, col);
  constexpr int kWideL = kL * kWideSamples;
  const int64_t n = block * kWideSamples + blockIdx.y % kWideSamples;
  if (n < a.samples)
    gate_grad<kWideL>(a, sh, n,
                      static_cast<int>(blockIdx.y) / kWideSamples * 4 * kWideL + 4 * (tid % kWideL));
}

}  // namespace

cudaError_t launch_finish(const FinishArgs& a, cudaStream_t st) {
  FinishArgs copy = a;
  void* args[] = {&copy};
  int64_t blocks = a.part_pre != nullptr ? 1 : 0, columns = (a.H + kFinishCols - 1) / kFinishCols;
  if (a.part_s != nullptr && a.samples == 1) blocks += 1;
  if (a.part_s != nullptr && a.samples > 1) {
    if (a.dw_post != nullptr) blocks += 4;
    if (wide_samples(a)) {
      blocks += (static_cast<int64_t>(a.samples) + kWideSamples - 1) / kWideSamples;
      columns = (columns + kWideSamples - 1) / kWideSamples * kWideSamples;
    } else {
      blocks += a.samples;
    }
  }
  return launch_pdl(reinterpret_cast<const void*>(&blk_finish_kernel),
                    dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(columns)),
                    dim3(kThreads), 0, st, args);
}

}  // namespace blk
