// gn_launch.h -- group norm kernel argument blocks, plans and launchers (host + device).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gnorm {

// A CTA owns a slab -- whole groups whose channels make whole 16-byte vectors -- of some
// consecutive places of one sample.  Its threads form `lanes` rows of `vecs` threads; thread
// (lane, vec) owns 16-byte vector vec of places lane, lane + lanes, ...  `ctas` CTAs of a
// cluster split a sample's (or a chunk's) places between them.
struct GnShape {
  int ev;        // elements a 16-byte vector
  int cg;        // channels a group
  int gs;        // groups a slab
  int cs;        // channels a slab = gs * cg
  int vecs;      // 16-byte vectors a slab = cs / ev
  int slabs;     // slabs a sample
  int lanes;     // rows of threads
  int threads;   // lanes * vecs, up to whole warps
  int ctas;      // CTAs a cluster
  int iters;     // most places a thread takes
  int on_chip;   // the slab stays in shared memory between statistics and output
  int lanes_n;   // on chip: clusters a slab (each takes samples lane, lane + lanes_n, ...)
  int chunks;    // two launches: chunks of places a sample's statistics are split into
  int samples;   // two launches: samples a pair of launches takes
  int parts;     // two launches: chunks of places of the second launch
  int part_iters;  // most places a thread of the second launch takes
  size_t smem;   // dynamic shared memory of the (first) launch
};

struct GnArgs {
  const void* x;
  const void* dy;        // backward
  const void* w;
  const void* b;
  void* out;             // y, or dx
  float* mean;           // [N, G]; backward: read
  float* rstd;
  float2* part;          // two launches: [N][chunks][G]: (mean, M2), or (sum g*xhat, sum g)
  float* cols;           // backward: [.][2][C] column sums (dw, then db)
  int64_t s_n, s_s;      // x's strides
  int64_t n0;            // first sample of this launch
  int64_t n1;            // end of its samples
  int64_t S;
  int32_t C, G;
  int32_t wb_dtype;
  float eps;
  GnShape s;
};

constexpr int kMaxThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = kMaxThreads / 32;

// Shared memory behind the staged vectors (floats unless said otherwise), in this order:
//   red    tensors * threads * ev: per-thread column values on their way to sums
//   parts  kMaxWarps + gs: per-warp partial sums of groups
//   gm     2 * gs: the CTA's group values, then
//   all    2 * gs * ctas: every CTA's (float2), gathered
//   gf     2 * gs: the sample's final group values
//   col    backward: 2 * cs column sums; on chip: + 4 * cs running totals (sum, compensation)
inline __host__ __device__ size_t gn_extra_floats(const GnShape& s, bool bwd) {
  size_t n = static_cast<size_t>(bwd ? 2 : 1) * s.threads * s.ev;
  n += kMaxWarps + s.gs;
  n += 2 * static_cast<size_t>(s.gs) + 2 * static_cast<size_t>(s.gs) * s.ctas +
       2 * static_cast<size_t>(s.gs);
  if (bwd) n += static_cast<size_t>(s.on_chip ? 6 : 2) * s.cs;
  return (n + 3) & ~static_cast<size_t>(3);
}
inline __host__ __device__ size_t gn_stage_bytes(const GnShape& s, bool bwd) {
  return s.on_chip ? static_cast<size_t>(bwd ? 2 : 1) * s.iters * s.threads * 16 : 0;
}

// CTAs of the launches over `samples` samples.
inline int64_t gn_stats_ctas(const GnShape& s, int64_t samples) {
  return static_cast<int64_t>(s.slabs) * s.ctas * (s.on_chip ? s.lanes_n : samples * s.chunks);
}
inline int64_t gn_out_ctas(const GnShape& s, int64_t samples) {
  return static_cast<int64_t>(s.slabs) * samples * s.parts;
}

// Launches fn over `ctas` CTAs in clusters of s.ctas, with programmatic dependent launch.
cudaError_t launch_cluster(const void* fn, int64_t ctas, const GnShape& s, const GnArgs& a,
                           cudaStream_t st);

// Launch the statistics (and, on chip, the output) of samples [a.n0, a.n1); then, for two
// launches, the output.  dtype and act: GROUPNORM_*.
cudaError_t launch_gn_fwd(const GnArgs& a, int dtype, int act, cudaStream_t st);
cudaError_t launch_gn_fwd_out(const GnArgs& a, int dtype, int act, cudaStream_t st);
cudaError_t launch_gn_bwd(const GnArgs& a, int dtype, int act, cudaStream_t st);
cudaError_t launch_gn_bwd_out(const GnArgs& a, int dtype, int act, cudaStream_t st);
// dw, db = the sums of `rows` column-sum rows [2][C] (rows == 0: zeros).
cudaError_t launch_gn_finish(const float* cols, float* dw, float* db, int64_t rows, int C,
                             cudaStream_t st);

}  // namespace gnorm
