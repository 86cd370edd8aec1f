// gn_launch.h -- group norm kernel argument blocks, plans and launchers (host + device).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gnorm {

// A CTA owns a slab -- whole groups whose channels make whole 16-byte vectors -- of some
// consecutive places of one sample.  Its threads form `lanes` rows of `vecs` threads; thread
// (lane, vec) owns 16-byte vector vec of places lane, lane + lanes, ...
// Two forms, one launch each:
//  on chip   `ctas` CTAs of a cluster split a sample's places and keep the slab in shared memory
//            between the statistics and the output
//  streamed  a cooperative grid takes units -- slabs of samples -- in turns of some tens of
//            megabytes, each split into `chunks` of places: statistics, a barrier of the grid, output
struct GnShape {
  int ev;        // elements a 16-byte vector
  int cg;        // channels a group
  int gs;        // groups a slab
  int cs;        // channels a slab = gs * cg
  int vecs;      // 16-byte vectors a slab = cs / ev
  int slabs;     // slabs a sample
  int lanes;     // rows of threads
  int threads;   // lanes * vecs, up to whole warps
  int on_chip;
  // on chip
  int ctas;      // CTAs a cluster, 1 << ctas_log2
  int ctas_log2;
  int iters;     // most places a thread takes
  int lanes_n;   // clusters a slab (each takes samples lane, lane + lanes_n, ...)
  int stages;    // samples a cluster has staged or on their way
  // streamed
  int units;     // units a turn takes, unit u the slab u % slabs of sample u / slabs
  int chunks;    // the first chunk_more of chunk_base + 1 places, the others of chunk_base
  int chunk_base, chunk_more;
  int seqs;      // backward: sequences of pieces that share a row of column sums (0: a row a piece)
  int grid;      // CTAs at most
  size_t smem;   // dynamic shared memory
};

struct GnArgs {
  const void* x;
  const void* dy;        // backward
  const void* w;
  const void* b;
  void* out;             // y, or dx
  float* mean;           // [N, G]; backward: read
  float* rstd;
  float2* part;          // streamed: [N][chunks][G]: (mean, M2), or (sum g*xhat, sum g)
  float* cols;           // backward: [.][2][C] column sums (dw, then db); of sequences, their
                         // compensations behind them
  int64_t s_n, s_s;      // x's strides
  int64_t N;
  int64_t S;
  int32_t C, G;
  int32_t wb_dtype;
  float eps;
  GnShape s;
};

// Two builds of every kernel, both with 128 registers a thread (enough for several vectors'
// independent work, which hides more latency here than a third CTA of 80 registers did: 5-15 %
// at every size measured): CTAs of up to kThreads threads, kCtas of them an SM, and, for slabs
// of more than kThreads vectors, up to kWideThreads threads, one CTA an SM.
constexpr int kThreads = 256, kWideThreads = 512;
constexpr int kCtas = 2;
constexpr int kMaxCluster = 8;
constexpr int max_threads(bool wide) { return wide ? kWideThreads : kThreads; }
constexpr int min_ctas(bool wide) { return wide ? 1 : kCtas; }

// Streamed: each thread's copies run through a ring of ring_groups groups of kRingPlaces places;
// on chip, `iters` places of each of `stages` samples are staged.  (Forward, bf16: 4 groups 135 us
// at 8 x 65536 x 256 and 90.8 at 64 x 4096 x 320, 6 groups 129 and 87.6, 8 groups 130 and 86.4 but
// 4 % more on the smallest streamed calls; backward, two tensors: 4 groups 227 and 155, 6 groups
// 235 and 159.)
constexpr int kRingPlaces = 2;
inline __host__ __device__ constexpr int ring_groups(int tensors) { return tensors == 1 ? 6 : 4; }
inline __host__ __device__ constexpr int ring_slots(int tensors) {
  return ring_groups(tensors) * kRingPlaces;
}
// Bytes of one staged sample, or of the ring.
inline __host__ __device__ size_t gn_stage_bytes(const GnShape& s, bool bwd) {
  const int tensors = bwd ? 2 : 1;
  return static_cast<size_t>(tensors) * (s.on_chip ? s.iters : ring_slots(tensors)) * s.threads *
         16;
}
// Shared memory of the kernels behind the staged vectors, in floats:
//   w, b  cs parameters each
//   c0, c1  cs channel constants each (forward: -mean and rstd * w; backward: nc1 and nc2)
//   col   2 * cs column values; on chip backward: + 4 * cs running totals (sum, compensation)
//   gm    2 * gs: the CTA's group values
//   ms    2 * gs: backward, the sample's mean and rstd of the slab's groups
//   red   2 planes [lanes][red_stride]: per-thread column values on their way to column sums
//         (forward: mean and M2; backward: A and B); streamed: over the ring, which is empty
//         then
// A row of red is padded so that four rows of eight columns fall on 32 different banks wherever
// the slab is a multiple of 32 channels.
inline __host__ __device__ int red_stride(const GnShape& s) { return s.cs + (s.cs % 32 ? 0 : 8); }
inline __host__ __device__ size_t gn_red_bytes(const GnShape& s) {
  return 2 * static_cast<size_t>(s.lanes) * red_stride(s) * sizeof(float);
}
inline __host__ __device__ size_t gn_front_bytes(const GnShape& s, bool bwd) {  // staged vectors
  const size_t stage = gn_stage_bytes(s, bwd), red = gn_red_bytes(s);
  if (s.on_chip) return stage * s.stages;
  return ((stage > red ? stage : red) + 15) & ~static_cast<size_t>(15);
}
inline __host__ __device__ size_t gn_stats_smem(const GnShape& s, bool bwd) {
  const size_t n = 6 * static_cast<size_t>(s.cs) + (bwd && s.on_chip ? 4 * s.cs : 0) +
                   4 * static_cast<size_t>(s.gs);
  return gn_front_bytes(s, bwd) + n * sizeof(float) + (s.on_chip ? gn_red_bytes(s) : 0);
}
// CTAs of the launch.
inline int64_t gn_ctas(const GnShape& s) {
  return s.on_chip ? static_cast<int64_t>(s.slabs) * s.ctas * s.lanes_n : s.grid;
}

// Launches fn: in clusters with programmatic dependent launch, or as a cooperative grid.
cudaError_t launch_gn(const void* fn, const GnArgs& a, cudaStream_t st);

// dtype and act: GROUPNORM_*.
cudaError_t launch_gn_fwd(const GnArgs& a, int dtype, int act, cudaStream_t st);
cudaError_t launch_gn_bwd(const GnArgs& a, int dtype, int act, cudaStream_t st);
// dw, db = the sums of `rows` column-sum rows [2][C] (rows == 0: zeros).
cudaError_t launch_gn_finish(const float* cols, float* dw, float* db, int64_t rows, int C,
                             cudaStream_t st);

}  // namespace gnorm
