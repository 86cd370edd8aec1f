// blk_launch.h -- argument blocks, launch shapes and launchers of a block's boundary
// (include/block_train.h) and of the norms that keep 8-bit activations (include/act8_train.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace blk {

constexpr int kMaxH = 8192;
// Most threads of a CTA, one CTA an SM.  A row costs a thread some 150 instructions (its waits,
// the sums' reduction, rstd, addresses) whatever its share of the row, so threads own 32 elements
// where the row has them, and as many threads run as have the registers for that: the waiting row
// and one weight in 128 (32768 x 4096 forward: 112 us with 512 threads, 128 with 384), two weights
// in 168 (with 512 threads of 24 elements 171 us against 177, but in 8 bits 240 against 218); in
// the backward column sums besides, of which one fits 168, two take 255 (with 512 threads of 16
// elements 265 us as well as 266).
enum { kKeep = 0, kPre = 1, kBoth = 2, kPost = 3 };
constexpr int fwd_threads(int form) { return form == kKeep ? 512 : 384; }
// From 8 bits the backward can keep a thread's column sums in tensor memory and run more threads with
// the registers that frees.  It does where that makes room for another row in a CTA: with both norms
// up to 6144 elements a row (65536 x 4096: 445 us against 464, 30720 x 6144 330 against 352, 65536 x
// 1536 175 against 202; wider rows are one at a time either way, 32768 x 8192 498 against 451), in the
// 8-bit norm past that (32768 x 8192 218 us against 278, with dh 317 against 318; 65536 x 4096 with dh 302
// against 296, though without 221 against 245).  From 16 bits it gains little or loses (65536 x 1536 199
// us against 202, 65536 x 512 87 against 81).
__host__ __device__ constexpr bool uses_tmem(int form, bool packed, int H) {
  return packed && (form == kBoth ? H <= 6144 : form == kKeep && H > 6144);
}
// The 8-bit norm's rows of three vectors a thread leave registers for a third more rows at a time.
// That pays where a row is one warp or two: without dh 65536 x 1536 102 us against 108, 262144 x 1536
// 356 against 397 (131072 x 768 96 against 93); with dh 120 against 119, 32768 x 1536 66 against 67 (FP16
// 66 against 70), 65536 x 768 67 against 70.  This form has three vectors only where every thread has
// all of them, so that is 768 and 1536 columns.  It does not pay where several rows lie in a warp
// (131072 x 384 57 against 53), with longer teams (65536 x 2304 with dh 180 against 171), or from 16
// bits (65536 x 1536 140 against 137, with dh 170 against 170); with both norms registers spill (65536
// x 1536 208 against 180).
constexpr bool more_rows(int form, bool packed, int vpt, int ntg) {
  return form == kKeep && packed && vpt == 3 && (ntg == 32 || ntg == 64);
}
__host__ __device__ constexpr int bwd_threads(int form, bool tmem, bool more) {
  return form == kKeep ? (tmem || more ? 512 : 384) : (tmem ? 384 : 256);
}
constexpr int kMaxWarps = 16;
constexpr int kMaxTensors = 4;    // staged
// CTAs of the backward at most, whatever the GPU: the rows' partition, and with it the order of
// every sum, is a function of the shape.  GB300 has 152 SMs: there it is one wave.
constexpr int kPartSMs = 152;
constexpr int kFinishCols = 32;

// What a kernel computes (the enumeration above).
//   kKeep  h = x [+ residual], rounded; norm before; h held in 8 bits    (rmsnorm_act8)
//   kPre   scales and gate, norm before
//   kBoth  norm behind, scales and gate, norm before
//   kPost  norm behind, scales and gate
// The backward has three forms with a norm before: kKeep (no x: no gate), kPre (x for the gate's
// gradient), kBoth; and kPost.

// A team of ntg threads (4, 8, 16: part of a warp, 32 / ntg rows side by side; 32; or several
// whole warps) takes one row (or those of its warp) at a time from its own ring of `stages` slots, each
// of `steps` such takes.
struct Shape {
  int vpt;      // 16-byte vectors (8 elements) a thread: 1 to 4
  int ntg;      // threads a row
  int teams;    // teams (of whole warps) a CTA
  int rows;     // rows a slot
  int stages;   // slots a team
  int threads;  // a CTA
  int P;        // CTAs
  bool factor;  // the branch's factors are in shared memory
  size_t slot;  // bytes
  size_t smem;  // bytes
};

struct Staged {
  const unsigned char* p;  // null: not staged
  int64_t stride;          // bytes between rows
  uint32_t bytes;          // of a row
  uint32_t off;            // within a slot
};

struct Args {
  Staged in[kMaxTensors];
  int32_t R, H;
  int32_t L;               // rows a sample
  int32_t samples;         // N
  const void* w_pre;
  const void* w_post;
  const void* gate;
  int32_t w_dtype, gate_dtype;
  float scale, residual_scale, eps;
  int32_t ntg, teams, rows, stages;
  uint32_t slot;
  unsigned* err;
};

// Forward: staged x, residual.
struct FwdArgs : Args {
  void* y;
  void* h;
  float* rstd_pre;
  float* rstd_post;
  unsigned char* x8;
  unsigned char* h8;
};

// Backward: staged h, dy, dh, x.
struct BwdArgs : Args {
  const float* rstd_pre;
  const float* rstd_post;
  void* dx;
  void* dres;
  int32_t fold;       // slots after which a thread's column sums go to their second level (0: never)
  uint32_t factor_at; // where the branch's factors lie in shared memory (factor_in_smem)
  float* part_pre;    // [P][H]: sums of dy * hhat, a row a CTA
  float* part_s;      // sums of t * xhat: [P][H], a row a CTA, or with several samples
                      // [P * teams + N - 1][H], a row a team and sample
};

// Whether every thread of a row has all its vectors, and every row of a warp is there: kernels are
// built for that case apart, without a predicate on any vector.
__host__ __device__ inline bool even_rows(int H, int vpt, int ntg) {
  return ntg >= 32 && H == 8 * vpt * ntg;
}

// Backward builds whose branch's factor (scale * gate * w_post of a thread's columns) is in shared
// memory: 4 bytes an element that a team's threads own, after everything else.  With both norms from
// 8 bits, whose kept vectors need the registers (65536 x 4096: 444 us against 607; 65536 x 1536 175
// against 176).  From 16 bits it gains nothing (65536 x 4096 523 us against 520, 30720 x 6144 358 against
// 359, 65536 x 1536 202 against 205, 30000 x 1000 82 against 77).
__host__ __device__ constexpr bool factor_in_smem(int form, bool packed) {
  return form == kBoth && packed;
}

// Builds of the backward: for column sums of one level, dh there or not; and for those of two (long
// runs of rows), with and without dh, each a build: told at run time the row's loop takes 3 % more
// instructions around the second level (65536 x 1536, both norms, 211 us against 205).
enum { kShort = 0, kLongNoDh = 1, kLongDh = 2 };

// First row of team k of n.
__host__ __device__ inline int32_t team_row(int64_t k, int64_t R, int64_t n) {
  return static_cast<int32_t>(k * R / n);
}
// The team that takes row r.
__host__ __device__ inline int64_t row_team(int64_t r, int64_t R, int64_t n) {
  return ((r + 1) * n - 1) / R;
}

cudaError_t launch_fwd(const FwdArgs& a, const Shape& s, int dtype, int form, bool pack,
                       cudaStream_t st);
cudaError_t launch_bwd(const BwdArgs& a, const Shape& s, int dtype, int form, bool packed,
                       cudaStream_t st);

// The sums' last step.
struct FinishArgs {
  const float* part_pre;   // null: no norm before
  float* part_s;           // null: neither norm behind nor gate
  int64_t ctas, teams;     // teams: of all CTAs
  int32_t R, H, samples;
  const void* w_post;
  const void* gate;
  int32_t w_dtype, gate_dtype;
  float scale;
  float* dw_pre;
  float* dw_post;          // null: no norm behind
  float* dgate;            // null: no gate
};
cudaError_t launch_finish(const FinishArgs& a, cudaStream_t st);

}  // namespace blk
