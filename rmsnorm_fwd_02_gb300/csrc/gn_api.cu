// gn_api.cu -- the group norm C ABI (include/groupnorm_train.h): argument checks, launch
// planning and kernel launches.  Never allocates, frees or synchronizes; every launch goes on
// the caller's stream.
#include <cmath>
#include <cstdint>
#include <numeric>

#include "gn_launch.h"
#include "groupnorm_train.h"  // include/ (on the include path)
#include "rmsn_common.cuh"

namespace gnorm {

namespace {

constexpr int kMaxC = 4096;
constexpr int64_t kMaxElements = int64_t{1} << 40;
constexpr size_t kMaxSmem = 227 * 1024;  // a CTA's
constexpr size_t kSmSmem = 220 * 1024;   // an SM's, over the CTAs it holds
// two CTAs an SM, so that one's loads overlap the other's exchange and stores
constexpr size_t kHalfSmem = kSmSmem / 2;
// The partition is a function of the shape, not of the GPU; its constants suit 152 SMs.
constexpr int kSMs = 152;
// CTAs that are resident together, `per_sm` an SM, in clusters of `ctas`: clusters keep within a
// GPC, so the larger ones leave SMs over (counts as cudaOccupancyMaxActiveClusters gives them).
int64_t resident(int per_sm, int ctas) {
  if (ctas <= 2) return static_cast<int64_t>(kSMs) * per_sm;
  static const int fours[4] = {144, 296, 440, 592}, eights[4] = {120, 288, 408, 576};
  const int* t = ctas == 4 ? fours : eights;
  return per_sm <= 4 ? t[per_sm - 1] : t[3] / 4 * per_sm;
}
// Bytes a place's slab aims at: at least a DRAM burst of two 64-byte halves.
constexpr int kSlabBytes = 128, kMinSlabBytes = 32;
constexpr int kSmallCta = 16 * 1024;  // staged bytes below which a CTA is not split further
constexpr int kMaxStages = 4;
// streamed: bytes of x (and dy) a turn takes at most.  Two turns are live at once, and L2 gives back
// part of that: 57 MB of a 67 MB sample's second read in the forward, 58 of a 134 MB one's,
// next to nothing in the backward, where what the turns buy is the hidden barrier (turns of 48 and
// of 100 MB were no faster).
constexpr int64_t kL2Bytes = int64_t{80} << 20;

int elem_bytes(int dtype) { return dtype == GROUPNORM_FP32 ? 4 : 2; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The slab of gs groups, and the threads for `rows` places a CTA at most, `least` a thread at
// least (fewer partial sums to combine, and room for other CTAs).
GnShape slab_shape(int dtype, int C, int G, int gs, int64_t rows, int least) {
  GnShape s{};
  s.ev = 16 / elem_bytes(dtype);
  s.cg = C / G;
  s.gs = gs;
  s.cs = gs * s.cg;
  s.vecs = s.cs / s.ev;
  s.slabs = G / gs;
  int64_t lanes = s.vecs >= kThreads ? 1 : kThreads / s.vecs;
  if (lanes > ceil_div(rows, least)) lanes = ceil_div(rows, least);
  s.iters = static_cast<int>(ceil_div(rows, lanes));
  s.lanes = static_cast<int>(ceil_div(rows, s.iters));  // evened out
  s.threads = (s.lanes * s.vecs + 31) / 32 * 32;
  s.ctas = 1;
  return s;
}

int least_groups(int dtype, int C, int G) {
  const int ev = 16 / elem_bytes(dtype);
  return ev / std::gcd(C / G, ev);
}

// The slab of at least `bytes` a place (fewest groups), or the widest there is.
int slab_groups(int dtype, int C, int G, int bytes) {
  const int gs0 = least_groups(dtype, C, G), units = G / gs0;
  const int one = gs0 * (C / G) * elem_bytes(dtype);
  int best = gs0;
  for (int m = 1; m <= units; ++m) {
    if (units % m != 0) continue;
    if (one * m / 16 > kWideThreads) break;
    best = gs0 * m;
    if (one * m >= bytes) break;
  }
  return best;
}

// One launch with the slab on chip: the fewest CTAs a cluster that let two CTAs share an SM
// (else one, which plan() takes for one place a sample alone), more while the GPU has idle SMs
// and the CTAs are not small; threads == 0 if a cluster of kMaxCluster cannot hold the slab.
GnShape on_chip_shape(int dtype, int64_t N, int64_t S, int C, int G, int gs, bool bwd) {
  GnShape best{};
  for (int k = 1; k <= kMaxCluster; k *= 2) {
    if (k > 1 && k > S) break;
    const int64_t rows = ceil_div(S, k);
    if (rows > (1 << 20)) continue;  // beyond any shared memory
    // many samples: throughput (measured at 1024 x 49 x 512: 35 us with 8, 55 with 4); few:
    // latency
    GnShape s = slab_shape(dtype, C, G, gs, rows, N * (G / gs) >= 8 * kSMs ? 8 : 4);
    s.ctas = k;
    s.ctas_log2 = k == 1 ? 0 : (k == 2 ? 1 : (k == 4 ? 2 : 3));
    s.on_chip = 1;
    s.stages = 1;
    const size_t stage = gn_stage_bytes(s, bwd);
    s.smem = gn_stats_smem(s, bwd);
    if (s.smem > kMaxSmem) continue;
    best = s;
    if (s.smem > kHalfSmem) continue;
    if (N * s.slabs * k >= kSMs || stage <= kSmallCta) break;
  }
  return best;
}

// How many clusters take a slab's samples, and how many samples each has staged: all at once
// while the SMs hold a CTA for every piece, else a loop over samples with the next ones on
// their way -- as many CTAs an SM as leave two stages each (two at least, while two fit).
void on_chip_loop(GnShape* s, int64_t N, bool bwd) {
  const size_t stage = gn_stage_bytes(*s, bwd), extra = s->smem - stage;
  const bool wide = s->vecs > kThreads;
  int most = min_ctas(wide) * max_threads(wide) / s->threads;  // by registers
  if (most > 16) most = 16;
  int ctas = static_cast<int>(kSmSmem / (2 * stage + extra));
  if (ctas < 2 && 2 * s->smem <= kSmSmem) ctas = 2;
  ctas = ctas < 1 ? 1 : (ctas > most ? most : ctas);
  const int64_t clusters = static_cast<int64_t>(s->slabs) * s->ctas;  // CTAs of one sample
  int64_t lanes = resident(ctas, s->ctas) / clusters;
  if (lanes < 1) lanes = 1;
  if (N <= lanes) {
    s->lanes_n = static_cast<int>(N);
    return;
  }
  s->lanes_n = static_cast<int>(lanes);
  const size_t room = kSmSmem / ctas;
  int stages = room > extra ? static_cast<int>((room - extra) / stage) : 1;
  s->stages = stages < 1 ? 1 : (stages > kMaxStages ? kMaxStages : stages);
  s->smem = stage * s->stages + extra;
}

GnShape plan(int dtype, int64_t N, int64_t S, int C, int G, bool bwd) {
  // on chip: from slabs of kSlabBytes, narrower while clusters do not hold them or leave SMs
  // idle
  GnShape chip{};
  const int gs0 = least_groups(dtype, C, G);
  const int one = gs0 * (C / G) * elem_bytes(dtype);
  for (int bytes = kSlabBytes; bytes >= kMinSlabBytes; bytes /= 2) {
    const int gs = slab_groups(dtype, C, G, bytes);
    const GnShape s = on_chip_shape(dtype, N, S, C, G, gs, bwd);
    if (s.threads != 0) {
      chip = s;
      if (N * s.slabs * s.ctas >= kSMs || gn_stage_bytes(s, bwd) <= kSmallCta) break;
    }
    if (gs == gs0 || one >= bytes) break;  // no narrower slab
  }
  // A backward over one place a sample stays on chip at one CTA an SM too, where the slab's constants
  // fill half an SM: streamed, it would have a row of sums a sample (65536 x 1 x 4096 bf16, one
  // group: 6.7 ms against 10.2).
  const bool one_place = bwd && S == 1;
  if (chip.threads != 0 && (chip.smem <= kHalfSmem || one_place)) {
    on_chip_loop(&chip, N, bwd);
    // a loop over samples has to have the next ones on their way: at 64 x 4096 x 320 bf16,
    // forward, one stage took 108 us and streaming 90
    if (chip.lanes_n == N || chip.stages > 1 || one_place) return chip;
  }
  // streamed
  int gs = slab_groups(dtype, C, G, kSlabBytes);
  auto slab_bytes = [&] { return S * gs * (C / G) * elem_bytes(dtype) * (bwd ? 2 : 1); };
  GnShape s = slab_shape(dtype, C, G, gs, S, 4);
  const int64_t all = N * s.slabs;
  // whole samples a turn, full lines of memory, unless one is far larger than L2 (measured: half
  // lines cost more than reading a quarter of the turn twice)
  const int64_t sample = slab_bytes() * s.slabs;
  int64_t units = sample <= 2 * kL2Bytes ? (sample < kL2Bytes ? kL2Bytes / sample : 1) * s.slabs
                                         : kL2Bytes / slab_bytes();
  units = units < 1 ? 1 : (units > all ? all : units);
  if (units >= s.slabs) {  // evened out
    const int64_t turns = ceil_div(N, units / s.slabs);
    units = ceil_div(N, turns) * s.slabs;
  }
  // (`all` fits 31 bits: N * S * C is below 2^40 and a streamed unit has more than 2^9 elements --
  // up to that, staged vectors, constants and partial sums are below 60 KB, so two CTAs share an
  // SM and stage several samples each)
  s.units = static_cast<int>(units);
  s.grid = kSMs * min_ctas(s.vecs > kThreads);
  // a piece a CTA, each thread 4 to 256 places
  int64_t chunks = s.grid / units;
  if (chunks > S / (4 * s.lanes)) chunks = S / (4 * s.lanes);
  if (chunks < ceil_div(S, 256 * static_cast<int64_t>(s.lanes)))
    chunks = ceil_div(S, 256 * static_cast<int64_t>(s.lanes));
  s.chunks = static_cast<int>(chunks);
  s.chunk_base = static_cast<int>(S / chunks);
  s.chunk_more = static_cast<int>(S % chunks);
  // A row of column sums a piece would be more than the piece itself (a few places in a wide slab):
  // a fixed number of sequences of pieces add theirs up, whatever grid runs them.
  if (bwd && S * elem_bytes(dtype) < 2 * static_cast<int64_t>(sizeof(float)) && N * chunks > s.grid)
    s.seqs = s.grid;
  if (units * chunks < s.grid) s.grid = static_cast<int>(units * chunks);
  s.iters = 0;  // nothing stays staged
  s.smem = gn_stats_smem(s, bwd);
  return s;
}

int check_sizes(int dtype, int64_t N, int64_t S, int32_t C, int32_t G) {
  if (dtype != GROUPNORM_BF16 && dtype != GROUPNORM_FP32 && dtype != GROUPNORM_FP16)
    return RMSN_ERR_INVALID_ARG;
  if (N < 0 || S < 0 || (N > 0 && S == 0) || C <= 0 || G <= 0 || C % 8 != 0 || C % G != 0)
    return RMSN_ERR_INVALID_ARG;
  if (C > kMaxC || N > INT32_MAX || S > INT32_MAX) return RMSN_ERR_UNSUPPORTED;
  if (least_groups(dtype, C, G) * (C / G) * elem_bytes(dtype) / 16 > kWideThreads)
    return RMSN_ERR_UNSUPPORTED;
  if (N > 0 && N > (kMaxElements - 1) / (S * C)) return RMSN_ERR_UNSUPPORTED;
  return RMSN_OK;
}

size_t part_bytes(const GnShape& s, int64_t N, int G) {
  if (s.on_chip) return 0;
  const size_t n = static_cast<size_t>(N) * s.chunks * G * sizeof(float2);
  return (n + 15) & ~static_cast<size_t>(15);
}
// Rows of column sums, and their bytes (those of sequences have compensations behind them).
int64_t col_rows(const GnShape& s, int64_t N) {
  if (s.on_chip) return static_cast<int64_t>(s.lanes_n) * s.ctas;
  return s.seqs > 0 ? s.seqs : N * s.chunks;
}
size_t col_bytes(const GnShape& s, int64_t N, int C) {
  return static_cast<size_t>(col_rows(s, N)) * (s.seqs > 0 ? 2 : 1) * 2 * C * sizeof(float);
}
size_t workspace_bytes(int dtype, int64_t N, int64_t S, int C, int G, bool bwd) {
  const GnShape s = plan(dtype, N, S, C, G, bwd);
  return part_bytes(s, N, G) + (bwd ? col_bytes(s, N, C) : 0);
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_common(int dtype, const void* x, const void* out, const void* w, const void* b,
                 int wb_dtype, const float* mean, const float* rstd, const void* workspace,
                 int64_t N, int64_t S, int32_t C, int32_t G, int64_t s_n, int64_t s_s, int act) {
  const int st = check_sizes(dtype, N, S, C, G);
  if (st != RMSN_OK) return st;
  if (wb_dtype != GROUPNORM_BF16 && wb_dtype != GROUPNORM_FP32 && wb_dtype != GROUPNORM_FP16)
    return RMSN_ERR_INVALID_ARG;
  if (act != GROUPNORM_ACT_NONE && act != GROUPNORM_ACT_SILU && act != GROUPNORM_ACT_GELU)
    return RMSN_ERR_INVALID_ARG;
  if (!w || !b || (N > 0 && (!x || !out || !mean || !rstd))) return RMSN_ERR_INVALID_ARG;
  const unsigned wa = static_cast<unsigned>(elem_bytes(wb_dtype));
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(w, wa) || !aligned(b, wa) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
    return RMSN_ERR_INVALID_ARG;
  const int ev = 16 / elem_bytes(dtype);
  if (s_n < 0 || s_s < 0 || s_n % ev != 0 || s_s % ev != 0) return RMSN_ERR_INVALID_ARG;
  return RMSN_OK;
}

GnArgs make_args(const void* x, const void* w, const void* b, int wb_dtype, void* out,
                 float* mean, float* rstd, void* workspace, int64_t N, int64_t S, int32_t C,
                 int32_t G, int64_t s_n, int64_t s_s, const GnShape& s) {
  GnArgs a{};
  a.x = x;
  a.w = w;
  a.b = b;
  a.out = out;
  a.mean = mean;
  a.rstd = rstd;
  a.part = static_cast<float2*>(workspace);
  a.cols = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + part_bytes(s, N, G));
  a.s_n = s_n;
  a.s_s = s_s;
  a.N = N;
  a.S = S;
  a.C = C;
  a.G = G;
  a.wb_dtype = wb_dtype;
  a.s = s;
  return a;
}

}  // namespace

cudaError_t launch_gn(const void* fn, const GnArgs& a, cudaStream_t st) {
  const GnShape& s = a.s;
  cudaError_t e = rmsn::prepare_kernel(fn, s.smem);
  if (e != cudaSuccess) return e;
  int64_t ctas = gn_ctas(s);
  if (!s.on_chip) {  // no more than are resident together (the pieces do not depend on it)
    int sms = 0;
    if (rmsn::check_device(&sms) != RMSN_OK) return cudaErrorInvalidDevice;
    const int64_t most = static_cast<int64_t>(sms) * rmsn::blocks_per_sm(fn, s.threads, s.smem);
    if (ctas > most) ctas = most;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(s.threads));
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (s.on_chip) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = s.ctas > 1 ? 2 : 1;
  } else {
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.numAttrs = 1;
  }
  GnArgs copy = a;
  void* args[] = {&copy};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace gnorm

using namespace gnorm;

extern "C" {

size_t groupnorm_train_fwd_workspace_bytes(int dtype, int64_t N, int64_t S, int32_t C,
                                           int32_t G) {
  if (check_sizes(dtype, N, S, C, G) != RMSN_OK || N == 0) return 0;
  return workspace_bytes(dtype, N, S, C, G, false);
}

size_t groupnorm_train_bwd_workspace_bytes(int dtype, int64_t N, int64_t S, int32_t C,
                                           int32_t G) {
  if (check_sizes(dtype, N, S, C, G) != RMSN_OK || N == 0) return 0;
  return workspace_bytes(dtype, N, S, C, G, true);
}

int groupnorm_train_fwd(const void* x, int dtype, const void* w, const void* b, int wb_dtype,
                        void* y, float* mean, float* rstd, void* workspace,
                        size_t workspace_bytes, int64_t N, int64_t S, int32_t C, int32_t G,
                        int64_t s_n, int64_t s_s, float eps, int act, void* stream) {
  int st = check_common(dtype, x, y, w, b, wb_dtype, mean, rstd, workspace, N, S, C, G, s_n, s_s,
                        act);
  if (st != RMSN_OK) return st;
  if (!std::isfinite(eps) || eps < 0.f) return RMSN_ERR_INVALID_ARG;
  if (N == 0) return RMSN_OK;
  const GnShape s = plan(dtype, N, S, C, G, false);
  const size_t need = part_bytes(s, N, G);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return RMSN_ERR_WORKSPACE;
  if ((st = rmsn::check_device()) != RMSN_OK) return st;
  const cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
  GnArgs a = make_args(x, w, b, wb_dtype, y, mean, rstd, workspace, N, S, C, G, s_n, s_s, s);
  a.eps = eps;
  return launch_gn_fwd(a, dtype, act, stream_) == cudaSuccess ? RMSN_OK : RMSN_ERR_CUDA;
}

int groupnorm_train_bwd(const void* x, const void* dy, int dtype, const float* mean,
                        const float* rstd, const void* w, const void* b, int wb_dtype, void* dx,
                        float* dw, float* db, void* workspace, size_t workspace_bytes, int64_t N,
                        int64_t S, int32_t C, int32_t G, int64_t s_n, int64_t s_s, int act,
                        void* stream) {
  int st = check_common(dtype, x, dx, w, b, wb_dtype, mean, rstd, workspace, N, S, C, G, s_n, s_s,
                        act);
  if (st != RMSN_OK) return st;
  if (!dw || !db || (N > 0 && !dy)) return RMSN_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(dw, 4) || !aligned(db, 4)) return RMSN_ERR_INVALID_ARG;
  GnShape s{};
  int64_t rows = 0;
  if (N > 0) {
    s = plan(dtype, N, S, C, G, true);
    rows = col_rows(s, N);
    const size_t need = part_bytes(s, N, G) + col_bytes(s, N, C);
    if (workspace == nullptr || workspace_bytes < need) return RMSN_ERR_WORKSPACE;
  }
  if ((st = rmsn::check_device()) != RMSN_OK) return st;
  const cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
  GnArgs a = make_args(x, w, b, wb_dtype, dx, const_cast<float*>(mean), const_cast<float*>(rstd),
                       workspace, N, S, C, G, s_n, s_s, s);
  a.dy = dy;
  if (N > 0 && launch_gn_bwd(a, dtype, act, stream_) != cudaSuccess) return RMSN_ERR_CUDA;
  return launch_gn_finish(a.cols, dw, db, rows, C, stream_) == cudaSuccess ? RMSN_OK
                                                                         : RMSN_ERR_CUDA;
}

int groupnorm_train_launch_plan(int dtype, int64_t N, int64_t S, int32_t C, int32_t G,
                                int backward, int64_t* out, int n_out) {
  if (!out || n_out < 0 || (backward != 0 && backward != 1)) return RMSN_ERR_INVALID_ARG;
  const int st = check_sizes(dtype, N, S, C, G);
  if (st != RMSN_OK) return st;
  if (N == 0) return RMSN_ERR_INVALID_ARG;
  const GnShape s = plan(dtype, N, S, C, G, backward != 0);
  const int64_t v[GROUPNORM_PLAN_FIELDS] = {
      s.on_chip, s.cs, s.threads, s.on_chip ? s.ctas : 1, gn_ctas(s),
      static_cast<int64_t>(s.smem), s.on_chip ? N * s.slabs : s.units, s.on_chip ? 1 : s.chunks};
  for (int i = 0; i < n_out && i < GROUPNORM_PLAN_FIELDS; ++i) out[i] = v[i];
  return RMSN_OK;
}

}  // extern "C"
