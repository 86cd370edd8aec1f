// blk_api.cu -- the C ABI of a block's boundary (include/block_train.h) and of the norm that keeps
// its input in 8 bits (include/act8_train.h): argument checks, launch shapes and launches.  Never
// allocates, frees or synchronizes (except the diagnostic rmsnorm_block_train_device_error); every
// launch goes on the caller's stream.
#include <cmath>
#include <cstdint>
#include <mutex>

#include "act8.cuh"
#include "blk_launch.h"
#include "block_train.h"  // include/ (on the include path)

namespace blk {

// Device error word of these kernels' bounded waits, one per device.
__device__ unsigned g_blk_err_word = 0u;

template <typename T>
cudaError_t launch_fwd_t(const FwdArgs& a, const Shape& s, int form, bool pack, cudaStream_t st);
template <typename T, int kLong>
cudaError_t launch_bwd_t(const BwdArgs& a, const Shape& s, int form, bool packed, cudaStream_t st);

cudaError_t launch_fwd(const FwdArgs& a, const Shape& s, int dtype, int form, bool pack,
                       cudaStream_t st) {
  return dtype == ACT8_BF16 ? launch_fwd_t<__nv_bfloat16>(a, s, form, pack, st)
                            : launch_fwd_t<__half>(a, s, form, pack, st);
}
cudaError_t launch_bwd(const BwdArgs& a, const Shape& s, int dtype, int form, bool packed,
                       cudaStream_t st) {
  const bool dh = a.in[2].p != nullptr;
  const auto launch =
      dtype == ACT8_BF16
          ? (a.fold == 0 ? launch_bwd_t<__nv_bfloat16, kShort>
             : dh        ? launch_bwd_t<__nv_bfloat16, kLongDh>
                         : launch_bwd_t<__nv_bfloat16, kLongNoDh>)
          : (a.fold == 0 ? launch_bwd_t<__half, kShort>
             : dh        ? launch_bwd_t<__half, kLongDh>
                         : launch_bwd_t<__half, kLongNoDh>);
  return launch(a, s, form, packed, st);
}

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxRows = (int64_t{1} << 31) - (int64_t{1} << 16);
constexpr size_t kSmemBytes = 226 * 1024;  // of the 227 KB that a CTA may take
constexpr size_t kCopyBytes = 2048;  // least bytes of a copy, where rows are narrow
// At most three slots a team: more reads on their way at a time than that needs cost both ways
// (65536 x 1536 forward: 136 us with three, 142 with four, 149 with two; backward 214 with three, 218
// with four).
constexpr int kMaxStages = 3;

std::mutex g_mu;
unsigned* g_err_ptr[kMaxDevices] = {};

// The error word's address on the current device, after the checks of every launch.
int device_setup(unsigned** err) {
  int st = rmsn::check_device();
  if (st != RMSN_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return RMSN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return RMSN_ERR_DEVICE;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_err_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_blk_err_word) != cudaSuccess || p == nullptr)
      return RMSN_ERR_CUDA;
    g_err_ptr[dev] = static_cast<unsigned*>(p);
  }
  *err = g_err_ptr[dev];
  return RMSN_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads a row, vectors a thread, teams a CTA and CTAs: functions of R, H and the kernel's form (the
// forward's also give the same results whether it packs or not).
Shape team_shape(int64_t R, int H, int form, bool bwd, bool packed) {
  const bool tmem = uses_tmem(form, packed, H);
  int threads_cta = bwd ? bwd_threads(form, tmem, false) : fwd_threads(form);
  Shape s{};
  const int nv = H / 8;
  auto threads = [&](int vpt) {
    const int per = (nv + vpt - 1) / vpt;
    return per <= 4 ? 4 : per <= 8 ? 8 : per <= 16 ? 16 : static_cast<int>(ceil_div(per, 32)) * 32;
  };
  auto teams = [&](int ntg) { return threads_cta / (ntg < 32 ? 32 : ntg); };
  auto busy = [&](int vpt) {  // threads of a CTA that have vectors
    const int ntg = threads(vpt), rows = ntg < 32 ? 32 / ntg : 1;
    return ntg > threads_cta ? 0 : teams(ntg) * rows * ((nv + vpt - 1) / vpt);
  };
  // Four vectors a thread, fewer in narrow rows, three where that keeps more threads busy (30720 x
  // 6144 backward, 256 threads against 192: 385 us against 423) -- but not where its threads are then
  // uneven and the numbers of 8 bits add to their work (32768 x 8192 backward with both norms 555
  // us against 476).
  const bool three = busy(3) > busy(4) && (nv == 3 * threads(3) || (form != kKeep && !packed));
  s.vpt = nv <= 4 ? 1 : nv <= 8 ? 2 : three ? 3 : 4;
  // one where the rows are so few that each then has a team at once: the shortest way through a row
  // (64 x 256 forward: 3.1 us against 5.6)
  if (nv > 16 && threads(1) <= threads_cta && R <= int64_t{kPartSMs} * teams(threads(1))) s.vpt = 1;
  s.ntg = threads(s.vpt);
  if (bwd) threads_cta = bwd_threads(form, tmem, more_rows(form, packed, s.vpt, s.ntg));
  s.teams = teams(s.ntg);
  // a row (or a warp's rows) a team at least, spread over the CTAs first
  const int side = s.ntg < 32 ? 32 / s.ntg : 1;
  const int64_t takes = ceil_div(R, side);
  const int64_t per = ceil_div(takes, kPartSMs);
  if (per < s.teams) s.teams = static_cast<int>(per < 1 ? 1 : per);
  const int64_t ctas = ceil_div(takes, s.teams);
  s.P = static_cast<int>(ctas < kPartSMs ? ctas : kPartSMs);
  s.threads = s.teams * (s.ntg < 32 ? 32 : s.ntg);
  return s;
}

// Bytes of the factors in shared memory, and of all of it but the teams' sums that take its place in
// the end.
size_t factor_bytes(const Shape& s) {
  return 32 * static_cast<size_t>(s.teams) * s.ntg * s.vpt;
}
size_t smem_bytes(const Shape& s) {
  const size_t n = static_cast<size_t>(s.teams) * s.stages;
  return (s.factor ? factor_bytes(s) : 0) + n * s.slot + ((8 * n + 15) & ~size_t{15}) +
         4 * 2 * kMaxWarps * static_cast<size_t>(s.teams) + 32;
}

// The ring for staged rows of `row` bytes, of which a copy moves at least `least` at once; the
// backward's teams' sums take its place in the end (`sums` rows a team).
void ring(Shape& s, int H, size_t row, size_t least, int sums) {
  const int side = s.ntg < 32 ? 32 / s.ntg : 1;
  int steps = 1;
  if (s.ntg <= 32)
    while (steps * side * least < kCopyBytes && steps < 64) steps *= 2;
  for (;; steps /= 2) {
    s.rows = steps * side;
    s.slot = row * s.rows;
    for (s.stages = kMaxStages; s.stages > 1 && smem_bytes(s) > kSmemBytes; --s.stages) {
    }
    if (steps == 1 || (s.stages >= 3 && smem_bytes(s) <= kSmemBytes)) break;
  }
  s.smem = smem_bytes(s);
  const size_t join = s.teams > 1 ? sizeof(float) * sums * s.teams * H : 0;
  if (s.smem < join) s.smem = join;
}

Shape plan(int64_t R, int H, int form, bool bwd, bool packed, size_t row, size_t least, int sums) {
  Shape s = team_shape(R, H, form, bwd, packed);
  s.factor = bwd && factor_in_smem(form, packed);
  ring(s, H, row, least, sums);
  return s;
}

// The forward's staged rows: x, and a residual.
Shape fwd_plan(int64_t R, int H, int form, bool residual) {
  const size_t row = 2 * static_cast<size_t>(H);
  return plan(R, H, form, false, false, residual ? 2 * row : row, row, 0);
}
// The backward's: with a norm before, h and dy; dh; but for kKeep, x.
Shape bwd_plan(int64_t R, int H, int form, bool packed, bool dh) {
  const bool pre = form != kPost, x = form != kKeep;
  const size_t wide = 2 * static_cast<size_t>(H);
  const size_t saved = packed ? static_cast<size_t>(rmsn::act8_row_size(H)) : wide;
  const size_t row = (pre ? saved + wide : 0) + (dh ? wide : 0) + (x ? saved : 0);
  return plan(R, H, form, true, packed, row, wide < saved ? wide : saved, (pre ? 1 : 0) + (x ? 1 : 0));
}
// Slots after which a thread's column sums go to their second level: rows of about the root of how many
// it adds up, where that is more than 64; else 0.
int32_t fold_slots(const Shape& s, int64_t R) {
  const int64_t side = s.ntg < 32 ? 32 / s.ntg : 1;
  const int64_t n = ceil_div(R, static_cast<int64_t>(s.P) * s.teams * side);
  if (n <= 64) return 0;
  int64_t fold = 16;
  while (fold * fold < n) fold *= 2;
  return static_cast<int32_t>(ceil_div(fold * side, s.rows));
}
int bwd_form(bool pre, bool post, bool gate) {
  return !post ? (gate ? kPre : kKeep) : (pre ? kBoth : kPost);
}

// A team of several warps starts a slot's next copies while it works on the slot behind it: the ring
// has two at least.  (Every size has; a shape without is not launched.)
bool runs(const Shape& s) {
  return s.stages >= 2 && s.smem <= kSmemBytes && s.teams >= 1 && s.threads <= 32 * kMaxWarps;
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool type_ok(int dtype, bool activation) {
  return dtype == ACT8_BF16 || dtype == ACT8_FP16 || (!activation && dtype == ACT8_FP32);
}

int check_sizes(int64_t R, int32_t H, int64_t N) {
  if (R < 0 || H <= 0 || H % 8 != 0 || N < 1) return RMSN_ERR_INVALID_ARG;
  if (H > kMaxH || R > kMaxRows) return RMSN_ERR_UNSUPPORTED;
  if (R % N != 0) return RMSN_ERR_INVALID_ARG;
  if (N > kMaxRows) return RMSN_ERR_UNSUPPORTED;
  return RMSN_OK;
}

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

void set_common(Args& a, const Shape& s, int64_t R, int32_t H, int64_t N, unsigned* err) {
  a.R = static_cast<int32_t>(R);
  a.H = H;
  a.samples = static_cast<int32_t>(N);
  a.L = static_cast<int32_t>(R / N);
  a.ntg = s.ntg;
  a.teams = s.teams;
  a.rows = s.rows;
  a.stages = s.stages;
  a.slot = static_cast<uint32_t>(s.slot);
  a.err = err;
}

// Places the staged tensors in a slot of `rows` rows.
void set_offsets(Args& a) {
  uint32_t off = 0;
  for (Staged& in : a.in) {
    if (in.p == nullptr) continue;
    in.off = off;
    off += in.bytes * static_cast<uint32_t>(a.rows);
  }
}

Staged staged(const void* p, int64_t stride_bytes, int64_t bytes) {
  return Staged{static_cast<const unsigned char*>(p), stride_bytes, static_cast<uint32_t>(bytes), 0};
}

struct Fwd {
  const void *x, *residual, *w_pre, *w_post, *gate;
  int dtype, w_dtype, gate_dtype, form;
  int64_t N, R;
  void *y, *h;
  float *rstd_pre, *rstd_post;
  void *x8, *h8;
  int32_t H;
  int64_t s_x, s_res;
  float scale, residual_scale, eps;
};

int run_fwd(const Fwd& f, void* stream) {
  unsigned* err = nullptr;
  const int st = device_setup(&err);
  if (st != RMSN_OK) return st;
  FwdArgs a{};
  const size_t row = 2 * static_cast<size_t>(f.H);
  const bool pack = f.x8 != nullptr || f.h8 != nullptr;
  const Shape s = fwd_plan(f.R, f.H, f.form, f.residual != nullptr);
  if (!runs(s)) return RMSN_ERR_UNSUPPORTED;
  set_common(a, s, f.R, f.H, f.N, err);
  a.in[0] = staged(f.x, f.R > 1 ? 2 * f.s_x : row, row);
  if (f.residual != nullptr) a.in[1] = staged(f.residual, f.R > 1 ? 2 * f.s_res : row, row);
  set_offsets(a);
  a.w_pre = f.w_pre;
  a.w_post = f.w_post;
  a.gate = f.gate;
  a.w_dtype = f.w_dtype;
  a.gate_dtype = f.gate_dtype;
  a.scale = f.scale;
  a.residual_scale = f.residual_scale;
  a.eps = f.eps;
  a.y = f.y;
  a.h = f.h;
  a.rstd_pre = f.rstd_pre;
  a.rstd_post = f.rstd_post;
  a.x8 = static_cast<unsigned char*>(f.x8);
  a.h8 = static_cast<unsigned char*>(f.h8);
  return launch_fwd(a, s, f.dtype, f.form, pack, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? RMSN_OK
             : RMSN_ERR_CUDA;
}

struct Bwd {
  const void *dy, *dh, *x, *h;
  bool packed;
  int dtype, form;
  const float *rstd_pre, *rstd_post;
  const void *w_pre, *w_post, *gate;
  int w_dtype, gate_dtype;
  int64_t N, R;
  void *dx, *dres;
  float *dw_pre, *dw_post, *dgate;
  void* workspace;
  size_t workspace_bytes;
  int32_t H;
  int64_t s_x;
  float scale, residual_scale;
};

// Floats of the sums' rows: of dw_pre's, a row a CTA; of S, too, or a row a team and sample.
size_t pre_floats(const Shape& s, int32_t H) { return static_cast<size_t>(s.P) * H; }
size_t s_floats(const Shape& s, int32_t H, int64_t N) {
  const int64_t rows = N == 1 ? s.P : static_cast<int64_t>(s.P) * s.teams + N - 1;
  return static_cast<size_t>(rows) * H;
}
size_t workspace_bytes(int64_t R, int32_t H, int64_t N) {
  size_t most = 0;
  for (int form : {kKeep, kPre, kBoth, kPost})
    for (bool packed : {false, true}) {
      if (form == kKeep && N > 1) continue;
      const Shape s = team_shape(R, H, form, true, packed);
      const size_t n = (form != kPost ? pre_floats(s, H) : 0) + (form != kKeep ? s_floats(s, H, N) : 0);
      if (n > most) most = n;
    }
  return sizeof(float) * most;
}

int run_bwd(const Bwd& b, void* stream) {
  const cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
  const bool pre = b.form != kPost, s_sums = b.form != kKeep;
  unsigned* err = nullptr;
  const int st = device_setup(&err);
  if (st != RMSN_OK) return st;
  if (b.R == 0) {
    for (float* p : {b.dw_pre, b.dw_post})
      if (p != nullptr && cudaMemsetAsync(p, 0, sizeof(float) * b.H, stream_) != cudaSuccess)
        return RMSN_ERR_CUDA;
    if (b.dgate != nullptr &&
        cudaMemsetAsync(b.dgate, 0, sizeof(float) * b.N * b.H, stream_) != cudaSuccess)
      return RMSN_ERR_CUDA;
    return RMSN_OK;
  }
  BwdArgs a{};
  const int64_t wide = 2 * static_cast<int64_t>(b.H);
  const int64_t saved = b.packed ? rmsn::act8_row_size(b.H) : wide;
  if (pre) {
    a.in[0] = staged(b.h, saved, saved);
    a.in[1] = staged(b.dy, wide, wide);
  }
  if (b.dh != nullptr) a.in[2] = staged(b.dh, wide, wide);
  if (s_sums) a.in[3] = staged(b.x, b.packed || b.R == 1 ? saved : 2 * b.s_x, saved);
  const Shape s = bwd_plan(b.R, b.H, b.form, b.packed, b.dh != nullptr);
  if (!runs(s)) return RMSN_ERR_UNSUPPORTED;
  set_common(a, s, b.R, b.H, b.N, err);
  set_offsets(a);
  const size_t need = sizeof(float) * ((pre ? pre_floats(s, b.H) : 0) +
                                       (s_sums ? s_floats(s, b.H, b.N) : 0));
  if (b.workspace == nullptr || b.workspace_bytes < need) return RMSN_ERR_WORKSPACE;
  float* ws = static_cast<float*>(b.workspace);
  a.w_pre = b.w_pre;
  a.w_post = b.w_post;
  a.gate = b.gate;
  a.w_dtype = b.w_dtype;
  a.gate_dtype = b.gate_dtype;
  a.scale = b.scale;
  a.residual_scale = b.residual_scale;
  a.rstd_pre = b.rstd_pre;
  a.rstd_post = b.rstd_post;
  a.fold = fold_slots(s, b.R);
  a.factor_at = static_cast<uint32_t>(smem_bytes(s) - (s.factor ? factor_bytes(s) : 0));
  a.dx = b.dx;
  a.dres = b.dres;
  a.part_pre = pre ? ws : nullptr;
  a.part_s = s_sums ? ws + (pre ? pre_floats(s, b.H) : 0) : nullptr;
  if (launch_bwd(a, s, b.dtype, b.form, b.packed, stream_) != cudaSuccess) return RMSN_ERR_CUDA;
  FinishArgs f{};
  f.part_pre = a.part_pre;
  f.part_s = a.part_s;
  f.ctas = s.P;
  f.teams = static_cast<int64_t>(s.P) * s.teams;
  f.R = a.R;
  f.H = b.H;
  f.samples = a.samples;
  f.w_post = b.w_post;
  f.gate = b.gate;
  f.w_dtype = b.w_dtype;
  f.gate_dtype = b.gate_dtype;
  f.scale = b.scale;
  f.dw_pre = b.dw_pre;
  f.dw_post = b.dw_post;
  f.dgate = b.dgate;
  return launch_finish(f, stream_) == cudaSuccess ? RMSN_OK : RMSN_ERR_CUDA;
}

}  // namespace

}  // namespace blk

using namespace blk;

extern "C" {

int rmsnorm_act8_train_fwd(const void* x, const void* residual, int dtype, const void* w,
                           int w_dtype, void* y, void* h_out, float* rstd, void* packed,
                           int64_t R, int32_t H, int64_t s_x, int64_t s_res, float eps,
                           void* stream) {
  const int st = check_sizes(R, H, 1);
  if (st != RMSN_OK) return st;
  if (!type_ok(dtype, true) || !type_ok(w_dtype, false) || !stride_ok(s_x) ||
      (residual != nullptr && !stride_ok(s_res)))
    return RMSN_ERR_INVALID_ARG;
  if (!w || (residual == nullptr && h_out != nullptr)) return RMSN_ERR_INVALID_ARG;
  if (R > 0 && (!x || !y || !rstd || !packed || (residual != nullptr && h_out == nullptr)))
    return RMSN_ERR_INVALID_ARG;
  for (const void* p : {x, residual, w, static_cast<const void*>(y), static_cast<const void*>(h_out),
                        static_cast<const void*>(packed)})
    if (!aligned(p, 16)) return RMSN_ERR_INVALID_ARG;
  if (!aligned(rstd, 4) || !std::isfinite(eps) || eps < 0.f) return RMSN_ERR_INVALID_ARG;
  if (R == 0) return RMSN_OK;
  Fwd f{};
  f.x = x;
  f.residual = residual;
  f.w_pre = w;
  f.dtype = dtype;
  f.w_dtype = w_dtype;
  f.form = kKeep;
  f.N = 1;
  f.R = R;
  f.y = y;
  f.h = h_out;
  f.rstd_pre = rstd;
  f.h8 = packed;
  f.H = H;
  f.s_x = s_x;
  f.s_res = s_res;
  f.eps = eps;
  return run_fwd(f, stream);
}

size_t rmsnorm_act8_train_bwd_workspace_bytes(int64_t R, int32_t H) {
  if (check_sizes(R, H, 1) != RMSN_OK || R == 0) return 0;
  return sizeof(float) * pre_floats(team_shape(R, H, kKeep, true, true), H);
}

int rmsnorm_act8_train_bwd(const void* packed, const void* dy, const void* dh, int dtype,
                           const float* rstd, const void* w, int w_dtype, void* dx, float* dw,
                           void* workspace, size_t workspace_bytes, int64_t R, int32_t H,
                           void* stream) {
  const int st = check_sizes(R, H, 1);
  if (st != RMSN_OK) return st;
  if (!type_ok(dtype, true) || !type_ok(w_dtype, false)) return RMSN_ERR_INVALID_ARG;
  if (!w || !dw || (R > 0 && (!packed || !dy || !rstd || !dx))) return RMSN_ERR_INVALID_ARG;
  for (const void* p : {packed, dy, dh, w, static_cast<const void*>(dx),
                        static_cast<const void*>(workspace)})
    if (!aligned(p, 16)) return RMSN_ERR_INVALID_ARG;
  if (!aligned(rstd, 4) || !aligned(dw, 4)) return RMSN_ERR_INVALID_ARG;
  Bwd b{};
  b.dy = dy;
  b.dh = dh;
  b.h = packed;
  b.packed = true;
  b.dtype = dtype;
  b.form = kKeep;
  b.rstd_pre = rstd;
  b.w_pre = w;
  b.w_dtype = w_dtype;
  b.N = 1;
  b.R = R;
  b.dres = dx;
  b.dw_pre = dw;
  b.workspace = workspace;
  b.workspace_bytes = workspace_bytes;
  b.H = H;
  b.scale = b.residual_scale = 1.f;
  return run_bwd(b, stream);
}

int rmsnorm_block_train_fwd(const void* x, const void* residual, int dtype, const void* w_pre,
                            const void* w_post, int w_dtype, const void* gate, int gate_dtype,
                            int64_t N, void* y, void* h, float* rstd_pre, float* rstd_post,
                            void* x8, void* h8, int64_t R, int32_t H, int64_t s_x, int64_t s_res,
                            float scale, float residual_scale, float eps, void* stream) {
  const int st = check_sizes(R, H, N);
  if (st != RMSN_OK) return st;
  if (!type_ok(dtype, true) || !type_ok(w_dtype, false) ||
      (gate != nullptr ? !type_ok(gate_dtype, false) : N != 1) || !stride_ok(s_x) ||
      !stride_ok(s_res) || (!w_pre && !w_post))
    return RMSN_ERR_INVALID_ARG;
  if (R > 0 && (!x || !residual || !h || (w_pre != nullptr) != (y != nullptr) ||
                (w_pre != nullptr) != (rstd_pre != nullptr) ||
                (w_post != nullptr) != (rstd_post != nullptr)))
    return RMSN_ERR_INVALID_ARG;
  // in 8 bits: all that the backward reads, or nothing
  const bool reads_x = w_post != nullptr || gate != nullptr, reads_h = w_pre != nullptr;
  if ((x8 != nullptr && !reads_x) || (h8 != nullptr && !reads_h) ||
      (reads_x && reads_h && (x8 != nullptr) != (h8 != nullptr)))
    return RMSN_ERR_INVALID_ARG;
  for (const void* p : {x, residual, w_pre, w_post, gate, static_cast<const void*>(y),
                        static_cast<const void*>(h), static_cast<const void*>(x8),
                        static_cast<const void*>(h8)})
    if (!aligned(p, 16)) return RMSN_ERR_INVALID_ARG;
  if (!aligned(rstd_pre, 4) || !aligned(rstd_post, 4) || !std::isfinite(scale) ||
      !std::isfinite(residual_scale) || !std::isfinite(eps) || eps < 0.f)
    return RMSN_ERR_INVALID_ARG;
  if (R == 0) return RMSN_OK;
  Fwd f{};
  f.x = x;
  f.residual = residual;
  f.w_pre = w_pre;
  f.w_post = w_post;
  f.gate = gate;
  f.dtype = dtype;
  f.w_dtype = w_dtype;
  f.gate_dtype = gate_dtype;
  f.form = w_post == nullptr ? kPre : (w_pre != nullptr ? kBoth : kPost);
  f.N = N;
  f.R = R;
  f.y = y;
  f.h = h;
  f.rstd_pre = rstd_pre;
  f.rstd_post = rstd_post;
  f.x8 = x8;
  f.h8 = h8;
  f.H = H;
  f.s_x = s_x;
  f.s_res = s_res;
  f.scale = scale;
  f.residual_scale = residual_scale;
  f.eps = eps;
  return run_fwd(f, stream);
}

size_t rmsnorm_block_train_bwd_workspace_bytes(int64_t R, int32_t H, int64_t N) {
  if (check_sizes(R, H, N) != RMSN_OK || R == 0) return 0;
  return workspace_bytes(R, H, N);
}

int rmsnorm_block_train_bwd(const void* dy, const void* dh, const void* x, const void* h,
                            int packed, int dtype, const float* rstd_pre, const float* rstd_post,
                            const void* w_pre, const void* w_post, int w_dtype, const void* gate,
                            int gate_dtype, int64_t N, void* dx, void* dresidual, float* dw_pre,
                            float* dw_post, float* dgate, void* workspace, size_t workspace_bytes,
                            int64_t R, int32_t H, int64_t s_x, float scale, float residual_scale,
                            void* stream) {
  const int st = check_sizes(R, H, N);
  if (st != RMSN_OK) return st;
  const bool pre = w_pre != nullptr, post = w_post != nullptr, gated = gate != nullptr;
  if (!type_ok(dtype, true) || !type_ok(w_dtype, false) ||
      (gated ? !type_ok(gate_dtype, false) : N != 1) || (packed != 0 && packed != 1) ||
      !stride_ok(s_x) || (!pre && !post))
    return RMSN_ERR_INVALID_ARG;
  if (pre != (dw_pre != nullptr) || post != (dw_post != nullptr) || gated != (dgate != nullptr))
    return RMSN_ERR_INVALID_ARG;
  if (R > 0 && (pre != (dy != nullptr) || (!pre && !dh) || (pre && (!h || !rstd_pre)) ||
                ((post || gated) && !x) || (post && !rstd_post) || !dx || !dresidual))
    return RMSN_ERR_INVALID_ARG;
  for (const void* p : {dy, dh, x, h, w_pre, w_post, gate, static_cast<const void*>(dx),
                        static_cast<const void*>(dresidual), static_cast<const void*>(workspace)})
    if (!aligned(p, 16)) return RMSN_ERR_INVALID_ARG;
  for (const float* p : {rstd_pre, rstd_post, static_cast<const float*>(dw_pre),
                         static_cast<const float*>(dw_post), static_cast<const float*>(dgate)})
    if (!aligned(p, 4)) return RMSN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(residual_scale)) return RMSN_ERR_INVALID_ARG;
  Bwd b{};
  b.dy = dy;
  b.dh = dh;
  b.x = x;
  b.h = h;
  b.packed = packed != 0;
  b.dtype = dtype;
  b.form = bwd_form(pre, post, gated);
  b.rstd_pre = rstd_pre;
  b.rstd_post = rstd_post;
  b.w_pre = w_pre;
  b.w_post = w_post;
  b.gate = gate;
  b.w_dtype = w_dtype;
  b.gate_dtype = gate_dtype;
  b.N = N;
  b.R = R;
  b.dx = dx;
  b.dres = dresidual;
  b.dw_pre = dw_pre;
  b.dw_post = dw_post;
  b.dgate = dgate;
  b.workspace = workspace;
  b.workspace_bytes = workspace_bytes;
  b.H = H;
  b.s_x = s_x;
  b.scale = scale;
  b.residual_scale = residual_scale;
  return run_bwd(b, stream);
}

int rmsnorm_block_train_launch_plan(int64_t R, int32_t H, int64_t N, int kernel, int packed,
                                    int64_t* out, int n_out) {
  constexpr int kAll = BLOCK_PLAN_BACKWARD | BLOCK_PLAN_NO_NORM_BEHIND | BLOCK_PLAN_NO_NORM_BEFORE |
                       BLOCK_PLAN_NO_GATE | BLOCK_PLAN_ONE_INPUT | BLOCK_PLAN_ACT8_NORM;
  if (!out || n_out < 0 || (kernel & ~kAll) != 0 || (packed != 0 && packed != 1))
    return RMSN_ERR_INVALID_ARG;
  const bool backward = kernel & BLOCK_PLAN_BACKWARD, post = !(kernel & BLOCK_PLAN_NO_NORM_BEHIND),
             pre = !(kernel & BLOCK_PLAN_NO_NORM_BEFORE), gate = !(kernel & BLOCK_PLAN_NO_GATE),
             one = kernel & BLOCK_PLAN_ONE_INPUT, norm8 = kernel & BLOCK_PLAN_ACT8_NORM;
  if (norm8 ? !(pre && post && gate) || (backward && !packed)
            : (!pre && !post) || (one && (!backward || !pre)))
    return RMSN_ERR_INVALID_ARG;
  const int st = check_sizes(R, H, N);
  if (st != RMSN_OK) return st;
  if (R == 0 || ((norm8 || !gate) && N != 1)) return RMSN_ERR_INVALID_ARG;
  const int form = norm8       ? kKeep
                   : backward  ? bwd_form(pre, post, gate)
                               : (!post ? kPre : pre ? kBoth : kPost);
  const Shape s = backward ? bwd_plan(R, H, form, packed != 0, !one)
                           : fwd_plan(R, H, form, !one);
  if (!runs(s)) return RMSN_ERR_UNSUPPORTED;
  const int64_t v[BLOCK_PLAN_FIELDS] = {s.vpt,    s.ntg,     s.teams, s.rows,
                                        s.stages, s.threads, s.P,     static_cast<int64_t>(s.smem)};
  for (int i = 0; i < n_out && i < BLOCK_PLAN_FIELDS; ++i) out[i] = v[i];
  return RMSN_OK;
}

int rmsnorm_block_train_device_error(unsigned int* flags, int reset) {
  if (!flags) return RMSN_ERR_INVALID_ARG;
  unsigned* err = nullptr;
  const int st = device_setup(&err);
  if (st != RMSN_OK) return st;
  if (cudaDeviceSynchronize() != cudaSuccess) return RMSN_ERR_CUDA;
  if (cudaMemcpyFromSymbol(flags, g_blk_err_word, sizeof(unsigned)) != cudaSuccess)
    return RMSN_ERR_CUDA;
  if (reset) {
    const unsigned zero = 0u;
    if (cudaMemcpyToSymbol(g_blk_err_word, &zero, sizeof(unsigned)) != cudaSuccess)
      return RMSN_ERR_CUDA;
  }
  return RMSN_OK;
}

}  // extern "C"
