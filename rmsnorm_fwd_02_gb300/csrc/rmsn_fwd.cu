// rmsn_fwd.cu -- the plain and residual builds of the RMSNorm training forward
// (rmsn_fwd_rows.cuh) and their launch.
#include "rmsn_fwd_rows.cuh"

namespace rmsn {

static const void* pick_fwd(const Shape& s, bool fp32w, bool res) {
  return res ? pick_fwd_rows<true, false>(s, fp32w) : pick_fwd_rows<false, false>(s, fp32w);
}

int fwd_blocks_per_sm(const Shape& s, bool fp32w) {
  return blocks_per_sm(pick_fwd(s, fp32w, s.tensors == 2), s.threads, s.smem);
}

cudaError_t launch_fwd(const FwdArgs& a, const Shape& s, bool fp32w, cudaStream_t st) {
  const void* fn = pick_fwd(s, fp32w, a.res != nullptr);
  cudaError_t e = prepare_kernel(fn, s.smem);
  if (e != cudaSuccess) return e;
  FwdArgs copy = a;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(static_cast<unsigned>(a.P)), dim3(static_cast<unsigned>(s.threads)),
                    s.smem, st, args);
}

}  // namespace rmsn
