// rmsn_drop_bwd.cu -- the builds of the RMSNorm training backward's row pass
// (rmsn_bwd_rows.cuh with kDrop = true) that return the gradients of both sides of a residual
// add whose added branch went through dropout.
#include "rmsn_bwd_rows.cuh"

namespace rmsn {

cudaError_t launch_bwd_rows_drop(const BwdDropArgs& a, const Shape& s, bool fp32w,
                                 cudaStream_t st) {
  const void* fn = pick_rows_kernel<false, true>(s, fp32w, a.dh != nullptr);
  cudaError_t e = prepare_kernel(fn, s.smem);
  if (e != cudaSuccess) return e;
  BwdDropArgs copy = a;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(static_cast<unsigned>(a.P)), dim3(static_cast<unsigned>(s.threads)),
                    s.smem, st, args);
}

}  // namespace rmsn
