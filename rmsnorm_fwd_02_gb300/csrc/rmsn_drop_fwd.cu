// rmsn_drop_fwd.cu -- the builds of the RMSNorm training forward (rmsn_fwd_rows.cuh) that add
// a dropped-out branch to the residual, in a translation unit of their own so that the builds
// compile in parallel.
#include "rmsn_fwd_rows.cuh"

namespace rmsn {

int fwd_drop_blocks_per_sm(const Shape& s, bool fp32w) {
  return blocks_per_sm(pick_fwd_rows<true, true>(s, fp32w), s.threads, s.smem);
}

cudaError_t launch_fwd_drop(const FwdDropArgs& a, const Shape& s, bool fp32w, cudaStream_t st) {
  const void* fn = pick_fwd_rows<true, true>(s, fp32w);
  cudaError_t e = prepare_kernel(fn, s.smem);
  if (e != cudaSuccess) return e;
  FwdDropArgs copy = a;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(static_cast<unsigned>(a.P)), dim3(static_cast<unsigned>(s.threads)),
                    s.smem, st, args);
}

}  // namespace rmsn
