// blk_fwd_fp16.cu -- the FP16 builds of blk_fwd.cuh, in a translation unit of their own so that the
// builds compile in parallel.
#include "blk_fwd.cuh"

namespace blk {

template cudaError_t launch_fwd_t<__half>(const FwdArgs&, const Shape&, int, bool, cudaStream_t);

}  // namespace blk
