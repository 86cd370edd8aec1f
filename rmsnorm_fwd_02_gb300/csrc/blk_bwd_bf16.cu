// blk_bwd_bf16.cu -- the BF16 builds of blk_bwd.cuh for column sums of one level, in a
// translation unit of their own so that the builds compile in parallel.
#include "blk_bwd.cuh"

namespace blk {

template cudaError_t launch_bwd_t<__nv_bfloat16, kShort>(const BwdArgs&, const Shape&, int, bool,
                                            cudaStream_t);

}  // namespace blk
