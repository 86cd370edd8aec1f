// blk_bwd_fp16_long_dh.cu -- the FP16 builds of blk_bwd.cuh for column sums of two levels with dh, in a
// translation unit of their own so that the builds compile in parallel.
#include "blk_bwd.cuh"

namespace blk {

template cudaError_t launch_bwd_t<__half, kLongDh>(const BwdArgs&, const Shape&, int, bool,
                                            cudaStream_t);

}  // namespace blk
