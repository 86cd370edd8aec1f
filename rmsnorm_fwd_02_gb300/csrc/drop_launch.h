// drop_launch.h -- the dropout parameter block and the dropout kernels' launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rmsn {

// One call's generator and probability, as its kernels take them (drop_philox.cuh).
struct DropParams {
  uint32_t rk[20];                 // round keys: key words of round r at 2r and 2r + 1
  unsigned long long offset;       // counter's upper half, before *step
  const unsigned long long* step;  // device, nullable
  uint32_t drop_below;             // 65536 t - 1 (t: the threshold; t = 0 drops nothing
                                   // and is told apart by `active`)
  float scale;                     // 65536 / (65536 - t); 0 when t = 65536
  int active;                      // t > 0
};

// Fills *d; false if p is not in [0, 1] or step is not 8-byte aligned.
bool drop_params(double p, uint64_t seed, uint64_t offset, const void* step, DropParams* d);

// y = [residual +] dropout(x) over n elements (dtype: DROPOUT_*).
cudaError_t launch_dropout(const void* x, const void* residual, void* y, int dtype, int64_t n,
                           const DropParams& d, cudaStream_t st);

}  // namespace rmsn
