// drop_philox.cuh -- the keep mask of the dropout kernels: a Philox4x32-10 block (Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011) per eight
// elements, 16 bits an element.
//
// Cost per block: ten rounds of two 32x32->64 multiplies and two three-input xors, so five
// integer instructions an element; 32 bits an element would take twice that, which a 16-bit
// activation's bandwidth does not leave room for.  The round keys depend on the seed alone
// and come from the host through the kernel's arguments (constant operands of the xors).
#pragma once

#include <stdint.h>

#include "drop_launch.h"

namespace rmsn {

// The counter's upper half: offset + *step.  Read once a thread, after the wait for the
// prior grid.
__device__ __forceinline__ uint2 drop_counter(const DropParams& d) {
  unsigned long long c = d.offset;
  if (d.step != nullptr) c += *d.step;
  return make_uint2(static_cast<uint32_t>(c), static_cast<uint32_t>(c >> 32));
}

// The block of eight-element group q.
__device__ __forceinline__ uint4 drop_block(const DropParams& d, uint2 c, uint64_t q) {
  uint32_t a0 = static_cast<uint32_t>(q), a1 = static_cast<uint32_t>(q >> 32);
  uint32_t a2 = c.x, a3 = c.y;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t u = static_cast<uint64_t>(a0) * 0xD2511F53u;
    const uint64_t v = static_cast<uint64_t>(a2) * 0xCD9E8D57u;
    a0 = static_cast<uint32_t>(v >> 32) ^ a1 ^ d.rk[2 * r];
    a1 = static_cast<uint32_t>(v);
    a2 = static_cast<uint32_t>(u >> 32) ^ a3 ^ d.rk[2 * r + 1];
    a3 = static_cast<uint32_t>(u);
  }
  return make_uint4(a0, a1, a2, a3);
}

// The eight-element group of vector c of a row of `vecs` vectors (row and vecs below 2^31; in
// 32-bit factors, which takes fewer registers than a 64-bit product).
__device__ __forceinline__ uint64_t drop_group(int32_t row, int vecs, int c) {
  return static_cast<uint64_t>(static_cast<uint32_t>(row)) * static_cast<uint32_t>(vecs) +
         static_cast<uint32_t>(c);
}

// Whether elements 2i (lo) and 2i+1 (hi) of a group are kept, from the block's word i.
// drop_below = 65536 t - 1 (modulo 2^32): for 1 <= t <= 65536 a 16-bit number u is at least
// t exactly when u * 65536 > drop_below, and the bits under an upper half do not matter.
__device__ __forceinline__ bool drop_keep_lo(const DropParams& d, uint32_t w) {
  return (w << 16) > d.drop_below;
}
__device__ __forceinline__ bool drop_keep_hi(const DropParams& d, uint32_t w) {
  return w > d.drop_below;
}

// The masks of a group's four words of 16-bit elements (all ones under a kept element, zeros
// under a dropped one).
__device__ __forceinline__ uint4 drop_masks(const DropParams& d, const uint4& b) {
  const uint32_t all = d.active ? 0u : 0xffffffffu;
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = drop_keep_hi(d, w[i]) ? 0xffff0000u : 0u;
    if (drop_keep_lo(d, w[i])) m[i] |= 0x0000ffffu;
    m[i] |= all;
  }
  return make_uint4(m[0], m[1], m[2], m[3]);
}

}  // namespace rmsn
