// A CTA's prefix sums.
#pragma once

#include "common.cuh"

namespace qd {

// Inclusive sum over the CTA's threads in thread order; total: the whole sum.
template <typename S>
QD_DEV S block_scan(S v, S* warp_sums, S& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();   // warp_sums of the scan before have been read
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const S x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  S before = 0, all = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    const S s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  total = all;
  return before + v;
}

}  // namespace qd
