// cta_scan.cuh -- prefix sums over the threads of a CTA.
#pragma once

#include <stdint.h>

namespace pkv {

// Exclusive prefix sums of N values per thread over the CTA (x), and their totals.
// warp_sums: shared memory for 32 warps; free again when the call returns.
template <int N>
__device__ __forceinline__ void scan_cta(int64_t (&x)[N], int64_t (&total)[N],
                                         int64_t (*warp_sums)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t incl[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    incl[i] = x[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl[i], o);
      if (lane >= o) incl[i] += y;
    }
    if (lane == 31) warp_sums[warp][i] = incl[i];
  }
  __syncthreads();
  // Every warp adds up the warps' sums by itself.
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int64_t y = lane < warps ? warp_sums[lane][i] : 0;
    int64_t mine = lane < warp ? y : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      y += __shfl_xor_sync(0xffffffffu, y, o);
      mine += __shfl_xor_sync(0xffffffffu, mine, o);
    }
    total[i] = y;
    x[i] = mine + incl[i] - x[i];
  }
  __syncthreads();
}

}  // namespace pkv
