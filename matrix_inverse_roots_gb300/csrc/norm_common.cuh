// Sums over a row that several warps hold.
#pragma once

#include "act_q8.cuh"

namespace dash {

// A row is held by W warps, J vectors of eight columns per thread: thread t of the row has
// columns 8 (j 32 W + t).

// Sums of N (1 or 2) values over the W warps of a row (W = 1: one warp; else the whole CTA,
// or the named barrier's group of warps), the same in every thread.  red holds 32 floats
// per value.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int W, int warp_in_row, float* red,
                                        int barrier) {
  const int lane = threadIdx.x & 31;
  if constexpr (N == 2) {
    // The lower half-warp goes on with the first value, the upper with the second.
    const bool up = lane >= 16;
    float x = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (W == 1) {
      v[0] = __shfl_sync(0xffffffffu, x, 0);
      v[1] = __shfl_sync(0xffffffffu, x, 16);
      return;
    }
    if ((lane & 15) == 0) red[(lane << 1) + warp_in_row] = x;
  } else {
    v[0] = warp_sum(v[0]);
    if (W == 1) return;
    if (lane == 0) red[warp_in_row] = v[0];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(W * 32) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (W <= 8) {
      // Up to eight partial sums: read by every thread, the missing ones as zeros.
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += w < W ? red[i * 32 + w] : 0.0f;
      v[i] = t;
    } else {
      v[i] = warp_sum(lane < W ? red[i * 32 + lane] : 0.0f);
    }
  }
}

}  // namespace dash
