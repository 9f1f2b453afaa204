// block_sums.cuh -- sums over the threads of a block of several values at once, always in the same order.
#pragma once
#include "ptx.cuh"

namespace mhc {

// Lane l gets the warp's total of value l % V.
template <int V>
__device__ __forceinline__ float warp_sums(float (&v)[V]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = V / 2; h >= 1; h /= 2) {
    const bool up = (lane & h) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float send = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, h);
    }
  }
#pragma unroll
  for (int o = V; o < 32; o *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}
// The block's totals from each warp's V sums (scratch [warps][V]; one barrier of the `nthreads`
// consumers): lane l of every warp gets that of value l % V. The next use of `scratch` has to come
// after another barrier.
template <int V>
__device__ __forceinline__ float group_sums(float (&v)[V], float* scratch, int warps, int nthreads) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float mine = warp_sums<V>(v);
  if (lane < V) scratch[warp * V + lane] = mine;
  named_bar_sync(1, nthreads);
  float t = 0.f;
  if (V <= 2) {   // at most 16 warps: every sum in a lane of its own, added by shuffles
    t = lane < warps * V ? scratch[lane] : 0.f;
#pragma unroll
    for (int o = 16; o >= V; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
  } else {
#pragma unroll 4
    for (int w = 0; w < warps; ++w) t += scratch[w * V + (lane & (V - 1))];
  }
  return t;
}
__device__ __forceinline__ float lane_value(float v, int lane) { return __shfl_sync(0xffffffffu, v, lane); }

}  // namespace mhc
