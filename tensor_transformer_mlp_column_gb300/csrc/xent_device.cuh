// xent_device.cuh — what the cross entropy's kernels share.
#pragma once

#include "device.cuh"
#include "train.h"

namespace tpmlp {

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What row t gives to the largest |dloss|: 0 where it does not count, and
// where its dloss is infinite (it spoils its own gradient, not the scale of the
// others).
__device__ __forceinline__ float finite_dloss(const float* dloss, const int64_t* targets, int64_t t, int64_t V) {
  const int64_t id = targets[t];
  const float a = fabsf(dloss[t]);
  return id >= 0 && id < V && a < INFINITY ? a : 0.f;
}

__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The largest finite |dloss| of the rows that count, from its parts (whole
// warp).
__device__ __forceinline__ float warp_dmax(const float* parts, int lane) {
  float m = 0.f;
  for (int i = lane; i < kXentDmaxParts; i += 32) m = fmaxf(m, parts[i]);
  return warp_max(m);
}

// The same from few rows themselves, without a launch before (whole warp);
// with `out` it is written there for the kernels after this one.
__device__ __forceinline__ float warp_dmax_of_rows(const XentDmax& d, int64_t V, int lane, bool write) {
  float m = 0.f;
#pragma unroll 4
  for (int t = lane; t < d.rows; t += 32) m = fmaxf(m, finite_dloss(d.dloss, d.targets, t, V));
  m = warp_max(m);
  if (write)
    for (int i = lane; i < kXentDmaxParts; i += 32) d.out[i] = m;
  return m;
}

}  // namespace tpmlp
