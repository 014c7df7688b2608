// attn_core.h — launchers of the attention on given queries, keys and values
// and its backward pass (attn_core.cu, attn_core_tc.cu), and of the norms and
// rotation of queries and keys (qk_rope.cu). Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"

namespace tpmlp {

// What the status word holds when a sequence's start and end are not in order,
// lie outside the T rows or are further apart than max_seq: the sequence is
// left out, and the next tpmlp_check_status() returns TPMLP_ERR_BOUNDS.
constexpr int kChkSequence = 10;

// A tensor [T][heads][dim]: element (t, h, e) at p[t * token + h * head + e].
struct HeadsView {
  void* p;
  int64_t token, head;
};

struct CoreShape {
  const int32_t* starts;  // device [batch + 1], or null: sequence b in rows b * max_seq ..
  int64_t T;
  int batch, max_seq;
  int heads, kv_heads, dim;
  float scale;
  int causal;
};

// A sequence's first row and length; length 0 (and a recorded failure) if the
// starts do not describe one.
__device__ __forceinline__ int core_sequence(const CoreShape& s, int b, int64_t& row0, int* status) {
  if (!s.starts) {
    row0 = int64_t(b) * s.max_seq;
    return s.max_seq;
  }
  const int64_t begin = s.starts[b], end = s.starts[b + 1];
  row0 = begin;
  if (begin >= 0 && end >= begin && end <= s.T && end - begin <= s.max_seq) return static_cast<int>(end - begin);
  atomicCAS(status, 0, kSiteBoundsBase + kChkSequence);
  return 0;
}

// Lets a kernel use `bytes` of dynamic shared memory, once per device and kernel.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t>& devices) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (devices.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Calls that compute nothing (no rows, or max_seq = 0) look at their sequences all the same: the ones that have tokens, or lie
// outside of the rows, are recorded.
cudaError_t check_core_sequences(const CoreShape& s, int* status, cudaStream_t stream);

struct CoreForward {
  CoreShape s;
  HeadsView q, k, v, o;
  float* lse;  // [heads][T]
  int bf16;
  int withhold;  // test hook, bf16: > 0: that load of every CTA's keys and values is never issued
  uint64_t wait_ns;
  int* status;
};
cudaError_t run_core_forward(const CoreForward& c, cudaStream_t stream);

struct CoreBackward {
  CoreShape s;
  HeadsView q, k, v, o, d_o, dq, dk, dv;
  const float* lse;
  int bf16;
  void* ws;
  int withhold;  // test hook, bf16: > 0: that load of every CTA's first ring is never issued
  uint64_t wait_ns;
  int* status;
};
size_t core_backward_workspace(int64_t T, int64_t batch, int64_t max_seq, int heads, int kv_heads, int dim, int bf16);
cudaError_t run_core_backward(const CoreBackward& c, cudaStream_t stream);
// The bf16 forms (attn_core_tc.cu). delta [heads][T]: the row sums of dO . O; part: where core_splits_tc() is above 1, that
// many times fp32 sums of dV and dK of batch x ceil(max_seq / 128) tiles of 128 keys.
int core_splits_tc(int64_t batch, int64_t max_seq, int heads, int kv_heads, int dim);
cudaError_t launch_core_forward_tc(const CoreForward& c, cudaStream_t stream);
cudaError_t launch_core_backward_tc(const CoreBackward& c, float* delta, float* part, cudaStream_t stream);

// ------------------------------------------------------------------ qk_rope.cu

constexpr int kRopeMaxDim = 256;

// Norm (where w is given) and rotation of the heads of q and k. The first
// `rot` elements of a head are turned in pairs: pair i by pos[axis[i]][t]
// times turn[i] / 2^64 of a full turn.
struct RopeShape {
  int64_t T;
  int heads[2], dim, rot;       // of q, of k
  int interleaved;              // pairs (2i, 2i + 1) in the place of (i, i + rot / 2)
  float eps;
  const int64_t* pos;           // device [axes][T]
  uint64_t turn[kRopeMaxDim / 2];
  uint8_t axis[kRopeMaxDim / 2];
};
struct RopeCall {
  RopeShape s;
  int backward;
  HeadsView x[2], y[2];         // forward: y from x; backward: y is dx, made from x and dy
  HeadsView dy[2];
  const void* w[2];             // [dim], or both null: no norm
  float* dw[2];                 // [dim]
  void* ws;
  int bf16;
  int* status;
};
size_t rope_backward_workspace(int64_t T, int heads, int kv_heads, int dim);
cudaError_t run_qk_rope(const RopeCall& c, cudaStream_t stream);

}  // namespace tpmlp
