// clip.cu — the global norm over many gradient tensors, and their clipping:
//
//   norm = sqrt(sum_i sum_j g_ij^2),   out_i = min(1, max_norm / (norm + 1e-6)) g_i.
//
// HBM-bound: one read for the norm, one read and one write for the scaling.
// Every tensor is cut into chunks of kChunk elements; a CTA walks the chunks
// b, b + grid, ... of all tensors together, so tensors of any sizes share the
// GPU evenly. A thread squares and adds in fp32 within one chunk (two sums of
// 32 terms) and across chunks in fp64 (one fp64 addition per 64 elements: the
// fp64 rate is too low for more), and the CTAs' fp64 sums are added in their
// order, so the norm is the same on every run. A chunk is 64 KB of fp32, all of
// which a scaling CTA has on its way at once, a squaring one as much as 34
// registers hold (chunks of half that: 339 and 665 us for the two passes over
// 2.1 GB instead of 322 and 653).
#include "device.cuh"
#include "internal.h"
#include "train.h"

namespace tpmlp {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16384;  // elements

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the CTA, in a fixed order; every thread gets it. `red` holds 32.
__device__ __forceinline__ double cta_sum_f64(double v, double* red) {
  v = warp_sum_f64(v);
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  __syncthreads();
  if (l == 0) red[w] = v;
  __syncthreads();
  return warp_sum_f64(l < (kThreads >> 5) ? red[l] : 0.0);
}

// Tensor that chunk c belongs to.
__device__ __forceinline__ int tensor_of(const ClipTensors& t, int64_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <typename E>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kElems = 4;
  __device__ static void unpack(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
  __device__ static uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ static float to_f(float v) { return v; }
  __device__ static float from_f(float v) { return v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kElems = 8;
  __device__ static void unpack(const uint4& w, float (&f)[8]) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 t = __bfloat1622float2(h[j]);
      f[2 * j] = t.x;
      f[2 * j + 1] = t.y;
    }
  }
  __device__ static uint4 pack(const float (&f)[8]) {
    uint4 w;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    return w;
  }
  __device__ static float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
  __device__ static __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
};

// This thread's share of the sum of squares of n <= kChunk elements at src
// (16-byte aligned).
template <typename E>
__device__ __forceinline__ float chunk_sumsq(const E* __restrict__ src, int n) {
  constexpr int K = Vec<E>::kElems, kPer = kChunk / K / kThreads;
  float s = 0.f;
  const int nv = n / K;
  uint4 w[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = threadIdx.x + i * kThreads;
    w[i] = v < nv ? reinterpret_cast<const uint4*>(src)[v] : make_uint4(0, 0, 0, 0);
  }
  float half = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    float f[K];
    Vec<E>::unpack(w[i], f);
#pragma unroll
    for (int j = 0; j < K; ++j) (i & 1 ? s : half) = fmaf(f[j], f[j], i & 1 ? s : half);
  }
  s += half;
  const int j = nv * K + threadIdx.x;  // the last, incomplete vector
  if (j < n) {
    const float f = Vec<E>::to_f(src[j]);
    s = fmaf(f, f, s);
  }
  return s;
}

template <typename E>
__device__ __forceinline__ void chunk_scale(const E* src, E* dst, int n, float c) {  // dst may be src
  constexpr int K = Vec<E>::kElems, kPer = kChunk / K / kThreads;
  const int nv = n / K;
  uint4 w[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = threadIdx.x + i * kThreads;
    if (v < nv) w[i] = reinterpret_cast<const uint4*>(src)[v];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int v = threadIdx.x + i * kThreads;
    float f[K];
    Vec<E>::unpack(w[i], f);
#pragma unroll
    for (int j = 0; j < K; ++j) f[j] *= c;
    if (v < nv) reinterpret_cast<uint4*>(dst)[v] = Vec<E>::pack(f);
  }
  const int j = nv * K + threadIdx.x;
  if (j < n) dst[j] = Vec<E>::from_f(Vec<E>::to_f(src[j]) * c);
}

__device__ __forceinline__ int elements_of(const ClipTensors& t, int i, int64_t at) {
  const int64_t left = t.count[i] - at;
  return left < kChunk ? static_cast<int>(left) : kChunk;
}

__global__ void __launch_bounds__(kThreads) sumsq_kernel(const __grid_constant__ ClipTensors t, double* __restrict__ part) {
  __shared__ double red[32];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t chunks = t.first[t.n];
  double sum = 0.0;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = (c - t.first[i]) * kChunk;
    const int n = elements_of(t, i, at);
    const float s = t.bf16[i] ? chunk_sumsq(static_cast<const __nv_bfloat16*>(t.src[i]) + at, n)
                              : chunk_sumsq(static_cast<const float*>(t.src[i]) + at, n);
    sum += static_cast<double>(s);
  }
  sum = cta_sum_f64(sum, red);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ float norm_of(const double* part, int nparts, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThreads) s += part[i];
  return static_cast<float>(sqrt(cta_sum_f64(s, red)));
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* part, int nparts, float* norm) {
  __shared__ double red[32];
  pdl_wait();
  pdl_launch_dependents();
  const float v = norm_of(part, nparts, red);
  if (threadIdx.x == 0) *norm = v;
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ ClipTensors t, const double* part, int nparts,
                                                         float max_norm, float* norm) {
  __shared__ double red[32];
  pdl_wait();
  pdl_launch_dependents();
  const float v = norm_of(part, nparts, red);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  const float q = max_norm / (v + 1e-6f);
  const float c = q > 1.f ? 1.f : q;  // a NaN norm makes every output NaN
  const int64_t chunks = t.first[t.n];
  for (int64_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const int i = tensor_of(t, k);
    if (c == 1.f && t.src[i] == t.dst[i]) continue;  // in place and nothing to clip
    const int64_t at = (k - t.first[i]) * kChunk;
    const int n = elements_of(t, i, at);
    if (t.bf16[i])
      chunk_scale(static_cast<const __nv_bfloat16*>(t.src[i]) + at, static_cast<__nv_bfloat16*>(t.dst[i]) + at, n, c);
    else
      chunk_scale(static_cast<const float*>(t.src[i]) + at, static_cast<float*>(t.dst[i]) + at, n, c);
  }
}

}  // namespace

int64_t clip_chunks(int64_t count) { return (count + kChunk - 1) / kChunk; }

int clip_grid(int64_t chunks) {
  int64_t cap = int64_t(num_sms()) * 4;
  if (cap > kClipMaxGrid) cap = kClipMaxGrid;
  return static_cast<int>(chunks < cap ? chunks : cap);
}

cudaError_t launch_clip_sumsq(const ClipTensors& t, double* part, cudaStream_t s) {
  return launch_pdl(sumsq_kernel, dim3(clip_grid(t.first[t.n])), dim3(kThreads), 0, s, t, part);
}

cudaError_t launch_clip_norm(const double* part, int nparts, float* norm, cudaStream_t s) {
  return launch_pdl(norm_kernel, dim3(1), dim3(kThreads), 0, s, part, nparts, norm);
}

cudaError_t launch_clip_scale(const ClipTensors& t, const double* part, int nparts, float max_norm, float* norm,
                              cudaStream_t s) {
  return launch_pdl(scale_kernel, dim3(clip_grid(t.first[t.n])), dim3(kThreads), 0, s, t, part, nparts, max_norm, norm);
}

}  // namespace tpmlp
