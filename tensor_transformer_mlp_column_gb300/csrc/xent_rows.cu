// xent_rows.cu — the cross entropy over the vocabulary for a few rows of X.
//
// With few rows every product is a pass over W (or a writing of dW) with
// little arithmetic, bound by HBM: a tensor-core tile of 256 rows would be
// nearly empty, and fp32 data would be split into planes that cost more
// traffic than W itself. Here W is streamed once per product through
// registers, in its own type, and the sums are fp32 FMAs:
//   dots    z = X W^T: a warp takes 4 R rows of W; eight lanes share a row, 16
//           bytes each, against X in shared memory as fp32. An X vector read
//           from shared memory serves R rows, which keeps those reads below
//           the FMAs. Its epilogue is that of the tensor-core form: (max, sum)
//           per row of X, or dz.
//   dX      a thread holds four columns of every row's sum and walks a slice of
//           the vocabulary; the slices' sums are added by a second kernel.
//   dW      a thread holds four columns of every row of X and writes four
//           columns of one row of dW after the other.
// dz is kept as [V][TP] fp32, the rows of X contiguous: one broadcast load
// per id.
#include "device.cuh"
#include "internal.h"
#include "train.h"

namespace tpmlp {

namespace {

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes of E as floats.
template <typename E>
struct V16;
template <>
struct V16<float> {
  static constexpr int K = 4;
  __device__ static void unpack(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
};
template <>
struct V16<__nv_bfloat16> {
  static constexpr int K = 8;
  __device__ static void unpack(const uint4& w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(u[j] << 16);
      f[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
};

constexpr int kDotThreads = 512;
constexpr int kDotWarps = kDotThreads / 32;

// X in shared memory: the columns in blocks of 8 K (what eight lanes take),
// within a block first every lane's first four columns, then (bf16) every
// lane's second four, so that a 16-byte read of eight lanes is 128 bytes.
template <typename E>
__device__ __forceinline__ int x_at(int col) {
  constexpr int K = V16<E>::K;
  const int block = col / (8 * K), in = col % (8 * K), lane = in / K, e = in % K;
  return block * 8 * K + (e / 4) * 32 + lane * 4 + e % 4;
}

struct RowsParams {
  const void* X;
  const void* W;
  const int64_t* targets;
  const float* lse;
  const float* dloss;
  float2* stats;  // [gridDim.x][T]
  float* zt;
  float* dz;      // [V][tp]
  int64_t V;
  int T, D, t0, tp;  // rows t0 .. of T
};

// Rows t0 .. t0 + TT - 1 of X (fewer at the end) against all of W.
template <typename E, int TT, int R, bool GRAD>
__global__ void __launch_bounds__(kDotThreads, 1) dots_kernel(const RowsParams p) {
  constexpr int K = V16<E>::K;
  extern __shared__ __align__(16) float xs[];  // [TT][Dp]
  __shared__ float2 red[kDotWarps][TT];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31, j = l & 7, g = l >> 3;
  const int Dp = (p.D + 8 * K - 1) / (8 * K) * (8 * K);
  const int rows = min(TT, p.T - p.t0);
  pdl_wait();
  pdl_launch_dependents();
  const E* X = static_cast<const E*>(p.X) + int64_t(p.t0) * p.D;
  for (int i = threadIdx.x; i < TT * (Dp / K); i += kDotThreads) {  // vectors of K
    const int t = i / (Dp / K), c = i % (Dp / K) * K;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t < rows && c < p.D) v = *reinterpret_cast<const uint4*>(X + int64_t(t) * p.D + c);
    float f[K];
    V16<E>::unpack(v, f);
#pragma unroll
    for (int q = 0; q < K / 4; ++q)
      *reinterpret_cast<float4*>(xs + t * Dp + x_at<E>(c + 4 * q)) = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
  }
  // Lane j of a group looks after the tokens j, j + 8.
  constexpr int TL = (TT + 7) / 8;
  int64_t target[TL];
  float lse[TL], dl[TL], mx[TL], sm[TL];
#pragma unroll
  for (int q = 0; q < TL; ++q) {
    const int t = p.t0 + j + 8 * q;
    const bool on = j + 8 * q < rows;
    target[q] = on ? p.targets[t] : -1;
    if (target[q] >= p.V) target[q] = -1;
    mx[q] = -INFINITY, sm[q] = 0.f;
    if constexpr (GRAD) {
      lse[q] = on ? p.lse[t] : 0.f;
      dl[q] = target[q] >= 0 ? p.dloss[t] : 0.f;
    }
  }
  __syncthreads();
  const E* W = static_cast<const E*>(p.W);
  const int64_t blocks = (p.V + 4 * R - 1) / (4 * R);
  const int steps = Dp / (8 * K);
  for (int64_t b = int64_t(blockIdx.x) + int64_t(w) * gridDim.x; b < blocks; b += int64_t(gridDim.x) * kDotWarps) {
    // This lane's rows: 4 R b + 4 r + g; past the end the last row again, unused.
    const E* src[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int64_t v = b * 4 * R + 4 * r + g;
      if (v >= p.V) v = p.V - 1;
      src[r] = W + v * p.D + j * K;
    }
    float acc[R][TT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[r][t] = 0.f;
#pragma unroll 2
    for (int s = 0; s < steps; ++s) {
      uint4 raw[R];
      const bool in = s * 8 * K + j * K < p.D;  // D is a multiple of 8
#pragma unroll
      for (int r = 0; r < R; ++r) raw[r] = in ? __ldcs(reinterpret_cast<const uint4*>(src[r] + s * 8 * K)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < K / 4; ++q) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const float4 x = *reinterpret_cast<const float4*>(xs + t * Dp + s * 8 * K + q * 32 + j * 4);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float f[K];
            V16<E>::unpack(raw[r], f);
            acc[r][t] = fmaf(f[4 * q], x.x, acc[r][t]);
            acc[r][t] = fmaf(f[4 * q + 1], x.y, acc[r][t]);
            acc[r][t] = fmaf(f[4 * q + 2], x.z, acc[r][t]);
            acc[r][t] = fmaf(f[4 * q + 3], x.w, acc[r][t]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t v = b * 4 * R + 4 * r + g;
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], o);
      if (v >= p.V) continue;
#pragma unroll
      for (int q = 0; q < TL; ++q) {
        float z = 0.f;
#pragma unroll
        for (int t = 8 * q; t < TT && t < 8 * q + 8; ++t) z = j == (t & 7) ? acc[r][t] : z;
        if (j + 8 * q >= rows) continue;
        if constexpr (GRAD) {
          const float d = expf(z - lse[q]) - (v == target[q] ? 1.f : 0.f);
          p.dz[v * p.tp + p.t0 + j + 8 * q] = dl[q] != 0.f ? d * dl[q] : 0.f;
        } else {
          if (v == target[q]) p.zt[p.t0 + j + 8 * q] = z;
          const float top = fmaxf(mx[q], z * kXentLog2e);
          const float base = top == -INFINITY ? 0.f : top;
          sm[q] = sm[q] * exp2_approx(mx[q] - base) + exp2_approx(fmaf(z, kXentLog2e, -base));
          mx[q] = top;
        }
      }
    }
  }
  if constexpr (!GRAD) {
    // The four groups of a warp, then the warps, each in their order.
    auto join = [](float& m, float& s, float m2, float s2) {
      const float top = fmaxf(m, m2);
      const float base = top == -INFINITY ? 0.f : top;
      s = s * exp2_approx(m - base) + s2 * exp2_approx(m2 - base);
      m = top;
    };
#pragma unroll
    for (int q = 0; q < TL; ++q) {
#pragma unroll
      for (int o = 8; o < 32; o <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, mx[q], o), s2 = __shfl_xor_sync(0xffffffffu, sm[q], o);
        join(mx[q], sm[q], m2, s2);
      }
      if (g == 0 && j + 8 * q < TT) red[w][j + 8 * q] = make_float2(mx[q], sm[q]);
    }
    __syncthreads();
    if (threadIdx.x < rows) {
      float m = red[0][threadIdx.x].x, s = red[0][threadIdx.x].y;
      for (int v = 1; v < kDotWarps; ++v) join(m, s, red[v][threadIdx.x].x, red[v][threadIdx.x].y);
      p.stats[int64_t(blockIdx.x) * p.T + p.t0 + threadIdx.x] = make_float2(m, s);
    }
  }
}

constexpr int kColThreads = 256;
constexpr int kIds = 4;  // ids on their way at a time

__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&f)[4]) {
  const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
  f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&f)[4]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&f)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)));
}

// part[slice][t][d] = sum over the slice's ids of dz[v][t] W[v][d]; TT = tp.
template <typename E, int TT>
__global__ void __launch_bounds__(kColThreads) rows_dx_kernel(const float* __restrict__ dz, const E* __restrict__ W, int64_t V,
                                                              int T, int D, int64_t per, float* __restrict__ part) {
  pdl_wait();
  pdl_launch_dependents();
  const int d = (blockIdx.x * kColThreads + threadIdx.x) * 4;
  if (d >= D) return;
  const int64_t from = blockIdx.y * per, to = from + per < V ? from + per : V;
  float acc[TT][4];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[t][c] = 0.f;
  for (int64_t v = from; v < to; v += kIds) {
    float w[kIds][4];
#pragma unroll
    for (int u = 0; u < kIds; ++u) {
      if (v + u < to) load4(W + (v + u) * D + d, w[u]);
    }
#pragma unroll
    for (int u = 0; u < kIds; ++u) {
      if (v + u >= to) break;
#pragma unroll
      for (int q = 0; q < TT; q += 4) {
        const float4 z = __ldg(reinterpret_cast<const float4*>(dz + (v + u) * TT + q));
        const float zz[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[q + t][c] = fmaf(zz[t], w[u][c], acc[q + t][c]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
    if (t < T) *reinterpret_cast<float4*>(part + (int64_t(blockIdx.y) * T + t) * D + d) = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
}

// dW[v][d] = sum over t of dz[v][t] X[t][d].
template <typename E, int TT>
__global__ void __launch_bounds__(kColThreads) rows_dw_kernel(const float* __restrict__ dz, const E* __restrict__ X, int64_t V,
                                                              int T, int D, int64_t per, E* __restrict__ dW) {
  pdl_wait();
  pdl_launch_dependents();
  const int d = (blockIdx.x * kColThreads + threadIdx.x) * 4;
  if (d >= D) return;
  const int64_t from = blockIdx.y * per, to = from + per < V ? from + per : V;
  float x[TT][4];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
    if (t < T) load4(X + int64_t(t) * D + d, x[t]);
  }
#pragma unroll 4
  for (int64_t v = from; v < to; ++v) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < TT; q += 4) {
      const float4 z = __ldg(reinterpret_cast<const float4*>(dz + v * TT + q));
      const float zz[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = fmaf(zz[t], x[q + t][c], acc[c]);
    }
    store4(dW + v * D + d, acc);
  }
}

template <typename E, int TT, int R, bool GRAD>
cudaError_t dots(RowsParams p, int grid, cudaStream_t s) {
  constexpr int K = V16<E>::K;
  const size_t smem = size_t(TT) * ((p.D + 8 * K - 1) / (8 * K) * (8 * K)) * 4;
  auto kern = dots_kernel<E, TT, R, GRAD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(kDotThreads), smem, s, p);
}

// Rows of X per pass: as many as fit shared memory in fp32, at most 16.
int group_of(int64_t T, int64_t D) {
  const int64_t Dp = (D + 63) / 64 * 64;
  int t = T > 8 ? 16 : T > 4 ? 8 : T > 2 ? 4 : T > 1 ? 2 : 1;
  while (t > 1 && t * Dp * 4 > kXentRowsSmem) t /= 2;
  return t;
}

template <typename E, bool GRAD>
cudaError_t all_dots(RowsParams p, cudaStream_t s) {
  const int tt = group_of(p.T, p.D), grid = xent_rows_parts(p.V);
  for (p.t0 = 0; p.t0 < p.T; p.t0 += tt) {
    const cudaError_t e = tt == 16  ? dots<E, 16, 4, GRAD>(p, grid, s)
                          : tt == 8 ? dots<E, 8, 4, GRAD>(p, grid, s)
                          : tt == 4 ? dots<E, 4, 4, GRAD>(p, grid, s)
                          : tt == 2 ? dots<E, 2, 4, GRAD>(p, grid, s)
                                    : dots<E, 1, 4, GRAD>(p, grid, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Ids of a slice, so that the slices and slabs of columns give every SM `ctas` CTAs.
int64_t ids_per(int64_t V, int64_t slabs, int ctas) {
  int64_t slices = (int64_t(num_sms()) * ctas + slabs - 1) / slabs;
  const int64_t per = (V + slices - 1) / slices;
  return (per + 7) / 8 * 8;
}

template <typename E, int TT>
cudaError_t backward(const float* dz, const E* X, const E* W, int64_t T, int64_t D, int64_t V, float* part, E* dW,
                     cudaStream_t s) {
  const int64_t slabs = (D / 4 + kColThreads - 1) / kColThreads;
  const int64_t per = xent_rows_ids(D, V);
  const dim3 grid(static_cast<unsigned>(slabs), static_cast<unsigned>((V + per - 1) / per));
  cudaError_t e = launch_pdl(rows_dx_kernel<E, TT>, grid, dim3(kColThreads), 0, s, dz, W, V, int(T), int(D), per, part);
  if (e != cudaSuccess) return e;
  const int64_t per_w = ids_per(V, slabs, 8);
  const dim3 grid_w(static_cast<unsigned>(slabs), static_cast<unsigned>((V + per_w - 1) / per_w));
  return launch_pdl(rows_dw_kernel<E, TT>, grid_w, dim3(kColThreads), 0, s, dz, X, V, int(T), int(D), per_w, dW);
}

template <typename E>
cudaError_t rows_backward(const float* dz, const void* X, const void* W, int64_t T, int64_t D, int64_t V, float* part,
                          void* dW, cudaStream_t s) {
  const E *x = static_cast<const E*>(X), *w = static_cast<const E*>(W);
  E* o = static_cast<E*>(dW);
  switch (xent_rows_tp(T)) {
    case 4:
      return backward<E, 4>(dz, x, w, T, D, V, part, o, s);
    case 8:
      return backward<E, 8>(dz, x, w, T, D, V, part, o, s);
    case 16:
      return backward<E, 16>(dz, x, w, T, D, V, part, o, s);
    default:
      return backward<E, 32>(dz, x, w, T, D, V, part, o, s);
  }
}

}  // namespace

int xent_rows_tp(int64_t T) { return T <= 4 ? 4 : T <= 8 ? 8 : T <= 16 ? 16 : 32; }

int xent_rows_parts(int64_t V) {
  const int64_t want = (V + 16 * 4 - 1) / (16 * 4), cap = num_sms();  // four blocks of 16 ids a CTA at least
  return static_cast<int>(want < cap ? want : cap);
}

int64_t xent_rows_ids(int64_t D, int64_t V) { return ids_per(V, (D / 4 + kColThreads - 1) / kColThreads, 3); }

cudaError_t launch_xent_rows_stats(const void* X, const void* W, const int64_t* targets, int64_t T, int64_t D, int64_t V,
                                   int is_bf16, float2* stats, float* zt, cudaStream_t s) {
  RowsParams p{};
  p.X = X, p.W = W, p.targets = targets, p.stats = stats, p.zt = zt, p.V = V, p.T = int(T), p.D = int(D);
  return is_bf16 ? all_dots<__nv_bfloat16, false>(p, s) : all_dots<float, false>(p, s);
}

cudaError_t launch_xent_rows_dz(const void* X, const void* W, const int64_t* targets, const float* lse, const float* dloss,
                                int64_t T, int64_t D, int64_t V, int is_bf16, float* dz, cudaStream_t s) {
  RowsParams p{};
  p.X = X, p.W = W, p.targets = targets, p.lse = lse, p.dloss = dloss, p.dz = dz, p.V = V, p.T = int(T), p.D = int(D);
  p.tp = xent_rows_tp(T);
  return is_bf16 ? all_dots<__nv_bfloat16, true>(p, s) : all_dots<float, true>(p, s);
}

cudaError_t launch_xent_rows_products(const float* dz, const void* X, const void* W, int64_t T, int64_t D, int64_t V,
                                      int is_bf16, float* part, void* dW, cudaStream_t s) {
  return is_bf16 ? rows_backward<__nv_bfloat16>(dz, X, W, T, D, V, part, dW, s)
                 : rows_backward<float>(dz, X, W, T, D, V, part, dW, s);
}

}  // namespace tpmlp
