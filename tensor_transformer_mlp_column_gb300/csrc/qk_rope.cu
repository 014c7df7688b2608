// qk_rope.cu — the norm of every head of the queries and keys and the rotation
// of its pairs by their positions, in one pass, and the gradients.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = r x,  z = n * w,
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t) for the pairs of z
//   back: g = dy turned back, dw = sum of g * n over tokens and heads,
//         dx = r (g * w - n mean(g * w * n))
//
// The angle of a pair is a number of turns, pos * f / (2 pi), of which only the
// fraction counts: with f / (2 pi) as a 64-bit binary fraction the product
// modulo 2^64 is that fraction to 2^-64 pos, at any position, without 64-bit
// floating point.
//
// Bound by memory: x is read once (backward: x and dy) and y written once. A
// head belongs to a group of 8, 16 or 32 lanes, eight elements a lane, held in
// registers between the sums and the result: the two runs of four whose pairs
// they are (4 i and rot / 2 + 4 i) or eight in a row. A group takes several
// heads of one token, so that a lane makes its four angles once for them, and
// has several heads' loads in flight. The gradients of the weights are summed by
// each lane over the heads it takes, then over the CTA's groups, then (in 64
// bits) over the CTAs, in an order that the sizes fix.
#include "attn_core.h"

#include <cuda_bf16.h>

#include "device.cuh"
#include "internal.h"
#include "trace.h"

namespace tpmlp {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxGrid = 152 * 4;  // of the backward: CTAs whose sums are added at the end

template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  using type = uint2;
};
template <>
struct Raw<float> {
  using type = uint4;
};

__device__ __forceinline__ void unpack(uint2 u, float* v) {
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(uint4 u, float* v) {
  v[0] = __uint_as_float(u.x);
  v[1] = __uint_as_float(u.y);
  v[2] = __uint_as_float(u.z);
  v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void pack(uint2& u, const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void pack(uint4& u, const float* v) {
  u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// What a lane does with a head: its elements at a .. a + 3 and b .. b + 3, and their four angles.
struct Lane {
  int a, b;
  bool on, turned;
  float cos[4], sin[4];
};

template <int G>
__device__ __forceinline__ Lane lane_of(const RopeShape& s, int u) {
  Lane l;
  l.on = 8 * u < s.dim;
  l.turned = 8 * u < s.rot;
  const bool halves = l.turned && !s.interleaved;
  l.a = halves ? 4 * u : 8 * u;
  l.b = halves ? s.rot / 2 + 4 * u : 8 * u + 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) l.cos[i] = 1.f, l.sin[i] = 0.f;  // of a lane that gets no token
  return l;
}

__device__ __forceinline__ void angles(const RopeShape& s, int64_t t, int u, Lane& l) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l.cos[i] = 1.f;
    l.sin[i] = 0.f;
    if (l.turned) {
      const uint64_t turn = static_cast<uint64_t>(s.pos[s.axis[4 * u + i] * s.T + t]) * s.turn[4 * u + i];
      // turn / 2^64 of a full turn, as half turns in [-1, 1).
      sincospif(static_cast<float>(static_cast<int64_t>(turn)) * 0x1p-63f, &l.sin[i], &l.cos[i]);
    }
  }
}

// The pairs of v (4 elements at a, 4 at b) turned by the angles, `back` by their negatives.
__device__ __forceinline__ void turn(float (&v)[8], const Lane& l, bool interleaved, bool back) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = l.cos[i], s = back ? -l.sin[i] : l.sin[i];
    if (interleaved) {
      const float x = v[2 * i], y = v[2 * i + 1];
      v[2 * i] = fmaf(x, c, -(y * s));
      v[2 * i + 1] = fmaf(x, s, y * c);
    } else {
      const float x = v[i], y = v[4 + i];
      v[i] = fmaf(x, c, -(y * s));
      v[4 + i] = fmaf(x, s, y * c);
    }
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Items: (token, run of heads); item i is token i / runs, and its j-th head is i % runs + j runs, q's heads first.
template <typename T, int G, bool BACK>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeCall c, int runs, int per,
                                                        float* part) {
  constexpr int kGroups = kThreads / G;
  constexpr int kAhead = BACK ? 2 : 4;  // heads whose loads are in flight
  using R = typename Raw<T>::type;
  __shared__ float sums[BACK ? kThreads / 32 : 1][BACK ? 2 : 1][BACK ? 8 * G : 1];
  const RopeShape& s = c.s;
  const int u = threadIdx.x % G;
  Lane l = lane_of<G>(s, u);
  const bool norm = c.w[0] != nullptr;
  const int all = s.heads[0] + s.heads[1];
  const float inv_dim = 1.f / static_cast<float>(s.dim);
  pdl_wait();
  pdl_launch_dependents();
  float w[2][8], dw[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) w[k][e] = 1.f, dw[k][e] = 0.f;
  if (norm && l.on) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      unpack(*reinterpret_cast<const R*>(static_cast<const T*>(c.w[k]) + l.a), w[k]);
      unpack(*reinterpret_cast<const R*>(static_cast<const T*>(c.w[k]) + l.b), w[k] + 4);
    }
  }
  const int64_t items = s.T * runs;
  // Every lane of a warp goes through the same number of items: the sums of a head are over the warp's shuffles.
  const int64_t step = int64_t(gridDim.x) * kGroups;
  for (int64_t base = int64_t(blockIdx.x) * kGroups; base < items; base += step) {
    const int64_t item = base + threadIdx.x / G;
    const bool live = item < items && l.on;
    const int64_t t = item < items ? item / runs : 0;
    const int h0 = static_cast<int>(item - t * runs);
    if (live) angles(s, t, u, l);
    for (int j0 = 0; j0 < per; j0 += kAhead) {
      R xa[kAhead], xb[kAhead], ga[kAhead], gb[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int h = h0 + (j0 + j) * runs;
        if (live && j0 + j < per && h < all) {
          const int k = h >= s.heads[0];
          const int hk = h - (k ? s.heads[0] : 0);
          const T* x = static_cast<const T*>(c.x[k].p) + t * c.x[k].token + hk * c.x[k].head;
          xa[j] = *reinterpret_cast<const R*>(x + l.a);
          xb[j] = *reinterpret_cast<const R*>(x + l.b);
          if (BACK) {
            const T* g = static_cast<const T*>(c.dy[k].p) + t * c.dy[k].token + hk * c.dy[k].head;
            ga[j] = *reinterpret_cast<const R*>(g + l.a);
            gb[j] = *reinterpret_cast<const R*>(g + l.b);
          }
        } else {
          xa[j] = xb[j] = R{};
          if (BACK) ga[j] = gb[j] = R{};
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int h = h0 + (j0 + j) * runs;
        const bool mine = live && j0 + j < per && h < all;
        const int k = h >= s.heads[0];
        float x[8], y[8];
        unpack(xa[j], x);
        unpack(xb[j], x + 4);
        if (!BACK) {
          float r = 1.f;
          if (norm) {
            float q = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) q = fmaf(x[e], x[e], q);
            r = 1.0f / sqrtf(fmaf(group_sum<G>(q), inv_dim, s.eps));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e] * r * (k ? w[1][e] : w[0][e]);
          if (l.turned) turn(y, l, s.interleaved, false);
        } else {
          unpack(ga[j], y);
          unpack(gb[j], y + 4);
          if (l.turned) turn(y, l, s.interleaved, true);
          if (norm) {
            float q = 0.f, d = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              q = fmaf(x[e], x[e], q);
              d = fmaf(y[e] * (k ? w[1][e] : w[0][e]), x[e], d);
            }
            const float root = sqrtf(fmaf(group_sum<G>(q), inv_dim, s.eps));
            const float r = mine ? 1.0f / root : 0.f;  // a lane without a head adds nothing to dw, even at eps = 0
            const float m = group_sum<G>(d) * r * inv_dim;  // mean(g * w * n)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float n = x[e] * r;
              if (k)
                dw[1][e] = fmaf(y[e], n, dw[1][e]);
              else
                dw[0][e] = fmaf(y[e], n, dw[0][e]);
              y[e] = r * fmaf(-n, m, y[e] * (k ? w[1][e] : w[0][e]));
            }
          }
        }
        if (mine) {
          const int hk = h - (k ? s.heads[0] : 0);
          T* o = static_cast<T*>(c.y[k].p) + t * c.y[k].token + hk * c.y[k].head;
          R v;
          pack(v, y);
          *reinterpret_cast<R*>(o + l.a) = v;
          pack(v, y + 4);
          *reinterpret_cast<R*>(o + l.b) = v;
        }
      }
    }
  }
  if constexpr (BACK) {
    if (!norm) return;
    // The groups of a warp, then the CTA's warps, in order.
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = dw[k][e];
#pragma unroll
        for (int o = G; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (threadIdx.x % 32 < G && l.on) sums[threadIdx.x / 32][k][(e < 4 ? l.a : l.b - 4) + e] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * s.dim; i += kThreads) {
      const int k = i / s.dim, e = i % s.dim;
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kThreads / 32; ++q) v += sums[q][k][e];
      part[int64_t(blockIdx.x) * 2 * s.dim + i] = v;
    }
  }
}

// dw[e] = the sum of the CTAs' parts: a CTA per 32 of the 2 dim columns.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* part, int parts, int dim, float* dwq, float* dwk) {
  __shared__ double rows[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  double v = 0.0;
  if (col < 2 * dim)
    for (int i = warp; i < parts; i += 32) v += part[int64_t(i) * 2 * dim + col];
  rows[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && col < 2 * dim) {
    double sum = 0.0;
    for (int i = 0; i < 32; ++i) sum += rows[i][lane];
    (col < dim ? dwq : dwk)[col < dim ? col : col - dim] = static_cast<float>(sum);
  }
}

struct RopePlan {
  int g, runs, per;
  int64_t grid;
};

// How the heads are handed out: a group takes up to 8 heads of a token, fewer
// where the GPU would not be full (2048 threads an SM).
RopePlan plan_rope(int64_t T, int heads, int kv_heads, int dim, int backward) {
  RopePlan p;
  p.g = dim <= 64 ? 8 : dim <= 128 ? 16 : 32;
  const int all = heads + kv_heads;
  const int64_t resident = int64_t(152) * 2048 / p.g;
  int64_t per = T * all / resident;
  per = per < 1 ? 1 : per > 8 ? 8 : per;
  p.runs = static_cast<int>((all + per - 1) / per);
  p.per = (all + p.runs - 1) / p.runs;
  const int groups = kThreads / p.g;
  const int64_t ctas = (T * p.runs + groups - 1) / groups;
  const int64_t most = backward ? kMaxGrid : 152 * 16;
  p.grid = ctas < most ? ctas : most;
  return p;
}

template <typename T, int G>
cudaError_t launch_rope(const RopeCall& c, const RopePlan& p, cudaStream_t s) {
  return launch_pdl(c.backward ? rope_kernel<T, G, true> : rope_kernel<T, G, false>, dim3(static_cast<unsigned>(p.grid)),
                    dim3(kThreads), 0, s, c, p.runs, p.per, static_cast<float*>(c.ws));
}

}  // namespace

size_t rope_backward_workspace(int64_t T, int heads, int kv_heads, int dim) {
  if (T == 0) return 0;
  return static_cast<size_t>(plan_rope(T, heads, kv_heads, dim, 1).grid) * 2 * dim * sizeof(float);
}

cudaError_t run_qk_rope(const RopeCall& c, cudaStream_t s) {
  TraceScope trace(c.backward ? "qk_rope_backward" : "qk_rope_forward", s);
  const bool norm = c.w[0] != nullptr;
  if (c.s.T == 0) {  // backward only
    for (int k = 0; k < 2 && norm; ++k) {
      cudaError_t e = cudaMemsetAsync(c.dw[k], 0, c.s.dim * sizeof(float), s);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  const RopePlan p = plan_rope(c.s.T, c.s.heads[0], c.s.heads[1], c.s.dim, c.backward);
  cudaError_t e;
  if (c.bf16)
    e = p.g == 8 ? launch_rope<__nv_bfloat16, 8>(c, p, s) : p.g == 16 ? launch_rope<__nv_bfloat16, 16>(c, p, s)
                                                                      : launch_rope<__nv_bfloat16, 32>(c, p, s);
  else
    e = p.g == 8 ? launch_rope<float, 8>(c, p, s) : p.g == 16 ? launch_rope<float, 16>(c, p, s)
                                                              : launch_rope<float, 32>(c, p, s);
  if (e != cudaSuccess || !c.backward || !norm) return e;
  return launch_pdl(rope_dw_kernel, dim3((2 * c.s.dim + 31) / 32), dim3(1024), 0, s, static_cast<const float*>(c.ws),
                    static_cast<int>(p.grid), c.s.dim, c.dw[0], c.dw[1]);
}

}  // namespace tpmlp
