// qk_rope.cu — the norm of every head of the queries and keys and the rotation
// of its pairs by their positions, in one pass, and the gradients.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = r x,  z = n * w,
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t) for the pairs of z
//   back: g = dy turned back, dw = sum of g * n over tokens and heads,
//         dx = r (g * w - n mean(g * w * n))
//
// The angle of a pair is a number of turns, pos * f / (2 pi), of which only the
// fraction counts: with f / (2 pi) as a 64-bit binary fraction (made by the host,
// off by less than 2^-64) the product modulo 2^64 is that fraction to 2^-64 pos, at
// any position, without 64-bit floating point here.
//
// Bound by memory: x is read once (backward: x and dy) and y written once (16384
// tokens, 32 + 8 heads of 128, bf16: 62 us, 5.4 TB/s, and 97 us, 5.2 TB/s; fp32 107
// and 162 us, 6.3 and 6.2); what costs beside it is the instructions. A head belongs to a group of lanes, 2 RUN
// elements a lane, held in registers between the sums and the result: two runs
// of RUN whose pairs they are (i and rot / 2 + i), or 2 RUN in a row. RUN is 8
// for bf16 where the halves begin on 16 bytes (rot and head_dim multiples of 16),
// else 4. A CTA has heads of q or of k; a group takes up to 8 heads of one token,
// so that a lane makes its angles once for them, and has several heads' loads in
// flight while it does. The gradients of the weights are summed by each lane over
// the heads it takes, then over the CTA's groups, then over the CTAs, in an order
// that the sizes fix.
#include "attn_core.h"

#include <cuda_bf16.h>

#include "device.cuh"
#include "internal.h"
#include "trace.h"

namespace tpmlp {

namespace {

constexpr int kThreads = 256;

template <typename T, int RUN>
struct RawOf {
  using type = uint4;  // 8 bf16 or 4 fp32
};
template <>
struct RawOf<__nv_bfloat16, 4> {
  using type = uint2;
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float* v) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[2 * i] = __uint_as_float(x[i] << 16);
      v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
    } else {
      v[i] = __uint_as_float(x[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ void unpack(const uint2& u, float* v) {
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void pack(uint4& u, const float* v) {
  if constexpr (sizeof(T) == 2)
    u = make_uint4(pack_pair(v[0], v[1]), pack_pair(v[2], v[3]), pack_pair(v[4], v[5]), pack_pair(v[6], v[7]));
  else
    u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <typename T>
__device__ __forceinline__ void pack(uint2& u, const float* v) {
  u = make_uint2(pack_pair(v[0], v[1]), pack_pair(v[2], v[3]));
}

// cos and sin of `turn` / 2^64 of a full turn. For bf16 the upper 32 bits and the special-function unit, off by at
// most 2^-20: a thousandth of the result's rounding.
template <typename T>
__device__ __forceinline__ void angle(uint64_t turn, float& cos, float& sin) {
  if constexpr (sizeof(T) == 2) {
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * (3.14159265358979f * 0x1p-31f);
    cos = __cosf(x);
    sin = __sinf(x);
  } else {
    sincospif(static_cast<float>(static_cast<int64_t>(turn)) * 0x1p-63f, &sin, &cos);
  }
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float cos, float sin) {
  const float x = a;
  a = fmaf(x, cos, -(b * sin));
  b = fmaf(x, sin, b * cos);
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A lane's weights, from shared memory: they would take 16 of the registers that loads in flight need.
template <int RUN>
__device__ __forceinline__ void weights(const float* s_w, int a, int b, float (&w)[2 * RUN]) {
#pragma unroll
  for (int i = 0; i < RUN; i += 4) {
    const float4 x = *reinterpret_cast<const float4*>(s_w + a + i), y = *reinterpret_cast<const float4*>(s_w + b + i);
    w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
    w[RUN + i] = y.x, w[RUN + i + 1] = y.y, w[RUN + i + 2] = y.z, w[RUN + i + 3] = y.w;
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// How the heads are handed out. Items of a kind (q, k): (token, run of heads); item i is token i / runs, and its j-th
// head is i % runs + j runs.
struct RopePlan {
  int run, group;  // elements of a run; lanes of a group
  int runs[2], per[2];
  int ctas[2];
};

template <typename T, int RUN, int G, bool BACK>
__global__ void __launch_bounds__(kThreads, BACK ? 2 : 3) rope_kernel(const __grid_constant__ RopeCall c,
                                                           const __grid_constant__ RopePlan plan, float* part) {
  constexpr int kGroups = kThreads / G;
  constexpr int kAhead = 2;  // heads whose loads are in flight
  constexpr int N = 2 * RUN;            // elements of a lane
  using R = typename RawOf<T, RUN>::type;
  __shared__ uint64_t s_turn[kRopeMaxDim / 2];
  __shared__ uint8_t s_axis[kRopeMaxDim / 2];
  __shared__ __align__(16) float s_w[kRopeMaxDim];
  __shared__ float sums[BACK ? kThreads / 32 : 1][BACK ? N * G : 1];
  const RopeShape& s = c.s;
  const int kind = static_cast<int>(blockIdx.x) >= plan.ctas[0];
  const int cta = blockIdx.x - (kind ? plan.ctas[0] : 0);
  const int heads = s.heads[kind], runs = plan.runs[kind], per = plan.per[kind];
  const int u = threadIdx.x % G;
  // A lane's elements: a .. a + RUN - 1 and b .. b + RUN - 1.
  const bool on = N * u < s.dim, turned = N * u < s.rot, halves = turned && !s.interleaved;
  const int a = halves ? RUN * u : N * u, b = halves ? s.rot / 2 + RUN * u : N * u + RUN;
  const float inv_dim = 1.f / static_cast<float>(s.dim);
  for (int i = threadIdx.x; i < s.rot / 2; i += kThreads) {
    s_turn[i] = s.turn[i];
    s_axis[i] = s.axis[i];
  }
  pdl_wait();
  const bool norm = c.w[0] != nullptr;
  for (int i = threadIdx.x; norm && i < kRopeMaxDim; i += kThreads)
    s_w[i] = i < s.dim ? to_float(static_cast<const T*>(c.w[kind])[i]) : 0.f;
  __syncthreads();
  bool alike = turned;  // one axis turns all pairs of this lane
#pragma unroll
  for (int i = 1; i < RUN; ++i) alike = alike && s_axis[RUN * u + i] == s_axis[RUN * u];
  float dw[N], cos[RUN], sin[RUN];
#pragma unroll
  for (int e = 0; e < N; ++e) dw[e] = 0.f;
#pragma unroll
  for (int e = 0; e < RUN; ++e) cos[e] = 1.f, sin[e] = 0.f;  // of a lane that gets no token or turns nothing
  const HeadsView xv = c.x[kind], gv = c.dy[kind], yv = c.y[kind];
  const int64_t items = s.T * runs;
  // Every lane of a warp goes through the same number of items: the sums of a head are over the warp's shuffles. The
  // item's token and run follow from the last one's, without a division.
  const int64_t step = int64_t(plan.ctas[kind]) * kGroups;
  const int64_t step_t = step / runs;
  const int step_r = static_cast<int>(step - step_t * runs);
  int64_t item = int64_t(cta) * kGroups + threadIdx.x / G;
  int64_t t = item / runs;
  int h0 = static_cast<int>(item - t * runs);
  for (int64_t base = int64_t(cta) * kGroups; base < items; base += step) {
    // The next kernel's CTAs come when this one's last items are begun: any earlier they take the places of its own (2000
    // tokens, 16 + 4 heads of 128, forward and gradients: 19.9 us with the trigger at the start, 18.7 here).
    if (base + step >= items) pdl_launch_dependents();
    const bool live = item < items && on &&
                      TPMLP_DCHECK(t >= 0 && t < s.T && h0 >= 0 && h0 < heads && a + RUN <= s.dim && b + RUN <= s.dim, c.status,
                                   kChkOutput);
    const int64_t pos = live && alike ? s.pos[s_axis[RUN * u] * s.T + t] : 0;
    const T* x = static_cast<const T*>(xv.p) + t * xv.token + h0 * xv.head;
    const T* g = BACK ? static_cast<const T*>(gv.p) + t * gv.token + h0 * gv.head : nullptr;
    T* y = static_cast<T*>(yv.p) + t * yv.token + h0 * yv.head;
    for (int j0 = 0; j0 < per; j0 += kAhead) {
      R xa[kAhead], xb[kAhead], ga[BACK ? kAhead : 1], gb[BACK ? kAhead : 1];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (live && j0 + j < per && h0 + (j0 + j) * runs < heads) {
          xa[j] = *reinterpret_cast<const R*>(x + a);
          xb[j] = *reinterpret_cast<const R*>(x + b);
          if constexpr (BACK) {
            ga[j] = *reinterpret_cast<const R*>(g + a);
            gb[j] = *reinterpret_cast<const R*>(g + b);
          }
        } else {
          xa[j] = xb[j] = R{};
          if constexpr (BACK) ga[j] = gb[j] = R{};
        }
        x += runs * xv.head;
        if constexpr (BACK) g += runs * gv.head;
      }
      if (j0 == 0 && live && turned) {  // while the first heads come
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
          const int64_t at = alike ? pos : s.pos[s_axis[RUN * u + i] * s.T + t];
          angle<T>(static_cast<uint64_t>(at) * s_turn[RUN * u + i], cos[i], sin[i]);
          if (BACK) sin[i] = -sin[i];
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const bool mine = live && j0 + j < per && h0 + (j0 + j) * runs < heads;
        float v[N], z[N];
        unpack<T>(xa[j], v);
        unpack<T>(xb[j], v + RUN);
        float r = 1.f;
        if (norm) {
          float q = 0.f;
#pragma unroll
          for (int e = 0; e < N; ++e) q = fmaf(v[e], v[e], q);
          r = rsqrtf(fmaf(group_sum<G>(q), inv_dim, s.eps));
        }
        if constexpr (BACK) {
          unpack<T>(ga[j], z);
          unpack<T>(gb[j], z + RUN);
        } else {
          if (norm) {
            float w[N];
            weights<RUN>(s_w, a, b, w);
#pragma unroll
            for (int e = 0; e < N; ++e) z[e] = v[e] * (r * w[e]);
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e) z[e] = v[e];
          }
        }
        if (turned) {
          if (s.interleaved) {
#pragma unroll
            for (int i = 0; i < RUN; ++i) turn_pair(z[2 * i], z[2 * i + 1], cos[i], sin[i]);
          } else {
#pragma unroll
            for (int i = 0; i < RUN; ++i) turn_pair(z[i], z[RUN + i], cos[i], sin[i]);
          }
        }
        if constexpr (BACK) {
          if (norm) {
            if (!mine) r = 0.f;  // a lane without a head adds nothing to dw, even at eps = 0
            float d = 0.f, w[N];
            weights<RUN>(s_w, a, b, w);
#pragma unroll
            for (int e = 0; e < N; ++e) {
              v[e] *= r;
              dw[e] = fmaf(z[e], v[e], dw[e]);
              z[e] *= w[e];
              d = fmaf(z[e], v[e], d);
            }
            const float m = group_sum<G>(d) * inv_dim;
#pragma unroll
            for (int e = 0; e < N; ++e) z[e] = r * fmaf(-v[e], m, z[e]);
          }
        }
        if (mine) {
          R o;
          pack<T>(o, z);
          *reinterpret_cast<R*>(y + a) = o;
          pack<T>(o, z + RUN);
          *reinterpret_cast<R*>(y + b) = o;
        }
        y += runs * yv.head;
      }
    }
    item += step;
    t += step_t;
    h0 += step_r;
    if (h0 >= runs) h0 -= runs, ++t;
  }
  if constexpr (BACK) {
    if (!norm) return;
    // The groups of a warp, then the CTA's warps, in order.
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float v = dw[e];
#pragma unroll
      for (int o = G; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (threadIdx.x % 32 < G && on) sums[threadIdx.x / 32][(e < RUN ? a : b - RUN) + e] = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < s.dim; e += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kThreads / 32; ++q) v += sums[q][e];
      part[int64_t(blockIdx.x) * s.dim + e] = v;
    }
  }
}

// dw[e] = the sum of the CTAs' parts: a CTA per 32 columns of a kind, ten parts at most to each of its 32 warps, whose
// sums are added in a tree (in 64 bits, of which this GPU adds a few a clock, the same took 4 to 8 us more).
constexpr int kMostParts = 10;
static_assert(152 * 2 <= 32 * kMostParts, "parts of the backward's CTAs");
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* part, int ctas_q, int ctas_k, int dim, float* dwq,
                                                       float* dwk, int* status) {
  __shared__ float rows[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kind = blockIdx.y, col = blockIdx.x * 32 + lane;
  const int first = kind ? ctas_q : 0, last = kind ? ctas_q + ctas_k : ctas_q;
  if (!TPMLP_DCHECK(last - first <= 32 * kMostParts, status, kChkReduce)) return;
  float x[kMostParts];
#pragma unroll
  for (int j = 0; j < kMostParts; ++j) {
    const int i = first + warp + 32 * j;
    x[j] = i < last && col < dim ? part[int64_t(i) * dim + col] : 0.f;
  }
#pragma unroll
  for (int n = kMostParts; n > 1; n = (n + 1) / 2)
#pragma unroll
    for (int j = 0; j < n / 2; ++j) x[j] += x[j + (n + 1) / 2];
  rows[warp][lane] = x[0];
  __syncthreads();
  // Warp w: column w of the 32, a row a lane.
  float v = rows[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int c = blockIdx.x * 32 + warp;
  if (lane == 0 && c < dim) (kind ? dwk : dwq)[c] = v;
}

// A group takes up to 8 heads of a token, fewer where the GPU would not be full; as many CTAs as run at once, each (of
// the backward) with a part of dw.
RopePlan plan_rope(int64_t T, const int (&heads)[2], int dim, int rot, int bf16, int backward) {
  RopePlan p{};
  p.run = bf16 && dim % 16 == 0 && rot % 16 == 0 ? 8 : 4;
  const int lanes = (dim + 2 * p.run - 1) / (2 * p.run);
  const int most = 32 / (p.run / 4);  // lanes of the longest head
  p.group = lanes <= most / 4 ? most / 4 : lanes <= most / 2 ? most / 2 : most;
  const int64_t all = heads[0] + heads[1];
  const int64_t resident = int64_t(152) * 512 / p.group;
  int64_t per = T * all / resident;
  per = per < 1 ? 1 : per > 8 ? 8 : per;
  const int groups = kThreads / p.group;
  for (int k = 0; k < 2; ++k) {
    p.runs[k] = static_cast<int>((heads[k] + per - 1) / per);
    p.per[k] = (heads[k] + p.runs[k] - 1) / p.runs[k];
    const int64_t ctas = (T * p.runs[k] + groups - 1) / groups;
    int64_t cap = int64_t(152 * (backward ? 2 : 3)) * heads[k] / all;
    if (cap < 1) cap = 1;
    p.ctas[k] = static_cast<int>(ctas < cap ? ctas : cap);
  }
  return p;
}

template <typename T, int RUN, int G>
cudaError_t launch_rope(const RopeCall& c, const RopePlan& p, cudaStream_t s) {
  return launch_pdl(c.backward ? rope_kernel<T, RUN, G, true> : rope_kernel<T, RUN, G, false>,
                    dim3(static_cast<unsigned>(p.ctas[0] + p.ctas[1])), dim3(kThreads), 0, s, c, p,
                    static_cast<float*>(c.ws));
}

template <typename T, int RUN>
cudaError_t launch_rope(const RopeCall& c, const RopePlan& p, cudaStream_t s) {
  constexpr int M = 32 / (RUN / 4);
  return p.group == M / 4   ? launch_rope<T, RUN, M / 4>(c, p, s)
         : p.group == M / 2 ? launch_rope<T, RUN, M / 2>(c, p, s)
                            : launch_rope<T, RUN, M>(c, p, s);
}

}  // namespace

size_t rope_backward_workspace(int64_t T, int heads, int kv_heads, int dim) {
  if (T == 0) return 0;
  // The most CTAs of any type and rot.
  const int h[2] = {heads, kv_heads};
  int ctas = 0;
  for (int bf16 = 0; bf16 < 2; ++bf16) {
    const RopePlan p = plan_rope(T, h, dim, 0, bf16, 1);
    if (p.ctas[0] + p.ctas[1] > ctas) ctas = p.ctas[0] + p.ctas[1];
  }
  return static_cast<size_t>(ctas) * dim * sizeof(float);
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
  const RopePlan p = plan_rope(c.s.T, c.s.heads, c.s.dim, c.s.rot, c.bf16, c.backward);
  cudaError_t e = !c.bf16      ? launch_rope<float, 4>(c, p, s)
                  : p.run == 8 ? launch_rope<__nv_bfloat16, 8>(c, p, s)
                               : launch_rope<__nv_bfloat16, 4>(c, p, s);
  if (e != cudaSuccess || !c.backward || !norm) return e;
  return launch_pdl(rope_dw_kernel, dim3((c.s.dim + 31) / 32, 2), dim3(1024), 0, s, static_cast<const float*>(c.ws),
                    p.ctas[0], p.ctas[1], c.s.dim, c.dw[0], c.dw[1], c.status);
}

}  // namespace tpmlp
