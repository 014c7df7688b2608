// xent.cu — softmax cross entropy over a large vocabulary, without keeping
// the logits, and its gradient:
//
//   z_tv = x_t . w_v,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,target(t),
//   dz_tv = dloss_t (exp(z_tv - lse_t) - [v = target(t)]),  dX = dz W,  dW = dz^T X.
//
// Forward: one tensor-core product whose epilogue reduces each row's 128
// columns to (max, sum of exponentials) while the next tile is computed, then
// one small kernel that joins the parts: 2 T V D operations, nothing of the
// size T x V is written (8 bytes per 128 logits).
//
// Backward, in pieces of the vocabulary: the logits of a piece are computed
// again (2 T V D) and leave the chip as dz in bf16, which the two products dX
// += dz W and dW = dz^T X read (4 T V D). dz is divided by the largest |dloss|
// before it is rounded and the products are multiplied by it: with the usual
// equal row gradients dz of a target is then -(1 - p), which bf16 holds
// closely where p is small, instead of a number whose rounding would scale
// every target's gradient by the same up to 2^-8. Of up to 64 rows dz is two
// bf16 pieces.
//
// fp32 data are split into three bf16 planes (24 bits in all) and every
// product is the sum of the six plane products that are not below fp32
// rounding, accumulated in fp32 (in runs over two accumulators, for few rows
// over three by the products' size): six times the bf16 work, where the CUDA
// cores would take about thirty times.
#include "device.cuh"
#include "internal.h"
#include "tpmlp.h"
#include "trace.h"
#include "xent_device.cuh"

namespace tpmlp {

namespace {

// A launcher's status, passed on; the step is timed under TPMLP_TRACE=1.
#define XENT_STEP(phase, s, expr)          \
  do {                                     \
    TraceScope trace_scope_(phase, s);     \
    const cudaError_t e_ = (expr);         \
    if (e_ != cudaSuccess) return e_;      \
  } while (0)

// Row t's parts joined. They hold every id but the target: with S 2^M their
// sum of exponentials (M in units of log2) and e = S 2^M / exp(z) of the
// target's z,
//   loss = log(1 + e),   lse = z + loss,
// which keeps its digits where the target is nearly certain and lse - z would
// lose them. A row that does not count has lse = (M + log2 S) / log2 e. log2 e
// is the same fp32 constant that scaled the logits. A CTA takes R rows, its
// warps (and the lanes that share a row) every so many parts each, joined in a
// fixed order.
// M - z log2 e is in fp64: a rounding to fp32 would weigh as much as one of z.
// With `rest` the loss's place holds what z's own rounding left out.
// R = 4 rows a CTA where there are few rows: 128 threads share a row's parts.
constexpr int kJoinWarps = 16;
template <int R>
__global__ void __launch_bounds__(32 * kJoinWarps) xent_join_kernel(const float2* __restrict__ stats, int parts, int64_t T,
                                                                    const int64_t* __restrict__ targets, int64_t V,
                                                                    const float* __restrict__ zt, float* __restrict__ loss,
                                                                    float* __restrict__ lse, int rest, int* status) {
  constexpr int S = 32 / R;  // lanes that share a row
  __shared__ float2 red[kJoinWarps][R];
  pdl_wait();
  pdl_launch_dependents();
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * R + l % R;
  float m = -INFINITY, s = 0.f;
  auto add = [&](float2 p) {
    const float top = fmaxf(m, p.x);
    const float base = top == -INFINITY ? 0.f : top;
    s = s * exp2f(m - base) + p.y * exp2f(p.x - base);
    m = top;
  };
  const int64_t target = t < T && w == 0 ? targets[t] : -1;
  const float z = target >= 0 && target < V ? zt[t] : 0.f;
  const float z_rest = rest && target >= 0 && target < V ? loss[t] : 0.f;
  if (t < T) {
#pragma unroll 8
    for (int i = w * S + l / R; i < parts; i += kJoinWarps * S) add(stats[int64_t(i) * T + t]);
  }
#pragma unroll
  for (int o = R; o < 32; o <<= 1)
    add(make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o)));
  if (l < R) red[w][l] = make_float2(m, s);
  __syncthreads();
  if (w != 0 || l >= R || t >= T) return;
  for (int i = 1; i < kJoinWarps; ++i) add(red[i][l]);
  if (target >= V) atomicCAS(status, 0, kSiteBoundsBase + kChkTarget);
  // log2 of s with its exponent apart, where a rounding to fp32 weighs less.
  const int k = s >= 1.f && s < INFINITY ? ilogbf(s) : 0;
  const double ln2 = 1.0 / double(kXentLog2e);
  double whole = (double(m) + double(k) + double(log2f(ldexpf(s, -k)))) * ln2, own = 0.0;
  if (target >= 0 && target < V) {
    const double zd = double(z) + double(z_rest);
    const double x = double(m) - zd * double(kXentLog2e);  // log2 (e / S)
    if (!(z < INFINITY)) {
      whole = own = double(z - z);
    } else if (s == 0.f) {
      whole = zd;  // there is no other id, or none that counts
    } else if (x < 30.0) {
      const double i = rint(fmax(x, -200.0));
      const float e = ldexpf(s * exp2f(static_cast<float>(fmax(x, -200.0) - i)), static_cast<int>(i));
      own = double(log1pf(e));
      whole = zd + own;
    } else {  // the target's own share of the sum is below the rounding
      own = whole - zd;
    }
  }
  lse[t] = static_cast<float>(whole);
  loss[t] = static_cast<float>(own);
}

// parts[b] = the largest finite |dloss| among CTA b's rows that count.
__global__ void __launch_bounds__(256) xent_dmax_kernel(const float* __restrict__ dloss, const int64_t* __restrict__ targets,
                                                        int64_t T, int64_t V, float* __restrict__ parts) {
  __shared__ float red[8];
  pdl_wait();
  pdl_launch_dependents();
  float m = 0.f;
  for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < T; t += int64_t(gridDim.x) * 256)
    m = fmaxf(m, finite_dloss(dloss, targets, t, V));
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
    parts[blockIdx.x] = m;
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A tensor's rows of d8 groups of 8 elements, copied into one (bf16) or three
// planes (fp32) with rows pitch8 groups apart, `plane` groups from one to the
// next.
struct PlaneCopy {
  const void* x;
  int64_t rows, d8, pitch8, plane;
  uint16_t* out;
};

// Planes of two tensors. fp32: x = high + middle + low, each the bf16 nearest
// to what the ones before leave, 24 bits in all.
template <bool F32>
__global__ void __launch_bounds__(256) xent_planes_kernel(PlaneCopy a, PlaneCopy b) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t na = a.rows * a.d8, n = na + b.rows * b.d8;
  for (int64_t k = int64_t(blockIdx.x) * 256 + threadIdx.x; k < n; k += int64_t(gridDim.x) * 256) {
    const PlaneCopy& c = k < na ? a : b;
    const int64_t i = k < na ? k : k - na;
    int64_t to = i;
    if (c.pitch8 != c.d8) to += (i >> 32 ? i / c.d8 : static_cast<uint32_t>(i) / static_cast<uint32_t>(c.d8)) * (c.pitch8 - c.d8);
    uint4* out = reinterpret_cast<uint4*>(c.out) + to;
    if constexpr (!F32) {
      *out = static_cast<const uint4*>(c.x)[i];
    } else {
      const float4 u = static_cast<const float4*>(c.x)[2 * i], v = static_cast<const float4*>(c.x)[2 * i + 1];
      float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int pl = 0; pl < kXentPlanes; ++pl) {
        out[pl * c.plane] =
            make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] -= __bfloat162float(__float2bfloat16_rn(f[j]));
      }
    }
  }
}

// out = dmax * (part[0] + part[1] + ...), n4 groups of 4 elements, slices
// stride4 groups apart. LANES threads share a group's slices, a consecutive
// part each, and their sums are added in order: with little output (few rows)
// one thread a group would leave most of the GPU idle behind a chain of loads.
template <typename E, int LANES>
__global__ void __launch_bounds__(256) xent_reduce_kernel(const float4* __restrict__ part, int slices, int64_t stride4,
                                                          int64_t n4, const float* __restrict__ dmax, E* __restrict__ out) {
  constexpr int kGroups = 256 / LANES;
  __shared__ float scale_s;
  __shared__ float4 red[LANES > 1 ? 256 : 1];
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < 32) {
    const float m = warp_dmax(dmax, threadIdx.x);
    if (threadIdx.x == 0) scale_s = m;
  }
  __syncthreads();
  const float scale = scale_s;
  const int lane = threadIdx.x / kGroups;  // which part of the slices
  const int per = (slices + LANES - 1) / LANES, from = lane * per, to = min(slices, from + per);
  for (int64_t i0 = int64_t(blockIdx.x) * kGroups; i0 < n4; i0 += int64_t(gridDim.x) * kGroups) {
    const int64_t i = i0 + threadIdx.x % kGroups;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n4) {
#pragma unroll 4
      for (int k = from; k < to; ++k) {
        const float4 a = part[k * stride4 + i];
        v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
      }
    }
    if constexpr (LANES > 1) {
      __syncthreads();
      red[threadIdx.x] = v;
      __syncthreads();
      if (lane == 0) {
#pragma unroll
        for (int k = 1; k < LANES; ++k) {
          const float4 a = red[k * kGroups + threadIdx.x];
          v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
        }
      }
    }
    if (lane != 0 || i >= n4) continue;
    v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
    if constexpr (sizeof(E) == 4)
      reinterpret_cast<float4*>(out)[i] = v;
    else
      reinterpret_cast<uint2*>(out)[i] = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
  }
}

// dW of up to T rows: out [n][D] = dmax * sum_t dz_tv X_t on the CUDA cores, a
// thread N columns of X's rows in registers, kOuterRows rows of out at a time.
// It is the writing of dW, where the tensor cores' tiles load and multiply 64
// rows (V = 64000, D = 1024, with the launch: fp32, T = 1 76 -> 43 us, T = 8 57
// -> 43, but T = 16 57 -> 69; bf16, T = 1 39 -> 24, T = 2 38 -> 24; the tensor
// cores need 31 from T = 3 on, this form 38 at T = 8).
constexpr int kOuterRows = 64;
int64_t outer_max(int is_bf16) { return is_bf16 ? 2 : 8; }
template <typename E, int T>
__global__ void __launch_bounds__(256) xent_outer_kernel(const __nv_bfloat16* __restrict__ dz, int planes, int64_t plane,
                                                         int64_t pitch, const E* __restrict__ X, int rows, int64_t D,
                                                         int64_t n, const float* __restrict__ dmax, E* __restrict__ out) {
  constexpr int N = 16 / sizeof(E);
  __shared__ __align__(16) float s_dz[kOuterRows][T];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  const int64_t col = (int64_t(blockIdx.y) * blockDim.x + threadIdx.x) * N;
  const float scale = warp_dmax(dmax, tid & 31);
  float x[T][N];
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int j = 0; j < N; ++j) x[t][j] = 0.f;
    if (t >= rows || col >= D) continue;
    const uint4 w = *reinterpret_cast<const uint4*>(X + t * D + col);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < N; ++j)
      x[t][j] = sizeof(E) == 4 ? __uint_as_float(u[j]) : __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
  }
  for (int64_t base = int64_t(blockIdx.x) * kOuterRows; base < n; base += int64_t(gridDim.x) * kOuterRows) {
    const int here = n - base < kOuterRows ? static_cast<int>(n - base) : kOuterRows;
    __syncthreads();
    for (int i = tid; i < T * kOuterRows; i += blockDim.x * blockDim.y) {
      const int t = i / kOuterRows, r = i % kOuterRows;
      float d = 0.f;
      if (t < rows && r < here)
        for (int pl = planes - 1; pl >= 0; --pl) d += __bfloat162float(dz[pl * plane + t * pitch + base + r]);
      s_dz[r][t] = d * scale;
    }
    __syncthreads();
    if (col >= D) continue;
#pragma unroll 4
    for (int r = threadIdx.y; r < here; r += blockDim.y) {
      float v[N];
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = s_dz[r][0] * x[0][j];
#pragma unroll
      for (int t = 1; t < T; ++t)
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = fmaf(s_dz[r][t], x[t][j], v[j]);
      uint4 w;
      if constexpr (sizeof(E) == 4)
        w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      else
        w = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
      *reinterpret_cast<uint4*>(out + (base + r) * D + col) = w;
    }
  }
}

int grid_for(int64_t items) {
  const int64_t want = (items + 255) / 256, cap = int64_t(num_sms()) * 8;
  return static_cast<int>(want < 1 ? 1 : want < cap ? want : cap);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
int64_t ceil_to(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Rows of one slice of a product's fp32 partial sums: a warp's store covers 32.
int64_t slice_rows(int64_t M) { return ceil_to(M, 32); }

// Into how many runs a product's K is cut: few output tiles leave most of the
// GPU idle for the whole of a long K, more runs cost their partial sums'
// traffic. Cost in K blocks of a tile's work: the rounds over the CTA pairs
// times (K blocks of a run + the fill of the pipeline and the epilogue, about
// 8 of them), and the partial sums written and read back, one K block being
// about 0.28 us, in which the GPU moves about 1.9 MB.
int choose_slices(int64_t M, int64_t N, int64_t K, int pairs) {
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  const int64_t kb = ((K + 63) / 64) * pairs;
  const int64_t units = num_sms() > 1 ? num_sms() / 2 : 1;
  int best = 1;
  double best_cost = 0;
  for (int s = 1; s <= 64 && s <= (K + 63) / 64; ++s) {
    const double rounds = double((tiles * s + units - 1) / units);
    double cost = rounds * (double(kb) / s + 8);
    if (s > 1) cost += 2.0 * s * double(M) * double(N) * 4 / 1.9e6 + 12;
    if (s == 1 || cost < 0.97 * best_cost) best = s, best_cost = cost;
  }
  return best;
}

bool operand_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch) {
  return make_operand_map(m, base, rows, cols, pitch, 128);
}
// MN-major operand (a row-major [rows][cols] tensor contracted over its rows).
bool mn_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch, bool is_b, int* major) {
  *major |= is_b ? kMnB : kMnA;
  if (cols % (is_b ? 256 : 64) == 0 && make_operand_map_mn3d(m, base, rows, cols, pitch)) {
    *major |= is_b ? kMnB3d : kMnA3d;
    return true;
  }
  return make_operand_map(m, base, rows, cols, pitch, 64);
}

template <typename T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}

// The bf16 planes of X [T][D] and W [V][D], rows pitch_x and pitch_w apart:
// the data themselves, or copies (of W only where the products read planes of
// it).
struct Planes {
  const uint16_t *x[kXentPlanes], *w[kXentPlanes];
  int64_t pitch_x, pitch_w;
  int n;
};
cudaError_t planes_of(const void* X, const void* W, int64_t T, int64_t D, int64_t V, int is_bf16, void* ws,
                      const XentPlan& p, Planes* out, cudaStream_t s) {
  out->n = is_bf16 ? 1 : kXentPlanes;
  out->pitch_x = p.pitch_x;
  out->pitch_w = p.pitch_w;
  const PlaneCopy x{X, p.copy_x ? T : 0, D / 8, p.pitch_x / 8, T * p.pitch_x / 8, at<uint16_t>(ws, p.planes_x)};
  const PlaneCopy w{W, p.copy_w ? V : 0, D / 8, p.pitch_w / 8, V * p.pitch_w / 8, at<uint16_t>(ws, p.planes_w)};
  if (p.copy_x || p.copy_w)
    XENT_STEP("xent_planes", s,
              launch_pdl(is_bf16 ? xent_planes_kernel<false> : xent_planes_kernel<true>,
                         dim3(grid_for((x.rows + w.rows) * x.d8)), dim3(256), 0, s, x, w));
  for (int i = 0; i < out->n; ++i) {
    out->x[i] = p.copy_x ? x.out + i * T * p.pitch_x : static_cast<const uint16_t*>(X);
    out->w[i] = p.copy_w ? w.out + i * V * p.pitch_w : static_cast<const uint16_t*>(W);
  }
  return cudaSuccess;
}

cudaError_t run_join(const float2* stats, int parts, int64_t T, const int64_t* targets, int64_t V, const float* zt,
                            float* loss, float* lse, int rest, int* status, cudaStream_t s) {
  const bool few = T < 2048;
  const dim3 grid(static_cast<unsigned>(few ? (T + 3) / 4 : (T + 31) / 32));
  XENT_STEP("xent_join", s,
            launch_pdl(few ? xent_join_kernel<4> : xent_join_kernel<32>, grid, dim3(32 * kJoinWarps), 0, s, stats, parts, T,
                       targets, V, zt, loss, lse, rest, status));
  return cudaSuccess;
}

cudaError_t run_reduce(const float* part, int slices, int64_t stride, int64_t n, const float* dmax, int is_bf16,
                              void* out, cudaStream_t s) {
  const float4* p4 = reinterpret_cast<const float4*>(part);
  const int64_t n4 = n / 4, stride4 = stride / 4;
  const bool shared = slices >= 8 && n4 < int64_t(num_sms()) * 1024;
  const dim3 grid(grid_for(shared ? 8 * n4 : n4));
  auto go = [&](auto kern, auto* o) { return launch_pdl(kern, grid, dim3(256), 0, s, p4, slices, stride4, n4, dmax, o); };
  XENT_STEP("xent_reduce", s,
            is_bf16 ? go(shared ? xent_reduce_kernel<__nv_bfloat16, 8> : xent_reduce_kernel<__nv_bfloat16, 1>,
                         static_cast<__nv_bfloat16*>(out))
                    : go(shared ? xent_reduce_kernel<float, 8> : xent_reduce_kernel<float, 1>, static_cast<float*>(out)));
  return cudaSuccess;
}

template <typename E>
cudaError_t run_outer(const uint16_t* dz, int planes, int64_t plane, int64_t pitch, const void* X, int64_t T, int64_t D,
                      int64_t n, const float* dmax, void* out, cudaStream_t s) {
  const int64_t threads = D / (16 / static_cast<int>(sizeof(E)));
  const int across = threads >= 256 ? 256 : static_cast<int>(ceil_to(threads, 32));
  const int64_t slabs = (threads + across - 1) / across, most = int64_t(num_sms()) * 16 / slabs + 1;
  int64_t blocks = (n + kOuterRows - 1) / kOuterRows;
  if (blocks > most) blocks = most;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(slabs)), block(across, 256 / across);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, block, 0, s, reinterpret_cast<const __nv_bfloat16*>(dz), planes, plane, pitch,
                      static_cast<const E*>(X), static_cast<int>(T), D, n, dmax, static_cast<E*>(out));
  };
  if constexpr (sizeof(E) == 4)
    if (T > 2) return T <= 4 ? go(xent_outer_kernel<E, 4>) : go(xent_outer_kernel<E, 8>);
  return T == 1 ? go(xent_outer_kernel<E, 1>) : go(xent_outer_kernel<E, 2>);
}

// The operands of the logits of ids [0, n) of W for the group of rows from t0.
bool thin_maps(XentThin* h, const void* W, const Planes& pl, int64_t t0, int64_t T, int64_t n, int64_t D) {
  const int64_t rows = T - t0 < kXentThinMax ? T - t0 : kXentThinMax;
  h->f32 = pl.n > 1;
  h->T = static_cast<int>(rows);
  h->M = static_cast<int>(n);
  h->K = static_cast<int>(D);
  h->slices = 1;
  for (int i = 0; i < pl.n; ++i)
    if (!make_operand_map(&h->map_b[i], pl.x[i] + t0 * pl.pitch_x, rows, D, pl.pitch_x, xent_thin_columns(rows))) return false;
  return h->f32 ? make_output_map_f32(&h->map_w, const_cast<void*>(W), n, D, D) : make_operand_map(&h->map_w, W, n, D, D, 128);
}

// out [M][N] = dmax * acc (is_bf16: rounded once), through fp32 partial sums
// where the K of g is cut.
cudaError_t product_out(XentGemm& g, void* out, float* part, int is_bf16, uint64_t wait_ns, cudaStream_t s,
                        const char* phase) {
  const int slices = xent_slices(g.K, g.slices);
  if (slices == 1) {
    if (!(is_bf16 ? make_output_map_bf16(&g.map_out[0], out, g.M, g.N, g.N)
                  : make_output_map_f32(&g.map_out[0], out, g.M, g.N, g.N)))
      return cudaErrorInvalidValue;
    g.epi = is_bf16 ? kXentOutBf16 : kXentOutF32;
    g.slices = 1;
    XENT_STEP(phase, s, launch_xent_gemm(g, wait_ns, s));
    return cudaSuccess;
  }
  const int64_t rows = slice_rows(g.M);
  if (!make_output_map_f32(&g.map_out[0], part, rows * slices, g.N, g.N)) return cudaErrorInvalidValue;
  const float* dmax = g.dmax;
  g.dmax = nullptr;
  g.epi = kXentOutF32;
  g.slice_rows = rows;
  XENT_STEP(phase, s, launch_xent_gemm(g, wait_ns, s));
  return run_reduce(part, slices, rows * g.N, int64_t(g.M) * g.N, dmax, is_bf16, out, s);
}

}  // namespace

// Columns of a piece of the vocabulary. A piece's dz takes at most 512 MB (all
// planes together), but a piece has at least 8192 columns: each piece adds its
// share of dX in fp32, 16 T D bytes of traffic against 4 T D 8192 operations.
// Among the pieces from half of that to all of it the one whose dW products,
// all pieces together, take the fewest rounds over the CTA pairs (T = 8000, D =
// 512, V = 100000: 33536 columns make 12, 29184 make 11 of at least 10.3).
int64_t choose_piece(int64_t T, int64_t D, int64_t V, int planes) {
  int64_t most = (int64_t(1) << 28) / (T * planes) / 256;
  if (most < 32) most = 32;
  const int64_t blocks = (V + 255) / 256, across = (D + 255) / 256, pairs = num_sms() > 1 ? num_sms() / 2 : 1;
  if (most >= blocks) return V;
  int64_t best = most, best_rounds = 0;
  for (int64_t b = most; b >= 32 && b >= most / 2; --b) {
    const int64_t full = blocks / b, rest = blocks - full * b;
    const int64_t rounds = full * ((b * across + pairs - 1) / pairs) + (rest * across + pairs - 1) / pairs;
    if (best_rounds == 0 || rounds < best_rounds) best = b, best_rounds = rounds;
  }
  return best * 256;
}

// Whether the products with W go by groups of kXentThinMax rows, each a pass
// over W. bf16: one group (64 rows, V = 128000, D = 1024: the logits 54 us
// either way, 32 rows 50 against 59). fp32, where the other form splits W into
// planes in memory first: up to three groups of a W that is more than a few
// launches' worth (V = 128000, D = 1024, a whole step: 64 rows 0.47 against
// 1.46 ms, 128 rows 0.86 / 1.46, 192 rows 1.23 / 1.6, 256 rows 1.61 / 1.64; V =
// 3000, D = 256, 128 rows: 150 us against 126).
static bool use_thin(int64_t T, int64_t D, int64_t V, int is_bf16) {
  static_assert(3 * kXentThinMax <= kXentDmaxRows, "the few-row kernel of dz finds the largest |dloss| itself");
  return T <= kXentThinMax || (!is_bf16 && T <= 3 * kXentThinMax && V * D >= (int64_t(1) << 24));
}

// Whether the products read a copy of bf16 X, on rows of whole 128-byte lines:
// rows that begin off the 32-byte sectors of the L2 slow TMA's loads. A copy
// costs a launch and T D, it saves a part of T V D (V = 30011, D = 1032, loss
// and gradients: T = 200 100 -> 98.5 us, 1000 245 -> 238, 8000 1.46 -> 1.40 ms;
// V = 3001, T = 1000 57 -> 59 us, 8000 192 -> 198). A copy of W saves less than
// it costs up to T = 8000.
static bool copies_x(int64_t T, int64_t D, int64_t V, int thin) {
  return !thin && D % 16 != 0 && V >= 8192 && T * V >= (int64_t(1) << 32) / D;
}

XentPlan plan_xent(int64_t T, int64_t D, int64_t V, int is_bf16, int backward) {
  XentPlan p{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t a = off;
    off = up256(off + bytes);
    return a;
  };
  const int planes = is_bf16 ? 1 : kXentPlanes, pairs = is_bf16 ? 1 : kXentPairs;
  p.thin = use_thin(T, D, V, is_bf16);
  p.copy_x = !is_bf16 || copies_x(T, D, V, p.thin);
  p.copy_w = !p.thin && !is_bf16;
  p.pitch_x = p.copy_x ? ceil_to(D, 64) : D;
  p.pitch_w = p.copy_w ? ceil_to(D, 64) : D;
  if (p.copy_x) p.planes_x = take(size_t(T) * p.pitch_x * 2 * planes);
  if (p.copy_w) p.planes_w = take(size_t(V) * p.pitch_w * 2 * planes);
  if (!backward) {
    const int64_t parts = p.thin ? xent_thin_parts(V) : (V + kXentPart - 1) / kXentPart;
    p.stats = take(size_t(parts) * T * sizeof(float2));
    p.zt = take(size_t(T) * 4);
    p.total = off;
    return p;
  }
  p.dz_planes = is_bf16 && p.thin ? kThinDzPlanes : planes;
  p.piece = choose_piece(T, D, V, p.dz_planes);
  const int64_t piece = p.piece;
  p.dz_pitch = ceil_to(piece, 64);
  p.dmax = take(kXentDmaxParts * 4);
  p.dz = take(size_t(T) * p.dz_pitch * 2 * p.dz_planes);
  p.slices_x = p.thin ? xent_thin_slices(D, p.dz_pitch)
                      : xent_slices(static_cast<int>(p.dz_pitch), choose_slices(T, D, p.dz_pitch, pairs));
  p.slices_w = xent_slices(static_cast<int>(T), choose_slices(piece, D, T, is_bf16 ? p.dz_planes : pairs));
  p.dx_part = piece < V || p.slices_x > 1 || p.thin;
  if (p.dx_part) p.dx = take(size_t(p.slices_x) * (p.thin ? T : slice_rows(T)) * D * 4);
  if (p.slices_w > 1) p.dw = take(size_t(p.slices_w) * slice_rows(piece) * D * 4);
  p.total = off;
  return p;
}

cudaError_t run_xent_forward(const void* X, const void* W, const int64_t* targets, int64_t T, int64_t D, int64_t V,
                             int is_bf16, float* loss, float* lse, void* ws, int* status, uint64_t wait_ns,
                             cudaStream_t s, int inject) {
  const XentPlan p = plan_xent(T, D, V, is_bf16, 0);
  Planes pl;
  cudaError_t e = planes_of(X, W, T, D, V, is_bf16, ws, p, &pl, s);
  if (e != cudaSuccess) return e;
  if (p.thin) {
    float2* stats = at<float2>(ws, p.stats);
    float* zt = at<float>(ws, p.zt);
    for (int64_t t0 = 0; t0 < T; t0 += kXentThinMax) {
      XentThin h{};
      if (!thin_maps(&h, W, pl, t0, T, V, D)) return cudaErrorInvalidValue;
      h.targets = targets + t0;
      h.V = V;
      h.stats = stats + t0 * xent_thin_parts(V);
      h.zt = zt + t0;
      h.zt_rest = loss + t0;
      h.inject = inject;
      XENT_STEP("xent_logits", s, launch_xent_thin_stats(h, wait_ns, s));
      if (inject > 0) return cudaSuccess;
      if ((e = run_join(h.stats, xent_thin_parts(V), h.T, h.targets, V, h.zt, loss + t0, lse + t0, is_bf16 && xent_thin_columns(h.T) == 32,
                        status, s)) != cudaSuccess)
        return e;
    }
    return cudaSuccess;
  }
  XentGemm g{};
  for (int i = 0; i < pl.n; ++i)
    if (!operand_map(&g.map_a[i], pl.x[i], T, D, pl.pitch_x) || !operand_map(&g.map_b[i], pl.w[i], V, D, pl.pitch_w))
      return cudaErrorInvalidValue;
  g.pairs = pl.n == 1 ? 1 : kXentPairs;
  g.M = static_cast<int>(T);
  g.N = static_cast<int>(V);
  g.K = static_cast<int>(D);
  g.slices = 1;
  g.group_m = 16;
  g.epi = kXentStats;
  g.targets = targets;
  g.V = V;
  g.stats = at<float2>(ws, p.stats);
  g.zt = at<float>(ws, p.zt);
  g.inject = inject;
  XENT_STEP("xent_logits", s, launch_xent_gemm(g, wait_ns, s));
  if (inject > 0) return cudaSuccess;
  const int parts = static_cast<int>((V + kXentPart - 1) / kXentPart);
  return run_join(g.stats, parts, T, targets, V, g.zt, loss, lse, 0, status, s);
}

cudaError_t run_xent_backward(const void* X, const void* W, const int64_t* targets, const float* loss, const float* lse,
                              const float* dloss, int64_t T, int64_t D, int64_t V, int is_bf16, void* dX, void* dW,
                              void* ws, uint64_t wait_ns, cudaStream_t s) {
  const XentPlan p = plan_xent(T, D, V, is_bf16, 1);
  Planes pl;
  cudaError_t e = planes_of(X, W, T, D, V, is_bf16, ws, p, &pl, s);
  if (e != cudaSuccess) return e;
  const int pairs = pl.n == 1 ? 1 : kXentPairs;
  const size_t es = is_bf16 ? 2 : 4;
  float* dmax = at<float>(ws, p.dmax);
  XentDmax rows{dloss, targets, static_cast<int>(T), dmax};
  if (T > kXentDmaxRows) {
    XENT_STEP("xent_dmax", s, launch_pdl(xent_dmax_kernel, dim3(kXentDmaxParts), dim3(256), 0, s, dloss, targets, T, V, dmax));
    rows.rows = 0;
  }
  uint16_t* dz[kXentPlanes];
  for (int i = 0; i < p.dz_planes; ++i) dz[i] = at<uint16_t>(ws, p.dz) + i * T * p.dz_pitch;
  for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
    const int64_t vc = V - v0 < p.piece ? V - v0 : p.piece, vp = ceil_to(vc, 64);
    const void* W0 = static_cast<const char*>(W) + v0 * D * es;
    // dz of the piece, from its logits computed again; columns vc .. vp are zeros.
    XentGemm g{};
    for (int64_t t0 = 0; p.thin && t0 < T; t0 += kXentThinMax) {
      XentThin h{};
      if (!thin_maps(&h, W0, pl, t0, T, vc, D)) return cudaErrorInvalidValue;
      h.targets = targets + t0;
      h.V = V;
      h.col0 = v0;
      h.lse = lse + t0;
      h.loss = loss ? loss + t0 : nullptr;
      h.dloss = dloss + t0;
      h.rows = rows;
      h.dz = reinterpret_cast<__nv_bfloat16*>(dz[0]) + t0 * p.dz_pitch;
      h.plane = T * p.dz_pitch;
      h.pitch = p.dz_pitch;
      h.dz_columns = vp;
      XENT_STEP("xent_dz", s, launch_xent_thin_dz(h, wait_ns, s));
    }
    for (int i = 0; !p.thin && i < pl.n; ++i)
      if (!operand_map(&g.map_a[i], pl.x[i], T, D, pl.pitch_x) ||
          !operand_map(&g.map_b[i], pl.w[i] + v0 * pl.pitch_w, vc, D, pl.pitch_w) ||
          !make_output_map_bf16(&g.map_out[i], dz[i], T, vp, p.dz_pitch))
        return cudaErrorInvalidValue;
    g.pairs = pairs;
    g.M = static_cast<int>(T);
    g.N = static_cast<int>(vc);
    g.K = static_cast<int>(D);
    g.slices = 1;
    g.group_m = 16;
    g.epi = is_bf16 ? kXentGrad : kXentGradF32;
    g.targets = targets;
    g.V = V;
    g.col0 = v0;
    g.lse = lse;
    g.loss = loss;
    g.dloss = dloss;
    g.dmax = dmax;
    g.rows = rows;
    if (!p.thin) XENT_STEP("xent_dz", s, launch_xent_gemm(g, wait_ns, s));

    // dW of the piece = dz^T X.
    if (T <= outer_max(is_bf16)) {
      void* out = static_cast<char*>(dW) + v0 * D * es;
      XENT_STEP("xent_dW", s,
                is_bf16 ? run_outer<__nv_bfloat16>(dz[0], p.dz_planes, T * p.dz_pitch, p.dz_pitch, X, T, D, vc, dmax, out, s)
                        : run_outer<float>(dz[0], p.dz_planes, T * p.dz_pitch, p.dz_pitch, X, T, D, vc, dmax, out, s));
    } else {
      g = XentGemm{};
      for (int i = 0; i < p.dz_planes; ++i)
        if (!mn_map(&g.map_a[i], dz[i], T, vp, p.dz_pitch, false, &g.mn_major)) return cudaErrorInvalidValue;
      for (int i = 0; i < pl.n; ++i)
        if (!mn_map(&g.map_b[i], pl.x[i], T, D, pl.pitch_x, true, &g.mn_major)) return cudaErrorInvalidValue;
      g.pairs = is_bf16 ? p.dz_planes : pairs;
      g.M = static_cast<int>(vc);
      g.N = static_cast<int>(D);
      g.K = static_cast<int>(T);
      g.slices = p.slices_w;
      g.group_m = 16;
      g.dmax = dmax;
      if ((e = product_out(g, static_cast<char*>(dW) + v0 * D * es, at<float>(ws, p.dw), is_bf16, wait_ns, s, "xent_dW")) !=
          cudaSuccess)
        return e;
    }

    // dX += dz W over the piece.
    if (p.thin) {
      const bool f32 = pl.n > 1;
      for (int64_t t0 = 0; t0 < T; t0 += kXentThinMax) {
        XentThin h{};
        h.f32 = f32;
        h.T = static_cast<int>(T - t0 < kXentThinMax ? T - t0 : kXentThinMax);
        h.M = static_cast<int>(D);
        h.K = static_cast<int>(vp);
        h.slices = p.slices_x;
        h.part = at<float>(ws, p.dx) + t0 * D;
        h.part_rows = T;
        h.add = v0 > 0;
        if (!(f32 ? make_output_map_f32(&h.map_w, const_cast<void*>(W0), vc, D, D)
                  : make_operand_map(&h.map_w, W0, vc, D, D, 64)))
          return cudaErrorInvalidValue;
        for (int i = 0; i < p.dz_planes; ++i)
          if (!make_operand_map(&h.map_b[i], dz[i] + t0 * p.dz_pitch, h.T, vp, p.dz_pitch, xent_thin_columns(h.T)))
            return cudaErrorInvalidValue;
        XENT_STEP("xent_dX", s, launch_xent_thin_dx(h, wait_ns, s));
      }
      if (v0 + vc < V) continue;
      if ((e = run_reduce(at<float>(ws, p.dx), p.slices_x, T * D, T * D, dmax, is_bf16, dX, s)) != cudaSuccess) return e;
      continue;
    }
    g = XentGemm{};
    for (int i = 0; i < pl.n; ++i)
      if (!operand_map(&g.map_a[i], dz[i], T, vp, p.dz_pitch) ||
          !mn_map(&g.map_b[i], pl.w[i] + v0 * pl.pitch_w, vc, D, pl.pitch_w, true, &g.mn_major))
        return cudaErrorInvalidValue;
    g.pairs = pairs;
    g.M = static_cast<int>(T);
    g.N = static_cast<int>(D);
    g.K = static_cast<int>(vp);
    g.group_m = 8;
    g.dmax = dmax;
    if (p.piece == V) {
      g.slices = p.slices_x;
      if ((e = product_out(g, dX, at<float>(ws, p.dx), is_bf16, wait_ns, s, "xent_dX")) != cudaSuccess) return e;
      continue;
    }
    // Several pieces: the first one's slices are stored, the later ones' added.
    const int64_t rows = slice_rows(T);
    const int slices = xent_slices(static_cast<int>(vp), p.slices_x);
    if (!make_output_map_f32(&g.map_out[0], at<float>(ws, p.dx), rows * p.slices_x, D, D)) return cudaErrorInvalidValue;
    g.slices = slices;
    g.dmax = nullptr;
    g.epi = kXentOutF32;
    g.add = v0 > 0;
    g.slice_rows = rows;
    XENT_STEP("xent_dX", s, launch_xent_gemm(g, wait_ns, s));
    if (v0 + vc < V) continue;
    if ((e = run_reduce(at<float>(ws, p.dx), p.slices_x, rows * D, T * D, dmax, is_bf16, dX, s)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tpmlp
