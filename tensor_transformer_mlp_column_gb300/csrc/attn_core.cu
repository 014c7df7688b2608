// attn_core.cu — attention on given queries, keys and values, and its backward
// pass: the row sums delta = dO . O, and the kernels on the CUDA cores.
//
//   s_ij = scale q_i . k_j (keys j of i's sequence; causal: j <= i)
//   lse_i = log sum_j exp(s_ij),  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   ds_ij = p_ij (do_i . v_j - delta_i),  delta_i = do_i . o_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// The scores are never stored: the forward keeps a running maximum and sum for
// each row, the backward makes the probabilities again from lse. dK and dV
// come from one kernel (a CTA per 64 keys of a kv head, walking over the
// queries of every head that shares them) and dQ from another (a CTA per 64
// queries), so every sum has one owner and a fixed order, without atomics.
//
// A CTA holds 64 x 64 scores, 4 x 4 for each of its 256 threads, and the 64 x
// dim tiles in shared memory, rows 4 words longer than dim so that 8 rows read
// 16 bytes each without a bank conflict. Rows behind a sequence's end are read
// as zero, whatever they hold.
#include "device.cuh"
#include "internal.h"

#include "attn_core.h"
#include "trace.h"

namespace tpmlp {

namespace {

constexpr int kTile = 64;
constexpr int kThreads = 256;
constexpr int kPitchP = kTile + 4;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

__device__ __forceinline__ float at(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ float* row_of(const HeadsView& v, int64_t row, int head) {
  return static_cast<float*>(v.p) + row * v.token + head * v.head;
}

// Rows first .. first + 63 of a sequence's tile, zero from row `len` on and from column `dim` on.
template <int DH>
__device__ __forceinline__ void load_tile(float* dst, const HeadsView& v, int64_t row0, int first, int len, int head,
                                          int dim) {
  for (int i = threadIdx.x; i < kTile * (DH / 4); i += kThreads) {
    const int r = i / (DH / 4), c = i % (DH / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (first + r < len && c < dim) x = load4(row_of(v, row0 + first + r, head) + c);
    *reinterpret_cast<float4*>(dst + r * (DH + 4) + c) = x;
  }
}

// acc[i][j] = a[4 ty + i] . b[tx + 16 j] over DH.
template <int DH>
__device__ __forceinline__ void dot_tiles(float (&acc)[4][4], const float* a, const float* b, int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 2
  for (int c = 0; c < DH; c += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * (DH + 4) + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * (DH + 4) + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, acc[i][j]))));
  }
}

// acc[i][:] += sum over k of m[4 ty + i][k] t[k][4 tx + 64 u ..]: rows of a 64 x 64 matrix times a tile.
template <int DH>
__device__ __forceinline__ void add_rows(float4 (&acc)[4][DH / 64], const float* m, const float* t, int ty, int tx) {
#pragma unroll 2
  for (int k = 0; k < kTile; k += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(m + (4 * ty + i) * kPitchP + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int u = 0; u < DH / 64; ++u) {
        const float4 x = *reinterpret_cast<const float4*>(t + (k + kk) * (DH + 4) + 4 * tx + 64 * u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = at(w[i], kk);
          acc[i][u].x = fmaf(c, x.x, acc[i][u].x);
          acc[i][u].y = fmaf(c, x.y, acc[i][u].y);
          acc[i][u].z = fmaf(c, x.z, acc[i][u].z);
          acc[i][u].w = fmaf(c, x.w, acc[i][u].w);
        }
      }
  }
}

// The same with the matrix's columns: acc[i][:] += sum over k of m[k][4 ty + i] t[k][..].
template <int DH>
__device__ __forceinline__ void add_columns(float4 (&acc)[4][DH / 64], const float* m, const float* t, int ty, int tx) {
#pragma unroll 4
  for (int k = 0; k < kTile; ++k) {
    const float4 w = *reinterpret_cast<const float4*>(m + k * kPitchP + 4 * ty);
#pragma unroll
    for (int u = 0; u < DH / 64; ++u) {
      const float4 x = *reinterpret_cast<const float4*>(t + k * (DH + 4) + 4 * tx + 64 * u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = at(w, i);
        acc[i][u].x = fmaf(c, x.x, acc[i][u].x);
        acc[i][u].y = fmaf(c, x.y, acc[i][u].y);
        acc[i][u].z = fmaf(c, x.z, acc[i][u].z);
        acc[i][u].w = fmaf(c, x.w, acc[i][u].w);
      }
    }
  }
}

template <int DH>
__device__ __forceinline__ void clear(float4 (&acc)[4][DH / 64]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < DH / 64; ++u) acc[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// Rows 4 ty .. of the accumulators, times a factor for each.
template <int DH>
__device__ __forceinline__ void store_rows(const HeadsView& v, int64_t row0, int first, int len, int head, int dim,
                                           const float4 (&acc)[4][DH / 64], const float (&f)[4], int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (first + 4 * ty + i >= len) continue;
    float* dst = row_of(v, row0 + first + 4 * ty + i, head);
#pragma unroll
    for (int u = 0; u < DH / 64; ++u)
      if (4 * tx + 64 * u < dim)
        store4(dst + 4 * tx + 64 * u,
               make_float4(acc[i][u].x * f[i], acc[i][u].y * f[i], acc[i][u].z * f[i], acc[i][u].w * f[i]));
  }
}

__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int DH>
constexpr size_t tile_bytes() {
  return sizeof(float) * kTile * (DH + 4);
}
constexpr size_t kMatrixBytes = sizeof(float) * kTile * kPitchP;

// Item i of a launch: tile, head and sequence. Causal: the tiles with the most
// work (`last_first`: the last ones) come first.
__device__ __forceinline__ void item_of(int64_t i, int tiles, int heads, bool last_first, int& tile, int& head, int& b) {
  const int64_t per = int64_t(heads) * (gridDim.x / (int64_t(tiles) * heads));  // items of one tile index
  tile = static_cast<int>(i / per);
  if (last_first) tile = tiles - 1 - tile;
  head = static_cast<int>(i % per % heads);
  b = static_cast<int>(i % per / heads);
}

template <int DH>
__global__ void __launch_bounds__(kThreads) core_forward_kernel(const __grid_constant__ CoreForward c) {
  extern __shared__ __align__(16) float smem[];
  float* sq = smem;
  float* sk = sq + kTile * (DH + 4);
  float* sv = sk + kTile * (DH + 4);
  float* sp = sv + kTile * (DH + 4);
  pdl_wait();
  pdl_launch_dependents();
  int tile, h, b;
  item_of(blockIdx.x, (c.s.max_seq + kTile - 1) / kTile, c.s.heads, c.s.causal, tile, h, b);
  int64_t row0;
  const int len = core_sequence(c.s, b, row0, c.status);
  const int q0 = tile * kTile;
  if (q0 >= len) return;
  const int kv = h / (c.s.heads / c.s.kv_heads);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_tile<DH>(sq, c.q, row0, q0, len, h, c.s.dim);
  float m[4], l[4];
  float4 acc[4][DH / 64];
  clear<DH>(acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
  const int k_end = c.s.causal ? min(len, q0 + kTile) : len;
  for (int k0 = 0; k0 < k_end; k0 += kTile) {
    __syncthreads();
    load_tile<DH>(sk, c.k, row0, k0, len, kv, c.s.dim);
    load_tile<DH>(sv, c.v, row0, k0, len, kv, c.s.dim);
    __syncthreads();
    float s[4][4];
    dot_tiles<DH>(s, sq, sk, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int qi = q0 + 4 * ty + i;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kj = k0 + tx + 16 * j;
        s[i][j] = kj < len && (!c.s.causal || kj <= qi) ? s[i][j] * c.s.scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      const float m_new = fmaxf(m[i], max16(mx));
      const float base = m_new == -INFINITY ? 0.f : m_new;  // no score above -inf yet: weights of zero, not NaN
      const float alpha = expf(m[i] - base);
      m[i] = m_new;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = expf(s[i][j] - base);
        sum += p;
        sp[(4 * ty + i) * kPitchP + tx + 16 * j] = p;
      }
      l[i] = l[i] * alpha + sum16(sum);
#pragma unroll
      for (int u = 0; u < DH / 64; ++u) {
        acc[i][u].x *= alpha;
        acc[i][u].y *= alpha;
        acc[i][u].z *= alpha;
        acc[i][u].w *= alpha;
      }
    }
    __syncwarp();  // a warp's rows of P are read by the same warp
    add_rows<DH>(acc, sp, sv, ty, tx);
  }
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = 1.0f / l[i];
    const int qi = q0 + 4 * ty + i;
    if (tx == 0 && qi < len) c.lse[int64_t(h) * c.s.T + row0 + qi] = m[i] + logf(l[i]);
  }
  store_rows<DH>(c.o, row0, q0, len, h, c.s.dim, acc, f, ty, tx);
}

// delta[h][t] = sum over the head of dO * O: eight lanes a row of a head.
__global__ void __launch_bounds__(256) core_delta_kernel(HeadsView o, HeadsView d_o, int64_t T_, int heads, int dim,
                                                         float* delta) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) / 8;  // head fastest: neighbours in memory
  if (i >= T_ * heads) return;  // all eight lanes of a row at once, and the shuffles name only them
  const int lane = threadIdx.x & 7, h = static_cast<int>(i % heads);
  const int64_t t = i / heads;
  const float* a = row_of(o, t, h);
  const float* b = row_of(d_o, t, h);
  float sum = 0.f;
  for (int c = 4 * lane; c < dim; c += 32) {
    const float4 x = load4(a + c), y = load4(b + c);
    sum = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, sum))));
  }
  const uint32_t mask = 0xffu << (threadIdx.x & 24);
#pragma unroll
  for (int x = 4; x > 0; x >>= 1) sum += __shfl_xor_sync(mask, sum, x);
  if (lane == 0) delta[int64_t(h) * T_ + t] = sum;
}

// p and ds of one 64 x 64 tile (rows: queries). Both are zero wherever a query
// or a key does not count.
__device__ __forceinline__ void probabilities(const CoreShape& c, float (&s)[4][4], const float (&dp)[4][4],
                                              const float (&lse)[4], const float (&delta)[4], int q0, int k0, int len,
                                              int ty, int tx, float (&ds)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int qi = q0 + 4 * ty + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kj = k0 + tx + 16 * j;
      const bool on = qi < len && kj < len && (!c.causal || kj <= qi);
      const float p = on ? expf(fmaf(s[i][j], c.scale, -lse[i])) : 0.f;
      ds[i][j] = on ? p * (dp[i][j] - delta[i]) : 0.f;
      s[i][j] = p;
    }
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads) core_dkv_kernel(const __grid_constant__ CoreBackward c, const float* delta) {
  extern __shared__ __align__(16) float smem[];
  float* sk = smem;
  float* sv = sk + kTile * (DH + 4);
  float* sq = sv + kTile * (DH + 4);
  float* sd = sq + kTile * (DH + 4);
  float* sp = sd + kTile * (DH + 4);
  float* ss = sp + kTile * kPitchP;
  pdl_wait();
  pdl_launch_dependents();
  int tile, kv, b;
  item_of(blockIdx.x, (c.s.max_seq + kTile - 1) / kTile, c.s.kv_heads, false, tile, kv, b);
  int64_t row0;
  const int len = core_sequence(c.s, b, row0, c.status);
  const int k0 = tile * kTile;
  if (k0 >= len) return;
  const int group = c.s.heads / c.s.kv_heads;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_tile<DH>(sk, c.k, row0, k0, len, kv, c.s.dim);
  load_tile<DH>(sv, c.v, row0, k0, len, kv, c.s.dim);
  float4 dk[4][DH / 64], dv[4][DH / 64];
  clear<DH>(dk);
  clear<DH>(dv);
  for (int h = kv * group; h < (kv + 1) * group; ++h) {
    for (int q0 = c.s.causal ? k0 : 0; q0 < len; q0 += kTile) {
      __syncthreads();
      load_tile<DH>(sq, c.q, row0, q0, len, h, c.s.dim);
      load_tile<DH>(sd, c.d_o, row0, q0, len, h, c.s.dim);
      float lse[4], del[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = int64_t(h) * c.s.T + row0 + min(q0 + 4 * ty + i, len - 1);
        lse[i] = c.lse[at];
        del[i] = delta[at];
      }
      __syncthreads();
      float s[4][4], dp[4][4], ds[4][4];
      dot_tiles<DH>(s, sq, sk, ty, tx);
      dot_tiles<DH>(dp, sd, sv, ty, tx);
      probabilities(c.s, s, dp, lse, del, q0, k0, len, ty, tx, ds);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sp[(4 * ty + i) * kPitchP + tx + 16 * j] = s[i][j];
          ss[(4 * ty + i) * kPitchP + tx + 16 * j] = ds[i][j];
        }
      __syncthreads();
      add_columns<DH>(dv, sp, sd, ty, tx);
      add_columns<DH>(dk, ss, sq, ty, tx);
    }
  }
  const float one[4] = {1.f, 1.f, 1.f, 1.f}, sc[4] = {c.s.scale, c.s.scale, c.s.scale, c.s.scale};
  store_rows<DH>(c.dv, row0, k0, len, kv, c.s.dim, dv, one, ty, tx);
  store_rows<DH>(c.dk, row0, k0, len, kv, c.s.dim, dk, sc, ty, tx);
}

template <int DH>
__global__ void __launch_bounds__(kThreads) core_dq_kernel(const __grid_constant__ CoreBackward c, const float* delta) {
  extern __shared__ __align__(16) float smem[];
  float* sq = smem;
  float* sd = sq + kTile * (DH + 4);
  float* sk = sd + kTile * (DH + 4);
  float* sv = sk + kTile * (DH + 4);
  float* ss = sv + kTile * (DH + 4);
  pdl_wait();
  pdl_launch_dependents();
  int tile, h, b;
  item_of(blockIdx.x, (c.s.max_seq + kTile - 1) / kTile, c.s.heads, c.s.causal, tile, h, b);
  int64_t row0;
  const int len = core_sequence(c.s, b, row0, c.status);
  const int q0 = tile * kTile;
  if (q0 >= len) return;
  const int kv = h / (c.s.heads / c.s.kv_heads);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_tile<DH>(sq, c.q, row0, q0, len, h, c.s.dim);
  load_tile<DH>(sd, c.d_o, row0, q0, len, h, c.s.dim);
  float lse[4], del[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = int64_t(h) * c.s.T + row0 + min(q0 + 4 * ty + i, len - 1);
    lse[i] = c.lse[at];
    del[i] = delta[at];
  }
  float4 dq[4][DH / 64];
  clear<DH>(dq);
  const int k_end = c.s.causal ? min(len, q0 + kTile) : len;
  for (int k0 = 0; k0 < k_end; k0 += kTile) {
    __syncthreads();
    load_tile<DH>(sk, c.k, row0, k0, len, kv, c.s.dim);
    load_tile<DH>(sv, c.v, row0, k0, len, kv, c.s.dim);
    __syncthreads();
    float s[4][4], dp[4][4], ds[4][4];
    dot_tiles<DH>(s, sq, sk, ty, tx);
    dot_tiles<DH>(dp, sd, sv, ty, tx);
    probabilities(c.s, s, dp, lse, del, q0, k0, len, ty, tx, ds);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) ss[(4 * ty + i) * kPitchP + tx + 16 * j] = ds[i][j];
    __syncwarp();  // a warp's rows of dS are read by the same warp
    add_rows<DH>(dq, ss, sk, ty, tx);
  }
  const float sc[4] = {c.s.scale, c.s.scale, c.s.scale, c.s.scale};
  store_rows<DH>(c.dq, row0, q0, len, h, c.s.dim, dq, sc, ty, tx);
}

template <auto Kernel, typename... Args>
cudaError_t launch(int64_t items, size_t smem, cudaStream_t s, Args... args) {
  static std::atomic<uint64_t> devices{0};
  cudaError_t e = allow_smem(Kernel, smem, devices);
  if (e != cudaSuccess) return e;
  return launch_pdl(Kernel, dim3(static_cast<unsigned>(items)), dim3(kThreads), smem, s, args...);
}

template <int DH>
cudaError_t simt_forward(const CoreForward& c, cudaStream_t s) {
  const int64_t tiles = (c.s.max_seq + kTile - 1) / kTile;
  return launch<core_forward_kernel<DH>>(tiles * c.s.heads * c.s.batch, 3 * tile_bytes<DH>() + kMatrixBytes, s, c);
}

template <int DH>
cudaError_t simt_backward(const CoreBackward& c, const float* delta, cudaStream_t s) {
  const int64_t tiles = (c.s.max_seq + kTile - 1) / kTile;
  {
    TraceScope trace("attn_core_dkv", s);
    cudaError_t e = launch<core_dkv_kernel<DH>>(tiles * c.s.kv_heads * c.s.batch, 4 * tile_bytes<DH>() + 2 * kMatrixBytes, s, c, delta);
    if (e != cudaSuccess) return e;
  }
  TraceScope trace("attn_core_dq", s);
  return launch<core_dq_kernel<DH>>(tiles * c.s.heads * c.s.batch, 4 * tile_bytes<DH>() + kMatrixBytes, s, c, delta);
}

}  // namespace

size_t core_backward_workspace(int64_t T, int heads) { return static_cast<size_t>(T) * heads * sizeof(float); }

cudaError_t run_core_forward(const CoreForward& c, cudaStream_t s) {
  TraceScope trace("attn_core_forward", s);
  if (c.bf16) return launch_core_forward_tc(c, s);
  return c.s.dim <= 64 ? simt_forward<64>(c, s) : simt_forward<128>(c, s);
}

cudaError_t run_core_backward(const CoreBackward& c, cudaStream_t s) {
  float* delta = static_cast<float*>(c.ws);
  if (c.bf16) return launch_core_backward_tc(c, delta, s);
  {
    TraceScope trace("attn_core_delta", s);
    const unsigned grid = static_cast<unsigned>((c.s.T * c.s.heads + 31) / 32);
    cudaError_t e = launch_pdl(core_delta_kernel, dim3(grid), dim3(256), 0, s, c.o, c.d_o, c.s.T, c.s.heads, c.s.dim, delta);
    if (e != cudaSuccess) return e;
  }
  return c.s.dim <= 64 ? simt_backward<64>(c, delta, s) : simt_backward<128>(c, delta, s);
}

}  // namespace tpmlp
