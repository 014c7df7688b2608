// attn_core.cu — attention on given queries, keys and values, and its backward
// pass: the calls, and the fp32 kernels on the CUDA cores.
//
//   s_ij = scale q_i . k_j (keys j of i's sequence; causal: j <= i)
//   lse_i = log sum_j exp(s_ij),  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   ds_ij = p_ij (do_i . v_j - delta_i),  delta_i = do_i . o_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// The scores are never stored: the forward keeps a running maximum and sum for
// each row, the backward makes the probabilities again from lse. dQ (with
// delta) comes from one kernel (a CTA per ROWS queries), dK and dV from the next (a
// CTA per ROWS keys of a kv head, walking over the queries of every head that
// shares them), so every sum has one owner and a fixed order, without atomics.
//
// A CTA holds ROWS x 64 scores, 4 x 4 for each of its 4 ROWS threads, and its
// tiles in shared memory, rows 4 words longer than the head so that 8 rows read
// 16 bytes each without a bank conflict. The tiles that it walks over come by
// cp.async, one ahead. Products go two at a time (packed fp32 pairs). Rows
// behind a sequence's end are read as zero, whatever they hold.
//
// The kernels do not let the stream's next one in early: its CTAs would wait in the
// places that this one's second round needs, unevenly (2 x 300 tokens, 8 heads of 64
// on 2, a step: 205 us so, 174 without; 4 x 384, 8 heads: 129 and 117).
//
// Bound by what shared memory returns to the registers, 16 bytes a lane eight times
// for 64 multiply-adds a lane (65 to 78 % of that path busy, 54 to 60 of the FMA pipe;
// which lanes read the same line makes no difference): 16 heads of 128, 4 x 1024 tokens, causal, 463,
// 706 (dQ) and 976 us (dK, dV), 37, 37 and 35 TFLOP/s of about 75; 16 heads of 64
// 239, 358 and 462. A key tile walks over all queries of its group by itself, so dK
// and dV take long where one kv head serves many (1024 tokens, 4 heads of 128 on 4:
// 272 us, on one: 1062; 4096 tokens, 32 on one: 33.7 ms, the bf16 kernel, which cuts
// such walks into runs, 0.2).
#include "attn_core.h"

#include <algorithm>

#include "attn_core_walk.cuh"
#include "device.cuh"
#include "internal.h"
#include "trace.h"

namespace tpmlp {

namespace {

constexpr int kWide = 64;  // rows of the tiles that a CTA walks over
constexpr int kPitchP = kWide + 4;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// Packed pairs of fp32.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float sum_of(uint64_t d) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
  return a + b;
}
__device__ __forceinline__ void unpair(uint64_t d, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ void fma_pair(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float* row_of(const HeadsView& v, int64_t row, int head) {
  return static_cast<float*>(v.p) + row * v.token + head * v.head;
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Starts the copy of rows first .. first + ROWS - 1 of a sequence, zero from row `len` on and from column `dim` on.
template <int DH, int ROWS, int THREADS>
__device__ __forceinline__ void copy_tile(float* dst, const HeadsView& v, int64_t row0, int first, int len, int head,
                                          int dim) {
#pragma unroll 4
  for (int i = threadIdx.x; i < ROWS * (DH / 4); i += THREADS) {
    const int r = i / (DH / 4), c = i % (DH / 4) * 4;
    const bool on = first + r < len && c < dim;
    const float* src = on ? row_of(v, row0 + first + r, head) + c : static_cast<const float*>(v.p);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst + r * (DH + 4) + c)), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
  }
}

// acc[i][j] = a[4 ty + i] . b[tx + TX j] over DH; even and odd elements are summed apart and added at the end.
template <int DH, int TX>
__device__ __forceinline__ void dot_tiles(float (&out)[4][4], const float* a, const float* b, int ty, int tx) {
  uint64_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;
#pragma unroll 2
  for (int c = 0; c < DH; c += 4) {
    ulonglong2 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(a + (4 * ty + i) * (DH + 4) + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2*>(b + (tx + TX * j) * (DH + 4) + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        fma_pair(acc[i][j], x[i].x, y[j].x);
        fma_pair(acc[i][j], x[i].y, y[j].y);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) out[i][j] = sum_of(acc[i][j]);
}

// Four rows of an output, columns 4 tx + 64 u ..
template <int DH>
struct Rows {
  uint64_t v[4][DH / 64][2];
};
template <int DH>
__device__ __forceinline__ void clear(Rows<DH>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < DH / 64; ++u) r.v[i][u][0] = r.v[i][u][1] = 0;
}
template <int DH>
__device__ __forceinline__ void scale_row(Rows<DH>& r, int i, float f) {
#pragma unroll
  for (int u = 0; u < DH / 64; ++u)
#pragma unroll
    for (int x = 0; x < 2; ++x) r.v[i][u][x] = mul_pair(r.v[i][u][x], pair(f, f));
}

__device__ __forceinline__ float at(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// acc row i += w[i] t[0 .. 63]'s columns: one row of the tile times a weight for each of the four rows.
template <int DH>
__device__ __forceinline__ void add_row(Rows<DH>& acc, const uint64_t (&w)[4], const float* t, int tx) {
#pragma unroll
  for (int u = 0; u < DH / 64; ++u) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(t + 4 * tx + 64 * u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fma_pair(acc.v[i][u][0], w[i], x.x);
      fma_pair(acc.v[i][u][1], w[i], x.y);
    }
  }
}
// acc row i += sum over k < K of m[4 ty + i][k] t[k].
template <int DH>
__device__ __forceinline__ void add_rows(Rows<DH>& acc, const float* m, const float* t, int ty, int tx) {
#pragma unroll 2
  for (int k = 0; k < kWide; k += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = load4(m + (4 * ty + i) * kPitchP + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint64_t f[4] = {pair(at(w[0], kk), at(w[0], kk)), pair(at(w[1], kk), at(w[1], kk)),
                             pair(at(w[2], kk), at(w[2], kk)), pair(at(w[3], kk), at(w[3], kk))};
      add_row<DH>(acc, f, t + (k + kk) * (DH + 4), tx);
    }
  }
}
// acc row i += sum over k < 64 of m[k][4 ty + i] t[k]: the matrix's columns, its rows `pitch` apart.
template <int DH>
__device__ __forceinline__ void add_columns(Rows<DH>& acc, const float* m, int pitch, const float* t, int ty, int tx) {
#pragma unroll 4
  for (int k = 0; k < kWide; ++k) {
    const float4 w = load4(m + k * pitch + 4 * ty);
    const uint64_t f[4] = {pair(w.x, w.x), pair(w.y, w.y), pair(w.z, w.z), pair(w.w, w.w)};
    add_row<DH>(acc, f, t + k * (DH + 4), tx);
  }
}

// Rows 4 ty .. of an output, times a factor for each.
template <int DH>
__device__ __forceinline__ void store_rows(const HeadsView& v, int64_t row0, int first, int len, int head, int dim,
                                           const Rows<DH>& acc, const float (&f)[4], int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (first + 4 * ty + i >= len) continue;
    float* dst = row_of(v, row0 + first + 4 * ty + i, head);
#pragma unroll
    for (int u = 0; u < DH / 64; ++u)
      if (4 * tx + 64 * u < dim) {
        float4 x;
        unpair(acc.v[i][u][0], x.x, x.y);
        unpair(acc.v[i][u][1], x.z, x.w);
        *reinterpret_cast<float4*>(dst + 4 * tx + 64 * u) = make_float4(x.x * f[i], x.y * f[i], x.z * f[i], x.w * f[i]);
      }
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

// What a CTA works on. Without WALK one item, given by its index: all heads and sequences of a tile index, causal the
// tiles with the most work (`last_first`: the last ones) first; a tile that its sequence does not have is no work. With it
// persistent CTAs walk over the tiles that there are.
template <bool WALK, int ROWS>
struct Work {
  SequenceWalk walk;
  int round = 0;
  __device__ __forceinline__ Work(const CoreShape& s, int* status, int heads, bool last_first)
      : walk(s, status, heads, ROWS, last_first, threadIdx.x & 31) {}
  __device__ __forceinline__ bool next(Item& it) {
    const CoreShape& s = walk.s;
    if constexpr (WALK) {
      if (!walk.find(walk_place(round++), it)) return false;
    } else {
      if (round++ > 0) return false;
      const int64_t i = blockIdx.x, per = int64_t(walk.heads) * s.batch;  // items of one tile index
      it.tile = static_cast<int>(i / per);
      if (walk.last_first && s.causal) it.tile = (s.max_seq + ROWS - 1) / ROWS - 1 - it.tile;
      it.head = static_cast<int>(i % per % walk.heads);
      it.seq = static_cast<int>(i % per / walk.heads);
    }
    it.len = core_sequence(s, it.seq, it.row0, walk.status);
    return it.tile * ROWS < it.len && in_bounds(s, it, walk.heads, ROWS, walk.status);
  }
};

template <int DH, int N>
__host__ __device__ constexpr int tile_floats() {
  return N * (DH + 4);
}

// Queries, then two buffers of keys and values, then the probabilities.
template <int DH, int ROWS, int BUFS>
constexpr size_t forward_smem() {
  return sizeof(float) * (tile_floats<DH, ROWS>() + 2 * BUFS * tile_floats<DH, kWide>() + ROWS * kPitchP);
}
template <int DH, int ROWS, int BUFS, bool WALK>
__global__ void __launch_bounds__(4 * ROWS) core_forward_kernel(const __grid_constant__ CoreForward c) {
  constexpr int THREADS = 4 * ROWS, W = tile_floats<DH, kWide>();
  extern __shared__ __align__(16) float smem[];
  float* sq = smem;
  float* skv = sq + tile_floats<DH, ROWS>();  // [BUFS][2]
  float* sp = skv + 2 * BUFS * W;
  pdl_wait();
  Item it;
  for (Work<WALK, ROWS> work(c.s, c.status, c.s.heads, true); work.next(it);) {
    const int64_t row0 = it.row0;
    const int h = it.head, len = it.len, q0 = it.tile * ROWS;
    const int kv = h / (c.s.heads / c.s.kv_heads);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    auto copy = [&](int n) {
      copy_tile<DH, kWide, THREADS>(skv + n % BUFS * 2 * W, c.k, row0, n * kWide, len, kv, c.s.dim);
      copy_tile<DH, kWide, THREADS>(skv + n % BUFS * 2 * W + W, c.v, row0, n * kWide, len, kv, c.s.dim);
      copies_commit();
    };
    copy_tile<DH, ROWS, THREADS>(sq, c.q, row0, q0, len, h, c.s.dim);
    copy(0);
    float m[4], l[4];
    Rows<DH> acc;
    clear<DH>(acc);
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
    const int tiles = ((c.s.causal ? min(len, q0 + ROWS) : len) + kWide - 1) / kWide;
    for (int n = 0; n < tiles; ++n) {
      if (BUFS == 1 && n > 0) copy(n);
      if (BUFS == 2 && n + 1 < tiles) {
        copy(n + 1);
        copies_wait<1>();
      } else {
        copies_wait<0>();
      }
      __syncthreads();
      const float* sk = skv + n % BUFS * 2 * W;
      const int k0 = n * kWide;
      float s[4][4];
      dot_tiles<DH, 16>(s, sq, sk, ty, tx);
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
        scale_row<DH>(acc, i, alpha);
      }
      __syncwarp();  // a warp's rows of P are read by the same warp
      add_rows<DH>(acc, sp, sk + W, ty, tx);
      __syncthreads();
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
}

// p and ds of a thread's 4 x 4 scores (rows: queries from q, columns: keys k, k + TX ..). Both are zero wherever a
// query or a key does not count.
template <int TX>
__device__ __forceinline__ void probabilities(const CoreShape& c, float (&s)[4][4], const float (&dp)[4][4],
                                              const float (&lse)[4], const float (&delta)[4], int q, int k, int len,
                                              float (&ds)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kj = k + TX * j;
      const bool on = q + i < len && kj < len && (!c.causal || kj <= q + i);
      const float p = on ? expf(fmaf(s[i][j], c.scale, -lse[i])) : 0.f;
      ds[i][j] = on ? p * (dp[i][j] - delta[i]) : 0.f;
      s[i][j] = p;
    }
  }
}

// Keys and values, then two buffers of queries and dO, then P, and in its place dS.
template <int DH, int ROWS, int BUFS>
constexpr size_t dkv_smem() {
  return sizeof(float) * (2 * tile_floats<DH, ROWS>() + 2 * BUFS * tile_floats<DH, kWide>() + kWide * (ROWS + 4));
}
template <int DH, int ROWS, int BUFS, bool WALK>
__global__ void __launch_bounds__(4 * ROWS) core_dkv_kernel(const __grid_constant__ CoreBackward c, const float* delta) {
  constexpr int THREADS = 4 * ROWS, TX = ROWS / 4, W = tile_floats<DH, kWide>(), PITCH = ROWS + 4;
  extern __shared__ __align__(16) float smem[];
  float* sk = smem;
  float* sv = sk + tile_floats<DH, ROWS>();
  float* sqd = sv + tile_floats<DH, ROWS>();  // [BUFS][2]
  float* sp = sqd + 2 * BUFS * W;
  pdl_wait();
  Item it;
  for (Work<WALK, ROWS> work(c.s, c.status, c.s.kv_heads, false); work.next(it);) {
    const int64_t row0 = it.row0;
    const int kv = it.head, len = it.len, k0 = it.tile * ROWS;
    const int group = c.s.heads / c.s.kv_heads;
    const int sx = threadIdx.x % TX, sy = threadIdx.x / TX;    // of the scores: 64 queries x ROWS keys
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;    // of the outputs: ROWS keys
    const int first = c.s.causal ? k0 / kWide : 0;
    const int per = (len + kWide - 1) / kWide - first, passes = per * group;
    auto copy = [&](int n) {
      const int h = kv * group + n / per, q0 = (first + n % per) * kWide;
      copy_tile<DH, kWide, THREADS>(sqd + n % BUFS * 2 * W, c.q, row0, q0, len, h, c.s.dim);
      copy_tile<DH, kWide, THREADS>(sqd + n % BUFS * 2 * W + W, c.d_o, row0, q0, len, h, c.s.dim);
      copies_commit();
    };
    copy_tile<DH, ROWS, THREADS>(sk, c.k, row0, k0, len, kv, c.s.dim);
    copy_tile<DH, ROWS, THREADS>(sv, c.v, row0, k0, len, kv, c.s.dim);
    copy(0);
    Rows<DH> dk, dv;
    clear<DH>(dk);
    clear<DH>(dv);
    for (int n = 0; n < passes; ++n) {
      const int h = kv * group + n / per, q0 = (first + n % per) * kWide;
      float lse[4], del[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = int64_t(h) * c.s.T + row0 + min(q0 + 4 * sy + i, len - 1);
        lse[i] = c.lse[at];
        del[i] = delta[at];
      }
      if (BUFS == 1 && n > 0) copy(n);
      if (BUFS == 2 && n + 1 < passes) {
        copy(n + 1);
        copies_wait<1>();
      } else {
        copies_wait<0>();
      }
      __syncthreads();
      const float* sq = sqd + n % BUFS * 2 * W;
      float s[4][4], dp[4][4], ds[4][4];
      dot_tiles<DH, TX>(s, sq, sk, sy, sx);
      dot_tiles<DH, TX>(dp, sq + W, sv, sy, sx);
      probabilities<TX>(c.s, s, dp, lse, del, q0 + 4 * sy, k0 + sx, len, ds);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sp[(4 * sy + i) * PITCH + sx + TX * j] = s[i][j];
      __syncthreads();
      add_columns<DH>(dv, sp, PITCH, sq + W, ty, tx);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sp[(4 * sy + i) * PITCH + sx + TX * j] = ds[i][j];
      __syncthreads();
      add_columns<DH>(dk, sp, PITCH, sq, ty, tx);
      __syncthreads();
    }
    const float one[4] = {1.f, 1.f, 1.f, 1.f}, sc[4] = {c.s.scale, c.s.scale, c.s.scale, c.s.scale};
    store_rows<DH>(c.dv, row0, k0, len, kv, c.s.dim, dv, one, ty, tx);
    store_rows<DH>(c.dk, row0, k0, len, kv, c.s.dim, dk, sc, ty, tx);
  }
}

// Queries and dO, then two buffers of keys and values, then dS.
template <int DH, int ROWS, int BUFS>
constexpr size_t dq_smem() {
  return sizeof(float) * (2 * tile_floats<DH, ROWS>() + 2 * BUFS * tile_floats<DH, kWide>() + ROWS * kPitchP);
}
template <int DH, int ROWS, int BUFS, bool WALK>
__global__ void __launch_bounds__(4 * ROWS) core_dq_kernel(const __grid_constant__ CoreBackward c, float* delta) {
  constexpr int THREADS = 4 * ROWS, W = tile_floats<DH, kWide>();
  extern __shared__ __align__(16) float smem[];
  float* sq = smem;
  float* sd = sq + tile_floats<DH, ROWS>();
  float* skv = sd + tile_floats<DH, ROWS>();  // [BUFS][2]
  float* ss = skv + 2 * BUFS * W;
  pdl_wait();
  Item it;
  for (Work<WALK, ROWS> work(c.s, c.status, c.s.heads, true); work.next(it);) {
    const int64_t row0 = it.row0;
    const int h = it.head, len = it.len, q0 = it.tile * ROWS;
    const int kv = h / (c.s.heads / c.s.kv_heads);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    auto copy = [&](int n) {
      copy_tile<DH, kWide, THREADS>(skv + n % BUFS * 2 * W, c.k, row0, n * kWide, len, kv, c.s.dim);
      copy_tile<DH, kWide, THREADS>(skv + n % BUFS * 2 * W + W, c.v, row0, n * kWide, len, kv, c.s.dim);
      copies_commit();
    };
    copy_tile<DH, ROWS, THREADS>(sq, c.q, row0, q0, len, h, c.s.dim);
    copy_tile<DH, ROWS, THREADS>(sd, c.d_o, row0, q0, len, h, c.s.dim);
    copies_commit();
    copy(0);
    // delta: four lanes a row, all of them in the warp that takes the row's scores below; O while dO comes.
    const int r = threadIdx.x >> 2;
    float4 o[DH / 16];
#pragma unroll
    for (int x = 0; x < DH / 16; ++x) {
      const int e = 16 * x + 4 * (threadIdx.x & 3);
      o[x] = q0 + r < len && e < c.s.dim ? load4(row_of(c.o, row0 + q0 + r, h) + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float lse[4], del[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) lse[i] = c.lse[int64_t(h) * c.s.T + row0 + min(q0 + 4 * ty + i, len - 1)];
    copies_wait<1>();
    __syncthreads();
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < DH / 16; ++x) {
      const float4 d = load4(sd + r * (DH + 4) + 16 * x + 4 * (threadIdx.x & 3));
      sum = fmaf(o[x].x, d.x, fmaf(o[x].y, d.y, fmaf(o[x].z, d.z, fmaf(o[x].w, d.w, sum))));
    }
    sum += __shfl_xor_sync(kAll, sum, 2);
    sum += __shfl_xor_sync(kAll, sum, 1);
    if ((threadIdx.x & 3) == 0 && q0 + r < len) delta[int64_t(h) * c.s.T + row0 + q0 + r] = sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) del[i] = __shfl_sync(kAll, sum, 16 * (ty & 1) + 4 * i);
    Rows<DH> dq;
    clear<DH>(dq);
    const int tiles = ((c.s.causal ? min(len, q0 + ROWS) : len) + kWide - 1) / kWide;
    for (int n = 0; n < tiles; ++n) {
      if (BUFS == 1 && n > 0) copy(n);
      if (BUFS == 2 && n + 1 < tiles) {
        copy(n + 1);
        copies_wait<1>();
      } else {
        copies_wait<0>();
      }
      __syncthreads();
      const float* sk = skv + n % BUFS * 2 * W;
      float s[4][4], dp[4][4], ds[4][4];
      dot_tiles<DH, 16>(s, sq, sk, ty, tx);
      dot_tiles<DH, 16>(dp, sd, sk + W, ty, tx);
      probabilities<16>(c.s, s, dp, lse, del, q0 + 4 * ty, n * kWide + tx, len, ds);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) ss[(4 * ty + i) * kPitchP + tx + 16 * j] = ds[i][j];
      __syncwarp();  // a warp's rows of dS are read by the same warp
      add_rows<DH>(dq, ss, sk, ty, tx);
      __syncthreads();
    }
    const float sc[4] = {c.s.scale, c.s.scale, c.s.scale, c.s.scale};
    store_rows<DH>(c.dq, row0, q0, len, h, c.s.dim, dq, sc, ty, tx);
  }
}

// Whether a launch over all tiles of the longest length would be mostly of tiles that no sequence has: of sequences back to
// back there are at most T / rows + batch. (Forward, one CTA a tile of the launch and walked. 1000 sequences in 65536 tokens,
// 8 heads of 64, max_seq left at T: 16529 and 553 us; 13 in 4096, 12 heads, at T: 109 and 101; the same with a tight
// max_seq: 91 and 101, as the GPU hands out CTAs when others end, and the walk does not know when that is.)
bool walked(const CoreShape& s, int rows, int heads) {
  const int64_t tiles = int64_t((s.max_seq + rows - 1) / rows) * s.batch;
  return s.starts && (tiles > 2 * (s.T / rows + s.batch) || tiles * heads > INT32_MAX);
}

template <auto Kernel, auto Walking, typename... Args>
cudaError_t launch(const CoreShape& s, int rows, int heads, size_t smem, cudaStream_t stream, Args... args) {
  static std::atomic<uint64_t> devices{0}, walking{0};
  const bool walk = walked(s, rows, heads);
  cudaError_t e = walk ? allow_smem(Walking, smem, walking) : allow_smem(Kernel, smem, devices);
  if (e != cudaSuccess) return e;
  int64_t items = int64_t((s.max_seq + rows - 1) / rows) * heads * s.batch;
  // As many as an SM's shared memory takes.
  if (walk) items = std::min(items, int64_t(num_sms()) * static_cast<int64_t>(228 * 1024 / (smem + 1024)));
  return launch_pdl(walk ? Walking : Kernel, dim3(static_cast<unsigned>(items)), dim3(4 * rows), smem, stream, args...);
}

template <int DH, int ROWS>
cudaError_t simt_forward(const CoreForward& c, cudaStream_t s) {
  return launch<core_forward_kernel<DH, ROWS, 2, false>, core_forward_kernel<DH, ROWS, 2, true>>(
      c.s, ROWS, c.s.heads, forward_smem<DH, ROWS, 2>(), s, c);
}

template <int DH, int ROWS, int BUFS>
cudaError_t simt_dkv(const CoreBackward& c, const float* delta, cudaStream_t s) {
  return launch<core_dkv_kernel<DH, ROWS, BUFS, false>, core_dkv_kernel<DH, ROWS, BUFS, true>>(
      c.s, ROWS, c.s.kv_heads, dkv_smem<DH, ROWS, BUFS>(), s, c, delta);
}
template <int DH, int ROWS, int BUFS>
cudaError_t simt_dq(const CoreBackward& c, float* delta, cudaStream_t s) {
  return launch<core_dq_kernel<DH, ROWS, BUFS, false>, core_dq_kernel<DH, ROWS, BUFS, true>>(
      c.s, ROWS, c.s.heads, dq_smem<DH, ROWS, BUFS>(), s, c, delta);
}

// The records of core_sequence() alone.
__global__ void __launch_bounds__(256) core_sequences_kernel(CoreShape s, int* status) {
  pdl_wait();
  for (int64_t b = int64_t(blockIdx.x) * 256 + threadIdx.x; b < s.batch; b += int64_t(gridDim.x) * 256) {
    int64_t row0;
    core_sequence(s, static_cast<int>(b), row0, status);
  }
}

// CTAs of `rows` tokens of each head and sequence that fill the GPU four times over.
bool many(const CoreShape& s, int rows, int heads) {
  return int64_t((s.max_seq + rows - 1) / rows) * heads * s.batch >= 4 * num_sms();
}

}  // namespace

namespace {
// delta, on whole lines, then the sums of splits.
size_t delta_bytes(int64_t T, int heads) { return (static_cast<size_t>(T) * heads * sizeof(float) + 255) / 256 * 256; }
}  // namespace

size_t core_backward_workspace(int64_t T, int64_t batch, int64_t max_seq, int heads, int kv_heads, int dim, int bf16) {
  if (T == 0 || batch == 0 || max_seq == 0) return 0;
  const int splits = bf16 ? core_splits_tc(batch, max_seq, heads, kv_heads, dim) : 1;
  const size_t keys = static_cast<size_t>(batch) * ((max_seq + 127) / 128) * 128 * kv_heads;
  return delta_bytes(T, heads) + (splits > 1 ? 2 * splits * keys * dim * sizeof(float) : 0);
}

cudaError_t check_core_sequences(const CoreShape& s, int* status, cudaStream_t stream) {
  const int64_t ctas = (int64_t(s.batch) + 255) / 256, most = 4 * num_sms();
  return launch_pdl(core_sequences_kernel, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), dim3(256), 0, stream, s,
                    status);
}

cudaError_t run_core_forward(const CoreForward& c, cudaStream_t s) {
  TraceScope trace("attn_core_forward", s);
  if (c.bf16) return launch_core_forward_tc(c, s);
  // 64 rows share the tiles that come in, 32 are more CTAs and a shorter last one. Of heads of up to 64, 16 heads, 4 x
  // 1024 tokens: 239 us with 64 rows, 282 with 32; 8 heads, 4 x 384: 40 and 33. Longer heads fill an SM's shared memory
  // either way, and 64 rows bring twice the warps (16 heads of 128, 4 x 1024: 461 us and 621; 8 heads, 2 x 512: 70 and 91).
  if (c.s.dim > 64) return simt_forward<128, 64>(c, s);
  return many(c.s, 64, c.s.heads) ? simt_forward<64, 64>(c, s) : simt_forward<64, 32>(c, s);
}

cudaError_t run_core_backward(const CoreBackward& c, cudaStream_t s) {
  float* delta = static_cast<float*>(c.ws);
  if (c.bf16)
    return launch_core_backward_tc(c, delta, delta + delta_bytes(c.s.T, c.s.heads) / sizeof(float), s);
  // As in the forward, but the backward of short heads stays ahead with 32 rows (16 heads of 64, 4 x 1024 tokens: 893 us
  // and 950 with 64; 16 heads of 128: 2050 with 32 and 1780 with 64). A second buffer takes the copies' time out of the
  // loop, but without it three CTAs fit an SM in the place of two, and the others' work hides the copies: better where there
  // are that many (the same 16 heads of 64: 815 us with one buffer, 893 with two; 8 heads, 4 x 384: 107 and 97).
  const bool small = c.s.dim <= 64;
  {  // makes delta as well, which dK needs
    TraceScope trace("attn_core_dq", s);
    cudaError_t e = !small                      ? simt_dq<128, 64, 2>(c, delta, s)
                    : many(c.s, 32, c.s.heads) ? simt_dq<64, 32, 1>(c, delta, s)
                                               : simt_dq<64, 32, 2>(c, delta, s);
    if (e != cudaSuccess) return e;
  }
  TraceScope trace("attn_core_dkv", s);
  return !small                         ? simt_dkv<128, 64, 2>(c, delta, s)
         : many(c.s, 32, c.s.kv_heads) ? simt_dkv<64, 32, 1>(c, delta, s)
                                       : simt_dkv<64, 32, 2>(c, delta, s);
}

}  // namespace tpmlp
