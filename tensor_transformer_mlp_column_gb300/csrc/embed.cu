// embed.cu — the embedding lookup and the gradient of its table:
//
//   out_t = s E[id_t],        dE_v = s * sum_{t: id_t = v} dout_t.
//
// Both are HBM-bound: the lookup reads and writes T rows, the gradient reads
// T rows and writes all V rows of the table.
//
// The gradient is a sum over equal ids. The tokens are sorted by id (a stable
// radix sort, so equal ids keep the order of t), which turns it into sums of
// consecutive entries with no atomics: the order of every addition is fixed
// by the ids alone. The sorted entries are cut into chunks of kRun; a CTA
// walks one chunk over a slab of columns, keeps the running sum in fp32
// registers, and writes a table row when the id changes. Where an id's
// entries cross a chunk's border the partial sums go to scratch, and a second
// kernel adds them in order: a chunk's work does not depend on how often its
// ids occur, so one id repeated T times is split like any other input.
#include "device.cuh"
#include "internal.h"
#include "train.h"

namespace tpmlp {

namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float& d, float v) { d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

// N consecutive elements as floats; N * sizeof(E) is 16 bytes or one element.
template <typename E, int N>
__device__ __forceinline__ void load_n(const E* p, float (&f)[N]) {
  if constexpr (N == 1) {
    f[0] = to_f(*p);
  } else {
    constexpr int kWords = N * sizeof(E) / 16;
    uint4 w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    const E* e = reinterpret_cast<const E*>(w);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = to_f(e[j]);
  }
}
template <typename E, int N>
__device__ __forceinline__ void store_n(E* p, const float (&f)[N]) {
  if constexpr (N == 1) {
    from_f(*p, f[0]);
  } else {
    constexpr int kWords = N * sizeof(E) / 16;
    uint4 w[kWords];
    E* e = reinterpret_cast<E*>(w);
#pragma unroll
    for (int j = 0; j < N; ++j) from_f(e[j], f[j]);
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
}

// ------------------------------------------------------------------ lookup

constexpr int kThreads = 256;

// A group of `lanes` threads takes one token: pieces of N elements, `lanes`
// apart. N = 8 where rows split into 16-byte pieces, else 1.
template <typename E, int N>
__global__ void __launch_bounds__(kThreads) embed_kernel(const E* __restrict__ table, const int64_t* __restrict__ ids,
                                                         int64_t T, int64_t D, int64_t V, float scale,
                                                         E* __restrict__ out, int lanes, int* status) {
  pdl_wait();
  pdl_launch_dependents();
  const int per_cta = kThreads / lanes;
  const int lane = threadIdx.x % lanes;
  const int64_t pieces = D / N;
  for (int64_t t = int64_t(blockIdx.x) * per_cta + threadIdx.x / lanes; t < T; t += int64_t(gridDim.x) * per_cta) {
    const int64_t id = ids[t];
    const bool on = id >= 0 && id < V;
    if (id >= V && lane == 0) atomicCAS(status, 0, kSiteBoundsBase + kChkToken);
    const E* src = table + (on ? id : 0) * D;
    E* dst = out + t * D;
    for (int64_t c = lane; c < pieces; c += lanes) {
      float f[N];
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = 0.f;
      if (on) load_n<E, N>(src + c * N, f);
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] *= scale;
      store_n<E, N>(dst + c * N, f);
    }
  }
}

// ------------------------------------------------------------------ stable radix sort of (id, t)

// 8 bits a pass. A CTA ranks kTile entries: warp w takes its own 256 in eight
// rounds of 32, so an entry's rank among equal digits follows its index.
constexpr int kDigits = 256;
constexpr int kRounds = 8;
constexpr int kTile = kThreads * kRounds;

// Key of token t: its id, or V (sorted last) where it has no row.
__device__ __forceinline__ uint32_t key_of(int64_t id, int64_t V) {
  return id >= 0 && id < V ? static_cast<uint32_t>(id) : static_cast<uint32_t>(V);
}

// counts[digit * tiles + tile] = entries of the tile with that digit.
__global__ void __launch_bounds__(kThreads) count_kernel(const int64_t* __restrict__ ids, const uint32_t* __restrict__ key,
                                                         int64_t T, int64_t V, int shift, int tiles,
                                                         uint32_t* __restrict__ counts, int* status) {
  __shared__ uint32_t hist[kDigits];
  pdl_wait();
  pdl_launch_dependents();
  hist[threadIdx.x] = 0;
  __syncthreads();
  const int64_t base = int64_t(blockIdx.x) * kTile;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * kThreads + threadIdx.x;
    if (i < T) {
      const uint32_t k = ids ? key_of(ids[i], V) : key[i];
      if (ids && ids[i] >= V) atomicCAS(status, 0, kSiteBoundsBase + kChkToken);
      atomicAdd(&hist[(k >> shift) & (kDigits - 1)], 1u);
    }
  }
  __syncthreads();
  counts[int64_t(threadIdx.x) * tiles + blockIdx.x] = hist[threadIdx.x];
}

// Exclusive prefix sum of n counts, by one CTA of 1024 threads.
__global__ void __launch_bounds__(1024) scan_kernel(uint32_t* __restrict__ counts, int64_t n) {
  __shared__ uint32_t sums[32];
  __shared__ uint32_t carry;
  pdl_wait();
  pdl_launch_dependents();
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  for (int64_t base = 0; base < n; base += 4096) {
    uint32_t v[4];
    const int64_t i = base + 4 * threadIdx.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < n ? counts[i + j] : 0u;
    const uint32_t mine = v[0] + v[1] + v[2] + v[3];
    uint32_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (l >= o) x += y;
    }
    if (l == 31) sums[w] = x;
    __syncthreads();
    if (w == 0) {
      uint32_t y = sums[l];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
        if (l >= o) y += z;
      }
      sums[l] = y;
    }
    __syncthreads();
    uint32_t run = carry + (w ? sums[w - 1] : 0u) + x - mine;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j < n) counts[i + j] = run;
      run += v[j];
    }
    __syncthreads();
    if (threadIdx.x == 0) carry += sums[31];
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kThreads) scatter_kernel(const int64_t* __restrict__ ids, const uint32_t* __restrict__ key,
                                                           const uint32_t* __restrict__ pos, int64_t T, int64_t V,
                                                           int shift, int tiles, const uint32_t* __restrict__ counts,
                                                           uint32_t* __restrict__ key_out,
                                                           uint32_t* __restrict__ pos_out) {
  __shared__ uint32_t seen[kThreads / 32][kDigits];
  pdl_wait();
  pdl_launch_dependents();
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  for (int d = l; d < kDigits; d += 32) seen[w][d] = 0;
  __syncwarp();
  const int64_t base = int64_t(blockIdx.x) * kTile + w * (32 * kRounds);
  uint32_t k[kRounds], p[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * 32 + l;
    const bool on = i < T;
    k[r] = on ? (ids ? key_of(ids[i], V) : key[i]) : 0u;
    p[r] = on ? (ids ? static_cast<uint32_t>(i) : pos[i]) : 0u;
    // Lanes past the end match only each other.
    const uint32_t d = on ? (k[r] >> shift) & (kDigits - 1) : kDigits;
    const uint32_t same = __match_any_sync(0xffffffffu, d);
    const uint32_t before = __popc(same & ((1u << l) - 1u));
    uint32_t at = 0;
    if (on) at = seen[w][d];
    __syncwarp();
    if (on && before == 0) seen[w][d] = at + __popc(same);
    __syncwarp();
    rank[r] = at + before;
  }
  __syncthreads();
  // seen[w][d] -> the global index of the warp's first entry with digit d.
  {
    uint32_t run = counts[int64_t(threadIdx.x) * tiles + blockIdx.x];
#pragma unroll
    for (int v = 0; v < kThreads / 32; ++v) {
      const uint32_t c = seen[v][threadIdx.x];
      seen[v][threadIdx.x] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * 32 + l;
    if (i >= T) continue;
    const uint32_t to = seen[w][(k[r] >> shift) & (kDigits - 1)] + rank[r];
    key_out[to] = k[r];
    pos_out[to] = p[r];
  }
}

// ------------------------------------------------------------------ sums of equal ids

constexpr int kRun = 64;  // sorted entries of a chunk

// Chunk blockIdx.x, columns of slab blockIdx.y: thread x holds N consecutive
// columns. A segment (run of equal ids) inside the chunk goes to its table
// row; the part of a segment that began in an earlier chunk goes to part[2 b],
// the part of one that goes on after this chunk (and began in it) to
// part[2 b + 1]; the whole chunk inside one segment counts as the former.
template <typename G, typename E, int N>
__global__ void __launch_bounds__(kThreads) segment_kernel(const G* __restrict__ dout, const uint32_t* __restrict__ key,
                                                           const uint32_t* __restrict__ pos, int64_t T, int64_t D,
                                                           int64_t V, float scale, E* __restrict__ dE, int accumulate,
                                                           float* __restrict__ part) {
  __shared__ uint32_t skey[kRun + 2], spos[kRun];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t first = int64_t(blockIdx.x) * kRun;
  const int n = static_cast<int>(T - first < kRun ? T - first : kRun);
  // skey[0] and skey[n + 1]: the neighbours' keys (all ones where there is none).
  for (int i = threadIdx.x; i < n + 2; i += blockDim.x) {
    const int64_t at = first + i - 1;
    skey[i] = at >= 0 && at < T ? key[at] : 0xffffffffu;
    if (i >= 1 && i <= n) spos[i - 1] = pos[at];
  }
  __syncthreads();
  const int64_t col = (int64_t(blockIdx.y) * blockDim.x + threadIdx.x) * N;
  if (col >= D) return;
  float sum[N];
#pragma unroll
  for (int j = 0; j < N; ++j) sum[j] = 0.f;
  bool began = skey[0] != skey[1];  // whether the running segment began in this chunk
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const uint32_t k = skey[i + 1];
    if (k >= V) break;  // entries without a row, sorted last
    float f[N];
    load_n<G, N>(dout + int64_t(spos[i]) * D + col, f);
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] += f[j];
    const bool last = skey[i + 2] != k;
    if (!last && i + 1 < n) continue;
    if (last && began) {
      E* row = dE + int64_t(k) * D + col;
      float old[N];
#pragma unroll
      for (int j = 0; j < N; ++j) old[j] = 0.f;
      if (accumulate) load_n<E, N>(row, old);
#pragma unroll
      for (int j = 0; j < N; ++j) sum[j] = fmaf(sum[j], scale, old[j]);
      store_n<E, N>(row, sum);
    } else {
      store_n<float, N>(part + (2 * int64_t(blockIdx.x) + (began ? 1 : 0)) * D + col, sum);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] = 0.f;
    began = true;
  }
}

// Chunk blockIdx.x where a segment begins that goes on after it: adds its
// parts in order and writes the table row.
template <typename E, int N>
__global__ void __launch_bounds__(kThreads) join_kernel(const uint32_t* __restrict__ key, int64_t T, int64_t D, int64_t V,
                                                        float scale, E* __restrict__ dE, int accumulate,
                                                        const float* __restrict__ part) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t b = blockIdx.x, end = (b + 1) * kRun;  // the chunk's end
  if (end >= T) return;
  const uint32_t k = key[end - 1];
  if (k >= V || key[end] != k) return;              // no segment goes on
  if (key[b * kRun] == k && b > 0 && key[b * kRun - 1] == k) return;  // it began earlier
  const int64_t col = (int64_t(blockIdx.y) * blockDim.x + threadIdx.x) * N;
  if (col >= D) return;
  float sum[N];
  load_n<float, N>(part + (2 * b + 1) * D + col, sum);
  for (int64_t c = b + 1; c * kRun < T && key[c * kRun] == k; ++c) {
    float f[N];
    load_n<float, N>(part + 2 * c * D + col, f);
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] += f[j];
  }
  E* row = dE + int64_t(k) * D + col;
  float old[N];
#pragma unroll
  for (int j = 0; j < N; ++j) old[j] = 0.f;
  if (accumulate) load_n<E, N>(row, old);
#pragma unroll
  for (int j = 0; j < N; ++j) sum[j] = fmaf(sum[j], scale, old[j]);
  store_n<E, N>(row, sum);
}

template <typename E>
cudaError_t embed_dispatch(const E* table, const int64_t* ids, int64_t T, int64_t D, int64_t V, float scale, E* out,
                           int* status, cudaStream_t s) {
  const bool vec = D * static_cast<int64_t>(sizeof(E)) % 16 == 0 && D % 8 == 0;
  const int64_t pieces = vec ? D / 8 : D;
  int lanes = 1;
  while (lanes < kThreads && lanes < pieces) lanes <<= 1;
  const int64_t want = (T + kThreads / lanes - 1) / (kThreads / lanes), cap = int64_t(num_sms()) * 8;
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
  return vec ? launch_pdl(embed_kernel<E, 8>, grid, dim3(kThreads), 0, s, table, ids, T, D, V, scale, out, lanes, status)
             : launch_pdl(embed_kernel<E, 1>, grid, dim3(kThreads), 0, s, table, ids, T, D, V, scale, out, lanes, status);
}

template <typename G, typename E, int N>
cudaError_t segments(const G* dout, const uint32_t* key, const uint32_t* pos, int64_t T, int64_t D, int64_t V,
                     float scale, E* dE, int accumulate, float* part, cudaStream_t s) {
  const int64_t pieces = D / N;
  int threads = 32;
  while (threads < kThreads && threads < pieces) threads <<= 1;
  const dim3 grid(static_cast<unsigned>((T + kRun - 1) / kRun), static_cast<unsigned>((pieces + threads - 1) / threads));
  cudaError_t e = launch_pdl(segment_kernel<G, E, N>, grid, dim3(threads), 0, s, dout, key, pos, T, D, V, scale, dE,
                             accumulate, part);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_kernel<E, N>, grid, dim3(threads), 0, s, key, T, D, V, scale, dE, accumulate,
                    static_cast<const float*>(part));
}

template <typename G, typename E>
cudaError_t segments_dispatch(const void* dout, const uint32_t* key, const uint32_t* pos, int64_t T, int64_t D, int64_t V,
                              float scale, void* dE, int accumulate, float* part, cudaStream_t s) {
  const G* g = static_cast<const G*>(dout);
  E* e = static_cast<E*>(dE);
  return D % 8 == 0 ? segments<G, E, 8>(g, key, pos, T, D, V, scale, e, accumulate, part, s)
                    : segments<G, E, 1>(g, key, pos, T, D, V, scale, e, accumulate, part, s);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_embed(const void* E, const int64_t* ids, int64_t T, int64_t D, int64_t V, int is_bf16, float scale,
                         void* out, int* status, cudaStream_t s) {
  if (is_bf16)
    return embed_dispatch(static_cast<const __nv_bfloat16*>(E), ids, T, D, V, scale, static_cast<__nv_bfloat16*>(out),
                          status, s);
  return embed_dispatch(static_cast<const float*>(E), ids, T, D, V, scale, static_cast<float*>(out), status, s);
}

EmbedPlan plan_embed(int64_t T, int64_t D, int64_t V) {
  (void)V;
  EmbedPlan p{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = up256(off + bytes);
    return at;
  };
  for (int i = 0; i < 2; ++i) {
    p.key[i] = take(size_t(T) * 4);
    p.pos[i] = take(size_t(T) * 4);
  }
  p.counts = take(size_t((T + kTile - 1) / kTile) * kDigits * 4);
  p.part = take(size_t((T + kRun - 1) / kRun) * 2 * size_t(D) * 4);
  p.total = off;
  return p;
}

cudaError_t launch_embed_grad(const void* dout, int dout_bf16, const int64_t* ids, int64_t T, int64_t D, int64_t V,
                              float scale, void* dE, int dE_bf16, int accumulate, void* ws, int* status,
                              cudaStream_t s) {
  cudaError_t e;
  if (!accumulate) {
    e = cudaMemsetAsync(dE, 0, size_t(V) * size_t(D) * (dE_bf16 ? 2 : 4), s);
    if (e != cudaSuccess || T == 0) return e;
  }
  const EmbedPlan p = plan_embed(T, D, V);
  char* base = static_cast<char*>(ws);
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(base + p.key[0]), reinterpret_cast<uint32_t*>(base + p.key[1])};
  uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(base + p.pos[0]), reinterpret_cast<uint32_t*>(base + p.pos[1])};
  uint32_t* counts = reinterpret_cast<uint32_t*>(base + p.counts);
  const int tiles = static_cast<int>((T + kTile - 1) / kTile);
  int at = 0;
  for (int shift = 0; shift == 0 || (V >> shift) != 0; shift += 8) {  // keys are 0 .. V
    const int64_t* from = shift == 0 ? ids : nullptr;
    if ((e = launch_pdl(count_kernel, dim3(tiles), dim3(kThreads), 0, s, from, static_cast<const uint32_t*>(key[at]), T, V,
                        shift, tiles, counts, status)) != cudaSuccess)
      return e;
    if ((e = launch_pdl(scan_kernel, dim3(1), dim3(1024), 0, s, counts, int64_t(tiles) * kDigits)) != cudaSuccess) return e;
    if ((e = launch_pdl(scatter_kernel, dim3(tiles), dim3(kThreads), 0, s, from, static_cast<const uint32_t*>(key[at]),
                        static_cast<const uint32_t*>(pos[at]), T, V, shift, tiles, static_cast<const uint32_t*>(counts),
                        key[at ^ 1], pos[at ^ 1])) != cudaSuccess)
      return e;
    at ^= 1;
  }
  float* part = reinterpret_cast<float*>(base + p.part);
  if (dout_bf16)
    return dE_bf16 ? segments_dispatch<__nv_bfloat16, __nv_bfloat16>(dout, key[at], pos[at], T, D, V, scale, dE, accumulate, part, s)
                   : segments_dispatch<__nv_bfloat16, float>(dout, key[at], pos[at], T, D, V, scale, dE, accumulate, part, s);
  return dE_bf16 ? segments_dispatch<float, __nv_bfloat16>(dout, key[at], pos[at], T, D, V, scale, dE, accumulate, part, s)
                 : segments_dispatch<float, float>(dout, key[at], pos[at], T, D, V, scale, dE, accumulate, part, s);
}

}  // namespace tpmlp
