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
// by the ids alone. The sorted entries are cut into chunks; a CTA walks one
// chunk over a slab of columns, keeps the running sum in fp32 registers, and
// writes a table row when the id changes. An id with more entries than two
// chunks hold leaves partial sums in scratch, which a last kernel adds in
// order, so that one id repeated T times is split like any other input.
//
// Most rows of a large table get no gradient and are cleared, by CTAs that
// alternate with the summing ones, all but a first part that fills the time
// of the sort.
#include <atomic>

#include "device.cuh"
#include "internal.h"
#include "trace.h"
#include "train.h"

namespace tpmlp {

namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float& d, float v) { d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

// A thread's N columns of a row. S = false: consecutive ones, loaded as 8, 16 or
// 32 bytes, or one element. S = true, where rows are not made of such pieces:
// `stride` columns apart (the threads that share the row), the first `count` of
// them within the row; a warp's access then covers 32 neighbours.
template <typename E, int N, bool S>
struct Raw {
  static constexpr int kBytes = N * sizeof(E);
  static constexpr int kWords = kBytes >= 16 ? kBytes / 16 : 1;
  uint4 w[kWords];
};
template <typename E, int N>
struct Raw<E, N, true> {
  E e[N];
};
struct Columns {
  int stride, count;
};
// Columns of thread `lane` of `lanes`, from its first one.
template <int N, bool S>
__device__ __forceinline__ Columns columns(int64_t first, int lanes, int64_t D) {
  Columns c{1, N};
  if constexpr (S) {
    c.stride = lanes;
    c.count = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) c.count += first + int64_t(j) * lanes < D;
  }
  return c;
}
template <typename E, int N, bool S>
__device__ __forceinline__ void fetch(const E* p, const Columns& c, Raw<E, N, S>& r) {
  if constexpr (S) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < c.count) r.e[j] = p[j * c.stride];
  } else if constexpr (N == 1) {
    *reinterpret_cast<E*>(r.w) = *p;
  } else if constexpr (Raw<E, N, S>::kBytes == 8) {
    *reinterpret_cast<uint2*>(r.w) = *reinterpret_cast<const uint2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < Raw<E, N, S>::kWords; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
}
template <typename E, int N, bool S>
__device__ __forceinline__ void unpack(const Columns& c, const Raw<E, N, S>& r, float (&f)[N]) {
  if constexpr (S) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = j < c.count ? to_f(r.e[j]) : 0.f;
  } else {
    const E* e = reinterpret_cast<const E*>(r.w);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = to_f(e[j]);
  }
}
template <typename E, int N, bool S>
__device__ __forceinline__ void load_n(const E* p, const Columns& c, float (&f)[N]) {
  Raw<E, N, S> r;
  fetch<E, N, S>(p, c, r);
  unpack<E, N, S>(c, r, f);
}
template <typename E, int N, bool S>
__device__ __forceinline__ void store_n(E* p, const Columns& c, const float (&f)[N]) {
  Raw<E, N, S> r;
  if constexpr (S) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      from_f(r.e[j], f[j]);
      if (j < c.count) p[j * c.stride] = r.e[j];
    }
  } else {
    E* e = reinterpret_cast<E*>(r.w);
#pragma unroll
    for (int j = 0; j < N; ++j) from_f(e[j], f[j]);
    if constexpr (N == 1) {
      *p = *e;
    } else if constexpr (Raw<E, N, S>::kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(r.w);
    } else {
#pragma unroll
      for (int i = 0; i < Raw<E, N, S>::kWords; ++i) reinterpret_cast<uint4*>(p)[i] = r.w[i];
    }
  }
}
// ------------------------------------------------------------------ lookup

constexpr int kThreads = 256;

// Columns of slab blockIdx.y: 2^log_lanes threads take a token's pieces of N
// elements (16 bytes; S: see Raw), K tokens, all loaded before one is written.
template <typename E, int N, bool S, int K>
__global__ void __launch_bounds__(kThreads) embed_kernel(const E* __restrict__ table, const int64_t* __restrict__ ids,
                                                         int64_t T, int64_t D, int64_t V, float scale,
                                                         E* __restrict__ out, int log_lanes, int* status) {
  pdl_wait();
  pdl_launch_dependents();
  const int groups = kThreads >> log_lanes;  // tokens side by side
  const int lanes = 1 << log_lanes, lane = threadIdx.x & (lanes - 1);
  const int64_t col = S ? int64_t(blockIdx.y) * lanes * N + lane : (int64_t(blockIdx.y) * lanes + lane) * N;
  if (col >= D) return;
  const Columns cols = columns<N, S>(col, lanes, D);
  const int64_t t0 = int64_t(blockIdx.x) * (groups * K) + (threadIdx.x >> log_lanes);
  int row[K];  // -1: zero, -2: zero and to be reported
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t id = t0 + k * groups < T ? ids[t0 + k * groups] : -1;
    row[k] = id < 0 ? -1 : id < V ? static_cast<int>(id) : -2;
  }
  Raw<E, N, S> r[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (row[k] >= 0) fetch<E, N, S>(table + row[k] * D + col, cols, r[k]);
  E* dst = out + t0 * D + col;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (t0 + k * groups >= T) break;
    float f[N];
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = 0.f;
    if (row[k] >= 0) {
      unpack<E, N, S>(cols, r[k], f);
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] *= scale;
    }
    store_n<E, N, S>(dst, cols, f);
    dst += groups * D;
  }
  if (col == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (row[k] == -2) atomicCAS(status, 0, kSiteBoundsBase + kChkToken);
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

// counts[digit * tiles + tile] = entries of the tile with that digit; the
// first pass (from the ids) also marks the ids in `present`.
__global__ void __launch_bounds__(kThreads) count_kernel(const int64_t* __restrict__ ids, const uint32_t* __restrict__ key,
                                                         int64_t T, int64_t V, int shift, int tiles,
                                                         uint32_t* __restrict__ counts, uint32_t* __restrict__ present,
                                                         int* status) {
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
      // Looked at first: a frequent id would keep all its marks waiting for one word.
      if (ids && k < V && !(*reinterpret_cast<volatile uint32_t*>(present + (k >> 5)) >> (k & 31) & 1u))
        atomicOr(present + (k >> 5), 1u << (k & 31));
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

// ------------------------------------------------------------------ the sort in one cluster

// CTA c of the first cluster holds the entries c P .. (c + 1) P - 1, P = 1024
// ITEMS, in shared memory. A pass reads them into registers, ranks them by a
// digit of up to 9 bits, puts them in the digit's order within the CTA, and
// copies them to their places in the cluster's shared memory (the last pass:
// to global memory), neighbours to neighbours: without the order within the
// CTA every 4 bytes were a transaction of their own, and 65536 tokens took 70
// us. Above the cluster's capacity a sort of three launches a digit follows.
// The other clusters clear the first clear_bytes of `clear` meanwhile.
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 512;
constexpr int kMaxItems = 8;
constexpr int64_t kClusterSortMax = int64_t(kSortCtas) * kSortThreads * kMaxItems;

__host__ __device__ constexpr size_t sort_smem(int items) {
  return 2 * size_t(items) * kSortThreads * 8 + size_t(kSortWarps) * kMaxBins * 2 + 3 * kMaxBins * 4 + 64 * 4;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint2 v) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const int64_t* __restrict__ ids, int64_t T, int64_t V,
                                                               int bits, int passes, uint32_t* __restrict__ key_out,
                                                               uint32_t* __restrict__ pos_out,
                                                               uint32_t* __restrict__ present, void* clear,
                                                               int64_t clear_bytes, int* status) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x >= kSortCtas) {
    // In consecutive blocks of 64 KB.
    constexpr int64_t kBlock = 4096;
    const int64_t n16 = clear_bytes / 16;
    for (int64_t b = int64_t(blockIdx.x - kSortCtas) * kBlock; b < n16; b += int64_t(gridDim.x - kSortCtas) * kBlock)
#pragma unroll
      for (int u = 0; u < kBlock / kSortThreads; ++u) {
        const int64_t i = b + u * kSortThreads + threadIdx.x;
        if (i < n16) reinterpret_cast<uint4*>(clear)[i] = make_uint4(0, 0, 0, 0);
      }
    return;
  }
  constexpr int P = ITEMS * kSortThreads;
  uint2* entry = reinterpret_cast<uint2*>(smem);  // (key, position)
  uint2* staged = entry + P;
  uint16_t* seen = reinterpret_cast<uint16_t*>(staged + P);                     // [warp][bin]
  uint32_t* count = reinterpret_cast<uint32_t*>(seen + kSortWarps * kMaxBins);  // this CTA's entries of a bin
  uint32_t* local = count + kMaxBins;  // place of the bin's first entry within the CTA
  uint32_t* move = local + kMaxBins;   // from there to its place in the cluster
  uint32_t* sums = move + kMaxBins;    // two scans of 16 warps
  const uint32_t cta = cluster_ctarank();
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31, tid = threadIdx.x;
  const int64_t left = T - int64_t(cta) * P;
  const int n = left < 0 ? 0 : left < P ? static_cast<int>(left) : P;  // this CTA's entries
  const int mine = w * (32 * ITEMS) + l;                               // this thread's: mine + 32 r
  const int bins = 1 << bits;
  for (int64_t i = int64_t(cta) * kSortThreads + tid; i < (V + 31) / 32; i += kSortCtas * kSortThreads) present[i] = 0;
  cluster_sync_all();  // orders the clearing of `present` before the cluster's marks
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    uint2 e[ITEMS];
    uint32_t place[ITEMS];
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
      const int i = mine + 32 * r;
      e[r] = make_uint2(0, 0);
      if (i >= n) continue;
      if (pass == 0) {
        const int64_t id = ids[int64_t(cta) * P + i];
        if (id >= V) atomicCAS(status, 0, kSiteBoundsBase + kChkToken);
        e[r] = make_uint2(key_of(id, V), cta * P + i);
      } else {
        e[r] = entry[i];
      }
    }
    for (int d = l; d < bins; d += 32) seen[w * kMaxBins + d] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
      const bool on = mine + 32 * r < n;
      const uint32_t d = (e[r].x >> shift) & (bins - 1);
      // Lanes with the same digit, bit by bit.
      uint32_t same = __ballot_sync(0xffffffffu, on);
      for (int bit = 0; bit < bits; ++bit) {
        const bool set = d >> bit & 1u;
        const uint32_t b = __ballot_sync(0xffffffffu, set);
        same &= set ? b : ~b;
      }
      const uint32_t before = __popc(same & ((1u << l) - 1u));
      uint32_t at = 0;
      if (on) at = seen[w * kMaxBins + d];
      __syncwarp();
      if (on && before == 0) seen[w * kMaxBins + d] = static_cast<uint16_t>(at + __popc(same));
      __syncwarp();
      place[r] = at + before;
    }
    __syncthreads();
    if (tid < bins) {  // the warps' counts -> the warps' first places within the bin
      uint32_t run = 0;
#pragma unroll 8
      for (int v = 0; v < kSortWarps; ++v) {
        const uint32_t c = seen[v * kMaxBins + tid];
        seen[v * kMaxBins + tid] = static_cast<uint16_t>(run);
        run += c;
      }
      count[tid] = run;
    }
    cluster_sync_all();  // every CTA's counts are there, every entry is in registers
    // Places: bin by bin in the cluster, within a bin CTA by CTA; and within this CTA.
    uint32_t total = 0, ahead = 0, own = 0, x = 0, y = 0;
    if (tid < kMaxBins) {
      if (tid < bins) {
        own = count[tid];
#pragma unroll
        for (uint32_t c = 0; c < kSortCtas; ++c) {
          const uint32_t v = ld_cluster_u32(map_to_cta(smem_addr(count + tid), c));
          if (c < cta) ahead += v;
          total += v;
        }
      }
      x = total, y = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
        if (l >= o) x += a, y += b;
      }
      if (l == 31) sums[w] = x, sums[16 + w] = y;
    }
    __syncthreads();
    if (tid < bins) {
      uint32_t lx = 0, ly = 0;
      for (int v = 0; v < w; ++v) lx += sums[v], ly += sums[16 + v];
      local[tid] = ly + y - own;
      move[tid] = (lx + x - total + ahead) - (ly + y - own);
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
      if (mine + 32 * r >= n) continue;
      const uint32_t d = (e[r].x >> shift) & (bins - 1);
      staged[local[d] + seen[w * kMaxBins + d] + place[r]] = e[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
      const int i = r * kSortThreads + tid;
      if (i >= n) continue;
      const uint2 v = staged[i];
      const uint32_t to = i + move[(v.x >> shift) & (bins - 1)];
      if (pass + 1 < passes) {
        st_cluster_v2(map_to_cta(smem_addr(entry + to % P), to / P), v);
      } else {
        key_out[to] = v.x;
        pos_out[to] = v.y;
        // In the last pass the CTA's entries are in the order of their keys: one mark for each.
        if (v.x < V && (i == 0 || staged[i - 1].x != v.x)) atomicOr(present + (v.x >> 5), 1u << (v.x & 31));
      }
    }
    cluster_sync_all();  // entries in place, counts read
  }
}

template <int ITEMS>
cudaError_t cluster_sort(const int64_t* ids, int64_t T, int64_t V, uint32_t* key, uint32_t* pos, uint32_t* present,
                         void* clear, int64_t clear_bytes, int* status, cudaStream_t s) {
  auto kern = sort_kernel<ITEMS>;
  constexpr size_t smem = sort_smem(ITEMS);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  int all = 1;
  while ((V >> all) != 0) ++all;  // bits of the keys 0 .. V
  const int passes = (all + 8) / 9, bits = (all + passes - 1) / passes;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSortCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSortCtas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  // Clearing takes as many clusters as 64 KB for each of their CTAs justify and
  // as run at once: not every SM finds seven others for one (15 clusters; two
  // more begin when the first are done, T = 4096, V = 50257, D = 768: the sort
  // 14.6 -> 18.7 us).
  int64_t clusters = 1 + (clear_bytes + 65536 * kSortCtas - 1) / (65536 * kSortCtas);
  if (clusters > 1) {
    static std::atomic<int> max_clusters[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    int cap = max_clusters[dev].load(std::memory_order_relaxed);
    if (!cap) {
      cfg.numAttrs = 1;  // the query takes the cluster shape only
      if ((e = cudaOccupancyMaxActiveClusters(&cap, kern, &cfg)) != cudaSuccess) return e;
      if (cap < 2) cap = 2;
      max_clusters[dev].store(cap, std::memory_order_relaxed);
    }
    if (clusters > cap) clusters = cap;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kSortCtas));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, ids, T, V, bits, passes, key, pos, present, clear, clear_bytes, status);
}

// ------------------------------------------------------------------ sums of equal ids

constexpr int kMaxRun = 64;
constexpr int kBatch = 8;
// Sorted entries of a chunk: few where there are few tokens, so that the
// chunks still spread over the SMs.
int run_of(int64_t T) { return T <= 16384 ? 16 : kMaxRun; }

// What the clearing CTAs of segment_kernel do: table rows from `row0` on that
// are not marked in `present`, in pieces of 16 bytes, kClearPieces a CTA, of the
// rows' bytes as a whole. A piece that holds parts of two rows, or the table's
// end, goes element by element. (One element at a time for all of a table with
// such rows: D = 1074, V = 111592, T = 391, fp32, the sums with the clearing 178
// us.)
constexpr int kClearUnroll = 8;
constexpr int kClearPieces = kThreads * kClearUnroll;
struct Clear {
  const uint32_t* present;
  int64_t row0, rows;   // rows [row0, rows); row0 rows are a multiple of 16 bytes
  int64_t bytes;        // of those
  uint32_t row_bytes;
  uint32_t magic;       // ceil(2^32 / row_bytes), where 1 < row_bytes < 16 kClearPieces, else 0
  int element;          // bytes
  int ctas;
  // The CTAs in their order: every `period`-th one is of the rarer kind, as
  // long as there are any. Rare summing CTAs are every second one at first:
  // theirs are the long chains of loads (T = 4096, V = 50257, D = 768: 30 us
  // spread over the grid, 26.5 so).
  int period, sums_rare;
};

__device__ __forceinline__ void clear_rows(const Clear& c, int64_t cta, char* dE) {
  const int64_t first = cta * (16 * kClearPieces);  // byte
  const int n = static_cast<int>(c.bytes - first < 16 * kClearPieces ? c.bytes - first : 16 * kClearPieces);
  const int64_t row = c.bytes >> 32 ? first / c.row_bytes : static_cast<uint32_t>(first) / c.row_bytes;
  const uint32_t skip = static_cast<uint32_t>(first - row * c.row_bytes);
  char* base = dE + c.row0 * c.row_bytes + first;
  auto marked = [&](int64_t v) { return v < c.rows ? __ldg(c.present + (v >> 5)) >> (v & 31) & 1u : 1u; };
  // How many rows below `row` byte skip + i is: long rows meet at most one border here, short ones divide by
  // multiplying (exact while numerator * row_bytes < 2^32).
  auto down_of = [&](uint32_t x) { return c.magic ? __umulhi(x, c.magic) : (x >= c.row_bytes ? 1u : 0u); };
  uint32_t marks[kClearUnroll];  // bit 0: the row is marked; bit 1: not of one whole row
#pragma unroll
  for (int u = 0; u < kClearUnroll; ++u) {
    const int i = (threadIdx.x + u * kThreads) * 16;
    const uint32_t x = skip + static_cast<uint32_t>(i), down = down_of(x);
    const bool whole = x - down * c.row_bytes + 16 <= c.row_bytes && i + 16 <= n;
    marks[u] = i >= n ? 1u : whole ? marked(c.row0 + row + down) : 2u;
  }
#pragma unroll
  for (int u = 0; u < kClearUnroll; ++u) {
    if (marks[u] & 1u) continue;
    const int i = (threadIdx.x + u * kThreads) * 16;
    if (marks[u] == 0) {
      *reinterpret_cast<uint4*>(base + i) = make_uint4(0, 0, 0, 0);
      continue;
    }
    for (int o = i; o < i + 16 && o < n; o += c.element) {
      if (marked(c.row0 + row + down_of(skip + static_cast<uint32_t>(o)))) continue;
      if (c.element == 4)
        *reinterpret_cast<uint32_t*>(base + o) = 0;
      else
        *reinterpret_cast<uint16_t*>(base + o) = 0;
    }
  }
}

// Chunk b (`run` sorted entries), columns of slab y: thread x holds N columns
// (S: see Raw). A segment (run of equal ids) of up to 2 run entries
// belongs to the chunk in which it begins, whose CTA follows it past the
// chunk's end. Of a longer one every chunk sums its part: the part of a segment
// that began in an earlier chunk goes to part[2 b], the part of one that
// begins in it to part[2 b + 1], and goes_on[b] says that there is such a
// one. The clearing CTAs alternate with these evenly over the grid.
template <typename G, typename E, int N, bool S>
__global__ void __launch_bounds__(kThreads, 4) segment_kernel(const G* __restrict__ dout, const uint32_t* __restrict__ key,
                                                           const uint32_t* __restrict__ pos, int64_t T, int64_t D,
                                                           int64_t V, float scale, E* __restrict__ dE, int accumulate,
                                                           float* __restrict__ part, uint8_t* __restrict__ goes_on,
                                                           int run, int slabs, const __grid_constant__ Clear clear) {
  __shared__ uint32_t skey[5 * kMaxRun], spos[3 * kMaxRun];
  __shared__ int s_start, s_stop, s_began;
  pdl_wait();
  pdl_launch_dependents();
  uint32_t job = blockIdx.x;
  if (clear.ctas > 0) {
    // q CTAs of the rarer kind before this one; is it one itself?
    const uint32_t rare = clear.sums_rare ? gridDim.x - clear.ctas : clear.ctas;
    const uint32_t turn = job / clear.period;
    const bool is_rare = job == turn * clear.period && turn < rare;
    const uint32_t q = min(turn + (job > turn * clear.period ? 1u : 0u), rare);
    const uint32_t index = is_rare ? turn : job - q;
    if (is_rare != static_cast<bool>(clear.sums_rare)) {
      clear_rows(clear, index, reinterpret_cast<char*>(dE));
      return;
    }
    job = index;
  }
  const uint32_t chunk32 = job / static_cast<uint32_t>(slabs);
  const int slab = job - chunk32 * slabs;
  const int64_t chunk = chunk32;
  const int64_t first = chunk * run;
  const int n = static_cast<int>(T - first < run ? T - first : run);
  const int most = 2 * run;
  // skey[most + i]: the key of entry first + i, from `most` entries before the
  // chunk to `most` after it (all ones past the end).
  for (int i = threadIdx.x; i < run + 2 * most; i += blockDim.x) {
    const int64_t at = first + i - most;
    skey[i] = at >= 0 && at < T ? key[at] : 0xffffffffu;
    if (i >= most && at < T) spos[i - most] = pos[at];
  }
  __syncthreads();
  const uint32_t* k_at = skey + most;
  // First index in [lo, hi) whose key is at least (after = 0) or above (1) k.
  auto bound = [&](int lo, int hi, uint32_t k, bool after) {
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (after ? k_at[mid] <= k : k_at[mid] < k)
        lo = mid + 1;
      else
        hi = mid;
    }
    return lo;
  };
  if (threadIdx.x < 32) {  // one warp looks, the others wait
    const int lowest = first < most ? -static_cast<int>(first) : -most;
    int start = 0, stop = n;
    bool began = true;  // whether the running segment began in this chunk
    const uint32_t k0 = k_at[0];
    const int a0 = bound(lowest, 0, k0, false);
    if (a0 < 0) {  // it began earlier: summed there, unless it is a long one
      began = a0 > -most && k_at[a0 + most] != k0;
      if (began) start = bound(0, n, k0, true);
    }
    bool long_on = false;
    if (start < n && n == run && k_at[n] == k_at[n - 1]) {
      const uint32_t k = k_at[n - 1];
      const int a = bound(lowest, n, k, false);
      if (a >= 0) {  // it begins in this chunk
        long_on = k_at[a + most] == k;
        if (!long_on) stop = bound(n, n + most, k, true);
      }
    }
    if (threadIdx.x == 0) {
      s_start = start, s_stop = stop, s_began = began;
      if (slab == 0) goes_on[chunk] = long_on && k_at[n - 1] < V;
    }
  }
  __syncthreads();
  const int start = s_start, stop = s_stop;
  bool began = s_began;
  const int64_t col =
      S ? int64_t(slab) * blockDim.x * N + threadIdx.x : (int64_t(slab) * blockDim.x + threadIdx.x) * N;
  if (col >= D) return;
  const Columns cols = columns<N, S>(col, blockDim.x, D);
  float sum[N];
#pragma unroll
  for (int j = 0; j < N; ++j) sum[j] = 0.f;
  // A ring of kBatch rows on their way: row i + kBatch is fetched when row i is added.
  Raw<G, N, S> r[kBatch];
  auto issue = [&](int i, Raw<G, N, S>& to) {
    if (i >= stop || k_at[i] >= V) return;
    fetch<G, N, S>(dout + int64_t(spos[i]) * D + col, cols, to);
    if (accumulate && k_at[i + 1] != k_at[i])
      asm volatile("prefetch.global.L2 [%0];" ::"l"(dE + int64_t(k_at[i]) * D + col));
  };
#pragma unroll
  for (int b = 0; b < kBatch; ++b) issue(start + b, r[b]);
  for (int i0 = start; i0 < stop; i0 += kBatch) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b;
      if (i >= stop) return;
      const uint32_t k = k_at[i];
      if (k >= V) return;  // entries without a row, sorted last
      float f[N];
      unpack<G, N, S>(cols, r[b], f);
      issue(i + kBatch, r[b]);
#pragma unroll
      for (int j = 0; j < N; ++j) sum[j] += f[j];
      const bool last = k_at[i + 1] != k;
      if (!last && i + 1 < stop) continue;
      if (last && began) {
        E* row = dE + int64_t(k) * D + col;
        float old[N];
#pragma unroll
        for (int j = 0; j < N; ++j) old[j] = 0.f;
        if (accumulate) load_n<E, N, S>(row, cols, old);
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] = fmaf(sum[j], scale, old[j]);
        store_n<E, N, S>(row, cols, sum);
      } else {
        store_n<float, N, S>(part + (2 * chunk + (began ? 1 : 0)) * D + col, cols, sum);
      }
#pragma unroll
      for (int j = 0; j < N; ++j) sum[j] = 0.f;
      began = true;
    }
  }
}

// The long segments that begin in one of `span` consecutive chunks: adds
// their parts in order and writes the table row. A CTA takes 32 N columns;
// its eight warps take consecutive eighths of a segment's parts and their
// sums are added in the warps' order, so that one id repeated T times is
// still spread over the GPU.
// Few chunks a CTA where that makes no more than a round or two of CTAs: the
// segments of one CTA go one after the other (T = 16384, D = 1024, bf16: 10.5
// us with 32, 8.4 with 4).
int join_span(int64_t chunks, int64_t columns) { return (chunks + 3) / 4 * columns <= 2048 ? 4 : 32; }
template <typename E, int N>
__global__ void __launch_bounds__(kThreads) join_kernel(const uint32_t* __restrict__ key, int64_t T, int64_t D, int run,
                                                        float scale, E* __restrict__ dE, int accumulate,
                                                        const float* __restrict__ part,
                                                        const uint8_t* __restrict__ goes_on, int64_t chunks, int span) {
  __shared__ float red[kThreads / 32][32 * N];
  pdl_wait();
  pdl_launch_dependents();
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  // Lane l looks at the CTA's chunk l (every warp alike).
  const int64_t mine = int64_t(blockIdx.x) * span + l;
  const bool owns = l < span && mine < chunks && goes_on[mine];
  uint32_t todo = __ballot_sync(0xffffffffu, owns);
  const int64_t col = (int64_t(blockIdx.y) * 32 + l) * N;
  for (; todo; todo &= todo - 1) {
    const int64_t b = int64_t(blockIdx.x) * span + __ffs(todo) - 1;
    const uint32_t k = key[(b + 1) * run - 1];
    // The chunks that the segment reaches are those after b whose first key is k.
    int64_t reach = b + 1;
    for (;;) {
      const int64_t c = reach + threadIdx.x;
      const int more = __syncthreads_count(c * run < T && key[c * run] == k);
      reach += more;
      if (more < kThreads) break;
    }
    // Parts: part[2 b + 1], then part[2 c] for c = b + 1 .. reach - 1.
    const int64_t parts = reach - b, per = (parts + 7) / 8;
    const int64_t from = w * per, to = from + per < parts ? from + per : parts;
    float sum[N];
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] = 0.f;
    if (col < D) {
#pragma unroll 4
      for (int64_t i = from; i < to; ++i) {
        float f[N];
        load_n<float, N, false>(part + (i == 0 ? 2 * b + 1 : 2 * (b + i)) * D + col, Columns{}, f);
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] += f[j];
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) red[w][l * N + j] = sum[j];
    __syncthreads();
    if (w == 0 && col < D) {
      for (int v = 1; v < kThreads / 32; ++v)
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] += red[v][l * N + j];
      E* row = dE + int64_t(k) * D + col;
      float old[N];
#pragma unroll
      for (int j = 0; j < N; ++j) old[j] = 0.f;
      if (accumulate) load_n<E, N, false>(row, Columns{}, old);
#pragma unroll
      for (int j = 0; j < N; ++j) sum[j] = fmaf(sum[j], scale, old[j]);
      store_n<E, N, false>(row, Columns{}, sum);
    }
    __syncthreads();
  }
}

template <typename E, int N, bool S>
cudaError_t lookup(const E* table, const int64_t* ids, int64_t T, int64_t D, int64_t V, float scale, E* out, int* status,
                   cudaStream_t s) {
  const int64_t pieces = (D + N - 1) / N;
  int log_lanes = 0;
  while ((1 << log_lanes) < kThreads && (1 << log_lanes) < pieces) ++log_lanes;
  const int64_t lanes = int64_t(1) << log_lanes;
  const int64_t slabs = (pieces + lanes - 1) / lanes, groups = kThreads / lanes;
  // Four tokens a thread where that still leaves eight CTAs an SM.
  const int64_t per4 = (T + groups * 4 - 1) / (groups * 4);
  const bool four = per4 * slabs >= int64_t(num_sms()) * 8;
  const int64_t x = four ? per4 : (T + groups - 1) / groups;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(slabs));
  return four ? launch_pdl(embed_kernel<E, N, S, 4>, grid, dim3(kThreads), 0, s, table, ids, T, D, V, scale, out, log_lanes, status)
              : launch_pdl(embed_kernel<E, N, S, 1>, grid, dim3(kThreads), 0, s, table, ids, T, D, V, scale, out, log_lanes, status);
}

template <typename E>
cudaError_t embed_dispatch(const E* table, const int64_t* ids, int64_t T, int64_t D, int64_t V, float scale, E* out,
                           int* status, cudaStream_t s) {
  constexpr int N = 16 / sizeof(E);
  return D % N == 0 ? lookup<E, N, false>(table, ids, T, D, V, scale, out, status, s)
                    : lookup<E, 4, true>(table, ids, T, D, V, scale, out, status, s);
}

template <typename G, typename E, int N, bool S>
cudaError_t segments(const G* dout, const uint32_t* key, const uint32_t* pos, int64_t T, int64_t D, int64_t V,
                     float scale, E* dE, int accumulate, float* part, uint8_t* goes_on, const Clear& clear,
                     cudaStream_t s) {
  const int run = run_of(T);
  const int64_t pieces = (D + N - 1) / N;
  int threads = 32;
  while (threads < kThreads && threads < pieces) threads <<= 1;
  if (clear.ctas > 0) threads = kThreads;  // the clearing CTAs'
  const int64_t slabs = (pieces + threads - 1) / threads, chunks = (T + run - 1) / run;
  const int64_t grid = chunks * slabs + clear.ctas;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  Clear c = clear;
  if (c.ctas > 0) {
    const int64_t sums = chunks * slabs;
    c.sums_rare = sums <= c.ctas;
    c.period = c.sums_rare ? 2 : static_cast<int>(sums / c.ctas) + 1;
  }
  {
    TraceScope trace("embed_segments", s);
    const cudaError_t e = launch_pdl(segment_kernel<G, E, N, S>, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, s, dout,
                                     key, pos, T, D, V, scale, dE, accumulate, part, goes_on, run, static_cast<int>(slabs), c);
    if (e != cudaSuccess) return e;
  }
  if (T <= 2 * run) return cudaSuccess;  // no segment is longer than that
  TraceScope trace("embed_join", s);
  // Four columns a thread where rows allow, whatever dout's pieces are.
  const unsigned columns = static_cast<unsigned>(D % 4 == 0 ? (D + 127) / 128 : (D + 31) / 32);
  const int span = join_span(chunks, columns);
  const dim3 join(static_cast<unsigned>((chunks + span - 1) / span), columns);
  const float* p = part;
  const uint8_t* on = goes_on;
  return D % 4 == 0
             ? launch_pdl(join_kernel<E, 4>, join, dim3(kThreads), 0, s, key, T, D, run, scale, dE, accumulate, p, on, chunks, span)
             : launch_pdl(join_kernel<E, 1>, join, dim3(kThreads), 0, s, key, T, D, run, scale, dE, accumulate, p, on, chunks, span);
}

template <typename G, typename E>
cudaError_t segments_dispatch(const void* dout, const uint32_t* key, const uint32_t* pos, int64_t T, int64_t D, int64_t V,
                              float scale, void* dE, int accumulate, float* part, uint8_t* goes_on, const Clear& clear, cudaStream_t s) {
  const G* g = static_cast<const G*>(dout);
  E* e = static_cast<E*>(dE);
  // Strided columns: eight bytes a thread (16 of fp32 spill beside the ring of rows: T = 65536, D = 1074, V = 50000,
  // 271 us, and 125 so; one element a thread 201).
  constexpr int N = 16 / sizeof(G);
  return D % N == 0 ? segments<G, E, N, false>(g, key, pos, T, D, V, scale, e, accumulate, part, goes_on, clear, s)
                    : segments<G, E, 8 / static_cast<int>(sizeof(G)), true>(g, key, pos, T, D, V, scale, e, accumulate, part, goes_on, clear, s);
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
  p.present = take(size_t((V + 31) / 32) * 4);
  p.counts = take(size_t((T + kTile - 1) / kTile) * kDigits * 4);
  const size_t chunks = size_t((T + run_of(T) - 1) / run_of(T));
  p.goes_on = take(chunks);
  p.part = take(chunks * 2 * size_t(D) * 4);
  p.total = off;
  return p;
}

cudaError_t launch_embed_grad(const void* dout, int dout_bf16, const int64_t* ids, int64_t T, int64_t D, int64_t V,
                              float scale, void* dE, int dE_bf16, int accumulate, void* ws, int* status,
                              cudaStream_t s) {
  cudaError_t e;
  const size_t bytes = size_t(V) * size_t(D) * (dE_bf16 ? 2 : 4);
  if (T == 0) return accumulate ? cudaSuccess : cudaMemsetAsync(dE, 0, bytes, s);
  const EmbedPlan p = plan_embed(T, D, V);
  char* base = static_cast<char*>(ws);
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(base + p.key[0]), reinterpret_cast<uint32_t*>(base + p.key[1])};
  uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(base + p.pos[0]), reinterpret_cast<uint32_t*>(base + p.pos[1])};
  uint32_t* counts = reinterpret_cast<uint32_t*>(base + p.counts);
  uint32_t* present = reinterpret_cast<uint32_t*>(base + p.present);
  const int64_t row_bytes = D * (dE_bf16 ? 2 : 4);
  Clear clear{};
  clear.present = present;
  clear.element = dE_bf16 ? 2 : 4;
  clear.row_bytes = static_cast<uint32_t>(row_bytes);
  clear.rows = V;
  const bool cluster = T <= kClusterSortMax;
  int items = 1;  // of a thread in the cluster's sort
  while (items < kMaxItems && T > int64_t(kSortCtas) * kSortThreads * items) items *= 2;
  if (!accumulate) {
    // The sort in the cluster takes about 6 + 3 items us, in which the other SMs write 7 MB a us (T = 40000, D =
    // 4096, V = 128000: 4 MB a us for 8 us and 2 more per 8192 tokens left 239 us in all, this 226).
    if (cluster) clear.row0 = int64_t(6 + 3 * items) * (7 << 20) / row_bytes;
    if (clear.row0 > V) clear.row0 = V;
    if (row_bytes % 16 != 0) clear.row0 &= ~int64_t(7);  // eight rows are a multiple of 16 bytes
    clear.bytes = (V - clear.row0) * row_bytes;
    const int64_t ctas = (clear.bytes + 16 * kClearPieces - 1) / (16 * kClearPieces);
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    clear.ctas = static_cast<int>(ctas);
    clear.magic =
        row_bytes < 16 * kClearPieces ? static_cast<uint32_t>(((1ull << 32) + clear.row_bytes - 1) / clear.row_bytes) : 0;
  }
  int at = 0;
  {
    TraceScope trace("embed_sort", s);
    if (cluster) {
      const int64_t first = clear.row0 * row_bytes;
      e = items == 1   ? cluster_sort<1>(ids, T, V, key[0], pos[0], present, dE, first, status, s)
          : items == 2 ? cluster_sort<2>(ids, T, V, key[0], pos[0], present, dE, first, status, s)
          : items == 4 ? cluster_sort<4>(ids, T, V, key[0], pos[0], present, dE, first, status, s)
                       : cluster_sort<kMaxItems>(ids, T, V, key[0], pos[0], present, dE, first, status, s);
      if (e != cudaSuccess) return e;
    } else {
      if ((e = cudaMemsetAsync(present, 0, size_t((V + 31) / 32) * 4, s)) != cudaSuccess) return e;
      const int tiles = static_cast<int>((T + kTile - 1) / kTile);
      for (int shift = 0; shift == 0 || (V >> shift) != 0; shift += 8) {  // keys are 0 .. V
        const int64_t* from = shift == 0 ? ids : nullptr;
        if ((e = launch_pdl(count_kernel, dim3(tiles), dim3(kThreads), 0, s, from, static_cast<const uint32_t*>(key[at]), T,
                            V, shift, tiles, counts, present, status)) != cudaSuccess)
          return e;
        if ((e = launch_pdl(scan_kernel, dim3(1), dim3(1024), 0, s, counts, int64_t(tiles) * kDigits)) != cudaSuccess)
          return e;
        if ((e = launch_pdl(scatter_kernel, dim3(tiles), dim3(kThreads), 0, s, from, static_cast<const uint32_t*>(key[at]),
                            static_cast<const uint32_t*>(pos[at]), T, V, shift, tiles,
                            static_cast<const uint32_t*>(counts), key[at ^ 1], pos[at ^ 1])) != cudaSuccess)
          return e;
        at ^= 1;
      }
    }
  }
  float* part = reinterpret_cast<float*>(base + p.part);
  uint8_t* goes_on = reinterpret_cast<uint8_t*>(base + p.goes_on);
  if (dout_bf16)
    return dE_bf16 ? segments_dispatch<__nv_bfloat16, __nv_bfloat16>(dout, key[at], pos[at], T, D, V, scale, dE, accumulate, part, goes_on, clear, s)
                   : segments_dispatch<__nv_bfloat16, float>(dout, key[at], pos[at], T, D, V, scale, dE, accumulate, part, goes_on, clear, s);
  return dE_bf16 ? segments_dispatch<float, __nv_bfloat16>(dout, key[at], pos[at], T, D, V, scale, dE, accumulate, part, goes_on, clear, s)
                 : segments_dispatch<float, float>(dout, key[at], pos[at], T, D, V, scale, dE, accumulate, part, goes_on, clear, s);
}

}  // namespace tpmlp
