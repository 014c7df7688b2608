// attn_core_tc.cu — attention on given queries, keys and values and its
// backward pass on the tensor cores (bf16, head sizes up to 128; the formulas
// stand in attn_core.cu).
//
// Three persistent kernels, tiles of 128 tokens, head sizes padded to DH = 64 or
// 128 by TMA's zero fill (products take the head in steps of 16):
//   forward  items of NQ query tiles of one head: S = Q K^T, P = exp(S - max),
//            O += P V, with a running maximum and sum for each row.
//   dQ       items of a query tile: S = Q K^T, dP = dO V^T, dS = P (dP - delta),
//            dQ += dS K, and P K, which puts dQ right for what delta is off.
//   dK, dV   items of a key tile of a kv head, over the query tiles of all heads
//            that share it: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.
// Making S and dP twice costs 7 products in the place of 5 (the mean key's is an
// eighth), but every sum has one owner: no atomics, no order that changes, no
// fp32 dQ in memory.
//
// All tiles come by TMA through a 3-D map (element, head, token) that knows any
// strides. P and dS never leave the SM: the threads that read S from tensor
// memory write them back there as bf16, and the next product takes them as its
// A operand from tensor memory. A tile in shared memory serves as a K-major
// operand (contraction over the head) and as an MN-major one (contraction over
// its tokens) without a copy.
//
// A tile's last rows can belong to the next sequence. Scores there are dropped
// by a comparison, and the rows of a tile that enters a contraction over its
// tokens are cleared in shared memory, so that no value of another sequence, not
// even a NaN, meets a weight of zero.
//
// Bound by the chain from S to P and dS: scores out of tensor memory, exponentials,
// bf16 numbers back into it. Beside it the tensor pipe is active for 49 % of the
// cycles (forward), 56 to 65 (dQ) and 60 (dK, dV) where heads are long, of the 75
// that a plain matrix product takes, and for 15 to 24 % where they are short (512
// tokens, heads of 64). 8192 tokens, 16 heads of 128, no mask: forward 386 us, 1.43
// PFLOP/s, dQ 614 us, 1.79 with the product of P and K, dK and dV 665 us, 1.65;
// heads of 64: 310, 463 and 578 us, 0.89, 1.19 and 0.95 PFLOP/s.
//
// The next kernel of the stream is let in by the loading warp when it has fetched its
// last item. Let in at the start, its CTAs waited in places beside the ones still at
// work, and unevenly (13 sequences of 1 to 1500 tokens, 12 heads of 80, a step: 202
// us, at the end 184; 8 x 512 tokens, 16 heads of 64: 78.5 and 74; 3 x 17 tokens: 23
// and 20).
//
// Warps: 4 or 8 for the softmax (warp w reads tensor memory lanes 32 (w % 4) ..),
// one issuing products, one issuing loads. Every wait is bounded; after a failure
// copies and products in flight are waited for and tensor memory is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <string.h>

#include <algorithm>

#include "attn_core.h"
#include "attn_core_walk.cuh"
#include "device.cuh"
#include "internal.h"
#include "trace.h"

namespace tpmlp {

namespace {

constexpr int kRows = 128;                   // tokens of a tile
constexpr uint32_t kChunk = kRows * 128;     // 64 elements of its rows
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ pieces

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// True in one lane of a converged warp. Under a branch on this the compiler knows that a single thread issues the
// products and keeps their operands in uniform registers; under `lane == 0` each tcgen05.mma cost 130 cycles of issue,
// with it 60, less than the 64 that a 128 x 128 x 16 product takes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

// Box of 64 elements x 1 head x 64 tokens.
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, int32_t x, int32_t head, int32_t token,
                                              uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(token), "r"(smem_addr(bar))
      : "memory");
}
// A tile of ROWS tokens, 64 elements of all of them after another; the barrier's arrival is the caller's.
template <int DH, int ROWS = kRows>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, int head, int64_t token, uint64_t* bar) {
#pragma unroll
  for (int c = 0; c < DH / 64; ++c)
#pragma unroll
    for (int r = 0; r < ROWS; r += 64)
      tma_load_rows(dst + (c * ROWS + r) * 128, map, 64 * c, head, static_cast<int32_t>(token) + r, bar);
}

// A in tensor memory (row i in lane i, two K in each 32-bit column), B in shared memory.
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A tile as an MN-major operand: 64 elements of N a line, 8 tokens (K) a group
// of 1024 bytes, the next 64 elements `chunk` bytes further.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t chunk) {
  return (static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4)) | (static_cast<uint64_t>(chunk >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (static_cast<uint64_t>(1u) << 46) | (static_cast<uint64_t>(2u) << 61);
}

// d = A B^T over the head's first 16 `steps` elements, both tiles K-major, A of 128 tokens, B of W: a 128 x W matrix.
template <int DH, int W = kRows>
__device__ __forceinline__ void product_rows(uint32_t d, const uint8_t* a, const uint8_t* b, int steps) {
  constexpr uint32_t id = idesc_bf16_f32(128, W);
  const uint32_t sa = smem_addr(a), sb = smem_addr(b);
#pragma unroll
  for (int k = 0; k < DH / 16; ++k)
    if (k < steps)
      tc_mma_bf16(d, smem_desc_sw128(sa + (k / 4) * kChunk + (k % 4) * 32),
                  smem_desc_sw128(sb + (k / 4) * (W * 128) + (k % 4) * 32), id, k > 0);
}
// d (+)= M B over W tokens, the first 16 `steps` elements of the head: M a 128 x W bf16 matrix in tensor memory, its
// columns in runs of RUN (of 16 bits) that begin `step` columns (of 32 bits) apart.
template <int W, int RUN>
__device__ __forceinline__ void product_tokens(uint32_t d, uint32_t m, const uint8_t* b, bool accumulate, uint32_t step,
                                               int steps) {
  const uint32_t id = idesc_bf16_f32(128, 16 * steps, 0, 1);
  const uint32_t sb = smem_addr(b);
#pragma unroll
  for (int k = 0; k < W / 16; ++k)
    mma_tmem_a(d, m + (k / (RUN / 16)) * step + (k % (RUN / 16)) * 8, desc_mn(sb + 2048 * k, W * 128), id,
               accumulate || k > 0);
}

// Clears a tile's rows from `from` on; all lanes of a warp, before a product by its lane 0.
template <int DH, int ROWS = kRows>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from, int lane) {
  for (int i = from * 8 + lane; i < ROWS * 8; i += 32)
#pragma unroll
    for (int c = 0; c < DH / 64; ++c) *reinterpret_cast<uint4*>(tile + c * ROWS * 128 + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

__device__ __forceinline__ void tmem_st_32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[32]) { tmem_st_32(taddr, v); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[16]) { tmem_st_16(taddr, v); }

// N columns, a multiple of 32, of this warp's lanes.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
  uint32_t r[N / 32][32];
#pragma unroll
  for (int x = 0; x < N / 32; ++x) tmem_ld_32cols_issue(taddr + 32 * x, r[x]);
#pragma unroll
  for (int x = 0; x < N / 32; ++x) {
    tmem_ld_wait(r[x]);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[32 * x + i] = __uint_as_float(r[x][i]);
  }
}

// Packed pairs of fp32.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitGuard& g, int site) {
  return __all_sync(kAll, wait_bounded(bar, parity, g, site));
}

// A ring of SLOTS buffers: position n is buffer n % SLOTS in its n / SLOTS-th use.
template <int SLOTS>
struct Ring {
  uint64_t *full, *empty;
  __device__ __forceinline__ void init(uint32_t full_count = 1, uint32_t empty_count = 1) const {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(full + i, full_count);
      mbar_init(empty + i, empty_count);
    }
  }
  __device__ __forceinline__ bool wait_full(int n, const WaitGuard& g) const {
    return warp_wait(full + n % SLOTS, (n / SLOTS) & 1, g, kSiteMmaFull);
  }
  __device__ __forceinline__ bool wait_empty(int n, const WaitGuard& g) const {
    return warp_wait(empty + n % SLOTS, ((n / SLOTS) & 1) ^ 1u, g, kSiteProducer);
  }
  // After a failure: the last fill of every buffer among the first n.
  __device__ __forceinline__ void drain(int n, uint64_t limit_ns) const {
    for (int i = n > SLOTS ? n - SLOTS : 0; i < n; ++i) wait_drain(full + i % SLOTS, (i / SLOTS) & 1, limit_ns);
  }
};

// A row's sums of all groups of columns.
template <int GROUPS>
__device__ __forceinline__ float row_sum(const float* s_sum, int row) {
  float v = 0.f;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) v += s_sum[g * kRows + row];
  return v;
}

// sum + the products of eight bf16 pairs.
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float sum) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), sum);
    sum = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), sum);
  }
  return sum;
}

// What rounding pairs of `v` to `w` left, as bf16.
template <int N>
__device__ __forceinline__ void rests(const float (&v)[N], uint32_t (&w)[N / 2]) {
#pragma unroll
  for (int e = 0; e < N; e += 2)
    w[e / 2] = pack_bf16(v[e] - __uint_as_float(w[e / 2] << 16), v[e + 1] - __uint_as_float(w[e / 2] & 0xffff0000u));
}

// The first `dim` of a row's columns at `column` .. column + 31 as bf16, times f.
__device__ __forceinline__ void store_row(__nv_bfloat16* dst, const float (&v)[32], float f, int column, int dim) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (column + 8 * u < dim)
      *reinterpret_cast<uint4*>(dst + column + 8 * u) =
          make_uint4(pack_bf16(v[8 * u] * f, v[8 * u + 1] * f), pack_bf16(v[8 * u + 2] * f, v[8 * u + 3] * f),
                     pack_bf16(v[8 * u + 4] * f, v[8 * u + 5] * f), pack_bf16(v[8 * u + 6] * f, v[8 * u + 7] * f));
}

// As fp32.
__device__ __forceinline__ void store_sums(float* dst, const float (&v)[32], int column, int dim) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (column + 4 * u < dim)
      *reinterpret_cast<float4*>(dst + column + 4 * u) = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
}

struct TcParams {
  CoreShape s;
  CUtensorMap q, k, v, d_o;
  HeadsView o, dq, dk, dv;
  float* lse;    // forward: written; backward: read
  float* delta;  // backward
  int splits;    // dK, dV: runs of a tile's passes
  float* part;   // where splits > 1: sums of dV, of dK, in the places that part_of() gives
  float scale_log2;
  int steps;       // of 16 elements: what products over or of the head take
  int tiles;       // tiles (forward: runs of NQ tiles) of the longest sequence
  uint32_t items;  // tiles x heads x sequences, or 2^31 - 1 where that is less (with starts only, which do not need it)
  int withhold;    // test hook: > 0: that load of the CTA's first ring is not issued
  uint64_t wait_ns;
  int* status;
};

// A split's sums of a row of a key tile: [dV, dK][splits][batch][tiles][kv_heads][128][dim].
__device__ __forceinline__ float* part_of(const TcParams& p, int z, int split, int seq, int tile, int kv, int row) {
  const int64_t at = ((int64_t(z * p.splits + split) * p.s.batch + seq) * p.tiles + tile) * p.s.kv_heads + kv;
  return p.part + (at * kRows + row) * p.s.dim;
}

// Debug build: whether there are such sums.
__device__ __forceinline__ bool part_exists(const TcParams& p, int split, int seq, int tile, int kv) {
  return TPMLP_DCHECK(split >= 0 && split < p.splits && seq >= 0 && seq < p.s.batch && tile >= 0 && tile < p.tiles && kv >= 0 &&
                          kv < p.s.kv_heads,
                      p.status, kChkReduce);
}

// The items of a CTA, found by its loading warp, in the order that attn_core_walk.cuh gives sequences of any lengths; equal
// sequences' are all tiles of one index after another, with a causal mask those with the most work first.
struct Walk {
  const TcParams& p;
  SequenceWalk sequences;
  bool last_first;
  uint64_t round = 0;

  __device__ __forceinline__ Walk(const TcParams& p_, int heads, int rows, bool last_first_, int lane)
      : p(p_), sequences(p_.s, p_.status, heads, rows, last_first_, lane), last_first(last_first_) {}
  // All lanes together.
  __device__ __forceinline__ bool next(Item& it) {
    const uint64_t at = walk_place(round++);
    if (!p.s.starts) {
      if (at >= p.items) return false;
      const uint32_t heads = sequences.heads, i = static_cast<uint32_t>(at), per = heads * p.s.batch, in = i % per;
      it.tile = static_cast<int>(i / per);
      if (last_first) it.tile = p.tiles - 1 - it.tile;
      it.head = static_cast<int>(in % heads);
      it.seq = static_cast<int>(in / heads);
    } else if (!sequences.find(at, it)) {
      return false;
    }
    it.len = core_sequence(p.s, it.seq, it.row0, p.status);
    return in_bounds(p.s, it, sequences.heads, sequences.rows, p.status);
  }
};

// Items on their way from the loading warp to the others.
constexpr int kItemSlots = 2;
constexpr size_t kItemBytes = kItemSlots * (sizeof(Item) + 16);
struct ItemRing {
  Item* items;
  uint64_t *full, *empty;
  __device__ __forceinline__ explicit ItemRing(void* at)
      : items(static_cast<Item*>(at)),
        full(reinterpret_cast<uint64_t*>(items + kItemSlots)),
        empty(full + kItemSlots) {}
  __device__ __forceinline__ void init(uint32_t readers) const {
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, readers);
    }
  }
  // The k-th item goes out; all lanes of the loading warp.
  __device__ __forceinline__ bool give(int k, const Item& it, int lane, const WaitGuard& g) const {
    if (!warp_wait(empty + k % kItemSlots, ((k / kItemSlots) & 1) ^ 1u, g, kSiteProducer)) return false;
    if (lane == 0) {
      items[k % kItemSlots] = it;
      mbar_arrive(full + k % kItemSlots);
    }
    return true;
  }
  // The k-th item, or false after the last one or a failure.
  __device__ __forceinline__ bool take(int k, Item& it, int lane, const WaitGuard& g) const {
    if (!hold(k, g)) return false;
    it = items[k % kItemSlots];
    release(k, lane);
    return true;
  }
  // The same for a warp that reads the item (held()) where it needs it, until it releases it.
  __device__ __forceinline__ bool hold(int k, const WaitGuard& g) const {
    return warp_wait(full + k % kItemSlots, (k / kItemSlots) & 1, g, kSiteMmaFull) && held(k).len > 0;
  }
  __device__ __forceinline__ const volatile Item& held(int k) const { return items[k % kItemSlots]; }
  __device__ __forceinline__ void release(int k, int lane) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + k % kItemSlots);
  }
};

// Shared memory of a kernel: tiles, then rows of floats, then barriers. There is no slack to align it in: the dynamic
// shared memory begins on a multiple of 1024 bytes, which the swizzled tiles need, and which is checked.
__device__ __forceinline__ bool misaligned(const uint8_t* smem, int* status) {
  if (!(smem_addr(smem) & 1023u)) return false;
  if (threadIdx.x == 0) atomicCAS(status, 0, kSiteSmemAlign);
  return true;
}

// Debug build: whether what follows the barriers ends within the kernel's `bytes` of shared memory.
__device__ __forceinline__ bool fits(const uint8_t* smem, size_t bytes, const volatile int* last, int* status) {
  return TPMLP_DCHECK(smem_addr(const_cast<const int*>(last + 1)) <= smem_addr(smem) + bytes, status, kChkArea);
}

// ------------------------------------------------------------------ forward

template <int DH, int NQ>
struct FwdCfg {
  static constexpr uint32_t TILE = DH / 64 * kChunk;
  static constexpr int SLOTS = 4;  // K_0, V_0, K_1, ..
  static constexpr uint32_t TMEM = NQ == 2 ? 512 : 256;
  static constexpr int CTAS = NQ == 1 && DH == 64 ? 2 : 1;  // an SM's
  static constexpr uint32_t O = NQ * 128;  // columns: S of each tile, then O of each
  static constexpr size_t BARS = 8 * (2 * SLOTS + 3 + 3 * NQ) + kItemBytes + 8;  // barriers, items, two words
  static constexpr size_t SMEM = (NQ + SLOTS) * TILE + BARS;
  static constexpr int THREADS = (4 * NQ + 2) * 32;
  static_assert(O + NQ * DH <= TMEM, "tensor memory");
};

// The row's maximum so far, raised where the tile's is above it by more than
// 2^8 in weight: until then weights stay below 2^8 and O needs no factor (a
// published method for attention on this generation of GPUs).
//
// Two query tiles take turns: one's products run while the other is in the
// softmax. An item's Q is fetched once the last item's scores are made, under its
// last softmax, product and output.
template <int DH, int NQ>
__global__ void __launch_bounds__(FwdCfg<DH, NQ>::THREADS, FwdCfg<DH, NQ>::CTAS) fwd_kernel(const __grid_constant__ TcParams p) {
  using C = FwdCfg<DH, NQ>;
  constexpr int kMma = 4 * NQ, kLoad = 4 * NQ + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (misaligned(smem, p.status)) return;
  uint8_t* s_q = smem;
  uint8_t* s_ring = smem + NQ * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_ring + C::SLOTS * C::TILE);
  const Ring<C::SLOTS> ring{bars, bars + C::SLOTS};
  uint64_t* q_full = bars + 2 * C::SLOTS;
  uint64_t* q_free = q_full + 1;   // the item's scores are all made
  uint64_t* s_full = q_free + 1;   // [NQ] scores of a tile are there
  uint64_t* p_full = s_full + NQ;  // [NQ] its probabilities are there, and O has the new maximum
  uint64_t* o_done = p_full + NQ;  // [NQ] an item's O is there
  uint64_t* drain = o_done + NQ;
  const ItemRing ring_i(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring_i.empty + kItemSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  if (!fits(smem, C::SMEM, abort_flag, p.status)) return;

  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ring.init();
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    for (int a = 0; a < NQ; ++a) {
      mbar_init(s_full + a, 1);
      mbar_init(p_full + a, 4);
      mbar_init(o_done + a, 1);
    }
    mbar_init(drain, 1);
    ring_i.init(4 * NQ + 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMma) tmem_alloc(tmem_slot, C::TMEM);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const WaitGuard guard{abort_flag, p.wait_ns, p.status};
  const int group = p.s.heads / p.s.kv_heads;
  // Key tiles of the item's query tile a.
  auto tiles_of = [&](const Item& it, int a) {
    const int first = (it.tile * NQ + a) * kRows;
    return first >= it.len ? 0 : ((p.s.causal ? min(it.len, first + kRows) : it.len) + kRows - 1) / kRows;
  };
  // Of any of them: causal, the last one that there is has the most.
  auto most_of = [&](const Item& it) {
    int n = tiles_of(it, 0);
#pragma unroll
    for (int a = 1; a < NQ; ++a) n = max(n, tiles_of(it, a));
    return n;
  };
  int issued = 0, items = 0;  // fills of the ring; items with work

  if (warp == kLoad) {
    bool ok = true;
    Item it;
    for (Walk walk(p, p.s.heads, NQ * kRows, true, lane); ok && walk.next(it);) {
      ok = ring_i.give(items, it, lane, guard);
      if (!ok) break;
      const int n = most_of(it), kv = it.head / group;
      ok = items == 0 || warp_wait(q_free, (items - 1) & 1, guard, kSiteProducer);
      if (!ok) break;
      if (elect_one()) {
        int tiles = 0;
        for (int a = 0; a < NQ; ++a) tiles += tiles_of(it, a) > 0;
        mbar_arrive_expect_tx(q_full, tiles * C::TILE);
        for (int a = 0; a < tiles; ++a)
          load_tile<DH>(s_q + a * C::TILE, &p.q, it.head, it.row0 + (it.tile * NQ + a) * kRows, q_full);
      }
      ++items;
      for (int i = 0; i < 2 * n; ++i) {
        ok = ring.wait_empty(issued, guard);
        if (!ok) break;
        if (issued + 1 != p.withhold && elect_one()) {
          mbar_arrive_expect_tx(ring.full + issued % C::SLOTS, C::TILE);
          load_tile<DH>(s_ring + (issued % C::SLOTS) * C::TILE, i & 1 ? &p.v : &p.k, kv, it.row0 + (i >> 1) * kRows,
                        ring.full + issued % C::SLOTS);
        }
        ++issued;
      }
    }
    pdl_launch_dependents();
    it.len = 0;
    if (ok) ring_i.give(items, it, lane, guard);
  } else if (warp == kMma) {
    bool ok = true;
    int at = 0;            // ring position of the item's first key tile
    int done[NQ] = {};     // tiles of each query tile so far
    Item it;
    for (int i = 0; ok && ring_i.take(i, it, lane, guard); ++i) {
      int n[NQ], n_max = 0;
#pragma unroll
      for (int a = 0; a < NQ; ++a) n[a] = tiles_of(it, a), n_max = max(n_max, n[a]);
      ok = warp_wait(q_full, items & 1, guard, kSiteMmaFull) && ring.wait_full(at, guard);
      if (!ok) break;
      ++items;
      if (elect_one()) {
#pragma unroll
        for (int a = 0; a < NQ; ++a)
          if (n[a] > 0) {
            product_rows<DH>(tmem + a * 128, s_q + a * C::TILE, s_ring + (at % C::SLOTS) * C::TILE, p.steps);
            tc_commit(s_full + a);
          }
        tc_commit(ring.empty + at % C::SLOTS);
        if (n_max == 1) tc_commit(q_free);
      }
      __syncwarp();
      for (int j = 0; j < n_max; ++j) {
        const int vn = at + 2 * j + 1, kn = vn + 1;
        uint8_t* v_tile = s_ring + (vn % C::SLOTS) * C::TILE;
        const uint8_t* k_next = s_ring + (kn % C::SLOTS) * C::TILE;
        ok = ring.wait_full(vn, guard);
        if (!ok) break;
        if (it.len - j * kRows < kRows) clear_rows<DH>(v_tile, it.len - j * kRows, lane);
        ok = j + 1 >= n_max || ring.wait_full(kn, guard);
        if (!ok) break;
#pragma unroll
        for (int a = 0; a < NQ; ++a) {
          if (j >= n[a]) continue;
          ok = ok && warp_wait(p_full + a, (done[a] + j) & 1, guard, kSiteMmaAcc);
          if (!ok) break;
          tc_fence_after_sync();
          if (elect_one()) {
            product_tokens<kRows, kRows>(tmem + C::O + a * DH, tmem + a * 128, v_tile, j > 0, 0, p.steps);
            if (j + 1 == n[a]) tc_commit(o_done + a);
            if (j + 1 < n[a]) {  // over P, whose product comes first
              product_rows<DH>(tmem + a * 128, s_q + a * C::TILE, k_next, p.steps);
              tc_commit(s_full + a);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) {
          tc_commit(ring.empty + vn % C::SLOTS);
          if (j + 1 < n_max) tc_commit(ring.empty + kn % C::SLOTS);
          if (j + 2 == n_max) tc_commit(q_free);
        }
        __syncwarp();
      }
      at += 2 * n_max;
#pragma unroll
      for (int a = 0; a < NQ; ++a) done[a] += n[a];
    }
  } else {
    const int a = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + a * 128, t_o = tmem + lanes + C::O + a * DH;
    const float c = p.scale_log2;
    bool ok = true;
    int done = 0;  // tiles so far
    Item it;
    for (int i = 0; ok && ring_i.take(i, it, lane, guard); ++i) {
      const int tiles = tiles_of(it, a), first = (it.tile * NQ + a) * kRows, qi = first + row;
      if (tiles == 0) continue;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < tiles; ++j) {
        ok = warp_wait(s_full + a, (done + j) & 1, guard, kSiteMmaFull);
        if (!ok) break;
        tc_fence_after_sync();
        float s[128];
        tmem_ld<128>(t_s, s);
        const int k0 = j * kRows;
        if (k0 + kRows > it.len || (p.s.causal && k0 + kRows > first)) {
          const int end = (p.s.causal ? min(it.len, qi + 1) : it.len) - k0;  // columns that count
#pragma unroll
          for (int e = 0; e < 128; ++e) s[e] = e < end ? s[e] : -INFINITY;
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 2)
          asm("max.f32 %0, %0, %1, %2;" : "+f"(m4[(e >> 1) & 3]) : "f"(s[e]), "f"(s[e + 1]));
        const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const float m_new = (top - m) * c > 8.f ? top : m;  // at a row's first finite score: top
        const float alpha = m_new == m ? 1.f : exp2_fast((m - m_new) * c);
        const float base = m_new == -INFINITY ? 0.f : m_new * c;  // no score above -inf yet: weights of zero, not NaN
        m = m_new;
        if (j > 0 && __any_sync(kAll, alpha != 1.f)) {
          // The scores' arrival came after the previous product's end: O holds still.
#pragma unroll 1
          for (int x = 0; x < DH && x < p.s.dim; x += 32) {
            float o[32];
            uint32_t w[32];
            tmem_ld_32cols(t_o + x, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * alpha);
            tmem_st_32(t_o + x, w);
          }
        }
        const uint64_t c2 = pair(c, c), b2 = pair(-base, -base);
        uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float e0, e1;
            unpair(fma_pair(pair(s[64 * x + e], s[64 * x + e + 1]), c2, b2), e0, e1);
            e0 = exp2_fast(e0);
            e1 = exp2_fast(e1);
            sum[(e >> 1) & 1] = add_pair(sum[(e >> 1) & 1], pair(e0, e1));
            w[e / 2] = pack_bf16(e0, e1);
          }
          tmem_st_32(t_s + 32 * x, w);
        }
        float x0, x1;
        unpair(add_pair(sum[0], sum[1]), x0, x1);
        l = l * alpha + (x0 + x1);
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + a);
      }
      if (!ok) break;
      done += tiles;
      ok = warp_wait(o_done + a, items & 1, guard, kSiteEpilogue);
      if (!ok) break;
      ++items;  // those with a query tile a
      tc_fence_after_sync();
      const float inv = 1.f / l;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o.p) + (it.row0 + qi) * p.o.token + it.head * p.o.head;
#pragma unroll 1
      for (int x = 0; x < DH && x < p.s.dim; x += 32) {
        float o[32];
        tmem_ld_32cols(t_o + x, o);
        if (qi < it.len) store_row(dst, o, inv, x, p.s.dim);
      }
      // O is in registers: the next item's first product, which waits for this warp's next probabilities, overwrites it.
      tc_fence_before_sync();
      if (qi < it.len) p.lse[int64_t(it.head) * p.s.T + it.row0 + qi] = m * p.s.scale + logf(l);
    }
  }
  __syncthreads();
  if (*abort_flag) {
    if (warp == kLoad && elect_one()) {
      if (items > 0) wait_drain(q_full, (items - 1) & 1, p.wait_ns);
      ring.drain(issued, p.wait_ns);
    }
    if (warp == kMma && elect_one()) {
      tc_commit(drain);
      wait_drain(drain, 0, p.wait_ns);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TMEM);
  }
}

// ------------------------------------------------------------------ dQ

template <int DH, int W>
struct DqCfg {
  static constexpr uint32_t TILE = DH / 64 * kChunk, NARROW = DH / 64 * W * 128;  // of the queries, of the keys
  static constexpr int KS = DH == 64 ? 4 : 3, VS = DH == 64 ? 3 : 2;
  static constexpr uint32_t S = 0, DP = W, DQ = 2 * W, KM = 2 * W + DH;  // columns: S, dP, dQ, the mean key
  static constexpr uint32_t TMEM = 2 * W + 2 * DH <= 256 ? 256 : 512;
  static constexpr int CTAS = TMEM == 256 ? 2 : 1;  // an SM's
  // Columns of a softmax warp: 64, but 32 for short heads, whose tiles are half as wide (8 x 2048 tokens, 32 heads of 128:
  // with 32 4 % slower; 16 heads of 64: with 64 4 % slower).
  static constexpr int COLUMNS = DH == 64 ? 32 : 64, GROUPS = W / COLUMNS, WARPS = 4 * GROUPS;
  static constexpr int THREADS = (WARPS + 2) * 32;
  static constexpr size_t BARS = 8 * (2 * KS + 2 * VS + 9) + kItemBytes + 8;
  static constexpr size_t SMEM = 2 * TILE + (KS + VS) * NARROW + (GROUPS + 1) * 512 + BARS;
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory");
};

// P goes over S, dS over dP; the scores of tile j + 1 are made while the threads
// work on dS of tile j, its dP while they work on P of tile j + 1.
//
// FINE: what rounding dS to bf16 leaves goes into dQ by a product of its own (and
// into dK by one there). Otherwise that rounding leaves dQ about as far off as the
// rounding of dQ itself, sqrt(2) of it together, more where a row's keys are alike:
// 0.0025 in the place of 0.0017 for heads of 8 and 16, and for the few numbers of
// short sequences, which are what it is for (dQ of heads below 64, dQ and dK where
// max_seq is within the tile of W). 8 x 2048 tokens, 16 heads of 32: 124 -> 142 us,
// 0.0024 -> 0.0017; 128 x 100 tokens, 32 heads of 128 on 8: 117 -> 131, dK and dV 94
// -> 104. With longer heads and sequences, where all sums are long, it is left out
// (8 x 2048 tokens, 32 heads of 128 on 8: 0.0024, and dQ 22 % slower with it).
//
// delta comes in as dO . O with the O that the forward rounded to bf16, which is
// as far off as dQ's own rounding. But the row's sum of dS, zero for the exact
// delta, says how far: e = sum of p dp - delta. dK's kernel gets delta + e, and dQ
// is put right with the row's mean key, dQ = sum of dS k - e sum of P k: a fourth
// product, for 0.0024 in the place of 0.0030 as dQ's error (8 x 2048 tokens, 32
// heads of 128; dQ 377 -> 407 us). Rows with a single key tile take their own sum of p dp from the
// start.
template <int DH, int W, bool FINE>
__global__ void __launch_bounds__(DqCfg<DH, W>::THREADS, DqCfg<DH, W>::CTAS) dq_kernel(const __grid_constant__ TcParams p) {
  using C = DqCfg<DH, W>;
  constexpr int H = C::COLUMNS, kMmaWarp = C::WARPS, kLoadWarp = C::WARPS + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (misaligned(smem, p.status)) return;
  uint8_t* s_q = smem;
  uint8_t* s_do = s_q + C::TILE;
  uint8_t* s_k = s_do + C::TILE;
  uint8_t* s_v = s_k + C::KS * C::NARROW;
  float* s_delta = reinterpret_cast<float*>(s_v + C::VS * C::NARROW);  // [128]
  float* s_sum = s_delta + kRows;                                      // [GROUPS][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_sum + C::GROUPS * kRows);
  const Ring<C::KS> ring_k{bars, bars + C::KS};
  bars += 2 * C::KS;
  const Ring<C::VS> ring_v{bars, bars + C::VS};
  bars += 2 * C::VS;
  uint64_t* q_full = bars;       // Q and dO
  uint64_t* q_free = bars + 1;   // the item's S and dP are all made
  uint64_t* s_full = bars + 2;
  uint64_t* p_full = bars + 3;
  uint64_t* dp_full = bars + 4;
  uint64_t* ds_full = bars + 5;
  uint64_t* done = bars + 6;     // an item's dQ and mean key are there
  uint64_t* meet = bars + 7;     // the softmax warps' sums are in shared memory
  uint64_t* drain = bars + 8;
  const ItemRing ring_i(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring_i.empty + kItemSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  if (!fits(smem, C::SMEM, abort_flag, p.status)) return;

  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ring_k.init();
    ring_v.init();
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, C::WARPS);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, C::WARPS);
    mbar_init(done, 1);
    mbar_init(meet, C::WARPS);
    mbar_init(drain, 1);
    ring_i.init(C::WARPS + 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, C::TMEM);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const WaitGuard guard{abort_flag, p.wait_ns, p.status};
  const int group = p.s.heads / p.s.kv_heads;
  // Key tiles of an item.
  auto tiles_of = [&](const Item& it) {
    const int q0 = it.tile * kRows;
    return q0 >= it.len ? 0 : ((p.s.causal ? min(it.len, q0 + kRows) : it.len) + W - 1) / W;
  };
  int items = 0, issued_k = 0, issued_v = 0;

  if (warp == kLoadWarp) {
    bool ok = true;
    Item it;
    for (Walk walk(p, p.s.heads, kRows, true, lane); ok && walk.next(it);) {
      ok = ring_i.give(items, it, lane, guard);
      if (!ok) break;
      const int n = tiles_of(it), kv = it.head / group;
      ok = items == 0 || warp_wait(q_free, (items - 1) & 1, guard, kSiteProducer);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(q_full, 2 * C::TILE);
        load_tile<DH>(s_q, &p.q, it.head, it.row0 + it.tile * kRows, q_full);
        load_tile<DH>(s_do, &p.d_o, it.head, it.row0 + it.tile * kRows, q_full);
      }
      ++items;
      for (int j = 0; j < n; ++j) {
        ok = ring_k.wait_empty(issued_k, guard);
        if (!ok) break;
        if (issued_k + 1 != p.withhold && elect_one()) {
          mbar_arrive_expect_tx(ring_k.full + issued_k % C::KS, C::NARROW);
          load_tile<DH, W>(s_k + (issued_k % C::KS) * C::NARROW, &p.k, kv, it.row0 + j * W, ring_k.full + issued_k % C::KS);
        }
        ++issued_k;
        ok = ring_v.wait_empty(issued_v, guard);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(ring_v.full + issued_v % C::VS, C::NARROW);
          load_tile<DH, W>(s_v + (issued_v % C::VS) * C::NARROW, &p.v, kv, it.row0 + j * W, ring_v.full + issued_v % C::VS);
        }
        ++issued_v;
      }
    }
    pdl_launch_dependents();
    it.len = 0;
    if (ok) ring_i.give(items, it, lane, guard);
  } else if (warp == kMmaWarp) {
    bool ok = true;
    int g = 0;  // tiles so far
    Item it;
    for (int i = 0; ok && ring_i.take(i, it, lane, guard); ++i) {
      const int n = tiles_of(it);
      ok = warp_wait(q_full, items & 1, guard, kSiteMmaFull);
      if (!ok) break;
      ++items;
      // Key tile j of the item at ring position i, its rows of the next sequence cleared.
      auto take_k = [&](int i, int j) {
        if (!ring_k.wait_full(i, guard)) return false;
        if (it.len - j * W < W) clear_rows<DH, W>(s_k + (i % C::KS) * C::NARROW, it.len - j * W, lane);
        return true;
      };
      ok = take_k(g, 0);
      if (!ok) break;
      if (elect_one()) {
        product_rows<DH, W>(tmem + C::S, s_q, s_k + (g % C::KS) * C::NARROW, p.steps);
        tc_commit(s_full);
      }
      __syncwarp();
      ok = ring_v.wait_full(g, guard);
      if (!ok) break;
      if (elect_one()) {
        product_rows<DH, W>(tmem + C::DP, s_do, s_v + (g % C::VS) * C::NARROW, p.steps);
        tc_commit(dp_full);
        tc_commit(ring_v.empty + g % C::VS);
        if (n == 1) tc_commit(q_free);
      }
      __syncwarp();
      for (int j = 0; j < n; ++j, ++g) {
        const uint8_t* k_tile = s_k + (g % C::KS) * C::NARROW;
        ok = warp_wait(p_full, g & 1, guard, kSiteMmaAcc);
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) product_tokens<W, H>(tmem + C::KM, tmem + C::S, k_tile, j > 0, H, p.steps);
        __syncwarp();
        if (j + 1 < n) {
          ok = take_k(g + 1, j + 1);
          if (!ok) break;
          if (elect_one()) {
            product_rows<DH, W>(tmem + C::S, s_q, s_k + ((g + 1) % C::KS) * C::NARROW, p.steps);
            tc_commit(s_full);
          }
          __syncwarp();
        }
        ok = warp_wait(ds_full, g & 1, guard, kSiteMmaAcc);
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
          product_tokens<W, H>(tmem + C::DQ, tmem + C::DP, k_tile, j > 0, H, p.steps);
          if constexpr (FINE) product_tokens<W, H>(tmem + C::DQ, tmem + C::DP + H / 2, k_tile, true, H, p.steps);
          tc_commit(ring_k.empty + g % C::KS);
          if (j + 1 == n) tc_commit(done);
        }
        __syncwarp();
        if (j + 1 < n) {
          ok = ring_v.wait_full(g + 1, guard);
          if (!ok) break;
          if (elect_one()) {
            product_rows<DH, W>(tmem + C::DP, s_do, s_v + ((g + 1) % C::VS) * C::NARROW, p.steps);
            tc_commit(dp_full);
            tc_commit(ring_v.empty + (g + 1) % C::VS);
            if (j + 2 == n) tc_commit(q_free);
          }
          __syncwarp();
        }
      }
    }
  } else {
    const int part = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + C::S + H * part, t_dp = tmem + lanes + C::DP + H * part;
    int g = 0, met = 0;  // tiles; uses of `meet`
    auto meet_all = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      return warp_wait(meet, met++ & 1, guard, kSiteEpilogue);
    };
    bool ok = true;
    for (int i = 0; ok && ring_i.hold(i, guard); ++i) {
      const volatile Item& it = ring_i.held(i);
      const int len = it.len, q0 = it.tile * kRows, qi = q0 + row;
      const int n = ((p.s.causal ? min(len, q0 + kRows) : len) + W - 1) / W;
      const float nl = -p.lse[int64_t(it.head) * p.s.T + it.row0 + min(qi, len - 1)] * kLog2e;
      float delta = 0.f;
      if (n > 1) {
        // delta of 128 / WARPS rows by each warp: eight lanes a row, whole lines of O from memory, dO from its tile. (Asked
        // for before the last item's output, O takes registers that the tiles' loop then lacks: 8 x 2048 tokens, 32 heads
        // of 128, 373 -> 393 us.)
        constexpr int R = kRows / C::WARPS / 4, N = R * (DH / 64);
        uint4 o[N];
#pragma unroll
        for (int x = 0; x < N; ++x) {
          const int y = (warp * R + x % R) * 4 + (lane >> 3), e = (x / R) * 64 + (lane & 7) * 8;
          o[x] = make_uint4(0, 0, 0, 0);
          if (q0 + y < len && e < p.s.dim)
            o[x] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.o.p) + (it.row0 + q0 + y) * p.o.token +
                                                   it.head * p.o.head + e);
        }
        ok = warp_wait(q_full, items & 1, guard, kSiteMmaFull);
        if (!ok) break;
        float sum[R];
#pragma unroll
        for (int x = 0; x < N; ++x) {
          const int y = (warp * R + x % R) * 4 + (lane >> 3);
          const uint4 d = *reinterpret_cast<const uint4*>(s_do + (x / R) * kChunk + y * 128 + (((lane & 7) ^ (y & 7)) << 4));
          sum[x % R] = dot8(o[x], d, x < R ? 0.f : sum[x % R]);
        }
#pragma unroll
        for (int x = 0; x < R; ++x) {
          sum[x] += __shfl_xor_sync(kAll, sum[x], 4);
          sum[x] += __shfl_xor_sync(kAll, sum[x], 2);
          sum[x] += __shfl_xor_sync(kAll, sum[x], 1);
          if ((lane & 7) == 0) s_delta[(warp * R + x) * 4 + (lane >> 3)] = sum[x];
        }
        fence_proxy_async_smem();  // the reads of dO, before the next item's comes there
        ok = meet_all();
        if (!ok) break;
        delta = s_delta[row];
      } else {
        ok = meet_all();  // s_sum is written in the loop: no warp reads the last item's any more
        if (!ok) break;
      }
      ++items;
      float total = 0.f;  // of dS
      for (int j = 0; j < n; ++j, ++g) {
        ok = warp_wait(s_full, g & 1, guard, kSiteMmaFull);
        if (!ok) break;
        tc_fence_after_sync();
        float s[H];
        tmem_ld<H>(t_s, s);
        const uint64_t c2 = pair(p.scale_log2, p.scale_log2), n2 = pair(nl, nl);
#pragma unroll
        for (int e = 0; e < H; e += 2) {
          unpair(fma_pair(pair(s[e], s[e + 1]), c2, n2), s[e], s[e + 1]);
          s[e] = exp2_fast(s[e]);
          s[e + 1] = exp2_fast(s[e + 1]);
        }
        const int k0 = j * W;
        const bool masked = k0 + W > len || (p.s.causal && k0 + W > q0);
        const int end = (p.s.causal ? min(len, qi + 1) : len) - k0 - H * part;  // columns that count
        if (masked) {
#pragma unroll
          for (int e = 0; e < H; ++e) s[e] = e < end ? s[e] : 0.f;
        }
        uint32_t w[H / 2];
#pragma unroll
        for (int e = 0; e < H; e += 2) w[e / 2] = pack_bf16(s[e], s[e + 1]);
        tmem_st(t_s, w);
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        ok = warp_wait(dp_full, g & 1, guard, kSiteMmaFull);
        if (!ok) break;
        tc_fence_after_sync();
        float dp[H];
        tmem_ld<H>(t_dp, dp);
        if (masked) {  // what stands there may be no number
#pragma unroll
          for (int e = 0; e < H; ++e) dp[e] = e < end ? dp[e] : 0.f;
        }
        if (n == 1) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < H; ++e) sum = fmaf(s[e], dp[e], sum);
          s_sum[part * kRows + row] = sum;
          ok = meet_all();
          if (!ok) break;
          delta = row_sum<C::GROUPS>(s_sum, row);
        }
        uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
        const uint64_t d2 = pair(-delta, -delta);
#pragma unroll
        for (int e = 0; e < H; e += 2) {
          const uint64_t ds = mul_pair(pair(s[e], s[e + 1]), add_pair(pair(dp[e], dp[e + 1]), d2));
          sum[(e >> 1) & 1] = add_pair(sum[(e >> 1) & 1], ds);
          unpair(ds, s[e], s[e + 1]);
          w[e / 2] = pack_bf16(s[e], s[e + 1]);
        }
        tmem_st(t_dp, w);
        if constexpr (FINE) {
          rests<H>(s, w);
          tmem_st(t_dp + H / 2, w);
        }
        float x0, x1;
        unpair(add_pair(sum[0], sum[1]), x0, x1);
        total += x0 + x1;
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      if (!ok) break;
      float off = 0.f;  // how far delta is
      if (n > 1) {
        s_sum[part * kRows + row] = total;
        ok = meet_all();
        if (!ok) break;
        off = row_sum<C::GROUPS>(s_sum, row);
      }
      const int64_t row0 = it.row0;
      const int head = it.head;
      ring_i.release(i, lane);
      if (part == 0 && qi < len) p.delta[int64_t(head) * p.s.T + row0 + qi] = delta + off;
      ok = warp_wait(done, (items - 1) & 1, guard, kSiteEpilogue);
      if (!ok) break;
      tc_fence_after_sync();
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.dq.p) + (row0 + qi) * p.dq.token + head * p.dq.head;
#pragma unroll 1
      for (int x = part * 32; x < DH && x < p.s.dim; x += C::GROUPS * 32) {
        float v[32], k[32];
        tmem_ld_32cols(tmem + lanes + C::DQ + x, v);
        tmem_ld_32cols(tmem + lanes + C::KM + x, k);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = fmaf(-off, k[e], v[e]);
        if (qi < len) store_row(dst, v, p.s.scale, x, p.s.dim);
      }
      tc_fence_before_sync();  // both are in registers; the next item's wait for this warp's next P and dS
    }
  }
  __syncthreads();
  if (*abort_flag) {
    if (warp == kLoadWarp && elect_one()) {
      if (items > 0) wait_drain(q_full, (items - 1) & 1, p.wait_ns);
      ring_k.drain(issued_k, p.wait_ns);
      ring_v.drain(issued_v, p.wait_ns);
    }
    if (warp == kMmaWarp && elect_one()) {
      tc_commit(drain);
      wait_drain(drain, 0, p.wait_ns);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TMEM);
  }
}

// ------------------------------------------------------------------ dK, dV

template <int DH, int W>
struct DkvCfg {
  static constexpr uint32_t TILE = DH / 64 * kChunk, NARROW = DH / 64 * W * 128;  // of the keys, of the queries
  static constexpr int QS = DH == 64 ? 4 : 3, DS = DH == 64 ? 4 : 2, RS = QS == 3 ? 2 : 4;
  static constexpr uint32_t S = 0, DP = W, DV = 2 * W, DK = 2 * W + DH;
  static constexpr uint32_t TMEM = 2 * W + 2 * DH <= 256 ? 256 : 512;
  static constexpr int CTAS = TMEM == 256 ? 2 : 1;  // an SM's
  // Columns of a softmax warp: 64 (8 x 2048 tokens, 32 heads of 128: 370 us, with 32 385; 16 heads of 64: 154 and 154).
  static constexpr int COLUMNS = 64, GROUPS = W / COLUMNS, WARPS = 4 * GROUPS;
  // Whether the next pass's tiles are waited for before this pass's P and dS: their rings are deep enough for short heads
  // (8192 tokens, 16 heads of 64: 486 -> 461 us), not for long ones (of 128: 635 -> 643).
  static constexpr bool EARLY = DH == 64;
  static constexpr int THREADS = (WARPS + 2) * 32;
  static constexpr size_t BARS = 8 * (2 * QS + 2 * DS + 2 * RS + 8) + kItemBytes + 8;
  static constexpr size_t SMEM = 2 * TILE + (QS + DS) * NARROW + RS * 2 * W * 4 + BARS;
  static_assert(SMEM <= 227 * 1024 && CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory");
};

// Query tile i: P^T goes over S^T, dS^T over dP^T. The scores of tile i + 1 are
// made while the threads work on dS of tile i, its dP while they work on P of
// tile i + 1.
//
// Few key tiles for many queries (one kv head for all heads, say) would leave SMs
// idle: then an item is one of p.splits runs of a tile's passes, which writes fp32
// sums, and a last kernel adds them in order.
template <int DH, int W, bool FINE>
__global__ void __launch_bounds__(DkvCfg<DH, W>::THREADS, DkvCfg<DH, W>::CTAS)
    dkv_kernel(const __grid_constant__ TcParams p) {
  using C = DkvCfg<DH, W>;
  constexpr int H = C::COLUMNS, kMmaWarp = C::WARPS, kLoadWarp = C::WARPS + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (misaligned(smem, p.status)) return;
  uint8_t* s_k = smem;
  uint8_t* s_v = s_k + C::TILE;
  uint8_t* s_q = s_v + C::TILE;
  uint8_t* s_do = s_q + C::QS * C::NARROW;
  float* s_row = reinterpret_cast<float*>(s_do + C::DS * C::NARROW);  // [RS][2][W]: -lse log2(e), -delta
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_row + C::RS * 2 * W);
  const Ring<C::QS> ring_q{bars, bars + C::QS};
  bars += 2 * C::QS;
  const Ring<C::DS> ring_d{bars, bars + C::DS};
  bars += 2 * C::DS;
  const Ring<C::RS> ring_r{bars, bars + C::RS};
  bars += 2 * C::RS;
  uint64_t* kv_full = bars;
  uint64_t* kv_free = bars + 1;  // the item's S and dP are all made
  uint64_t* s_full = bars + 2;
  uint64_t* p_full = bars + 3;
  uint64_t* dp_full = bars + 4;
  uint64_t* ds_full = bars + 5;
  uint64_t* done = bars + 6;  // an item's dK and dV are there
  uint64_t* drain = bars + 7;
  const ItemRing ring_i(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring_i.empty + kItemSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  if (!fits(smem, C::SMEM, abort_flag, p.status)) return;

  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ring_q.init();
    ring_d.init();
    ring_r.init(32, C::WARPS);
    mbar_init(kv_full, 1);
    mbar_init(kv_free, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, C::WARPS);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, C::WARPS);
    mbar_init(done, 1);
    mbar_init(drain, 1);
    ring_i.init(C::WARPS + 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, C::TMEM);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const WaitGuard guard{abort_flag, p.wait_ns, p.status};
  const int group = p.s.heads / p.s.kv_heads;
  // Passes of an item: the query tiles `first` .. `first` + `per` - 1 of every head of the group, head by head; of these n
  // from head `head`, tile `first` + `x` on. An item's head counts the splits of a kv head.
  struct Passes {
    int first, per, n, head, x;
  };
  auto passes_of = [&](int tile, int split_head, int len) {
    Passes y;
    y.first = p.s.causal ? tile * kRows / W : 0;
    y.per = (len + W - 1) / W - y.first;
    const int kv = split_head / p.splits, split = split_head % p.splits;
    const int64_t all = int64_t(y.per) * group;
    const int begin = static_cast<int>(all * split / p.splits);
    y.n = static_cast<int>(all * (split + 1) / p.splits) - begin;
    y.head = kv * group + begin / y.per;
    y.x = begin % y.per;
    return y;
  };
  int given = 0, items = 0, issued_q = 0, issued_d = 0;  // items, those with passes

  if (warp == kLoadWarp) {
    bool ok = true;
    Item it;
    for (Walk walk(p, p.s.kv_heads * p.splits, kRows, false, lane); ok && walk.next(it);) {
      ok = ring_i.give(given++, it, lane, guard);
      if (!ok) break;
      const Passes ps = passes_of(it.tile, it.head, it.len);
      if (ps.n == 0) continue;
      const int kv = it.head / p.splits;
      ok = items == 0 || warp_wait(kv_free, (items - 1) & 1, guard, kSiteProducer);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
        load_tile<DH>(s_k, &p.k, kv, it.row0 + it.tile * kRows, kv_full);
        load_tile<DH>(s_v, &p.v, kv, it.row0 + it.tile * kRows, kv_full);
      }
      ++items;
      // lse and delta of a tile's queries: they begin on any 4 bytes, so threads copy them, a pass ahead of their store.
      float nl[W / 32], nd[W / 32];
      auto fetch = [&](int h, int x) {
        const int q0 = (ps.first + x) * W;
        const int64_t at = int64_t(h) * p.s.T + it.row0 + q0;
#pragma unroll
        for (int y = 0; y < W / 32; ++y) {
          const int q = y * 32 + lane;
          const bool on = q0 + q < it.len;
          nl[y] = on ? -p.lse[at + q] * kLog2e : 0.f;
          nd[y] = on ? -p.delta[at + q] : 0.f;
        }
      };
      int h = ps.head, x = ps.x;  // head and query tile of pass i
      fetch(h, x);
      for (int i = 0; i < ps.n; ++i) {
        const int64_t row = it.row0 + (ps.first + x) * W;
        ok = TPMLP_DCHECK(h < (kv + 1) * group && (ps.first + x) * W < it.len, p.status, kChkAttnTile);
        if (!ok) {
          *abort_flag = 1;
          break;
        }
        ok = ring_q.wait_empty(issued_q, guard);
        if (!ok) break;
        if (issued_q + 1 != p.withhold && elect_one()) {
          mbar_arrive_expect_tx(ring_q.full + issued_q % C::QS, C::NARROW);
          load_tile<DH, W>(s_q + (issued_q % C::QS) * C::NARROW, &p.q, h, row, ring_q.full + issued_q % C::QS);
        }
        __syncwarp();
        ++issued_q;
        ok = ring_d.wait_empty(issued_d, guard);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(ring_d.full + issued_d % C::DS, C::NARROW);
          load_tile<DH, W>(s_do + (issued_d % C::DS) * C::NARROW, &p.d_o, h, row, ring_d.full + issued_d % C::DS);
        }
        __syncwarp();
        ok = ring_r.wait_empty(issued_d, guard);
        if (!ok) break;
        float* rows = s_row + (issued_d % C::RS) * 2 * W;
#pragma unroll
        for (int y = 0; y < W / 32; ++y) {
          rows[y * 32 + lane] = nl[y];
          rows[W + y * 32 + lane] = nd[y];
        }
        mbar_arrive(ring_r.full + issued_d % C::RS);
        ++issued_d;
        if (++x == ps.per) x = 0, ++h;
        if (i + 1 < ps.n) fetch(h, x);
      }
    }
    pdl_launch_dependents();
    it.len = 0;
    if (ok) ring_i.give(given, it, lane, guard);
  } else if (warp == kMmaWarp) {
    bool ok = true;
    int g = 0;  // passes so far
    Item it;
    for (int i = 0; ok && ring_i.take(i, it, lane, guard); ++i) {
      const Passes ps = passes_of(it.tile, it.head, it.len);
      if (ps.n == 0) continue;
      // Position i of a ring (query tile x), its rows of the next sequence cleared.
      auto take_q = [&](int i, int x) {
        if (!ring_q.wait_full(i, guard)) return false;
        const int rows = it.len - (ps.first + x) * W;
        if (rows < W) clear_rows<DH, W>(s_q + (i % C::QS) * C::NARROW, rows, lane);
        return true;
      };
      auto take_d = [&](int i, int x) {
        if (!ring_d.wait_full(i, guard)) return false;
        const int rows = it.len - (ps.first + x) * W;
        if (rows < W) clear_rows<DH, W>(s_do + (i % C::DS) * C::NARROW, rows, lane);
        return true;
      };
      ok = warp_wait(kv_full, items & 1, guard, kSiteMmaFull) && take_q(g, ps.x);
      if (!ok) break;
      ++items;
      if (elect_one()) {
        product_rows<DH, W>(tmem + C::S, s_k, s_q + (g % C::QS) * C::NARROW, p.steps);
        tc_commit(s_full);
      }
      __syncwarp();
      ok = take_d(g, ps.x);
      if (!ok) break;
      if (elect_one()) {
        product_rows<DH, W>(tmem + C::DP, s_v, s_do + (g % C::DS) * C::NARROW, p.steps);
        tc_commit(dp_full);
        if (ps.n == 1) tc_commit(kv_free);
      }
      __syncwarp();
      int x = ps.x;  // query tile of pass i + 1
      for (int i = 0; i < ps.n; ++i, ++g) {
        if (++x == ps.per) x = 0;
        ok = (!C::EARLY || i + 1 == ps.n || take_q(g + 1, x)) && warp_wait(p_full, g & 1, guard, kSiteMmaAcc);
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
          product_tokens<W, H>(tmem + C::DV, tmem + C::S, s_do + (g % C::DS) * C::NARROW, i > 0, H, p.steps);
          tc_commit(ring_d.empty + g % C::DS);
        }
        __syncwarp();
        if (i + 1 < ps.n) {
          ok = C::EARLY || take_q(g + 1, x);
          if (!ok) break;
          if (elect_one()) {
            product_rows<DH, W>(tmem + C::S, s_k, s_q + ((g + 1) % C::QS) * C::NARROW, p.steps);
            tc_commit(s_full);
          }
          __syncwarp();
        }
        ok = (!C::EARLY || i + 1 == ps.n || take_d(g + 1, x)) && warp_wait(ds_full, g & 1, guard, kSiteMmaAcc);
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
          product_tokens<W, H>(tmem + C::DK, tmem + C::DP, s_q + (g % C::QS) * C::NARROW, i > 0, H, p.steps);
          if constexpr (FINE)
            product_tokens<W, H>(tmem + C::DK, tmem + C::DP + H / 2, s_q + (g % C::QS) * C::NARROW, true, H, p.steps);
          tc_commit(ring_q.empty + g % C::QS);
          if (i + 1 == ps.n) tc_commit(done);
        }
        __syncwarp();
        if (i + 1 < ps.n) {
          ok = C::EARLY || take_d(g + 1, x);
          if (!ok) break;
          if (elect_one()) {
            product_rows<DH, W>(tmem + C::DP, s_v, s_do + ((g + 1) % C::DS) * C::NARROW, p.steps);
            tc_commit(dp_full);
            if (i + 2 == ps.n) tc_commit(kv_free);
          }
          __syncwarp();
        }
      }
    }
  } else {
    const int part = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + C::S + H * part, t_dp = tmem + lanes + C::DP + H * part;
    bool ok = true;
    int g = 0;  // passes so far
    for (int i = 0; ok && ring_i.hold(i, guard); ++i) {
      const volatile Item& it = ring_i.held(i);
      const int len = it.len, k0 = it.tile * kRows, kj = k0 + row;
      const int first = p.s.causal ? k0 : 0;  // a multiple of W
      int q0, n;                              // the first query of this warp's columns; passes
      {
        const Passes ps = passes_of(it.tile, it.head, len);
        q0 = (ps.first + ps.x) * W + H * part;
        n = ps.n;
      }
      for (int left = n; left > 0; --left, ++g) {
        const float* rows = s_row + (g % C::RS) * 2 * W + H * part;
        ok = ring_r.wait_full(g, guard) && warp_wait(s_full, g & 1, guard, kSiteMmaFull);
        if (!ok) break;
        tc_fence_after_sync();
        const uint64_t c2 = pair(p.scale_log2, p.scale_log2);
        float s[H];
        tmem_ld<H>(t_s, s);
#pragma unroll
        for (int e = 0; e < H; e += 4) {
          const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(rows + e);
          unpair(fma_pair(pair(s[e], s[e + 1]), c2, nl.x), s[e], s[e + 1]);
          unpair(fma_pair(pair(s[e + 2], s[e + 3]), c2, nl.y), s[e + 2], s[e + 3]);
#pragma unroll
          for (int y = 0; y < 4; ++y) s[e + y] = exp2_fast(s[e + y]);
        }
        const int begin = p.s.causal ? kj - q0 : 0, end = len - q0;  // columns that count
        const bool masked = end < H || (p.s.causal && q0 < k0 + kRows);
        if (masked) {
#pragma unroll
          for (int e = 0; e < H; ++e) s[e] = e >= begin && e < end ? s[e] : 0.f;
        }
        uint32_t w[H / 2];
#pragma unroll
        for (int e = 0; e < H; e += 2) w[e / 2] = pack_bf16(s[e], s[e + 1]);
        tmem_st(t_s, w);
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        ok = warp_wait(dp_full, g & 1, guard, kSiteMmaFull);
        if (!ok) break;
        tc_fence_after_sync();
        float dp[H];
        tmem_ld<H>(t_dp, dp);
        if (masked) {  // what stands there may be no number
#pragma unroll
          for (int e = 0; e < H; ++e) dp[e] = e >= begin && e < end ? dp[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < H; e += 4) {
          const ulonglong2 nd = *reinterpret_cast<const ulonglong2*>(rows + W + e);
          unpair(mul_pair(pair(s[e], s[e + 1]), add_pair(pair(dp[e], dp[e + 1]), nd.x)), s[e], s[e + 1]);
          unpair(mul_pair(pair(s[e + 2], s[e + 3]), add_pair(pair(dp[e + 2], dp[e + 3]), nd.y)), s[e + 2], s[e + 3]);
          w[e / 2] = pack_bf16(s[e], s[e + 1]);
          w[e / 2 + 1] = pack_bf16(s[e + 2], s[e + 3]);
        }
        tmem_st(t_dp, w);
        if constexpr (FINE) {
          rests<H>(s, w);
          tmem_st(t_dp + H / 2, w);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ds_full);
          mbar_arrive(ring_r.empty + g % C::RS);
        }
        q0 += W;
        if (q0 - H * part >= len) q0 = first + H * part;  // the next head's first
      }
      if (!ok) break;
      const int64_t at = it.row0 + kj;
      const int head = it.head, seq = it.seq;
      ring_i.release(i, lane);
      if (n > 0) {
        ok = warp_wait(done, items & 1, guard, kSiteEpilogue);
        if (!ok) break;
        ++items;
        tc_fence_after_sync();
      }
      const int kv = head / p.splits;
      __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(p.dv.p) + at * p.dv.token + kv * p.dv.head;
      __nv_bfloat16* dk = static_cast<__nv_bfloat16*>(p.dk.p) + at * p.dk.token + kv * p.dk.head;
#pragma unroll 1
      for (int y = part * 32; y < DH && y < p.s.dim; y += C::GROUPS * 32) {
#pragma unroll 1
        for (int z = 0; z < 2; ++z) {  // dV, dK
          float o[32];
          if (n > 0) {
            tmem_ld_32cols(tmem + lanes + (z ? C::DK : C::DV) + y, o);
          } else {  // a split without a pass
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
          if (kj >= len) continue;
          if (p.splits == 1)
            store_row(z ? dk : dv, o, z ? p.s.scale : 1.f, y, p.s.dim);
          else if (part_exists(p, head % p.splits, seq, k0 / kRows, kv))
            store_sums(part_of(p, z, head % p.splits, seq, k0 / kRows, kv, row), o, y, p.s.dim);
        }
      }
      tc_fence_before_sync();  // both are in registers; the next item's wait for this warp's next P and dS
    }
  }
  __syncthreads();
  if (*abort_flag) {
    if (warp == kLoadWarp && elect_one()) {
      if (items > 0) wait_drain(kv_full, (items - 1) & 1, p.wait_ns);
      ring_q.drain(issued_q, p.wait_ns);
      ring_d.drain(issued_d, p.wait_ns);
    }
    if (warp == kMmaWarp && elect_one()) {
      tc_commit(drain);
      wait_drain(drain, 0, p.wait_ns);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TMEM);
  }
}

// dV and dK of a tile of keys as the sums of their splits, in order. Eight elements a thread; blockIdx.y a 256th of theirs.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ TcParams p) {
  pdl_wait();
  const int64_t per = int64_t(p.s.kv_heads) * p.s.batch;
  const int tile = static_cast<int>(blockIdx.x / per), in = static_cast<int>(blockIdx.x % per);
  const int kv = in % p.s.kv_heads, seq = in / p.s.kv_heads;
  int64_t row0;
  const int len = core_sequence(p.s, seq, row0, p.status);
  const int units = p.s.dim / 8, i = blockIdx.y * 256 + threadIdx.x;  // of 2 x 128 x units
  const int z = i / (kRows * units), row = i / units % kRows, e = i % units * 8;
  if (tile * kRows + row >= len || !part_exists(p, p.splits - 1, seq, tile, kv)) return;
  const int64_t at = row0 + tile * kRows + row;
  const float* from = part_of(p, z, 0, seq, tile, kv, row) + e;
  const int64_t step = int64_t(p.s.batch) * p.tiles * p.s.kv_heads * kRows * p.s.dim;
  float sum[8] = {};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s, from += step) {
    const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + 4);
    sum[0] += a.x, sum[1] += a.y, sum[2] += a.z, sum[3] += a.w;
    sum[4] += b.x, sum[5] += b.y, sum[6] += b.z, sum[7] += b.w;
  }
  const HeadsView& v = z ? p.dk : p.dv;
  const float f = z ? p.s.scale : 1.f;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(v.p) + at * v.token + kv * v.head + e) =
      make_uint4(pack_bf16(sum[0] * f, sum[1] * f), pack_bf16(sum[2] * f, sum[3] * f), pack_bf16(sum[4] * f, sum[5] * f),
                 pack_bf16(sum[6] * f, sum[7] * f));
}

// Runs that a key tile's passes are cut into: where the key tiles do not fill the GPU, enough for one and a half items a
// CTA, of four tiles of 128 queries at least. (One sequence, causal, heads of 128, whole -> in runs: 4096 tokens, 32 heads on
// one kv head 1418 -> 209 us, 8192 tokens, 2 on one 186 -> 68; 512 tokens, 8 on one 61 -> 24; 1024 tokens, 4 on 4 22.5 ->
// 23.4. Two runs where the tiles do fill it, for more even CTAs, gain 3 % at 16384 tokens, 8 heads on 2, and lose 60 % at
// 4096, 8 on 8.) The tiles are those that max_seq gives every sequence, as the sums' places are: with max_seq far above the
// lengths there are no runs (8 x 512 tokens, 32 heads of 128 on one kv head: 64 us with max_seq = 512, 211 with 4096).
constexpr int kMaxSplits = 32;
int splits_of(int64_t items, int64_t passes, int ctas) {
  const int64_t full = int64_t(num_sms()) * ctas;
  int64_t n = items < full ? (3 * full + 2 * items - 1) / (2 * items) : 1;
  if (n > passes / 4) n = passes / 4;
  return static_cast<int>(n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n);
}

// ------------------------------------------------------------------ launches

bool heads_map(CUtensorMap* map, const HeadsView& v, int64_t T, int heads, int dim) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(v.head * 2), static_cast<cuuint64_t>(v.token * 2)};
  const cuuint32_t box[3] = {64, 1, 64};
  const cuuint32_t step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <typename C>
cudaError_t params_of(const C& c, TcParams* p) {
  memset(p, 0, sizeof(*p));
  p->s = c.s;
  p->o = c.o;
  p->lse = const_cast<float*>(c.lse);
  p->scale_log2 = c.s.scale * kLog2e;
  p->steps = (c.s.dim + 15) / 16;
  p->withhold = c.withhold;
  p->wait_ns = c.wait_ns;
  p->status = c.status;
  return heads_map(&p->q, c.q, c.s.T, c.s.heads, c.s.dim) && heads_map(&p->k, c.k, c.s.T, c.s.kv_heads, c.s.dim) &&
                 heads_map(&p->v, c.v, c.s.T, c.s.kv_heads, c.s.dim)
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <auto Kernel>
cudaError_t launch(TcParams& p, int rows, int heads, int threads, size_t smem, int ctas, cudaStream_t s) {
  static std::atomic<uint64_t> devices{0};
  p.tiles = (p.s.max_seq + rows - 1) / rows;
  cudaError_t e = allow_smem(Kernel, smem, devices);
  if (e != cudaSuccess) return e;
  p.items = static_cast<uint32_t>(std::min(int64_t(p.tiles) * heads * p.s.batch, int64_t(INT32_MAX)));
  const uint32_t most = static_cast<uint32_t>(num_sms()) * ctas;
  return launch_pdl(Kernel, dim3(p.items < most ? p.items : most), dim3(threads), smem, s, p);
}

template <int DH, int NQ>
cudaError_t launch_fwd(TcParams& p, cudaStream_t s) {
  using C = FwdCfg<DH, NQ>;
  return launch<fwd_kernel<DH, NQ>>(p, NQ * kRows, p.s.heads, C::THREADS, C::SMEM, C::CTAS, s);
}

template <int DH, int W>
cudaError_t launch_dq(TcParams& p, cudaStream_t s) {
  using C = DqCfg<DH, W>;
  return p.s.dim < 64 || p.s.max_seq <= W
             ? launch<dq_kernel<DH, W, true>>(p, kRows, p.s.heads, C::THREADS, C::SMEM, C::CTAS, s)
             : launch<dq_kernel<DH, W, false>>(p, kRows, p.s.heads, C::THREADS, C::SMEM, C::CTAS, s);
}
template <int DH, int W>
cudaError_t launch_dkv(TcParams& p, cudaStream_t s) {
  using C = DkvCfg<DH, W>;
  const int heads = p.s.kv_heads * p.splits;
  cudaError_t e = p.s.max_seq <= W ? launch<dkv_kernel<DH, W, true>>(p, kRows, heads, C::THREADS, C::SMEM, C::CTAS, s)
                                   : launch<dkv_kernel<DH, W, false>>(p, kRows, heads, C::THREADS, C::SMEM, C::CTAS, s);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_pdl(join_kernel, dim3(static_cast<unsigned>(p.items / p.splits), p.s.dim / 8), dim3(256), 0, s, p);
}

}  // namespace

cudaError_t launch_core_forward_tc(const CoreForward& c, cudaStream_t s) {
  TcParams p;
  cudaError_t e = params_of(c, &p);
  if (e != cudaSuccess) return e;
  // Short heads: one tile a CTA and two CTAs an SM. Long ones: two tiles that take turns, but one where the pairs do not
  // fill the GPU (8192 tokens, 2 heads of 128: 96 -> 90 us; 1024 tokens, 4 heads: 22 -> 18.5).
  if (c.s.dim <= 64) return launch_fwd<64, 1>(p, s);
  const int64_t pairs = int64_t((c.s.max_seq + 2 * kRows - 1) / (2 * kRows)) * c.s.heads * c.s.batch;
  return pairs < num_sms() ? launch_fwd<128, 1>(p, s) : launch_fwd<128, 2>(p, s);
}

int core_splits_tc(int64_t batch, int64_t max_seq, int heads, int kv_heads, int dim) {
  const int64_t tiles = (max_seq + kRows - 1) / kRows;
  return splits_of(tiles * kv_heads * batch, tiles * (heads / kv_heads),
                   dim <= 64 ? DkvCfg<64, 64>::CTAS : DkvCfg<128, 128>::CTAS);
}

cudaError_t launch_core_backward_tc(const CoreBackward& c, float* delta, float* part, cudaStream_t s) {
  TcParams p;
  cudaError_t e = params_of(c, &p);
  if (e != cudaSuccess) return e;
  if (!heads_map(&p.d_o, c.d_o, c.s.T, c.s.heads, c.s.dim)) return cudaErrorInvalidValue;
  p.dq = c.dq;
  p.dk = c.dk;
  p.dv = c.dv;
  p.delta = delta;
  p.part = part;
  p.splits = core_splits_tc(c.s.batch, c.s.max_seq, c.s.heads, c.s.kv_heads, c.s.dim);
  // Heads of up to 64 elements: 64 keys (queries) at a time and half of the tensor memory, so that two CTAs share an SM.
  const bool small = c.s.dim <= 64;
  {
    TraceScope trace("attn_core_dq", s);
    e = small ? launch_dq<64, 64>(p, s) : launch_dq<128, 128>(p, s);
  }
  if (e != cudaSuccess) return e;
  TraceScope trace("attn_core_dkv", s);
  return small ? launch_dkv<64, 64>(p, s) : launch_dkv<128, 128>(p, s);
}

}  // namespace tpmlp
