// xent_gemm.cu — the tensor-core products of the cross entropy over the
// vocabulary: logits tiles that never leave the chip, and the products that
// turn their gradient into dX and dW.
//
// A CTA pair (cta_group::2) computes 256 x 256 tiles, three 64 KB stages of
// two 64-deep K blocks filled by TMA, fp32 accumulators in tensor memory (two,
// so that one tile's epilogue runs under the next one's products):
//   every CTA, warp 0 lane 0 : TMA producer of its own 128 + 128 operand rows
//   even CTA, warp 1 lane 0  : issues the pair's MMAs
//   every CTA, warps 4..11   : epilogue, two warps per tensor-memory lane
//                              quarter, each 32 rows x 128 columns
// The logits' epilogues take one exponential per element, 256 x 256 / 2 a CTA
// at 16 a clock: 2048 clocks a tile, which four warps could not hide under
// the 6144 clocks of a K = 768 tile's products once the loads from tensor
// memory, the conversions and the stores are added; eight can.
//
// The tensor core cuts off what an addition to its fp32 accumulator shifts
// out, always towards zero, so the error of a long sum grows with its length
// (measured on the loss, one sum: 8.8e-7 at D = 1024, 1.7e-6 at 2056, 4.1e-6
// at 3496, against 3e-7 to 4e-7 of an fp32 product). Where an fp32 result is
// wanted a long sum is therefore cut into runs, alternating between the two
// accumulators, and the epilogue warps add the runs in registers with
// rounding to nearest: 128 sums a thread, for which the epilogue's two
// warpgroups take registers over from the first one (384 x 168 at launch =
// 128 x 56 + 256 x 224). A run read back keeps the tensor core from its
// accumulators, about 500 clocks when the warps read all of it at once; spread
// over the next run it costs a third of that (T = 8192, D = 4096, V = 128000:
// one sum 4.71 ms, runs of 512 5.30 ms at once and 5.09 ms spread, runs of
// 1024 4.84 ms spread).
//
// The last column of tiles of the gradients' products is as wide as it has to
// be (32 columns up): its MMAs and, of an MN-major operand, its loads shrink
// with it (bf16, T = 4000, V = 32000, D = 1056: dW 199 -> 188, dX 231 -> 219 us;
// fp32, T = 1000, D = 320: dW 140 -> 136, dX 130 -> 132 us). Not so of the
// logits, where V has one such column in hundreds and the widths cost every tile
// (D = 264: 72 -> 77 us).
//
// Waits are bounded; on a timeout the roles of both CTAs leave their loops,
// copies and MMAs in flight are drained and tensor memory is freed.
#include "gemm_common.cuh"
#include "xent_device.cuh"

#include <atomic>
#include <cstring>

namespace tpmlp {

namespace {

constexpr int kXThreads = 384;  // warp 0 TMA, warp 1 MMA, warps 2, 3 idle, warps 4..11 epilogue
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr int kRunsRegsFirst = 56, kRunsRegsEpi = 224;  // registers of a thread of the first four warps, of the epilogue's
constexpr int kRunsRegs = 128 * kRunsRegsFirst + 256 * kRunsRegsEpi;
constexpr int kSub = 2;         // K blocks of a stage
constexpr uint32_t kSubBytes = 128 * BK * 2;
constexpr uint32_t kOutBlock = 32 * 128;  // staging: 32 rows of 128 bytes
constexpr int BN = 256;
// K blocks of a run, at most. Of bf16 data 16, sums of up to 1024 products; 8
// where there is one row of tiles, which waits for W anyway (T = 200, V = 32000,
// D = 1024: 24.6 -> 25.3 us, the losses off by 3.8e-7 in the place of 8.0e-7; T =
// 1000 48.4 -> 52.4). Of fp32 data's high planes 8, where more is wanted; 128 of
// the five other plane pairs, which come first and whose sums are at most 2^-7
// of the sum of magnitudes (cut like the high planes' they made six runs of K =
// 512 instead of two: T = 1000, V = 32001, logits 124 -> 114 us).
constexpr int kRunLong = 16, kRunShort = 8, kRunSmall = 128;
// What is rounded to bf16 afterwards stays one sum up to kWhole K blocks: over N
// additions of 16 products of one sign it loses 1.4 N 2^-24 of itself. dz: 4096
// products, 2.1e-5 of a logit, so 6e-4 of a share of softmax at logits of 30,
// where the rounding of dz is up to 3.9e-3 (uncut, D = 262144 put them off by 9
// %). dX and dW: 65536, 3.4e-4.
constexpr int kWholeGrad = 64, kWholeOut = 1024, kRunOut = 256;
constexpr int kDrainPauseNs = 25;  // per K block of a run, between a warp's reads of it

template <int EPI, bool RUNS>
struct Cfg {
  static constexpr int kOutBlocks = EPI == kXentStats ? 0 : 1;  // staging blocks of an epilogue warp
  static constexpr int STAGES = 3;
  static constexpr uint32_t A_BYTES = kSub * kSubBytes;
  static constexpr uint32_t STAGE_BYTES = 2 * A_BYTES;
  static constexpr uint32_t STAGING = kEpiWarps * kOutBlocks * kOutBlock;
  static constexpr size_t SMEM = 1024 + size_t(STAGES) * STAGE_BYTES + STAGING + 256;
};

struct XParams {
  XentGemm g;
  int k_blocks, kb_per_slice, slices;
  int m_blocks, n_blocks, tiles;
  int run;  // RUNS: K blocks of a run, even
  uint64_t wait_ns;
  int* status;
};

// The plane pairs in the order in which they are added: small terms first, so
// that they are not lost against the large ones. Plane 0 is the high one.
__device__ __forceinline__ void plane_pair(int pairs, int i, int& a, int& b) {
  if (pairs < kXentPairs) {  // A's planes, the small one first
    a = pairs - 1 - i;
    b = 0;
    return;
  }
  // (1,1) (0,2) (2,0) (0,1) (1,0) (0,0)
  constexpr uint32_t kA = 1u | 0u << 4 | 2u << 8 | 0u << 12 | 1u << 16 | 0u << 20;
  constexpr uint32_t kB = 1u | 2u << 4 | 0u << 8 | 1u << 12 | 0u << 16 | 0u << 20;
  a = (kA >> (4 * i)) & 15;
  b = (kB >> (4 * i)) & 15;
}

constexpr float kLog2e = kXentLog2e;

__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, const void* src, int32_t x, int32_t y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_addr(src)), "r"(x), "r"(y)
               : "memory");
}

// Columns of tile column nb: 256, the last one's (kXentOut*) rounded up to 32.
template <int EPI>
__device__ __forceinline__ int tile_width(int nb, int N) {
  return EPI == kXentOutBf16 || EPI == kXentOutF32 ? min(BN, (N - nb * BN + 31) / 32 * 32) : BN;
}

// End of the run that begins at K block q of the `total` of a tile's plane
// pairs. Runs end where stages of kSub = 2 K blocks do: q and `run` are even.
__device__ __forceinline__ int run_end(int q, int total, int pairs, int run) {
  const int small = pairs > 1 ? total / kXentPairs * (kXentPairs - 1) & ~1 : 0;
  return q < small ? min(q + kRunSmall, small) : min(q + run, total);
}

// RUNS: a tile's sum may have several runs; else it has one.
template <int EPI, bool RUNS>
__global__ void __launch_bounds__(kXThreads, 1) xent_gemm_kernel(const __grid_constant__ XParams p) {
  using C = Cfg<EPI, RUNS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::STAGES * C::A_BYTES;
  uint8_t* s_out = smem + C::STAGES * C::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_out + C::STAGING);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t pos = rank & 1u;
  const int cluster = static_cast<int>(cluster_id_x());
  const int nclusters = static_cast<int>(cluster_count_x());

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      // Even CTA: its producer's arrival (and the pair's bytes). The test hook's stage waits for one that never comes.
      mbar_init(full + s, p.g.inject == s + 1 ? 2 : 1);
      mbar_init(empty + s, 1);  // the pair's commit once its MMAs have read the stage
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, 2 * kEpiWarps);  // even CTA: one arrival per epilogue warp of the pair
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before_sync();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();
  const WaitGuard guard{abort_flag, p.wait_ns, p.status};
  const uint32_t abort_addr = smem_addr(const_cast<int*>(abort_flag));
  auto raise_abort_in_cluster = [&]() { st_cluster_u32(map_to_cta(abort_addr, rank ^ 1u), 1u); };
  const TileGrid grid{0, kSharedNone, p.slices, p.m_blocks, p.n_blocks, p.g.group_m};
  // First K block of a slice and their number.
  auto k_first = [&](int slice) { return slice * p.kb_per_slice; };
  auto k_count = [&](int slice) { return min(p.kb_per_slice, p.k_blocks - slice * p.kb_per_slice); };
  bool aborted = false;

  if (warp < kEpiWarp0) {
    if constexpr (RUNS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRunsRegsFirst));
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed = 0, parity_bits = 0;
      const uint64_t pol = l2_policy(1);
      const int mn = p.g.mn_major;
      for (int tile = cluster; !aborted && tile < p.tiles; tile += nclusters) {
        int slice, mb, nb;
        decode_tile(grid, tile, slice, mb, nb);
        if (!tile_ok(grid, p.status, slice, mb, nb)) continue;
        const int m0 = mb * 256 + static_cast<int>(pos) * 128;
        const int width = tile_width<EPI>(nb, p.g.N);  // each CTA brings in half of it
        const int n0 = nb * BN + static_cast<int>(pos) * (width / 2);
        const bool one_chunk = (mn & kMnB) && !(mn & kMnB3d) && width <= 128;
        const uint32_t sub_bytes = kSubBytes + (one_chunk ? kMnChunkBytes : kSubBytes);
        const int kbs = k_count(slice), k0 = k_first(slice);
        const int total = p.g.pairs * kbs;
        int pair = 0, kk = 0, a, b;
        plane_pair(p.g.pairs, 0, a, b);
        for (int q = 0; q < total; q += kSub) {
          if (!wait_bounded(empty + stage, phase ^ 1u, guard, kSiteProducer)) {
            aborted = true;
            break;
          }
          const uint32_t full_lead = map_to_cta(smem_addr(full + stage), 0);
          const int nsub = total - q < kSub ? total - q : kSub;
          if (pos == 0) {
            mbar_arrive_expect_tx(full + stage, 2 * nsub * sub_bytes);  // both CTAs' A and B
            armed |= 1u << stage;
            parity_bits = (parity_bits & ~(1u << stage)) | (phase << stage);
          }
          for (int u = 0; u < nsub; ++u) {
            uint8_t* da = sA + stage * C::A_BYTES + u * kSubBytes;
            uint8_t* db = sB + stage * C::A_BYTES + u * kSubBytes;
            const CUtensorMap* ma = &p.g.map_a[a];
            const CUtensorMap* mbp = &p.g.map_b[b];
            const int kx = (k0 + kk) * BK;
            if (mn & kMnA3d) {
              tma_load_3d_pair_hint(da, ma, 0, kx, m0 / 64, full_lead, pol);
            } else if (mn & kMnA) {
              tma_load_2d_pair_hint(da, ma, m0, kx, full_lead, pol);
              tma_load_2d_pair_hint(da + kMnChunkBytes, ma, m0 + 64, kx, full_lead, pol);
            } else {
              tma_load_2d_pair_hint(da, ma, kx, m0, full_lead, pol);
            }
            if (mn & kMnB3d) {
              tma_load_3d_pair_hint(db, mbp, 0, kx, n0 / 64, full_lead, pol);
            } else if (mn & kMnB) {
              tma_load_2d_pair_hint(db, mbp, n0, kx, full_lead, pol);
              if (!one_chunk) tma_load_2d_pair_hint(db + kMnChunkBytes, mbp, n0 + 64, kx, full_lead, pol);
            } else {
              tma_load_2d_pair_hint(db, mbp, kx, n0, full_lead, pol);
            }
            if (++kk == kbs) {
              kk = 0;
              if (++pair < p.g.pairs) plane_pair(p.g.pairs, pair, a, b);
            }
          }
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (aborted) {
        raise_abort_in_cluster();
        if (pos == 0) {
          for (int s = 0; s < C::STAGES; ++s)
            if (armed >> s & 1u) wait_drain(full + s, (parity_bits >> s) & 1u, p.wait_ns);
        } else {
          // This CTA's copies are counted on the even CTA's barriers; give any
          // copy still in flight time to land before shared memory is released.
          const uint64_t t0 = global_timer_ns();
          while (global_timer_ns() - t0 < 200000ull) {
          }
        }
      }
    }
    if (warp == 1 && lane == 0 && pos == 0) {
      // ---------------- MMA issuer
      const bool a_mn = (p.g.mn_major & kMnA) != 0, b_mn = (p.g.mn_major & kMnB) != 0;
      constexpr uint16_t kPairMask = 0x3;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      for (int tile = cluster; !aborted && tile < p.tiles; tile += nclusters) {
        int slice, mb, nb;
        decode_tile(grid, tile, slice, mb, nb);
        if (!tile_ok(grid, p.status, slice, mb, nb)) continue;
        const int total = p.g.pairs * k_count(slice);
        const uint32_t idesc = idesc_bf16_f32(256, tile_width<EPI>(nb, p.g.N), a_mn, b_mn);
        for (int run = 0, end; !aborted && run < total; run = end) {
          end = RUNS ? run_end(run, total, p.g.pairs, p.run) : total;
          if (!wait_bounded(acc_empty + acc, acc_phase ^ 1u, guard, kSiteMmaAcc)) {
            aborted = true;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
          for (int q = run; q < end; q += kSub) {
            if (!wait_bounded(full + stage, phase, guard, kSiteMmaFull)) {
              aborted = true;
              break;
            }
            tc_fence_after_sync();
            const int nsub = total - q < kSub ? total - q : kSub;
            for (int u = 0; u < nsub; ++u) {
              const uint32_t a0 = smem_addr(sA + stage * C::A_BYTES + u * kSubBytes);
              const uint32_t b0 = smem_addr(sB + stage * C::A_BYTES + u * kSubBytes);
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)
                tc_mma_bf16_pair(d_tmem, operand_desc(a0, k, a_mn), operand_desc(b0, k, b_mn), idesc,
                                 (q != run || (u | k) != 0) ? 1u : 0u);
            }
            tc_commit_pair_multicast(empty + stage, kPairMask);
            if (++stage == C::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (aborted) break;
          tc_commit_pair_multicast(acc_full + acc, kPairMask);
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      if (aborted) {
        raise_abort_in_cluster();
        tc_commit_pair_multicast(drain, static_cast<uint16_t>(1u << rank));
        wait_drain(drain, 0, p.wait_ns);
      }
    }
  } else {
    if constexpr (RUNS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRunsRegsEpi));
    // ---------------- epilogue (warps 4..11 of every CTA)
    const int quarter = warp & 3;         // its tensor-memory lane quarter: rows quarter*32 .. +31 of this CTA's 128
    const int half = (warp - kEpiWarp0) >> 2;     // columns half*128 .. +127 of the tile
    uint8_t* stage_out = s_out + (warp - kEpiWarp0) * C::kOutBlocks * kOutBlock;
    const uint32_t acc_empty_lead = map_to_cta(smem_addr(acc_empty), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    float scale = 1.f, dmax = 0.f;  // kXentOut*: dmax or 1; kXentGrad*: dmax
    if constexpr (EPI == kXentOutBf16 || EPI == kXentOutF32) {
      if (p.g.dmax) scale = warp_dmax(p.g.dmax, lane);
    }
    if constexpr (EPI == kXentGrad || EPI == kXentGradF32) {
      dmax = p.g.rows.rows ? warp_dmax_of_rows(p.g.rows, p.g.V, lane, blockIdx.x == 0 && warp == kEpiWarp0)
                           : warp_dmax(p.g.dmax, lane);
    }
    for (int tile = cluster; tile < p.tiles; tile += nclusters) {
      int slice, mb, nb;
      decode_tile(grid, tile, slice, mb, nb);
      if (!tile_ok(grid, p.status, slice, mb, nb)) continue;
      const int64_t m_warp = int64_t(mb) * 256 + int64_t(pos) * 128 + quarter * 32;
      const int64_t m = m_warp + lane;
      const bool row_ok = m < p.g.M;
      const int nh = nb * BN + half * 128;  // first column of this warp
      // Rows' own values, loaded while the products run.
      int64_t hot = -1;  // the target's column, or none
      float lse2 = 0.f, rs = 0.f;
      // The target's dz / rs = exp(z - lse) - 1, or from the loss, of which it is -(1 - p) = expm1(-loss): where the row
      // is nearly certain, the former has only the digits that lse's rounding leaves (loss 1e-6 at z = 40: none).
      float own = -1.f;
      if constexpr (EPI == kXentStats || EPI == kXentGrad || EPI == kXentGradF32) {
        if (row_ok) {
          const int64_t t = p.g.targets[m];
          const bool counts = t >= 0 && t < p.g.V;
          hot = counts ? t - p.g.col0 : -1;
          if constexpr (EPI != kXentStats) {
            // fp32: lse itself, see below.
            lse2 = EPI == kXentGrad ? p.g.lse[m] * kLog2e : p.g.lse[m];
            if (counts && p.g.loss) own = expm1f(-p.g.loss[m]);
            const float d = p.g.dloss[m];
            rs = counts && d != 0.f ? d / dmax : 0.f;
          }
        }
      }
      const bool work = m_warp < p.g.M && nh < p.g.N;  // warp-uniform
      float run_max = -INFINITY, run_sum = 0.f;  // kXentStats, in units of log2
      // 32 columns of this thread's row, as bf16, into a half of the staging block (128-byte swizzle).
      auto stage_half = [&](int hb, const float (&v)[32]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(stage_out + lane * 128 + (((4 * hb + j) ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                         pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
      };
      // kXentGradF32: the planes of columns nh + c .. + 63, one after the other through the staging block.
      auto store_planes = [&](int c, float (&a)[32], float (&b)[32]) {
        if (!work || nh + c >= p.g.N) return;  // warp-uniform
        if (nh + c + 32 >= p.g.N) {            // finish() left the second half alone
#pragma unroll
          for (int i = 0; i < 32; ++i) b[i] = 0.f;
        }
#pragma unroll
        for (int pl = 0; pl < kXentPlanes; ++pl) {
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
          stage_half(0, a);
          stage_half(1, b);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.g.map_out[pl], stage_out, nh + c, static_cast<int32_t>(m_warp));
            bulk_commit_group();
          }
          if (pl + 1 < kXentPlanes) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              a[i] -= __bfloat162float(__float2bfloat16_rn(a[i]));
              b[i] -= __bfloat162float(__float2bfloat16_rn(b[i]));
            }
          }
        }
      };
      // Columns n0 .. n0+31 of this thread's row.
      auto finish = [&](int c, float (&v)[32]) {
        const int n0 = nh + c;
        if (!work || n0 >= p.g.N) return;  // warp-uniform
        if constexpr (EPI == kXentStats) {
          const int64_t h = hot - n0;
          if (h >= 0 && h < 32) {
            float z = v[0];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              z = h == i ? v[i] : z;
              v[i] = h == i ? -INFINITY : v[i];  // left to the join
            }
            p.g.zt[m] = z;
          }
          if (n0 + 32 > p.g.N) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (n0 + i >= p.g.N) v[i] = -INFINITY;
          }
          // Maximum, then the sum of the chunk's exponentials; the running sum
          // is rescaled once per chunk.
          float mx = v[0];
#pragma unroll
          for (int i = 1; i < 32; ++i) mx = fmaxf(mx, v[i]);
          const float top = fmaxf(run_max, mx * kLog2e);
          const float base = top == -INFINITY ? 0.f : top;  // a row of -inf so far: every term is 0, not NaN
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            s0 += exp2_approx(fmaf(v[i], kLog2e, -base));
            s1 += exp2_approx(fmaf(v[i + 1], kLog2e, -base));
          }
          run_sum = fmaf(run_sum, exp2_approx(run_max - base), s0 + s1);
          run_max = top;
        } else if constexpr (EPI == kXentGrad || EPI == kXentGradF32) {
          // dz = rs (softmax - [target]), rs = dloss / max |dloss|: exactly 0 in rows that do not count and past N.
          // In fp32 the difference comes first and the library's expf follows: lse scaled and rounded
          // would be off by 2^-24 of some 20, the same for the whole row.
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = EPI == kXentGrad ? exp2_approx(fmaf(v[i], kLog2e, -lse2)) : expf(v[i] - lse2);
          const int64_t h = hot - n0;
          if (h >= 0 && h < 32) {
            const float keep = p.g.loss ? 0.f : 1.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = h == i ? fmaf(v[i], keep, own) : v[i];
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = rs != 0.f ? v[i] * rs : 0.f;
          if (n0 + 32 > p.g.N) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (n0 + i >= p.g.N) v[i] = 0.f;
          }
          if constexpr (EPI == kXentGradF32) return;  // stored by store_planes
          const int hb = (c >> 5) & 1;  // half of the 64-column block
          if (hb == 0) {
            if (lane == 0) bulk_wait_group_read<0>();  // the staging block's previous store has read it
            __syncwarp();
          }
          stage_half(hb, v);
          // The block is stored when its second half is in, or when there is none.
          if (hb == 1 || n0 + 32 >= p.g.N) {
            if (hb == 0) {
              float none[32] = {};
              stage_half(1, none);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&p.g.map_out[0], stage_out, n0 - 32 * hb, static_cast<int32_t>(m_warp));
              bulk_commit_group();
            }
          }
        } else if constexpr (EPI == kXentOutBf16) {
          const int hb = (c >> 5) & 1;
          if (hb == 0) {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= scale;
          stage_half(hb, v);
          if (hb == 1 || n0 + 32 >= p.g.N) {  // columns past N are clipped by the store
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&p.g.map_out[0], stage_out, n0 - 32 * hb, static_cast<int32_t>(m_warp));
              bulk_commit_group();
            }
          }
        } else {
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(stage_out + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(__float_as_uint(v[4 * j] * scale), __float_as_uint(v[4 * j + 1] * scale),
                           __float_as_uint(v[4 * j + 2] * scale), __float_as_uint(v[4 * j + 3] * scale));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int32_t row = static_cast<int32_t>(m_warp + slice * p.g.slice_rows);
            if (p.g.add)
              tma_reduce_add_2d(&p.g.map_out[0], stage_out, n0, row);
            else
              tma_store_2d(&p.g.map_out[0], stage_out, n0, row);
            bulk_commit_group();
          }
        }
      };
      // Waits for the accumulator of the tile's next run; false: give up.
      auto acc_ready = [&]() {
        const bool ok = wait_bounded(acc_full + acc, acc_phase, guard, kSiteEpilogue);
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) raise_abort_in_cluster();
          return false;
        }
        tc_fence_after_sync();
        return true;
      };
      // This warp's columns are in registers: hand them back to the MMA issuer.
      auto acc_release = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_lead + 8u * static_cast<uint32_t>(acc));
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      };
      auto t_row = [&](int c) {
        return tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * BN + half * 128 + c);
      };
      if constexpr (RUNS) {
        float sum[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[c][i] = 0.f;
        const int total = p.g.pairs * k_count(slice);
        bool ok = true;
        for (int run = 0, end; (end = run_end(run, total, p.g.pairs, p.run)) < total; run = end) {
          if (!(ok = acc_ready())) break;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c) __nanosleep(kDrainPauseNs * p.run);
            float v[32];
            __syncwarp();
            tmem_ld_32cols(t_row(32 * c), v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c][i] += v[i];
          }
          acc_release();
        }
        if (!ok || !acc_ready()) break;
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32cols_issue(t_row(0), r);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait(r);
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[c][i] += __uint_as_float(r[i]);
          if (c < 3)
            tmem_ld_32cols_issue(t_row(32 * c + 32), r);  // in flight while this chunk is finished
          else
            acc_release();
          finish(32 * c, sum[c]);
          if constexpr (EPI == kXentGradF32) {
            if (c & 1) store_planes(32 * c - 32, sum[c - 1], sum[c]);
          }
          __syncwarp();
        }
      } else {
        if (!acc_ready()) break;
        uint32_t ra[32], rb[32];
        auto values = [&](int c, const uint32_t (&r)[32]) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          finish(c, v);
        };
        __syncwarp();
        tmem_ld_32cols_issue(t_row(0), ra);
        tmem_ld_wait(ra);
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          __syncwarp();
          tmem_ld_32cols_issue(t_row(c + 32), rb);
          values(c, ra);
          __syncwarp();
          tmem_ld_wait(rb);
          if (c + 64 == 128)
            acc_release();
          else
            tmem_ld_32cols_issue(t_row(c + 64), ra);
          values(c + 32, rb);
          if (c + 64 < 128) {
            __syncwarp();
            tmem_ld_wait(ra);
          }
        }
      }
      if constexpr (EPI == kXentStats) {
        if (work && row_ok) p.g.stats[int64_t(nh / kXentPart) * p.g.M + m] = make_float2(run_max, run_sum);
      }
    }
    if constexpr (EPI != kXentStats) {
      if (lane == 0) bulk_wait_group_all();
      __syncwarp();
    }
  }

  tc_fence_before_sync();
  __syncwarp();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <int EPI, bool RUNS>
cudaError_t launch_epi(const XParams& p, cudaStream_t s) {
  using C = Cfg<EPI, RUNS>;
  auto kern = xent_gemm_kernel<EPI, RUNS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::SMEM));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kXThreads, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  static std::atomic<int> max_clusters[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  int cached = max_clusters[dev].load(std::memory_order_relaxed);
  if (!cached) {
    // The epilogue's registers come out of what the block was launched with: with less, setmaxnreg would wait for ever.
    cudaFuncAttributes a;
    if (RUNS && (e = cudaFuncGetAttributes(&a, kern)) != cudaSuccess) return e;
    if (RUNS && a.numRegs * kXThreads < kRunsRegs) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3(2 * (num_sms() / 2), 1, 1);
    int n = 0;
    cfg.numAttrs = 1;  // the query takes the cluster shape only
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    cfg.numAttrs = 2;
    if (e != cudaSuccess) return e;
    cached = n > 0 ? n : 1;
    max_clusters[dev].store(cached, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3(2 * (p.tiles < cached ? p.tiles : cached), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

int xent_slices(int K, int slices) {
  const int kb = (K + BK - 1) / BK;
  const int per = (kb + slices - 1) / slices;
  return (kb + per - 1) / per;
}

cudaError_t launch_xent_gemm(const XentGemm& g, uint64_t wait_ns, cudaStream_t s) {
  XParams p;
  memset(&p, 0, sizeof(p));
  p.g = g;
  p.k_blocks = (g.K + BK - 1) / BK;
  p.kb_per_slice = (p.k_blocks + g.slices - 1) / g.slices;
  p.slices = (p.k_blocks + p.kb_per_slice - 1) / p.kb_per_slice;
  p.m_blocks = (g.M + 255) / 256;
  p.n_blocks = (g.N + BN - 1) / BN;
  const int64_t tiles = int64_t(p.m_blocks) * p.n_blocks * p.slices;
  if (tiles <= 0 || tiles > 0x7fffffff) return cudaErrorInvalidValue;
  p.tiles = static_cast<int>(tiles);
  p.wait_ns = wait_ns;
  p.status = device_status_word();
  if (!p.status) return cudaErrorInvalidSymbol;
  // Runs of a sum longer than one where an fp32 result is wanted (the statistics
  // and all of fp32), and of one longer than `whole` elsewhere, cut evenly.
  const int total = g.pairs * p.kb_per_slice;
  const bool f32 = g.pairs == kXentPairs;
  int most = f32 || g.M <= 256 ? kRunShort : kRunLong, whole = most;
  if (!f32 && g.epi == kXentGrad) most = kRunLong, whole = kWholeGrad;
  if (!f32 && (g.epi == kXentOutBf16 || g.epi == kXentOutF32)) most = kRunOut, whole = kWholeOut;
  const int runs = (total + most - 1) / most;
  p.run = ((total + runs - 1) / runs + 1) / 2 * 2;
  const bool cut = total > whole;
  switch (g.epi) {
    case kXentStats:
      return cut ? launch_epi<kXentStats, true>(p, s) : launch_epi<kXentStats, false>(p, s);
    case kXentGrad:
      return cut ? launch_epi<kXentGrad, true>(p, s) : launch_epi<kXentGrad, false>(p, s);
    case kXentGradF32:
      return launch_epi<kXentGradF32, true>(p, s);  // it holds a warp's columns in registers anyway
    case kXentOutBf16:
      return cut ? launch_epi<kXentOutBf16, true>(p, s) : launch_epi<kXentOutBf16, false>(p, s);
    case kXentOutF32:
      return cut ? launch_epi<kXentOutF32, true>(p, s) : launch_epi<kXentOutF32, false>(p, s);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace tpmlp
