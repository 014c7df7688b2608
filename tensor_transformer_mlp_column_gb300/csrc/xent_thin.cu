// xent_thin.cu — the products of the cross entropy over the vocabulary with W
// for up to 64 rows of X, on the tensor cores with W's side as the 128 rows of
// a tile and the rows of X (or of dz) as its N = 32 or 64 columns.
//
// With so few rows each product is a pass over W, bound by HBM: 256 x 256
// tiles would multiply mostly nothing, and planes of an fp32 W written to
// memory beforehand would cost more traffic than W. Here W is read once, by
// TMA, in its own type; fp32 tiles are split into their three bf16 planes on
// the way from shared memory to tensor memory, where they are the products'
// first operand.
//
//   logits, dz : A = W [V][D] K-major, B = X planes [T][D], tiles of 128 ids
//   dX^T       : A = W^T (128 columns of W), B = dz planes [T][V], the ids cut
//                into slices, each its own fp32 partial sum [T][D]
//
// One CTA per SM:
//   warp 0       : TMA of W (fp32: tiles of 32 K; bf16: of 64 K, with B)
//   warp 1       : issues the MMAs
//   warp 2       : fp32: TMA of the B planes
//   warps 4..11  : fp32: convert, a thread one row of A; warps 4..7 the first
//                  32 of every 64 K, warps 8..11 the second
//   warps 12..15 : epilogue
// The planes of B lie one below the other as one operand of 3 N rows, and a
// plane of A meets as many of them as matter in one MMA:
//   A_0 x (B_0, B_1, B_2) -> accumulators 0, 1, 2
//   A_1 x (B_0, B_1)      -> accumulators    1, 2
//   A_2 x (B_0)           -> accumulator        2
// so that products of one size share an accumulator, the small ones are not
// cut off against the large sum, and 3 MMAs do what 6 of N = 32 columns did,
// whose cost hardly depends on N. Runs of sums as in xent_gemm.cu: 512 fp32
// products; of bf16 16384 for dX, 1024 for dz and the logits' statistics, there in four
// accumulators by turns (HBM is the bound, and a quarter of the length is a
// quarter of what is cut off). Few rows have no mean over many to hide an error
// in: up to 32 of fp32 256 products (V = 64000, D = 1024: dz 60.6 us with 512,
// 61.8 with 256, 69.9 with 128); of bf16 512, up to two rows 256, with what
// each addition of a run leaves out carried over (the largest error of 64
// losses, T = 1: 2.4e-6 in runs of 1024, 1.4e-6 of 512, 8.6e-7 of 256; V =
// 64000, D = 4096: 98 us without, 100, 103 and 113).
#include "gemm_common.cuh"
#include "xent_device.cuh"

#include <atomic>
#include <climits>
#include <cstring>

namespace tpmlp {

namespace {

constexpr int kTThreads = 512;
constexpr int kConvWarp0 = 4, kConvWarps = 8, kEpiWarp0 = 12;
constexpr uint32_t kRawBytes = 128 * 32 * 4;    // fp32: 128 x 32 of W
constexpr uint32_t kPlaneBytes = 128 * 64 * 2;  // bf16: 128 x 64 of W

enum ThinKind : int { kThinStats = 0, kThinGrad = 1, kThinDx = 2 };

template <bool F32, int N, int KIND>
struct TCfg {
  static constexpr int TURNS = !F32 && KIND == kThinStats ? 4 : 1;
  static constexpr int PL = F32 ? kXentPlanes : 1;                               // planes of A
  static constexpr int PLB = F32 ? kXentPlanes : KIND == kThinDx ? kThinDzPlanes : 1;  // of B
  static constexpr int RAW = F32 ? 8 : 0;                                        // stages of raw W
  static constexpr uint32_t A_BYTES = F32 ? 0 : kPlaneBytes;                     // of A in shared memory
  static constexpr uint32_t B_BYTES = N * 64 * 2;                                // one plane of B, 64 K
  static constexpr uint32_t STAGE = A_BYTES + PLB * B_BYTES;                     // operands of 64 K
  static constexpr int STAGES = F32 ? 3 : STAGE > 24576 ? 6 : 8;
  static constexpr uint32_t ACC = PLB * TURNS * N;                               // columns of the accumulators of a run
  // Two sets, so that a run's epilogue goes on beside the next run; at N = 64
  // of fp32 tensor memory holds one.
  static constexpr int SETS = F32 && N > 32 ? 1 : 2;
  static constexpr uint32_t A_COLS = PL * 32;                                    // fp32: planes of 64 K of A
  static constexpr uint32_t USED = SETS * ACC + (F32 ? STAGES * A_COLS : 0);
  static constexpr uint32_t TMEM = USED <= 64 ? 64 : USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
  static constexpr size_t SMEM = 1024 + size_t(RAW) * kRawBytes + size_t(STAGES) * STAGE + 512;
  static_assert(USED <= 512, "tensor memory");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct TParams {
  XentThin g;
  int tiles_m, slices, kb_per_slice, k_blocks, tiles;
  int run;
  uint64_t wait_ns;
  int* status;
};

// D[tmem] (+)= A[tmem] * B[smem]^T: row i of A in lane i, two K in each 32-bit column.
__device__ __forceinline__ void mma_a_in_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 columns of this warp's lanes.
__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// The reductions of 32 columns over the 32 lanes: lane l ends up with column
// l's. 31 shuffles: each step halves the columns that a lane still holds.
template <bool MAX>
__device__ __forceinline__ float reduce_columns(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
      const float got = __shfl_xor_sync(0xffffffffu, give, o);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}

// Whether `ok` holds in all 128 epilogue threads.
__device__ __forceinline__ bool all_of_epilogue(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

template <bool F32, int N, int KIND>
__global__ void __launch_bounds__(kTThreads, 1) thin_kernel(const __grid_constant__ TParams p) {
  using C = TCfg<F32, N, KIND>;
  constexpr bool MN = KIND == kThinDx;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_stage = smem;                                // [STAGES][planes of A, planes of B]
  uint8_t* s_raw = smem + C::STAGES * C::STAGE;           // [RAW]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_raw + C::RAW * kRawBytes);
  uint64_t* empty = full + C::STAGES;
  uint64_t* raw_full = empty + C::STAGES;
  uint64_t* raw_empty = raw_full + C::RAW;
  uint64_t* acc_full = raw_empty + C::RAW;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ int s_issued, s_arrived[kConvWarps];  // fp32: K blocks of B issued, converted by each warp
  __shared__ int s_target[64];
  __shared__ float s_lse[64], s_rs[64], s_own[64];  // own: as in xent_gemm.cu
  __shared__ float s_ref[4][64], s_sum[4][64], s_base[64];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    // The test hook's stage of W's ring waits for an arrival that never comes.
    auto more = [&](int s) { return p.g.inject == s + 1 ? 1 : 0; };
#pragma unroll 1
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full + s, F32 ? 1 + kConvWarps : 1 + more(s));  // B's (or all) bytes; the converters
      mbar_init(empty + s, 1);                                  // commit of the MMAs that read it
    }
#pragma unroll 1
    for (int s = 0; s < C::RAW; ++s) {
      mbar_init(raw_full + s, 1 + more(s));
      mbar_init(raw_empty + s, kConvWarps / 2);  // one half's warps take a stage
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    for (int w = 0; w < kConvWarps; ++w) s_arrived[w] = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::TMEM);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();
  const WaitGuard guard{abort_flag, p.wait_ns, p.status};
  // Tile -> rows m0 .. of the A side, K blocks k0 .. k0 + kbs.
  auto decode = [&](int tile, int& slice, int& m0, int& k0, int& kbs) {
    slice = tile / p.tiles_m;
    m0 = (tile - slice * p.tiles_m) * 128;
    k0 = slice * p.kb_per_slice;
    kbs = min(p.kb_per_slice, p.k_blocks - k0);
  };
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA of W (and, bf16, of B)
      constexpr int ST = F32 ? C::RAW : C::STAGES;
      uint64_t* f = F32 ? raw_full : full;
      uint64_t* e = F32 ? raw_empty : empty;
      int st = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      const uint64_t keep = l2_policy(1), stream = l2_policy(0);
      for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x) {
        int slice, m0, k0, kbs;
        decode(tile, slice, m0, k0, kbs);
        for (int q = 0; ok && q < kbs * (F32 ? 2 : 1); ++q) {
          if (!(ok = wait_bounded(e + st, phase ^ 1u, guard, kSiteProducer))) break;
          issued |= 1u << st;
          parity = (parity & ~(1u << st)) | (phase << st);
          if constexpr (F32) {
            // Four boxes of 32 x 32, 4 KB each.
            mbar_arrive_expect_tx(f + st, kRawBytes);
            uint8_t* dst = s_raw + st * kRawBytes;
            const int kx = k0 * 64 + q * 32;
            for (int b = 0; b < 4; ++b)
              if constexpr (MN)
                tma_load_2d_hint(dst + b * 4096, &p.g.map_w, m0 + 32 * b, kx, f + st, stream);
              else
                tma_load_2d_hint(dst + b * 4096, &p.g.map_w, kx, m0 + 32 * b, f + st, stream);
          } else {
            mbar_arrive_expect_tx(f + st, C::STAGE);
            uint8_t* dst = s_stage + st * C::STAGE;
            const int kx = (k0 + q) * 64;
            if constexpr (MN) {
              tma_load_2d_hint(dst, &p.g.map_w, m0, kx, f + st, stream);
              tma_load_2d_hint(dst + kMnChunkBytes, &p.g.map_w, m0 + 64, kx, f + st, stream);
            } else {
              tma_load_2d_hint(dst, &p.g.map_w, kx, m0, f + st, stream);
            }
            for (int b = 0; b < C::PLB; ++b)
              tma_load_2d_hint(dst + kPlaneBytes + b * C::B_BYTES, &p.g.map_b[b], kx, 0, f + st, keep);
          }
          if (++st == ST) st = 0, phase ^= 1u;
        }
      }
      if (!ok)
#pragma unroll 1
        for (int s = 0; s < ST; ++s)
          if (issued >> s & 1u) wait_drain(f + s, (parity >> s) & 1u, p.wait_ns);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer
      int st = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x) {
        int slice, m0, k0, kbs;
        decode(tile, slice, m0, k0, kbs);
        for (int r = 0; ok && r < kbs; r += p.run) {
          if (!(ok = wait_bounded(acc_empty + acc, acc_phase ^ 1u, guard, kSiteMmaAcc))) break;
          tc_fence_after_sync();
          const uint32_t d0 = tmem_base + static_cast<uint32_t>(acc) * C::ACC;
          const int end = min(kbs, r + p.run);
          for (int q = r; q < end; ++q) {
            if (!(ok = wait_bounded(full + st, phase, guard, kSiteMmaFull))) break;
            tc_fence_after_sync();
            const uint32_t a0 = smem_addr(s_stage + st * C::STAGE), b0 = a0 + C::A_BYTES;
            const uint32_t a_tmem = tmem_base + C::SETS * C::ACC + st * C::A_COLS;
            // Plane pa of A and the first PLB - pa planes of B.
#pragma unroll
            for (int pa = 0; pa < C::PL; ++pa) {
              const uint32_t idesc = idesc_bf16_f32(128, (C::PLB - pa) * N, MN && !F32 ? 1 : 0, 0);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t accumulate = (C::TURNS == 1 && (pa | k) != 0) || q != r ? 1u : 0u;
                const uint64_t b_desc = operand_desc(b0, k, false);
                if constexpr (F32)
                  mma_a_in_tmem(d0 + pa * N, a_tmem + pa * 32 + k * 8, b_desc, idesc, accumulate);
                else
                  tc_mma_bf16(d0 + (k % C::TURNS) * N, operand_desc(a0, k, MN), b_desc, idesc, accumulate);
              }
            }
            tc_commit(empty + st);
            if (++st == C::STAGES) st = 0, phase ^= 1u;
          }
          if (!ok) break;
          tc_commit(acc_full + acc);
          if (++acc == C::SETS) acc = 0, acc_phase ^= 1u;
        }
      }
      if (!ok) {
        tc_commit(drain);
        wait_drain(drain, 0, p.wait_ns);
      }
    }
  } else if (warp == 2) {
    if (F32 && lane == 0) {
      // ---------------- TMA of the B planes
      int st = 0, issued = 0;
      uint32_t phase = 0;
      const uint64_t keep = l2_policy(1);
      for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x) {
        int slice, m0, k0, kbs;
        decode(tile, slice, m0, k0, kbs);
        for (int q = 0; ok && q < kbs; ++q) {
          if (!(ok = wait_bounded(empty + st, phase ^ 1u, guard, kSiteProducer))) break;
          ++issued;
          mbar_arrive_expect_tx(full + st, C::PLB * C::B_BYTES);
          uint8_t* dst = s_stage + st * C::STAGE;
          for (int b = 0; b < C::PLB; ++b)
            tma_load_2d_hint(dst + b * C::B_BYTES, &p.g.map_b[b], (k0 + q) * 64, 0, full + st, keep);
          if (++st == C::STAGES) st = 0, phase ^= 1u;
        }
      }
      s_issued = issued;
    }
  } else if (warp >= kConvWarp0 && warp < kEpiWarp0) {
    if constexpr (F32) {
      // ---------------- converters: fp32 tiles into planes
      const int quarter = warp & 3, half = (warp - kConvWarp0) >> 2;
      int st = 0, rs = half;  // raw stages alternate between the halves
      uint32_t phase = 0, raw_phase = 0;
      for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x) {
        int slice, m0, k0, kbs;
        decode(tile, slice, m0, k0, kbs);
        for (int q = 0; q < kbs; ++q) {
          ok = __all_sync(0xffffffffu, wait_bounded(raw_full + rs, raw_phase, guard, kSiteMmaFull));
          if (!ok) break;
          // This thread's row of A, 32 K, in shared memory as TMA's swizzle put it.
          const uint8_t* raw = s_raw + rs * kRawBytes + quarter * 4096;
          float f[32];
          if constexpr (MN) {
#pragma unroll
            for (int v = 0; v < 32; ++v)
              f[v] = *reinterpret_cast<const float*>(raw + v * 128 + (((lane >> 2) ^ (v & 7)) << 4) + (lane & 3) * 4);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 x = *reinterpret_cast<const float4*>(raw + lane * 128 + ((c ^ (lane & 7)) << 4));
              f[4 * c] = x.x, f[4 * c + 1] = x.y, f[4 * c + 2] = x.z, f[4 * c + 3] = x.w;
            }
          }
          // TMA writes this stage next: its writes are ordered behind these reads by the fence, not by the barrier alone.
          // (Without it a lane's last 16 bytes came, once in some thousand calls, from the stage's next fill.)
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(raw_empty + rs);
          if ((rs += 2) >= C::RAW) rs = half, raw_phase ^= 1u;
          ok = __all_sync(0xffffffffu, wait_bounded(empty + st, phase ^ 1u, guard, kSiteProducer));
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t to = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + C::SETS * C::ACC + st * C::A_COLS + half * 16;
#pragma unroll
          for (int pl = 0; pl < C::PL; ++pl) {
            uint32_t h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              h[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
              if (pl + 1 < C::PL) {
                f[2 * i] -= __uint_as_float(h[i] << 16);
                f[2 * i + 1] -= __uint_as_float(h[i] & 0xffff0000u);
              }
            }
            tmem_st_16cols(to + pl * 32, h);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(full + st);
            atomicAdd(&s_arrived[warp - kConvWarp0], 1);  // here, not in a register of each thread
          }
          if (++st == C::STAGES) st = 0, phase ^= 1u;
        }
      }
    }
  } else if (warp >= kEpiWarp0) {
    // ---------------- epilogue: lane = row of the tile's quarter, columns = rows of X
    const int quarter = warp & 3, et = threadIdx.x - kEpiWarp0 * 32;
    if constexpr (KIND != kThinDx) {
      float dmax = 0.f;
      if constexpr (KIND == kThinGrad)
        dmax = warp_dmax_of_rows(p.g.rows, p.g.V, lane, blockIdx.x == 0 && warp == kEpiWarp0);
      if (et < 64) {
        const bool in = et < p.g.T;
        const int64_t t = in ? p.g.targets[et] : -1;
        const bool counts = t >= 0 && t < p.g.V;
        s_target[et] = counts ? static_cast<int>(t - p.g.col0) : INT_MIN;  // below 0 too for an earlier piece's
        if constexpr (KIND == kThinGrad) {
          const float d = in ? p.g.dloss[et] : 0.f;
          s_lse[et] = in ? p.g.lse[et] : 0.f;
          s_rs[et] = counts && d != 0.f ? d / dmax : 0.f;
          s_own[et] = in && p.g.loss ? expm1f(-p.g.loss[et]) : -1.f;
        }
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    float run_max = -INFINITY, run_sum = 0.f;  // kThinStats: of row et of X, in units of log2
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x) {
      int slice, m0, k0, kbs;
      decode(tile, slice, m0, k0, kbs);
      // What the additions of runs to `sum` have left out.
      constexpr bool CARRY = !F32 && KIND == kThinStats && N == 32;
      float sum[N / 32][32], rest[CARRY ? 32 : 1];
#pragma unroll
      for (int c = 0; c < N / 32; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[c][i] = 0.f;
#pragma unroll
      for (int i = 0; i < (CARRY ? 32 : 1); ++i) rest[i] = 0.f;
      for (int r = 0; r < kbs; r += p.run) {
        // The four warps go on, or give up, together: they meet at barriers below.
        ok = all_of_epilogue(wait_bounded(acc_full + acc, acc_phase, guard, kSiteEpilogue));
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t t0 = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc) * C::ACC;
#pragma unroll
        for (int c = 0; c < static_cast<int>(C::ACC / 32); ++c) {
          float v[32];
          __syncwarp();
          tmem_ld_32cols(t0 + 32 * c, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if constexpr (CARRY) {
              const float add = v[i] + rest[i], s = sum[0][i] + add;
              rest[i] = fabsf(s) < INFINITY ? add - (s - sum[0][i]) : 0.f;
              sum[0][i] = s;
            } else {
              sum[c % (N / 32)][i] += v[i];
            }
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(acc_empty + acc);
        if (++acc == C::SETS) acc = 0, acc_phase ^= 1u;
      }
      if (!ok) break;
      const int m = m0 + quarter * 32 + lane;  // id, or column of dX
      if constexpr (KIND == kThinDx) {
        if (m < p.g.M) {
          float* out = p.g.part + int64_t(slice) * p.g.part_rows * p.g.M + m;
#pragma unroll
          for (int c = 0; c < N / 32; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i < p.g.T) {
                float* o = out + int64_t(32 * c + i) * p.g.M;
                *o = p.g.add ? *o + sum[c][i] : sum[c][i];
              }
        }
      } else if constexpr (KIND == kThinGrad) {
        if (m < p.g.dz_columns) {
          const float keep = p.g.loss ? 0.f : 1.f;
          // Once for both halves of N = 64: the code of 64 columns in a row does not fit the instruction cache
          // (T = 64, V = 128000, D = 1024, fp32: 158 us, and 124 so).
#pragma unroll 1
          for (int c = 0; c < N / 32; ++c) {
            __nv_bfloat16* dz = p.g.dz + int64_t(32 * c) * p.g.pitch + m;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int t = 32 * c + i;
              if (t < p.g.T) {
                const float z = c == 0 ? sum[0][i] : sum[N / 32 - 1][i], rs = s_rs[t];
                float d = F32 ? expf(z - s_lse[t]) : exp2_approx((z - s_lse[t]) * kXentLog2e);
                if (m == s_target[t]) d = fmaf(d, keep, s_own[t]);
                d = rs != 0.f && m < p.g.M ? d * rs : 0.f;
#pragma unroll
                for (int pl = 0; pl < (F32 ? kXentPlanes : kThinDzPlanes); ++pl) {
                  const __nv_bfloat16 h = __float2bfloat16_rn(d);
                  dz[pl * p.g.plane] = h;
                  d -= __bfloat162float(h);
                }
              }
              dz += p.g.pitch;
            }
          }
        }
      } else {
        // (max, sum of exponentials) of each column over the tile's 128 ids, the target's left to the join.
#pragma unroll
        for (int c = 0; c < N / 32; ++c) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const bool hot = m == s_target[32 * c + i];
            if (hot) {
              p.g.zt[32 * c + i] = sum[c][i];
              if constexpr (CARRY) p.g.zt_rest[i] = rest[i];
            }
            if (hot || m >= p.g.M) sum[c][i] = -INFINITY;
            v[i] = sum[c][i];
          }
          s_ref[quarter][32 * c + lane] = reduce_columns<true>(v, lane);
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        float top_tile = 0.f;
        if (et < N) {
          top_tile = fmaxf(fmaxf(s_ref[0][et], s_ref[1][et]), fmaxf(s_ref[2][et], s_ref[3][et])) * kXentLog2e;
          s_base[et] = top_tile == -INFINITY ? 0.f : top_tile;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int c = 0; c < N / 32; ++c) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = exp2_approx(fmaf(sum[c][i], kXentLog2e, -s_base[32 * c + i]));
          s_sum[quarter][32 * c + lane] = reduce_columns<false>(v, lane);
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (et < N) {
          const float add = (s_sum[0][et] + s_sum[1][et]) + (s_sum[2][et] + s_sum[3][et]);
          const float top = fmaxf(run_max, top_tile);
          const float base = top == -INFINITY ? 0.f : top;
          run_sum = run_sum * exp2_approx(run_max - base) + add * exp2_approx((top_tile == -INFINITY ? 0.f : top_tile) - base);
          run_max = top;
        }
        // The next tile's writes of s_ref, s_base and s_sum each come a barrier or more after their last reads here.
      }
    }
    if constexpr (KIND == kThinStats) {
      if (et < p.g.T) p.g.stats[int64_t(blockIdx.x) * p.g.T + et] = make_float2(run_max, run_sum);
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (F32 && threadIdx.x == 0 && *abort_flag) {
    // B's copies in flight: their stages' barriers lack the converters that gave up, whose arrivals are made here.
#pragma unroll 1
    for (int s = 0; s < C::STAGES; ++s) {
      if (s_issued <= s) break;
      const int last = s_issued - 1 - (s_issued - 1 - s) % C::STAGES;  // the stage's last K block
#pragma unroll 1
      for (int w = 0; w < kConvWarps; ++w)
        if (s_arrived[w] <= last) mbar_arrive(full + s);
      wait_drain(full + s, static_cast<uint32_t>(last / C::STAGES) & 1u, p.wait_ns);
    }
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::TMEM);
  }
}

template <bool F32, int N, int KIND>
cudaError_t launch_kind(const TParams& p, cudaStream_t s) {
  using C = TCfg<F32, N, KIND>;
  auto kern = thin_kernel<F32, N, KIND>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::SMEM));
  if (e != cudaSuccess) return e;
  const int grid = p.tiles < num_sms() ? p.tiles : num_sms();
  return launch_pdl(kern, dim3(grid), dim3(kTThreads), C::SMEM, s, p);
}

template <bool F32, int N>
cudaError_t launch_n(const TParams& p, int kind, cudaStream_t s) {
  return kind == kThinStats  ? launch_kind<F32, N, kThinStats>(p, s)
         : kind == kThinGrad ? launch_kind<F32, N, kThinGrad>(p, s)
                             : launch_kind<F32, N, kThinDx>(p, s);
}

cudaError_t launch_thin(const XentThin& g, int kind, uint64_t wait_ns, cudaStream_t s) {
  TParams p;
  memset(&p, 0, sizeof(p));
  p.g = g;
  p.tiles_m = static_cast<int>((g.M + 127) / 128);
  p.k_blocks = static_cast<int>((g.K + 63) / 64);
  p.slices = g.slices;
  p.kb_per_slice = (p.k_blocks + g.slices - 1) / g.slices;
  p.slices = (p.k_blocks + p.kb_per_slice - 1) / p.kb_per_slice;
  p.tiles = p.tiles_m * p.slices;
  if (g.f32)
    p.run = g.T <= 32 ? 4 : 8;
  else if (kind == kThinStats)
    p.run = g.T <= 2 ? 4 : g.T <= 32 ? 8 : 16;
  else
    p.run = kind == kThinGrad ? 16 : 256;
  p.wait_ns = wait_ns;
  p.status = device_status_word();
  if (!p.status) return cudaErrorInvalidSymbol;
  if (g.T <= 32) return g.f32 ? launch_n<true, 32>(p, kind, s) : launch_n<false, 32>(p, kind, s);
  return g.f32 ? launch_n<true, 64>(p, kind, s) : launch_n<false, 64>(p, kind, s);
}

}  // namespace

int xent_thin_columns(int64_t T) { return T <= 32 ? 32 : 64; }

int xent_thin_parts(int64_t V) {
  const int64_t tiles = (V + 127) / 128;
  return static_cast<int>(tiles < num_sms() ? tiles : num_sms());
}

int xent_thin_slices(int64_t D, int64_t K) {
  const int64_t tiles = (D + 127) / 128, kb = (K + 63) / 64, sms = num_sms();
  // The shortest rounds over the SMs, of slices of at least eight K blocks (V =
  // 64000, D = 4096, one row: ten slices in three rounds 239 us of fp32 and 118
  // of bf16; nine in two 181 and 97).
  int64_t best = kb, best_cost = INT64_MAX;
  for (int64_t s = 1; s == 1 || (s <= kb / 8 && s <= 4 * sms / tiles + 1); ++s) {
    const int64_t per = (kb + s - 1) / s, cost = (tiles * ((kb + per - 1) / per) + sms - 1) / sms * (per + 6);
    if (cost < best_cost) best = per, best_cost = cost;
  }
  return static_cast<int>((kb + best - 1) / best);
}

cudaError_t launch_xent_thin_stats(const XentThin& g, uint64_t wait_ns, cudaStream_t s) {
  return launch_thin(g, kThinStats, wait_ns, s);
}
cudaError_t launch_xent_thin_dz(const XentThin& g, uint64_t wait_ns, cudaStream_t s) {
  return launch_thin(g, kThinGrad, wait_ns, s);
}
cudaError_t launch_xent_thin_dx(const XentThin& g, uint64_t wait_ns, cudaStream_t s) {
  return launch_thin(g, kThinDx, wait_ns, s);
}

}  // namespace tpmlp
