// train.h — kernel launchers of the two ends of a training step: the
// cross entropy over the vocabulary (xent.cu, xent_gemm.cu), the embedding
// and its gradient (embed.cu), and the gradients' global norm and clipping
// (clip.cu). Not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tpmlp {

// What the status word holds when an id (a target or a token) was at or above
// V: its row is left out, as a negative id's is, and the next
// tpmlp_check_status() returns TPMLP_ERR_BOUNDS.
constexpr int kChkTarget = 8;
constexpr int kChkToken = 9;

// ------------------------------------------------------------------ clip.cu

// One launch's worth of tensors, passed by value as a kernel parameter (so a
// captured graph carries its own copy and nothing is copied to the device).
constexpr int kClipBatch = 256;
struct ClipTensors {
  const void* src[kClipBatch];
  void* dst[kClipBatch];
  int64_t count[kClipBatch];       // elements, >= 1
  int64_t first[kClipBatch + 1];   // index of the tensor's first chunk; first[n] = all chunks
  uint8_t bf16[kClipBatch];
  int n;
};
// Chunks of a tensor: the unit of work of one CTA.
int64_t clip_chunks(int64_t count);
// CTAs of a launch over `chunks` chunks (a function of the sizes alone, so the
// order of the sums is too).
int clip_grid(int64_t chunks);
// part[b] = the sum of squares of CTA b's chunks.
constexpr int kClipMaxGrid = 1024;
cudaError_t launch_clip_sumsq(const ClipTensors& t, double* part, cudaStream_t s);
// norm[0] = sqrt(sum of part[0 .. nparts)).
cudaError_t launch_clip_norm(const double* part, int nparts, float* norm, cudaStream_t s);
// dst = min(1, max_norm / (norm + 1e-6)) src; writes norm[0] too when it is given.
cudaError_t launch_clip_scale(const ClipTensors& t, const double* part, int nparts, float max_norm, float* norm,
                              cudaStream_t s);

// ------------------------------------------------------------------ embed.cu

// out[t] = scale * E[ids[t]], zero for a negative id; E and out of one type.
cudaError_t launch_embed(const void* E, const int64_t* ids, int64_t T, int64_t D, int64_t V, int is_bf16, float scale,
                         void* out, int* status, cudaStream_t s);

// Byte offsets of the gradient's scratch.
struct EmbedPlan {
  size_t key[2], pos[2];  // int32 [T] each, twice: the sort's source and destination
  size_t present;         // one bit for each id: whether it occurs
  size_t counts;          // the sort's digit counts
  size_t goes_on;         // a byte for each chunk of sorted entries: whether a long segment begins in it
  size_t part;            // fp32 [2 chunks][D]: the chunks' parts of long segments
  size_t total;
};
EmbedPlan plan_embed(int64_t T, int64_t D, int64_t V);
// dE[v] (+)= scale * sum over t with ids[t] = v of dout[t], in the order of t.
cudaError_t launch_embed_grad(const void* dout, int dout_bf16, const int64_t* ids, int64_t T, int64_t D, int64_t V,
                              float scale, void* dE, int dE_bf16, int accumulate, void* ws, int* status,
                              cudaStream_t s);

// ------------------------------------------------------------------ xent.cu, xent_gemm.cu

// One tensor-core product of the cross entropy (CTA pairs, 256 x 256 tiles):
//   acc[m, n] = sum over the plane pairs (a, b), in order, of
//               sum_k A_a[m, k] B_b[n, k]
// with bf16 operands and fp32 accumulation. bf16 data have one plane and one
// pair; fp32 data are split into three bf16 planes (high, middle, low) and
// take the six pairs whose product is not below fp32 rounding. With slices >
// 1 the K blocks are cut into that many runs, each its own output.
enum XentEpilogue : int {
  kXentStats = 0,    // per row and 128 columns: (max, sum of exponentials) of the logits; the target's logit
  kXentGrad = 1,     // dz, bf16
  kXentGradF32 = 2,  // dz in three bf16 planes
  kXentOutBf16 = 3,  // out bf16 = scale * acc
  kXentOutF32 = 4,   // out fp32 = scale * acc, or (add) out += acc
};
constexpr float kXentLog2e = 1.4426950408889634f;
constexpr int kXentPlanes = 3;
constexpr int kXentPairs = 6;
constexpr int kXentPart = 128;    // columns of one (max, sum) part
constexpr int kXentDmaxParts = 64;
// Up to kXentDmaxRows rows the kernels of dz find the largest |dloss| themselves.
constexpr int kXentDmaxRows = 512;
struct XentDmax {
  const float* dloss;      // [rows]
  const int64_t* targets;  // [rows]
  int rows;                // 0: read it from the parts
  float* out;              // [kXentDmaxParts], for the products
};
struct XentGemm {
  CUtensorMap map_a[kXentPlanes], map_b[kXentPlanes];
  CUtensorMap map_out[kXentPlanes];  // bf16: make_output_map_bf16; fp32: make_output_map_f32, slices stacked by rows
  int pairs;                         // of planes: 1; kThinDzPlanes of A with one of B; kXentPairs
  int M, N, K;
  int slices;                        // >= 1; more than the K blocks allow are not used
  int64_t slice_rows;                // rows between two slices of the output map
  int mn_major;                      // TcMajor bits; kMnB3d only where N is a multiple of 256 (tiles of other widths
                                     // do not begin at its 64-column chunks)
  int group_m;
  int epi;
  int add;                           // kXentOutF32
  int inject;                        // test hook: > 0: that stage (1-based) of every CTA's ring is never complete
  // kXentStats, kXentGrad*
  const int64_t* targets;            // [M]
  int64_t V, col0;                   // all ids; the id of column 0
  float2* stats;                     // [ceil(N / kXentPart)][M]: max in units of log2, sum of 2^(z - max)
  float* zt;                         // [M]: the target's logit
  const float* lse;                  // [M]
  const float* loss;                 // [M] or null: of a target dz from it, see kXentGrad
  const float* dloss;                // [M]
  const float* dmax;                 // [kXentDmaxParts] parts of the largest |dloss|; as the scale of kXentOut* (may be null)
  XentDmax rows;                     // kXentGrad*: in the place of dmax
};
// Slices that K is really cut into when `slices` are asked for.
int xent_slices(int K, int slices);
cudaError_t launch_xent_gemm(const XentGemm& g, uint64_t wait_ns, cudaStream_t s);

// The products with W for up to kXentThinMax rows of X at a time (xent_thin.cu).
constexpr int kXentThinMax = 64;
// Planes of their dz of bf16 data: a single row's gradient of a target would
// carry the rounding of its dz as a whole (up to 2^-8), where those of many rows
// and ids average out, and the products are bound by W either way.
constexpr int kThinDzPlanes = 2;
struct XentThin {
  CUtensorMap map_w;                // W: fp32, make_output_map_f32 (32 x 32 boxes); bf16, make_operand_map (K-major: 128
                                    // rows; for dX: 64 rows)
  CUtensorMap map_b[kXentPlanes];   // planes of X [T][D] or dz [T][V]: make_operand_map, xent_thin_columns(T) rows
  int f32, T;
  int M, K;                         // ids and D; for dX: D and ids
  int slices;                       // dX: runs of ids
  const int64_t* targets;
  int64_t V, col0;                  // all ids; the id of the first row of W
  float2* stats;                    // [xent_thin_parts(M)][T]
  float* zt;
  float* zt_rest;                   // bf16, up to 32 rows: what zt's rounding left out
  const float *lse, *loss, *dloss;  // loss may be null
  XentDmax rows;                    // of all groups: 3 kXentThinMax rows at most
  __nv_bfloat16* dz;                // rows [T][pitch] of planes that are `plane` apart
  int64_t plane, pitch, dz_columns; // of dz's columns dz_columns are written (zeros from M on)
  float* part;                      // dX: rows [T][M] of slices that are part_rows rows apart
  int64_t part_rows;
  int add;                          // dX: add to part
  int inject;                       // test hook, as in XentGemm, of W's ring
};
int xent_thin_columns(int64_t T);
int xent_thin_parts(int64_t V);
int xent_thin_slices(int64_t D, int64_t K);
cudaError_t launch_xent_thin_stats(const XentThin& g, uint64_t wait_ns, cudaStream_t s);
cudaError_t launch_xent_thin_dz(const XentThin& g, uint64_t wait_ns, cudaStream_t s);
cudaError_t launch_xent_thin_dx(const XentThin& g, uint64_t wait_ns, cudaStream_t s);

struct XentPlan {
  bool thin;                  // the products with W by groups of kXentThinMax rows
  bool copy_x, copy_w;        // the products read planes of X, of W (else the data themselves)
  int64_t pitch_x, pitch_w;   // elements from one of their rows to the next
  size_t planes_x, planes_w;  // the planes: [3][T][pitch_x], [3][V][pitch_w] of fp32 data, else one
  size_t stats, zt;           // forward
  size_t dmax, dz, dx, dw;    // backward
  size_t total;
  int64_t piece;              // columns of a piece of the vocabulary (a multiple of 256, or V)
  int64_t dz_pitch;           // columns of dz's rows
  int dz_planes;
  int slices_x, slices_w;     // slices of the dX and dW products
  bool dx_part;               // dX goes through fp32 partial sums
};
XentPlan plan_xent(int64_t T, int64_t D, int64_t V, int is_bf16, int backward);
// inject > 0 (test hook): only the first launch of the logits' product, with that stage never complete.
cudaError_t run_xent_forward(const void* X, const void* W, const int64_t* targets, int64_t T, int64_t D, int64_t V,
                             int is_bf16, float* loss, float* lse, void* ws, int* status, uint64_t wait_ns,
                             cudaStream_t s, int inject = 0);
// loss: as the forward wrote it, or null.
cudaError_t run_xent_backward(const void* X, const void* W, const int64_t* targets, const float* loss, const float* lse,
                              const float* dloss, int64_t T, int64_t D, int64_t V, int is_bf16, void* dX, void* dW,
                              void* ws, uint64_t wait_ns, cudaStream_t s);

}  // namespace tpmlp
