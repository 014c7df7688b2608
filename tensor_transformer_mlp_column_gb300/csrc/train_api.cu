// train_api.cu — C ABI of the two ends of a training step (include/tpmlp.h):
// the cross entropy over the vocabulary, the embedding, and the clipping of
// gradients. Argument checks and workspace sizes; the work is launched by
// xent.cu, embed.cu and clip.cu.
#include "tpmlp.h"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <new>
#include <vector>

#include "internal.h"
#include "trace.h"
#include "train.h"

using namespace tpmlp;

namespace {

#define TRAIN_TRY(expr)                                                                                 \
  do {                                                                                                  \
    cudaError_t e_ = (expr);                                                                            \
    if (e_ != cudaSuccess) return set_error(TPMLP_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(e_));   \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool al16(const void* p) { return aligned(p, 16); }
// Ids and one value a row are loaded one at a time: targets may be ids + 1.
bool al_ids(const int64_t* p) { return aligned(p, 8); }
bool al_rows(const float* p) { return aligned(p, 4); }

uint64_t wait_ns() {
  const char* s = getenv("TPMLP_WAIT_LIMIT_MS");
  long ms = s ? atol(s) : 0;
  if (ms <= 0 || ms > 600000) ms = 4000;
  return static_cast<uint64_t>(ms) * 1000000ull;
}

// The current device is a GB300 (asked once per device) whose status word is known.
int current_sm103() {
  static std::atomic<bool> seen[64] = {};
  int dev = -1, major = 0, minor = 0;
  TRAIN_TRY(cudaGetDevice(&dev));
  if (dev >= 0 && dev < 64 && seen[dev].load(std::memory_order_relaxed)) return TPMLP_OK;
  TRAIN_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
  TRAIN_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
  if (major != 10 || minor != 3)
    return set_error(TPMLP_ERR_DEVICE, "device %d is sm_%d%d; this library is built for sm_103a (GB300)", dev, major,
                     minor);
  if (!device_status_word()) return set_error(TPMLP_ERR_CUDA, "the device status word is not available");
  if (dev >= 0 && dev < 64) seen[dev].store(true, std::memory_order_relaxed);
  return TPMLP_OK;
}

bool known(tpmlp_dtype dt) { return dt == TPMLP_F32 || dt == TPMLP_BF16; }

// Sizes of the cross entropy and of the embedding: ids, rows and tile
// coordinates fit 32 bits, slabs of columns a grid's second dimension.
constexpr int64_t kMaxSize = int64_t(1) << 30, kMaxD = int64_t(1) << 20;
int check_sizes(int64_t T, int64_t D, int64_t V) {
  if (T < 0 || T > kMaxSize) return set_error(TPMLP_ERR_ARG, "T = %lld must be in [0, 2^30]", static_cast<long long>(T));
  if (D < 1 || D > kMaxD || V < 1 || V > kMaxSize)
    return set_error(TPMLP_ERR_ARG, "D = %lld must be in [1, 2^20] and V = %lld in [1, 2^30]", static_cast<long long>(D),
                     static_cast<long long>(V));
  return TPMLP_OK;
}
int check_xent(int64_t T, int64_t D, int64_t V, tpmlp_dtype dt) {
  int rc = check_sizes(T, D, V);
  if (rc) return rc;
  if (!known(dt)) return set_error(TPMLP_ERR_ARG, "unknown dtype %d", int(dt));
  if (D % 8 != 0) return set_error(TPMLP_ERR_SHAPE, "D = %lld must be a multiple of 8", static_cast<long long>(D));
  return TPMLP_OK;
}

// The gradients of one call: the tensors that are not empty, in batches of
// one launch each.
struct ClipCall {
  std::vector<ClipTensors> batches;
  std::vector<int> grids;
  int parts = 0;
};

size_t clip_workspace(int64_t tensors) {
  const int64_t batches = (tensors + kClipBatch - 1) / kClipBatch;
  return static_cast<size_t>(batches < 1 ? 1 : batches) * kClipMaxGrid * sizeof(double);
}

int check_clip(const void* const* grads, const int64_t* counts, const tpmlp_dtype* dts, int n, void* const* out) {
  if (n < 0) return set_error(TPMLP_ERR_ARG, "n = %d must be >= 0", n);
  if (n > 0 && (!grads || !counts || !dts)) return set_error(TPMLP_ERR_ARG, "grads, counts and dts must not be NULL");
  for (int i = 0; i < n; ++i) {
    if (counts[i] < 0) return set_error(TPMLP_ERR_ARG, "counts[%d] = %lld must be >= 0", i, static_cast<long long>(counts[i]));
    if (!known(dts[i])) return set_error(TPMLP_ERR_ARG, "unknown dtype %d of tensor %d", int(dts[i]), i);
    if (counts[i] == 0) continue;
    if (!grads[i] || (out && !out[i])) return set_error(TPMLP_ERR_ARG, "tensor %d has a NULL pointer", i);
    if (!al16(grads[i]) || (out && !al16(out[i])))
      return set_error(TPMLP_ERR_ALIGN, "tensor %d must be 16-byte aligned", i);
  }
  return TPMLP_OK;
}

// A tensor that is written may overlap no other one: two CTAs would scale the
// same elements, once or twice as they happen to run. (A tensor may be its
// own output.)
int check_overlap(const void* const* grads, const int64_t* counts, const tpmlp_dtype* dts, int n, void* const* out) {
  struct Span {
    uintptr_t begin, end;
    bool written;
    int i;
  };
  std::vector<Span> v;
  v.reserve(2 * static_cast<size_t>(n));
  for (int i = 0; i < n; ++i) {
    if (counts[i] == 0) continue;
    const uintptr_t bytes = static_cast<uintptr_t>(counts[i]) * (dts[i] == TPMLP_BF16 ? 2 : 4);
    const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]), b = reinterpret_cast<uintptr_t>(out ? out[i] : grads[i]);
    if (a != b) v.push_back({a, a + bytes, false, i});
    v.push_back({b, b + bytes, true, i});
  }
  std::sort(v.begin(), v.end(), [](const Span& x, const Span& y) { return x.begin < y.begin; });
  uintptr_t end_all = 0, end_written = 0;
  for (const Span& s : v) {
    if (s.begin < (s.written ? end_all : end_written))
      return set_error(TPMLP_ERR_ARG, "tensor %d overlaps another one that the call reads or writes", s.i);
    end_all = std::max(end_all, s.end);
    if (s.written) end_written = std::max(end_written, s.end);
  }
  return TPMLP_OK;
}

ClipCall plan_clip(const void* const* grads, const int64_t* counts, const tpmlp_dtype* dts, int n, void* const* out) {
  ClipCall c;
  for (int i = 0; i < n; ++i) {
    if (counts[i] == 0) continue;
    if (c.batches.empty() || c.batches.back().n == kClipBatch) {
      c.batches.emplace_back();
      c.batches.back().n = 0;
      c.batches.back().first[0] = 0;
    }
    ClipTensors& t = c.batches.back();
    const int k = t.n++;
    t.src[k] = grads[i];
    t.dst[k] = out ? out[i] : const_cast<void*>(grads[i]);
    t.count[k] = counts[i];
    t.bf16[k] = dts[i] == TPMLP_BF16;
    t.first[k + 1] = t.first[k] + clip_chunks(counts[i]);
  }
  for (const ClipTensors& t : c.batches) {
    c.grids.push_back(clip_grid(t.first[t.n]));
    c.parts += c.grids.back();
  }
  return c;
}

int64_t nonempty(const int64_t* counts, int n) {
  int64_t k = 0;
  for (int i = 0; i < n; ++i) k += counts[i] != 0;
  return k;
}

// The squares of every batch into ws.
int run_sumsq(const ClipCall& c, double* part, cudaStream_t s) {
  TraceScope trace("grad_sumsq", s);
  int at = 0;
  for (size_t b = 0; b < c.batches.size(); ++b) {
    TRAIN_TRY(launch_clip_sumsq(c.batches[b], part + at, s));
    at += c.grids[b];
  }
  return TPMLP_OK;
}

int grad_call(const void* const* grads, const int64_t* counts, const tpmlp_dtype* dts, int n, bool clip, float max_norm,
              void* const* out, float* norm, void* ws, size_t ws_bytes, cudaStream_t s) {
  int rc = check_clip(grads, counts, dts, n, out);
  if (rc) return rc;
  if (clip && !(max_norm >= 0.f && std::isfinite(max_norm)))
    return set_error(TPMLP_ERR_ARG, "max_norm = %g must be finite and >= 0", double(max_norm));
  if (!norm || !ws) return set_error(TPMLP_ERR_ARG, "norm and workspace must not be NULL");
  if (!al_rows(norm) || !al16(ws)) return set_error(TPMLP_ERR_ALIGN, "workspace must be 16-byte aligned, norm 4");
  const size_t need = clip_workspace(nonempty(counts, n));
  if (ws_bytes < need) return set_error(TPMLP_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  if (clip && (rc = check_overlap(grads, counts, dts, n, out))) return rc;
  if ((rc = current_sm103())) return rc;
  const ClipCall c = plan_clip(grads, counts, dts, n, out);
  double* part = static_cast<double*>(ws);
  if ((rc = run_sumsq(c, part, s))) return rc;
  if (!clip || c.batches.empty()) {
    TraceScope trace("grad_norm", s);
    TRAIN_TRY(launch_clip_norm(part, c.parts, norm, s));
    return TPMLP_OK;
  }
  TraceScope trace("grad_scale", s);
  for (size_t b = 0; b < c.batches.size(); ++b)
    TRAIN_TRY(launch_clip_scale(c.batches[b], part, c.parts, max_norm, b == 0 ? norm : nullptr, s));
  return TPMLP_OK;
}

int xent_forward(const void* X, const void* W, const int64_t* targets, int64_t T, int64_t D, int64_t V, tpmlp_dtype dt,
                 float* loss, float* lse, void* ws, size_t ws_bytes, uint64_t limit_ns, int inject, cudaStream_t stream) {
  int rc = check_xent(T, D, V, dt);
  if (rc) return rc;
  if (T == 0) return TPMLP_OK;
  if (!X || !W || !targets || !loss || !lse || !ws) return set_error(TPMLP_ERR_ARG, "a required pointer is NULL");
  if (!al16(X) || !al16(W) || !al_ids(targets) || !al_rows(loss) || !al_rows(lse) || !al16(ws))
    return set_error(TPMLP_ERR_ALIGN, "X, W and workspace must be 16-byte aligned, targets 8, loss and lse 4");
  const size_t need = plan_xent(T, D, V, dt == TPMLP_BF16, 0).total;
  if (ws_bytes < need) return set_error(TPMLP_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  if ((rc = current_sm103())) return rc;
  TRAIN_TRY(run_xent_forward(X, W, targets, T, D, V, dt == TPMLP_BF16, loss, lse, ws, device_status_word(), limit_ns,
                             stream, inject));
  return TPMLP_OK;
}

// loss: the forward's, or null.
int xent_backward(const void* X, const void* W, const int64_t* targets, const float* loss, const float* lse,
                  const float* dloss, int64_t T, int64_t D, int64_t V, tpmlp_dtype dt, void* dX, void* dW, void* ws,
                  size_t ws_bytes, cudaStream_t stream) {
  int rc = check_xent(T, D, V, dt);
  if (rc) return rc;
  if (!dW || !al16(dW))
    return set_error(dW ? TPMLP_ERR_ALIGN : TPMLP_ERR_ARG, "dW must not be NULL and must be 16-byte aligned");
  if (T == 0) {
    if ((rc = current_sm103())) return rc;
    TRAIN_TRY(cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * D * (dt == TPMLP_BF16 ? 2 : 4), stream));
    return TPMLP_OK;
  }
  if (!X || !W || !targets || !lse || !dloss || !dX || !ws) return set_error(TPMLP_ERR_ARG, "a required pointer is NULL");
  if (!al16(X) || !al16(W) || !al_ids(targets) || !al_rows(lse) || !al_rows(dloss) || !al16(dX) || !al16(ws))
    return set_error(TPMLP_ERR_ALIGN, "X, W, dX and workspace must be 16-byte aligned, targets 8, lse and dloss 4");
  const size_t need = plan_xent(T, D, V, dt == TPMLP_BF16, 1).total;
  if (ws_bytes < need) return set_error(TPMLP_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  if ((rc = current_sm103())) return rc;
  TRAIN_TRY(run_xent_backward(X, W, targets, loss, lse, dloss, T, D, V, dt == TPMLP_BF16, dX, dW, ws, wait_ns(),
                              stream));
  return TPMLP_OK;
}

}  // namespace

extern "C" {

size_t tpmlp_xent_workspace_bytes(int64_t T, int64_t D, int64_t V, tpmlp_dtype dt, int backward) {
  if (check_xent(T, D, V, dt) || backward < 0 || backward > 1) return 0;
  return T == 0 ? 0 : plan_xent(T, D, V, dt == TPMLP_BF16, backward).total;
}

int tpmlp_xent_forward(const void* X, const void* W, const int64_t* targets, int64_t T, int64_t D, int64_t V,
                       tpmlp_dtype dt, float* loss, float* lse, void* ws, size_t ws_bytes, tpmlp_stream_t stream) {
  return xent_forward(X, W, targets, T, D, V, dt, loss, lse, ws, ws_bytes, wait_ns(), 0, stream);
}

int tpmlp_selftest_xent_stage_timeout(const void* X, const void* W, const int64_t* targets, int64_t T, int64_t D,
                                      int64_t V, tpmlp_dtype dt, float* loss, float* lse, int stage, int limit_ms,
                                      void* ws, size_t ws_bytes, tpmlp_stream_t stream) {
  if (T < 1) return set_error(TPMLP_ERR_ARG, "T = %lld must be >= 1", static_cast<long long>(T));
  if (stage < 1 || stage > 3) return set_error(TPMLP_ERR_ARG, "stage = %d outside 1..3", stage);
  if (limit_ms < 1 || limit_ms > 10000) return set_error(TPMLP_ERR_ARG, "limit_ms = %d outside 1..10000", limit_ms);
  return xent_forward(X, W, targets, T, D, V, dt, loss, lse, ws, ws_bytes, static_cast<uint64_t>(limit_ms) * 1000000ull,
                      stage, stream);
}

int tpmlp_xent_backward(const void* X, const void* W, const int64_t* targets, const float* lse, const float* dloss,
                        int64_t T, int64_t D, int64_t V, tpmlp_dtype dt, void* dX, void* dW, void* ws, size_t ws_bytes,
                        tpmlp_stream_t stream) {
  return xent_backward(X, W, targets, nullptr, lse, dloss, T, D, V, dt, dX, dW, ws, ws_bytes, stream);
}

int tpmlp_xent_backward_saved(const void* X, const void* W, const int64_t* targets, const float* loss, const float* lse,
                              const float* dloss, int64_t T, int64_t D, int64_t V, tpmlp_dtype dt, void* dX, void* dW,
                              void* ws, size_t ws_bytes, tpmlp_stream_t stream) {
  if (T > 0 && !loss) return set_error(TPMLP_ERR_ARG, "loss must not be NULL");
  if (T > 0 && !al_rows(loss)) return set_error(TPMLP_ERR_ALIGN, "loss must be 4-byte aligned");
  return xent_backward(X, W, targets, loss, lse, dloss, T, D, V, dt, dX, dW, ws, ws_bytes, stream);
}

int tpmlp_embed_forward(const void* E, const int64_t* ids, int64_t T, int64_t D, int64_t V, tpmlp_dtype dt, float scale,
                        void* out, tpmlp_stream_t stream) {
  int rc = check_sizes(T, D, V);
  if (rc) return rc;
  if (!known(dt)) return set_error(TPMLP_ERR_ARG, "unknown dtype %d", int(dt));
  if (T == 0) return TPMLP_OK;
  if (!E || !ids || !out) return set_error(TPMLP_ERR_ARG, "E, ids and out must not be NULL");
  if (!al16(E) || !al_ids(ids) || !al16(out)) return set_error(TPMLP_ERR_ALIGN, "E and out must be 16-byte aligned, ids 8");
  if ((rc = current_sm103())) return rc;
  TraceScope trace("embed", stream);
  TRAIN_TRY(launch_embed(E, ids, T, D, V, dt == TPMLP_BF16, scale, out, device_status_word(), stream));
  return TPMLP_OK;
}

size_t tpmlp_embed_workspace_bytes(int64_t T, int64_t D, int64_t V) {
  if (check_sizes(T, D, V) || T == 0) return 0;
  return plan_embed(T, D, V).total;
}

int tpmlp_embed_backward(const void* dout, tpmlp_dtype dout_dt, const int64_t* ids, int64_t T, int64_t D, int64_t V,
                         float scale, void* dE, tpmlp_dtype dE_dt, int accumulate, void* ws, size_t ws_bytes,
                         tpmlp_stream_t stream) {
  int rc = check_sizes(T, D, V);
  if (rc) return rc;
  if (!known(dout_dt) || !known(dE_dt)) return set_error(TPMLP_ERR_ARG, "unknown dtype %d or %d", int(dout_dt), int(dE_dt));
  if (!dE || !al16(dE))
    return set_error(dE ? TPMLP_ERR_ALIGN : TPMLP_ERR_ARG, "dE must not be NULL and must be 16-byte aligned");
  if (T > 0) {
    if (!dout || !ids || !ws) return set_error(TPMLP_ERR_ARG, "dout, ids and workspace must not be NULL");
    if (!al16(dout) || !al_ids(ids) || !al16(ws))
      return set_error(TPMLP_ERR_ALIGN, "dout and workspace must be 16-byte aligned, ids 8");
    const size_t need = plan_embed(T, D, V).total;
    if (ws_bytes < need) return set_error(TPMLP_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  } else if (accumulate) {
    return TPMLP_OK;
  }
  if ((rc = current_sm103())) return rc;
  TRAIN_TRY(launch_embed_grad(dout, dout_dt == TPMLP_BF16, ids, T, D, V, scale, dE, dE_dt == TPMLP_BF16,
                              accumulate != 0, ws, device_status_word(), stream));
  return TPMLP_OK;
}

size_t tpmlp_grad_workspace_bytes(int n) { return n < 0 ? 0 : clip_workspace(n); }

int tpmlp_grad_norm(const void* const* grads, const int64_t* counts, const tpmlp_dtype* dts, int n, float* norm, void* ws,
                    size_t ws_bytes, tpmlp_stream_t stream) {
  try {
    return grad_call(grads, counts, dts, n, false, 0.f, nullptr, norm, ws, ws_bytes, stream);
  } catch (const std::bad_alloc&) {
    return set_error(TPMLP_ERR_ARG, "out of host memory for %d tensors", n);
  }
}

int tpmlp_grad_clip(const void* const* grads, const int64_t* counts, const tpmlp_dtype* dts, int n, float max_norm,
                    void* const* out, float* norm, void* ws, size_t ws_bytes, tpmlp_stream_t stream) {
  try {
    return grad_call(grads, counts, dts, n, true, max_norm, out, norm, ws, ws_bytes, stream);
  } catch (const std::bad_alloc&) {
    return set_error(TPMLP_ERR_ARG, "out of host memory for %d tensors", n);
  }
}

}  // extern "C"
