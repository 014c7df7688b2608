// attn_core_api.cu — C ABI of the attention of a training step
// (include/tpmlp.h, "The attention of a training step"): argument checks and
// workspace sizes; the work is launched by attn_core.cu and qk_rope.cu.
#include "tpmlp.h"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>

#include "attn_core.h"
#include "internal.h"

using namespace tpmlp;

namespace {

#define CORE_TRY(expr)                                                                                  \
  do {                                                                                                  \
    cudaError_t e_ = (expr);                                                                            \
    if (e_ != cudaSuccess) return set_error(TPMLP_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(e_));   \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known(tpmlp_dtype dt) { return dt == TPMLP_F32 || dt == TPMLP_BF16; }
int64_t esz(tpmlp_dtype dt) { return dt == TPMLP_BF16 ? 2 : 4; }

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
  CORE_TRY(cudaGetDevice(&dev));
  if (dev >= 0 && dev < 64 && seen[dev].load(std::memory_order_relaxed)) return TPMLP_OK;
  CORE_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
  CORE_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
  if (major != 10 || minor != 3)
    return set_error(TPMLP_ERR_DEVICE, "device %d is sm_%d%d; this library is built for sm_103a (GB300)", dev, major,
                     minor);
  if (!device_status_word()) return set_error(TPMLP_ERR_CUDA, "the device status word is not available");
  if (dev >= 0 && dev < 64) seen[dev].store(true, std::memory_order_relaxed);
  return TPMLP_OK;
}

constexpr int64_t kMaxT = int64_t(1) << 30, kMaxStride = int64_t(1) << 36;
constexpr int kMaxHeads = 4096;

int check_heads(int64_t T, int heads, int kv_heads, int dim, int max_dim, tpmlp_dtype dt) {
  if (!known(dt)) return set_error(TPMLP_ERR_ARG, "unknown dtype %d", int(dt));
  if (T < 0 || T > kMaxT) return set_error(TPMLP_ERR_ARG, "T = %lld must be in [0, 2^30]", static_cast<long long>(T));
  if (heads < 1 || heads > kMaxHeads || kv_heads < 1 || kv_heads > kMaxHeads)
    return set_error(TPMLP_ERR_ARG, "heads = %d and kv_heads = %d must be in [1, %d]", heads, kv_heads, kMaxHeads);
  if (dim < 8 || dim > max_dim || dim % 8 != 0)
    return set_error(TPMLP_ERR_SHAPE, "head_dim = %d must be a multiple of 8 in [8, %d]", dim, max_dim);
  return TPMLP_OK;
}

// The view of tensor number `i` of a call, its strides from the caller's list.
// A stride over a single token or head is not used and becomes a regular one.
int make_view(HeadsView* v, const void* p, const int64_t* strides, int i, const char* name, int64_t T, int heads, int dim,
              tpmlp_dtype dt) {
  if (!p) return set_error(TPMLP_ERR_ARG, "%s must not be NULL", name);
  if (!aligned(p, 16)) return set_error(TPMLP_ERR_ALIGN, "%s must be 16-byte aligned", name);
  int64_t token = strides[2 * i], head = strides[2 * i + 1];
  if (heads == 1) head = dim;
  if (T <= 1) token = dim;
  const int64_t per = 16 / esz(dt);
  if (token < 1 || head < 1 || token > kMaxStride || head > kMaxStride || token % per != 0 || head % per != 0)
    return set_error(TPMLP_ERR_ALIGN, "the strides of %s (token %lld, head %lld) must be positive multiples of %lld elements",
                     name, static_cast<long long>(token), static_cast<long long>(head), static_cast<long long>(per));
  // Rows of heads lie apart: all heads of a token before the next token, or all tokens of a head before the next head.
  const auto span = [dim](int64_t n, int64_t stride) { return static_cast<__int128>(n - 1) * stride + dim; };
  if (!((head >= dim && token >= span(heads, head)) || (token >= dim && head >= span(T, token))))
    return set_error(TPMLP_ERR_ARG, "the strides of %s (token %lld, head %lld) let its rows overlap", name,
                     static_cast<long long>(token), static_cast<long long>(head));
  *v = HeadsView{const_cast<void*>(p), token, head};
  return TPMLP_OK;
}

#define VIEW(dst, ptr, i, name, nheads)                                                                   \
  do {                                                                                                    \
    int rc_ = make_view(&(dst), ptr, strides, i, name, T, nheads, head_dim, dt);                          \
    if (rc_) return rc_;                                                                                  \
  } while (0)

int check_shape(int64_t T, int64_t batch, int64_t max_seq, int heads, int kv_heads, int head_dim, tpmlp_dtype dt) {
  int rc = check_heads(T, heads, kv_heads, head_dim, 128, dt);
  if (rc) return rc;
  if (heads % kv_heads != 0)
    return set_error(TPMLP_ERR_DIVISIBILITY, "heads = %d must be divisible by kv_heads = %d", heads, kv_heads);
  if (batch < 0 || max_seq < 0 || batch > kMaxT || max_seq > T)
    return set_error(TPMLP_ERR_ARG, "batch = %lld must be in [0, 2^30] and max_seq = %lld in [0, T]",
                     static_cast<long long>(batch), static_cast<long long>(max_seq));
  // Tiles of 32 rows: as many as the longest length gives every sequence, but no more than T rows back to back can have.
  const int64_t tiles = std::min((max_seq + 31) / 32 * batch, T / 32 + batch);
  if (tiles > ((int64_t(1) << 31) - 1) / heads || T > (int64_t(1) << 35) / heads)
    return set_error(TPMLP_ERR_ARG, "too many sequences, heads and rows for one call");
  return TPMLP_OK;
}

int check_core(const int64_t* strides, const int32_t* starts, int64_t T, int64_t batch, int64_t max_seq, int heads,
               int kv_heads, int head_dim, float scale, tpmlp_dtype dt) {
  int rc = check_shape(T, batch, max_seq, heads, kv_heads, head_dim, dt);
  if (rc) return rc;
  if (!starts && batch * max_seq != T)
    return set_error(TPMLP_ERR_ARG, "without starts T = %lld must be batch * max_seq = %lld * %lld", static_cast<long long>(T),
                     static_cast<long long>(batch), static_cast<long long>(max_seq));
  if (!(scale > 0.f) || !std::isfinite(scale)) return set_error(TPMLP_ERR_ARG, "scale = %g must be finite and > 0", double(scale));
  if (T > 0 && !strides) return set_error(TPMLP_ERR_ARG, "strides must not be NULL");
  if (!aligned(starts, 4)) return set_error(TPMLP_ERR_ALIGN, "starts must be 4-byte aligned");
  return TPMLP_OK;
}

CoreShape core_shape(const int32_t* starts, int64_t T, int64_t batch, int64_t max_seq, int heads, int kv_heads,
                     int head_dim, float scale, int causal) {
  return CoreShape{starts, T, static_cast<int>(batch), static_cast<int>(max_seq), heads, kv_heads, head_dim, scale,
                   causal != 0};
}

// A call without rows or with max_seq = 0: nothing to compute, but sequences that are given are looked at.
int nothing_to_compute(const CoreShape& s, cudaStream_t stream) {
  if (!s.starts || s.batch == 0) return TPMLP_OK;
  int rc = current_sm103();
  if (rc) return rc;
  CORE_TRY(check_core_sequences(s, device_status_word(), stream));
  return TPMLP_OK;
}

// The load that every CTA withholds (test hook; 0: none), and the limit of a wait.
struct Hook {
  int withhold;
  uint64_t limit_ns;
};

int core_forward(const void* q, const void* k, const void* v, const int64_t* strides, const int32_t* starts,
                            int64_t T, int64_t batch, int64_t max_seq, int heads, int kv_heads, int head_dim, float scale,
                            int causal, tpmlp_dtype dt, void* o, float* lse, Hook hook, cudaStream_t stream) {
  int rc = check_core(strides, starts, T, batch, max_seq, heads, kv_heads, head_dim, scale, dt);
  if (rc) return rc;
  const CoreShape shape = core_shape(starts, T, batch, max_seq, heads, kv_heads, head_dim, scale, causal);
  if (T == 0 || batch == 0 || max_seq == 0) return nothing_to_compute(shape, stream);
  CoreForward c{};
  VIEW(c.q, q, 0, "q", heads);
  VIEW(c.k, k, 1, "k", kv_heads);
  VIEW(c.v, v, 2, "v", kv_heads);
  VIEW(c.o, o, 3, "o", heads);
  if (!lse || !aligned(lse, 4)) return set_error(lse ? TPMLP_ERR_ALIGN : TPMLP_ERR_ARG, "lse must not be NULL and 4-byte aligned");
  if ((rc = current_sm103())) return rc;
  c.s = shape;
  c.lse = lse;
  c.bf16 = dt == TPMLP_BF16;
  c.withhold = hook.withhold;
  c.wait_ns = hook.limit_ns;
  c.status = device_status_word();
  CORE_TRY(run_core_forward(c, stream));
  return TPMLP_OK;
}

int core_backward(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* d_o,
                             const int64_t* strides, const int32_t* starts, int64_t T, int64_t batch, int64_t max_seq,
                             int heads, int kv_heads, int head_dim, float scale, int causal, tpmlp_dtype dt, void* dq,
                             void* dk, void* dv, void* ws, size_t ws_bytes, Hook hook, cudaStream_t stream) {
  int rc = check_core(strides, starts, T, batch, max_seq, heads, kv_heads, head_dim, scale, dt);
  if (rc) return rc;
  const CoreShape shape = core_shape(starts, T, batch, max_seq, heads, kv_heads, head_dim, scale, causal);
  if (T == 0 || batch == 0 || max_seq == 0) return nothing_to_compute(shape, stream);
  CoreBackward c{};
  VIEW(c.q, q, 0, "q", heads);
  VIEW(c.k, k, 1, "k", kv_heads);
  VIEW(c.v, v, 2, "v", kv_heads);
  VIEW(c.o, o, 3, "o", heads);
  VIEW(c.d_o, d_o, 4, "do", heads);
  VIEW(c.dq, dq, 5, "dq", heads);
  VIEW(c.dk, dk, 6, "dk", kv_heads);
  VIEW(c.dv, dv, 7, "dv", kv_heads);
  if (!lse || !ws) return set_error(TPMLP_ERR_ARG, "lse and workspace must not be NULL");
  if (!aligned(lse, 4) || !aligned(ws, 16)) return set_error(TPMLP_ERR_ALIGN, "workspace must be 16-byte aligned, lse 4");
  const size_t need = core_backward_workspace(T, batch, max_seq, heads, kv_heads, head_dim, dt == TPMLP_BF16);
  if (ws_bytes < need) return set_error(TPMLP_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  if ((rc = current_sm103())) return rc;
  c.s = shape;
  c.lse = lse;
  c.bf16 = dt == TPMLP_BF16;
  c.ws = ws;
  c.withhold = hook.withhold;
  c.wait_ns = hook.limit_ns;
  c.status = device_status_word();
  CORE_TRY(run_core_backward(c, stream));
  return TPMLP_OK;
}

// f / (2 pi) modulo 1 as a 64-bit binary fraction, off by less than 2^-64 for |f| up to 2^40: the quotient as the sum of two
// doubles, 1 / (2 pi) being two (together off by 2^-110), each without its whole part, which is taken off exactly.
uint64_t turn_of(double f) {
  const double inv = 0x1.45f306dc9c883p-3, inv_rest = -0x1.6b01ec5417056p-57, unit = 18446744073709551616.0;
  const volatile double rounded = f * inv;  // volatile: the product is not to be fused with what follows
  const double product = rounded, rest = std::fma(f, inv_rest, std::fma(f, inv, -product));
  const double x = (product - std::rint(product)) * unit, y = (rest - std::rint(rest)) * unit;  // each at most 2^63
  const double whole = std::floor(x);
  return static_cast<uint64_t>(static_cast<__int128>(whole) + static_cast<__int128>(std::rint((x - whole) + y)));
}

// Both forms of the rotation: dy, dq.. are the backward's. strides: q, k, (dyq, dyk,) and the two outputs.
int qk_rope(int backward, const void* dyq, const void* dyk, const void* q, const void* k, const int64_t* strides,
            const void* wq, const void* wk, float eps, const int64_t* pos, const double* freqs, const uint8_t* axis,
            int64_t T, int heads, int kv_heads, int head_dim, int rot, int axes, int interleaved, tpmlp_dtype dt, void* yq,
            void* yk, float* dwq, float* dwk, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = check_heads(T, heads, kv_heads, head_dim, kRopeMaxDim, dt);
  if (rc) return rc;
  if (rot < 0 || rot > head_dim || rot % 8 != 0)
    return set_error(TPMLP_ERR_SHAPE, "rot = %d must be a multiple of 8 in [0, head_dim]", rot);
  if (axes < 1 || axes > 8) return set_error(TPMLP_ERR_ARG, "axes = %d must be in [1, 8]", axes);
  if (!wq != !wk) return set_error(TPMLP_ERR_ARG, "wq and wk must both be given or both be NULL");
  if (wq && (!(eps >= 0.f) || !std::isfinite(eps))) return set_error(TPMLP_ERR_ARG, "eps = %g must be finite and >= 0", double(eps));
  if (!aligned(wq, 16) || !aligned(wk, 16)) return set_error(TPMLP_ERR_ALIGN, "wq and wk must be 16-byte aligned");
  RopeCall c{};
  if (rot > 0 && !freqs) return set_error(TPMLP_ERR_ARG, "freqs must not be NULL");
  for (int i = 0; i < rot / 2; ++i) {
    if (!std::isfinite(freqs[i])) return set_error(TPMLP_ERR_ARG, "freqs[%d] must be finite", i);
    if (axis && axis[i] >= axes) return set_error(TPMLP_ERR_ARG, "axis[%d] = %d must be below axes = %d", i, int(axis[i]), axes);
    c.s.turn[i] = turn_of(freqs[i]);
    c.s.axis[i] = axis ? axis[i] : 0;
  }
  if (backward && wq && (!dwq || !dwk || !aligned(dwq, 4) || !aligned(dwk, 4)))
    return set_error(!dwq || !dwk ? TPMLP_ERR_ARG : TPMLP_ERR_ALIGN, "dwq and dwk must not be NULL and 4-byte aligned");
  c.s.T = T;
  c.s.heads[0] = heads;
  c.s.heads[1] = kv_heads;
  c.s.dim = head_dim;
  c.s.rot = rot;
  c.s.interleaved = interleaved != 0;
  c.s.eps = eps;
  c.s.pos = pos;
  c.backward = backward;
  c.w[0] = wq;
  c.w[1] = wk;
  c.dw[0] = dwq;
  c.dw[1] = dwk;
  c.ws = ws;
  c.bf16 = dt == TPMLP_BF16;
  if (T == 0 && !(backward && wq)) return TPMLP_OK;
  if (T > 0) {
    if (!strides) return set_error(TPMLP_ERR_ARG, "strides must not be NULL");
    VIEW(c.x[0], q, 0, "q", heads);
    VIEW(c.x[1], k, 1, "k", kv_heads);
    const int out = backward ? 4 : 2;
    if (backward) {
      VIEW(c.dy[0], dyq, 2, "dyq", heads);
      VIEW(c.dy[1], dyk, 3, "dyk", kv_heads);
    }
    VIEW(c.y[0], yq, out, backward ? "dq" : "yq", heads);
    VIEW(c.y[1], yk, out + 1, backward ? "dk" : "yk", kv_heads);
    if (rot > 0 && !pos) return set_error(TPMLP_ERR_ARG, "pos must not be NULL");
    if (!aligned(pos, 8)) return set_error(TPMLP_ERR_ALIGN, "pos must be 8-byte aligned");
    if (backward && wq) {
      if (!ws) return set_error(TPMLP_ERR_ARG, "workspace must not be NULL");
      if (!aligned(ws, 16)) return set_error(TPMLP_ERR_ALIGN, "workspace must be 16-byte aligned");
      const size_t need = rope_backward_workspace(T, heads, kv_heads, head_dim);
      if (ws_bytes < need) return set_error(TPMLP_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    }
  }
  for (int i = 0; T > 0 && i < 2; ++i)
    for (const HeadsView* in : {&c.x[i], &c.dy[i]})
      if (in->p == c.y[i].p && (in->token != c.y[i].token || in->head != c.y[i].head))
        return set_error(TPMLP_ERR_ARG, "an output in the place of its input must have the input's strides");
  if ((rc = current_sm103())) return rc;
  c.status = device_status_word();
  CORE_TRY(run_qk_rope(c, stream));
  return TPMLP_OK;
}

}  // namespace

extern "C" {

int tpmlp_qk_rope_forward(const void* q, const void* k, const int64_t* strides, const void* wq, const void* wk, float eps,
                          const int64_t* pos, const double* freqs, const uint8_t* axis, int64_t T, int heads, int kv_heads,
                          int head_dim, int rot, int axes, int interleaved, tpmlp_dtype dt, void* yq, void* yk,
                          tpmlp_stream_t stream) {
  return qk_rope(0, nullptr, nullptr, q, k, strides, wq, wk, eps, pos, freqs, axis, T, heads, kv_heads, head_dim, rot, axes,
                 interleaved, dt, yq, yk, nullptr, nullptr, nullptr, 0, stream);
}

size_t tpmlp_qk_rope_workspace_bytes(int64_t T, int heads, int kv_heads, int head_dim) {
  return check_heads(T, heads, kv_heads, head_dim, kRopeMaxDim, TPMLP_F32) ? 0
                                                                           : rope_backward_workspace(T, heads, kv_heads, head_dim);
}

int tpmlp_qk_rope_backward(const void* dyq, const void* dyk, const void* q, const void* k, const int64_t* strides,
                           const void* wq, const void* wk, float eps, const int64_t* pos, const double* freqs,
                           const uint8_t* axis, int64_t T, int heads, int kv_heads, int head_dim, int rot, int axes,
                           int interleaved, tpmlp_dtype dt, void* dq, void* dk, float* dwq, float* dwk, void* ws,
                           size_t ws_bytes, tpmlp_stream_t stream) {
  return qk_rope(1, dyq, dyk, q, k, strides, wq, wk, eps, pos, freqs, axis, T, heads, kv_heads, head_dim, rot, axes,
                 interleaved, dt, dq, dk, dwq, dwk, ws, ws_bytes, stream);
}

int tpmlp_attn_core_forward(const void* q, const void* k, const void* v, const int64_t* strides, const int32_t* starts,
                            int64_t T, int64_t batch, int64_t max_seq, int heads, int kv_heads, int head_dim, float scale,
                            int causal, tpmlp_dtype dt, void* o, float* lse, tpmlp_stream_t stream) {
  return core_forward(q, k, v, strides, starts, T, batch, max_seq, heads, kv_heads, head_dim, scale, causal, dt, o, lse,
                      Hook{0, wait_ns()}, stream);
}

size_t tpmlp_attn_core_workspace_bytes(int64_t T, int64_t batch, int64_t max_seq, int heads, int kv_heads, int head_dim,
                                       tpmlp_dtype dt) {
  if (check_shape(T, batch, max_seq, heads, kv_heads, head_dim, dt)) return 0;
  return core_backward_workspace(T, batch, max_seq, heads, kv_heads, head_dim, dt == TPMLP_BF16);
}

int tpmlp_attn_core_backward(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* d_o,
                             const int64_t* strides, const int32_t* starts, int64_t T, int64_t batch, int64_t max_seq,
                             int heads, int kv_heads, int head_dim, float scale, int causal, tpmlp_dtype dt, void* dq,
                             void* dk, void* dv, void* ws, size_t ws_bytes, tpmlp_stream_t stream) {
  return core_backward(q, k, v, o, lse, d_o, strides, starts, T, batch, max_seq, heads, kv_heads, head_dim, scale, causal, dt,
                       dq, dk, dv, ws, ws_bytes, Hook{0, wait_ns()}, stream);
}

int tpmlp_selftest_attn_core_timeout(const void* q, const void* k, const void* v, void* o, float* lse, const void* d_o,
                                     int64_t T, int heads, int head_dim, void* dq, void* dk, void* dv, void* ws,
                                     size_t ws_bytes, int backward, int load, int limit_ms, tpmlp_stream_t stream) {
  if (load < 1) return set_error(TPMLP_ERR_ARG, "load = %d must be >= 1", load);
  if (limit_ms < 1 || limit_ms > 10000) return set_error(TPMLP_ERR_ARG, "limit_ms = %d outside 1..10000", limit_ms);
  if (T < 1) return set_error(TPMLP_ERR_ARG, "T = %lld must be >= 1", static_cast<long long>(T));
  int64_t strides[16];
  for (int i = 0; i < 8; ++i) strides[2 * i] = int64_t(heads) * head_dim, strides[2 * i + 1] = head_dim;
  const Hook hook{load, static_cast<uint64_t>(limit_ms) * 1000000ull};
  const float scale = 1.f / sqrtf(static_cast<float>(head_dim));
  return backward ? core_backward(q, k, v, o, lse, d_o, strides, nullptr, T, 1, T, heads, heads, head_dim, scale, 0,
                                  TPMLP_BF16, dq, dk, dv, ws, ws_bytes, hook, stream)
                  : core_forward(q, k, v, strides, nullptr, T, 1, T, heads, heads, head_dim, scale, 0, TPMLP_BF16, o, lse,
                                 hook, stream);
}

}  // extern "C"
