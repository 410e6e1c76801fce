// api.cu -- the extern "C" boundary of libgdn_gb300.so: host-side validation,
// workspace sizing, dispatch to the kernels, and error reporting.
//
// Every check runs before anything is launched, so a rejected call leaves all
// device memory untouched ("Add request-owned eight-way MTP serving for Qwen
// 35B", Clean-install public launch verification: an incomplete launch
// contract fails before any work; "MTP inference: review and commit
// structure", Review fixes: grouped replay checks all inputs before combining
// layers).
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <cmath>
#include <initializer_list>
#include <mutex>
#include <string>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include "gdn_common.cuh"
#include "kv4.cuh"
#include "sample.cuh"

using namespace gdn;

namespace {

thread_local std::string t_err;

// An NVTX range around each entry point (what a profiler timeline shows as
// the call's host-side extent; a no-op unless a tool is attached).
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange &) = delete;
  NvtxRange &operator=(const NvtxRange &) = delete;
};

int fail(int code, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_err = buf;
  return code;
}

int ok() {
  t_err.clear();
  return GDN_OK;
}

constexpr int kMaxPrefillLen = 1 << 20;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_dims(const gdn_dims *d) {
  if (!d) return fail(GDN_ERR_INVALID_ARG, "dims is NULL");
  if (d->B < 0 || d->B > 65535) return fail(GDN_ERR_UNSUPPORTED, "B=%d outside [0, 65535]", d->B);
  if (d->T < 1 || d->T > d->T_max || d->T_max > kMaxT)
    return fail(GDN_ERR_UNSUPPORTED, "need 1 <= T (%d) <= T_max (%d) <= %d", d->T, d->T_max, kMaxT);
  if (d->H_k < 1 || d->H_v < 1 || d->H_v % d->H_k != 0 || d->H_v > 65535)
    return fail(GDN_ERR_UNSUPPORTED, "need H_k >= 1 and H_v (%d) a multiple of H_k (%d), H_v <= 65535",
                d->H_v, d->H_k);
  if (d->d_k != d->d_v || (d->d_k != 32 && d->d_k != 64 && d->d_k != 128))
    return fail(GDN_ERR_UNSUPPORTED, "need d_k == d_v in {32, 64, 128} (got %d, %d)", d->d_k, d->d_v);
  if (d->width != kWidth) return fail(GDN_ERR_UNSUPPORTED, "conv width must be 4 (got %d)", d->width);
  if (d->act != GDN_ACT_NONE && d->act != GDN_ACT_SILU)
    return fail(GDN_ERR_INVALID_ARG, "act must be GDN_ACT_NONE or GDN_ACT_SILU (got %d)", d->act);
  const long long C = (2LL * d->H_k + d->H_v) * d->d_k;
  if (C > (1LL << 30)) return fail(GDN_ERR_UNSUPPORTED, "too many conv channels (%lld)", C);
  return GDN_OK;
}

int check_mode(int mode) {
  if (mode != GDN_COMMIT_RECOMPUTE && mode != GDN_COMMIT_SNAPSHOT && mode != GDN_COMMIT_DEFERRED)
    return fail(GDN_ERR_INVALID_ARG,
                "mode must be GDN_COMMIT_RECOMPUTE, GDN_COMMIT_SNAPSHOT or GDN_COMMIT_DEFERRED (got %d)", mode);
  return GDN_OK;
}

size_t layer_ws_bytes(const gdn_dims *d, int mode) {
  if (mode == GDN_COMMIT_RECOMPUTE) return recompute_ws(d->B, d->T, d->H_k, d->H_v, d->d_k).total;
  if (mode == GDN_COMMIT_DEFERRED) return deferred_ws(d->B, d->T, d->H_k, d->H_v, d->d_k).total;
  return snapshot_ws(d->B, d->T, d->H_v, d->d_k);
}

// Host arrays of per-layer device pointers for gdn_commit / gdn_flush.
int fill_layers(CommitParams &p, int n_layers, float *const *state, gdn_bf16 *const *ring, void *const *layer_ws) {
  if (n_layers < 1 || n_layers > kMaxLayers)
    return fail(GDN_ERR_INVALID_ARG, "n_layers=%d outside [1, %d]", n_layers, kMaxLayers);
  if (!state || !layer_ws) return fail(GDN_ERR_INVALID_ARG, "state / layer_ws host arrays are NULL");
  for (int l = 0; l < n_layers; ++l) {
    if (!state[l] || !layer_ws[l]) return fail(GDN_ERR_INVALID_ARG, "layer %d: NULL state or workspace", l);
    if (!aligned(state[l], 16)) return fail(GDN_ERR_MISALIGNED, "layer %d: state not 16-byte aligned", l);
    if (!aligned(layer_ws[l], 256))
      return fail(GDN_ERR_MISALIGNED, "layer %d: workspace not 256-byte aligned", l);
    p.state[l] = state[l];
    p.ws[l] = static_cast<float *>(layer_ws[l]);
    if (ring) {
      if (!ring[l]) return fail(GDN_ERR_INVALID_ARG, "layer %d: NULL ring", l);
      if (!aligned(ring[l], 16)) return fail(GDN_ERR_MISALIGNED, "layer %d: ring not 16-byte aligned", l);
      p.ring[l] = reinterpret_cast<uint16_t *>(ring[l]);
    }
  }
  p.n_layers = n_layers;
  return GDN_OK;
}

#define GDN_NEED_PTR(ptr, align)                                                             \
  do {                                                                                       \
    if (!(ptr)) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", #ptr);                        \
    if (!aligned((ptr), (align)))                                                            \
      return fail(GDN_ERR_MISALIGNED, "%s is not %d-byte aligned", #ptr, int(align));        \
  } while (0)

// An array of a call, and whether the call writes it.
struct Span {
  const char *name;
  const void *p;
  size_t bytes;
  bool written;
};

// Refuses an array that is written and lies over another one.
int check_apart(const char *call, std::initializer_list<Span> spans) {
  for (const Span *a = spans.begin(); a != spans.end(); ++a)
    for (const Span *b = spans.begin(); b != a; ++b) {
      const char *x = static_cast<const char *>(a->p), *y = static_cast<const char *>(b->p);
      if ((a->written || b->written) && x && y && x < y + b->bytes && y < x + a->bytes)
        return fail(GDN_ERR_INVALID_ARG, "%s: %s and %s overlap", call, b->name, a->name);
    }
  return GDN_OK;
}

int cuda_fail(cudaError_t e, const char *what) {
  return fail(GDN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

static_assert(sizeof(CUtensorMap) == sizeof(TmaDesc), "TmaDesc holds one CUtensorMap");

// cuTensorMapEncodeTiled, looked up once through the runtime (thread-safe
// static initialisation); nullptr if the driver does not provide it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// The tensor map of one layer's state for the d = 128 tensor-core verify:
// fp32 [rows][128] (rows = B * H_v * d_v), boxes of 128 rows x 32 columns,
// 128-byte swizzle (the layout the kind::tf32 products read).
int encode_state_map(TmaDesc &m, const float *state, long long rows) {
  if (rows > (1LL << 31) - 1)
    return fail(GDN_ERR_UNSUPPORTED, "B * H_v * d_v = %lld state rows exceed the 2^31 - 1 a tensor map addresses", rows);
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return fail(GDN_ERR_CUDA, "the driver provides no cuTensorMapEncodeTiled");
  CUtensorMap map;
  const cuuint64_t dim[2] = {128, cuuint64_t(rows)};
  const cuuint64_t stride[1] = {128 * sizeof(float)};
  const cuuint32_t box[2] = {32, 128};
  const cuuint32_t estride[2] = {1, 1};
  const CUresult r = enc(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float *>(state), dim, stride, box,
                         estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled of the state failed (CUresult %d)", int(r));
  std::memcpy(&m, &map, sizeof map);
  return GDN_OK;
}

}  // namespace

extern "C" {

__attribute__((visibility("default"))) const char *gdn_version(void) {
  return "gdn_gb300 1.0 (sm_103a)";
}

__attribute__((visibility("default"))) const char *gdn_last_error(void) { return t_err.c_str(); }

__attribute__((visibility("default"))) size_t gdn_layer_workspace_bytes(const gdn_dims *dims, int mode) {
  if (check_dims(dims) != GDN_OK || check_mode(mode) != GDN_OK) return 0;
  return layer_ws_bytes(dims, mode);
}

namespace {

int verify_impl(const gdn_dims *dims, int mode, const gdn_bf16 *x, const gdn_bf16 *conv_w, const float *g,
                const float *beta, const float *state, gdn_bf16 *ring, const int32_t *offsets,
                const uint8_t *active, const gdn_bf16 *gate_z, const gdn_bf16 *norm_w, float eps, gdn_bf16 *out,
                void *layer_ws, size_t layer_ws_bytes_given, void *stream, uint32_t test_extra_tx = 0,
                uint32_t wait_limit = kWaitLimit) {
  NvtxRange range(gate_z ? "gdn_conv_verify_gated" : "gdn_conv_verify");
  int rc = check_dims(dims);
  if (rc) return rc;
  if (mode & ~(GDN_VERIFY_OVERLAP | GDN_VERIFY_OVERLAP_STATE | 0xff))
    return fail(GDN_ERR_INVALID_ARG, "unknown flag bits in mode 0x%x", mode);
  if ((mode & GDN_VERIFY_OVERLAP) && (mode & GDN_VERIFY_OVERLAP_STATE))
    return fail(GDN_ERR_INVALID_ARG, "GDN_VERIFY_OVERLAP and GDN_VERIFY_OVERLAP_STATE exclude each other");
  int overlap = (mode & GDN_VERIFY_OVERLAP) ? 1 : (mode & GDN_VERIFY_OVERLAP_STATE) ? 2 : 0;
  mode &= 0xff;
  // the state-only level exists in the d = 128 tensor-core verify; elsewhere
  // it is the same as no flag
  if (overlap == 2 && (dims->d_k != 128 || mode == GDN_COMMIT_SNAPSHOT)) overlap = 0;
  if ((rc = check_mode(mode))) return rc;
  if (dims->B == 0) return ok();
  GDN_NEED_PTR(x, 16);
  GDN_NEED_PTR(conv_w, 16);
  GDN_NEED_PTR(g, 16);
  GDN_NEED_PTR(beta, 16);
  GDN_NEED_PTR(state, 16);
  GDN_NEED_PTR(ring, 16);
  GDN_NEED_PTR(active, 1);
  GDN_NEED_PTR(out, 16);
  GDN_NEED_PTR(layer_ws, 256);
  (void)offsets;  // the committed window lives at fixed ring slots
  const size_t need = layer_ws_bytes(dims, mode);
  if (layer_ws_bytes_given < need)
    return fail(GDN_ERR_WORKSPACE, "layer workspace has %zu bytes, needs %zu", layer_ws_bytes_given, need);

  VerifyParams p{};
  p.x = x;
  p.w = conv_w;
  p.g = g;
  p.beta = beta;
  p.state = state;
  p.ring = ring;
  p.active = active;
  p.out = out;
  p.B = dims->B;
  p.T = dims->T;
  p.H_k = dims->H_k;
  p.H_v = dims->H_v;
  p.C = (2 * dims->H_k + dims->H_v) * dims->d_k;
  p.R = kHist + dims->T_max;
  p.act = dims->act;
  p.overlap = overlap;
  p.gz = gate_z;
  p.gw = norm_w;
  p.geps = eps;
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  p.wait_limit = wait_limit;
  p.test_extra_tx = test_extra_tx;
  if (dims->d_k == 128 && mode != GDN_COMMIT_SNAPSHOT &&
      (rc = encode_state_map(p.tmap_state, state, (long long)dims->B * dims->H_v * 128)))
    return rc;
  char *ws = static_cast<char *>(layer_ws);
  if (mode == GDN_COMMIT_RECOMPUTE) {
    const RecomputeWs w = recompute_ws(dims->B, dims->T, dims->H_k, dims->H_v, dims->d_k);
    p.ws_e = reinterpret_cast<float *>(ws + w.e);
    p.ws_k = reinterpret_cast<float *>(ws + w.k);
    p.ws_G = reinterpret_cast<float *>(ws + w.G);
  } else if (mode == GDN_COMMIT_SNAPSHOT) {
    p.ws_snap = reinterpret_cast<float *>(ws);
  } else {
    const DeferredWs w = deferred_ws(dims->B, dims->T, dims->H_k, dims->H_v, dims->d_k);
    const RecomputeWs r = recompute_ws(dims->B, dims->T, dims->H_v, dims->H_v, dims->d_k);
    p.ws_pend = reinterpret_cast<int *>(ws + w.pend);
    p.ws_e = reinterpret_cast<float *>(ws + w.cap + r.e);
    p.ws_k = reinterpret_cast<float *>(ws + w.cap + r.k);
    p.ws_G = reinterpret_cast<float *>(ws + w.cap + r.G);
    p.state_w = const_cast<float *>(state);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (dims->d_k) {
    case 32: e = launch_verify_32(p, dims->T, mode, s); break;
    case 64: e = launch_verify_64(p, dims->T, mode, s); break;
    default: e = launch_verify_128(p, dims->T, mode, s); break;
  }
  if (e != cudaSuccess) return cuda_fail(e, "gdn_conv_verify launch");
  return ok();
}

}  // namespace

__attribute__((visibility("default"))) int gdn_conv_verify(
    const gdn_dims *dims, int mode, const gdn_bf16 *x, const gdn_bf16 *conv_w, const float *g,
    const float *beta, const float *state, gdn_bf16 *ring, const int32_t *offsets,
    const uint8_t *active, gdn_bf16 *out, void *layer_ws, size_t layer_ws_bytes_given, void *stream) {
  return verify_impl(dims, mode, x, conv_w, g, beta, state, ring, offsets, active, nullptr, nullptr, 0.f, out,
                     layer_ws, layer_ws_bytes_given, stream);
}

__attribute__((visibility("default"))) int gdn_test_verify_timeout(
    const gdn_dims *dims, int mode, const gdn_bf16 *x, const gdn_bf16 *conv_w, const float *g,
    const float *beta, const float *state, gdn_bf16 *ring, const int32_t *offsets,
    const uint8_t *active, gdn_bf16 *out, void *layer_ws, size_t layer_ws_bytes_given, uint32_t wait_limit,
    void *stream) {
  if (check_dims(dims) == GDN_OK && (dims->d_k != 128 || (mode & 0xff) == GDN_COMMIT_SNAPSHOT))
    return fail(GDN_ERR_UNSUPPORTED, "gdn_test_verify_timeout: d = 128, RECOMPUTE or DEFERRED only");
  if (wait_limit < 1) return fail(GDN_ERR_INVALID_ARG, "gdn_test_verify_timeout: wait_limit must be >= 1");
  return verify_impl(dims, mode, x, conv_w, g, beta, state, ring, offsets, active, nullptr, nullptr, 0.f, out,
                     layer_ws, layer_ws_bytes_given, stream, 16u, wait_limit);
}

__attribute__((visibility("default"))) int gdn_conv_verify_gated(
    const gdn_dims *dims, int mode, const gdn_bf16 *x, const gdn_bf16 *conv_w, const float *g,
    const float *beta, const float *state, gdn_bf16 *ring, const int32_t *offsets,
    const uint8_t *active, const gdn_bf16 *gate_z, const gdn_bf16 *norm_w, float eps, gdn_bf16 *out,
    void *layer_ws, size_t layer_ws_bytes_given, void *stream) {
  if (check_dims(dims) == GDN_OK && dims->B > 0) {
    GDN_NEED_PTR(gate_z, 16);
    GDN_NEED_PTR(norm_w, 16);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(GDN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  }
  return verify_impl(dims, mode, x, conv_w, g, beta, state, ring, offsets, active, gate_z, norm_w, eps, out,
                     layer_ws, layer_ws_bytes_given, stream);
}

__attribute__((visibility("default"))) int gdn_commit(const gdn_dims *dims, int mode, int n_layers,
                                                      float *const *state, gdn_bf16 *const *ring,
                                                      void *const *layer_ws, const int32_t *keep,
                                                      const uint8_t *active, int32_t *offsets, void *stream) {
  NvtxRange range("gdn_commit");
  int rc = check_dims(dims);
  if (rc) return rc;
  if ((rc = check_mode(mode))) return rc;
  if (!ring) return fail(GDN_ERR_INVALID_ARG, "ring host array is NULL");
  CommitParams p{};
  if ((rc = fill_layers(p, n_layers, state, ring, layer_ws))) return rc;
  if (dims->B == 0) return ok();
  GDN_NEED_PTR(keep, 4);
  GDN_NEED_PTR(active, 1);
  GDN_NEED_PTR(offsets, 4);
  p.keep = keep;
  p.active = active;
  p.offsets = offsets;
  p.B = dims->B;
  p.T = dims->T;
  p.H_k = dims->H_k;
  p.H_v = dims->H_v;
  p.C = (2 * dims->H_k + dims->H_v) * dims->d_k;
  p.R = kHist + dims->T_max;
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = launch_commit(p, dims->d_k, mode, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_commit launch");
  return ok();
}

__attribute__((visibility("default"))) int gdn_flush(const gdn_dims *dims, int mode, int n_layers,
                                                     float *const *state, void *const *layer_ws, void *stream) {
  NvtxRange range("gdn_flush");
  int rc = check_dims(dims);
  if (rc) return rc;
  if ((rc = check_mode(mode))) return rc;
  CommitParams p{};
  if ((rc = fill_layers(p, n_layers, state, nullptr, layer_ws))) return rc;
  if (dims->B == 0 || mode != GDN_COMMIT_DEFERRED) return ok();
  p.B = dims->B;
  p.T = dims->T;
  p.H_k = dims->H_k;
  p.H_v = dims->H_v;
  cudaError_t e = launch_flush(p, dims->d_k, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_flush launch");
  return ok();
}

__attribute__((visibility("default"))) size_t gdn_prefill_workspace_bytes(const gdn_dims *dims, int L) {
  if (check_dims(dims) != GDN_OK || L < 1 || L > kMaxPrefillLen) return 0;
  return prefill_workspace_bytes(dims->B, L, dims->H_k, dims->H_v, dims->d_k);
}

__attribute__((visibility("default"))) int gdn_prefill_chunked(
    const gdn_dims *dims, int L, const gdn_bf16 *x, const gdn_bf16 *conv_w, const float *g,
    const float *beta, float *state, gdn_bf16 *ring, int32_t *offsets, gdn_bf16 *out, void *ws,
    size_t ws_bytes, void *stream) {
  NvtxRange range("gdn_prefill_chunked");
  int rc = check_dims(dims);
  if (rc) return rc;
  if (L < 0 || L > kMaxPrefillLen)
    return fail(GDN_ERR_UNSUPPORTED, "prompt length L=%d outside [0, %d]", L, kMaxPrefillLen);
  if (dims->B == 0 || L == 0) return ok();
  GDN_NEED_PTR(x, 16);
  GDN_NEED_PTR(conv_w, 16);
  GDN_NEED_PTR(g, 16);
  GDN_NEED_PTR(beta, 16);
  GDN_NEED_PTR(state, 16);
  GDN_NEED_PTR(ring, 16);
  GDN_NEED_PTR(offsets, 4);
  GDN_NEED_PTR(out, 16);
  GDN_NEED_PTR(ws, 256);
  const size_t need = prefill_workspace_bytes(dims->B, L, dims->H_k, dims->H_v, dims->d_k);
  if (ws_bytes < need) return fail(GDN_ERR_WORKSPACE, "prefill workspace has %zu bytes, needs %zu", ws_bytes, need);
  cudaError_t e = launch_prefill(x, conv_w, g, beta, state, ring, offsets, out, ws, dims->B, L, dims->H_k,
                                 dims->H_v, dims->d_k, kHist + dims->T_max, dims->act,
                                 static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_prefill_chunked launch");
  return ok();
}

__attribute__((visibility("default"))) int gdn_get_status(int clear, uint32_t *status) {
  if (!status) return fail(GDN_ERR_INVALID_ARG, "status is NULL");
  uint32_t *dev = status_word_address();
  if (!dev) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "gdn_get_status synchronize");
  e = cudaMemcpy(status, dev, sizeof(uint32_t), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "gdn_get_status read");
  if (clear) {
    e = cudaMemset(dev, 0, sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "gdn_get_status clear");
  }
  return ok();
}

__attribute__((visibility("default"))) size_t gdn_accept_workspace_bytes(int B, int T, int V) {
  if (B < 0 || T < 1 || T > kMaxAcceptT || V < 1) return 0;
  return accept_workspace_bytes(B, T, V);
}

__attribute__((visibility("default"))) int gdn_accept_greedy(int B, int T, int V, const gdn_bf16 *logits,
                                                             const int32_t *draft, const uint8_t *active,
                                                             int32_t *keep, int32_t *next, void *ws,
                                                             size_t ws_bytes, void *stream) {
  NvtxRange range("gdn_accept_greedy");
  if (B < 0 || T < 1 || V < 1) return fail(GDN_ERR_INVALID_ARG, "accept: B=%d T=%d V=%d", B, T, V);
  if (T > kMaxAcceptT) return fail(GDN_ERR_UNSUPPORTED, "accept: T=%d above %d", T, kMaxAcceptT);
  if ((long long)B * T > 65535) return fail(GDN_ERR_UNSUPPORTED, "accept: B*T=%lld above 65535", (long long)B * T);
  if (B == 0) return ok();
  GDN_NEED_PTR(logits, 16);
  GDN_NEED_PTR(draft, 16);
  GDN_NEED_PTR(active, 16);
  GDN_NEED_PTR(keep, 16);
  GDN_NEED_PTR(next, 16);
  GDN_NEED_PTR(ws, 256);
  const size_t need = accept_workspace_bytes(B, T, V);
  if (ws_bytes < need) return fail(GDN_ERR_WORKSPACE, "accept workspace has %zu bytes, needs %zu", ws_bytes, need);
  cudaError_t e = launch_accept(logits, draft, active, keep, next, ws, B, T, V, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_accept_greedy launch");
  return ok();
}

__attribute__((visibility("default"))) int gdn_move_rows(
    const gdn_dims *src_dims, const gdn_dims *dst_dims, int mode, int n_layers, const float *const *src_state,
    const gdn_bf16 *const *src_ring, const int32_t *src_offsets, float *const *dst_state, gdn_bf16 *const *dst_ring,
    int32_t *dst_offsets, void *const *dst_layer_ws, const int32_t *src_rows, const int32_t *dst_rows, int n_rows,
    void *stream) {
  NvtxRange range("gdn_move_rows");
  int rc = check_dims(src_dims);
  if (rc) return rc;
  if ((rc = check_dims(dst_dims))) return rc;
  if ((rc = check_mode(mode))) return rc;
  if (src_dims->H_k != dst_dims->H_k || src_dims->H_v != dst_dims->H_v || src_dims->d_k != dst_dims->d_k ||
      src_dims->T_max != dst_dims->T_max || src_dims->width != dst_dims->width)
    return fail(GDN_ERR_INVALID_ARG, "move_rows: the cohorts differ in heads, head size or T_max");
  if (n_layers < 1 || n_layers > kMaxLayers)
    return fail(GDN_ERR_INVALID_ARG, "n_layers=%d outside [1, %d]", n_layers, kMaxLayers);
  if (n_rows < 0) return fail(GDN_ERR_INVALID_ARG, "n_rows=%d", n_rows);
  if (!src_state || !src_ring || !dst_state || !dst_ring) return fail(GDN_ERR_INVALID_ARG, "NULL layer array");
  if (mode == GDN_COMMIT_DEFERRED && !dst_layer_ws)
    return fail(GDN_ERR_INVALID_ARG, "DEFERRED: the destination layer workspaces are needed");
  if (n_rows == 0) return ok();
  GDN_NEED_PTR(src_offsets, 16);
  GDN_NEED_PTR(dst_offsets, 16);
  GDN_NEED_PTR(src_rows, 16);
  GDN_NEED_PTR(dst_rows, 16);
  MoveParams p{};
  for (int l = 0; l < n_layers; ++l) {
    if (!src_state[l] || !src_ring[l] || !dst_state[l] || !dst_ring[l])
      return fail(GDN_ERR_INVALID_ARG, "layer %d: NULL state or ring", l);
    if (!aligned(src_state[l], 16) || !aligned(src_ring[l], 16) || !aligned(dst_state[l], 16) ||
        !aligned(dst_ring[l], 16))
      return fail(GDN_ERR_MISALIGNED, "layer %d: state or ring not 16-byte aligned", l);
    p.src_state[l] = src_state[l];
    p.src_ring[l] = reinterpret_cast<const uint16_t *>(src_ring[l]);
    p.dst_state[l] = dst_state[l];
    p.dst_ring[l] = reinterpret_cast<uint16_t *>(dst_ring[l]);
    if (mode == GDN_COMMIT_DEFERRED) {
      if (!dst_layer_ws[l] || !aligned(dst_layer_ws[l], 256))
        return fail(GDN_ERR_MISALIGNED, "layer %d: NULL or misaligned destination workspace", l);
      p.dst_ws[l] = dst_layer_ws[l];
    }
  }
  const int C = (2 * src_dims->H_k + src_dims->H_v) * src_dims->d_k;
  p.src_offsets = src_offsets;
  p.dst_offsets = dst_offsets;
  p.src_rows = src_rows;
  p.dst_rows = dst_rows;
  p.state_bytes = size_t(src_dims->H_v) * src_dims->d_v * src_dims->d_k * sizeof(float);
  p.ring_bytes = size_t(kHist + src_dims->T_max) * C * sizeof(uint16_t);
  p.pend_bytes = mode == GDN_COMMIT_DEFERRED ? size_t(dst_dims->H_v) * sizeof(int) : 0;
  p.n_layers = n_layers;
  p.n_rows = n_rows;
  p.src_B = src_dims->B;
  p.dst_B = dst_dims->B;
  p.H_v = dst_dims->H_v;
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = launch_move_rows(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_move_rows launch");
  return ok();
}

// ---- sampled decoding ----------------------------------------------------------
namespace {

int check_sample(int B, int T, int V, long long stride) {
  if (B < 0 || T < 1 || V < 1) return fail(GDN_ERR_INVALID_ARG, "sample: B=%d T=%d V=%d", B, T, V);
  if (T > kMaxAcceptT) return fail(GDN_ERR_UNSUPPORTED, "sample: T=%d above %d", T, kMaxAcceptT);
  if ((long long)B * T > 65535) return fail(GDN_ERR_UNSUPPORTED, "sample: B*T=%lld above 65535", (long long)B * T);
  if (V > kMaxSampleV) return fail(GDN_ERR_UNSUPPORTED, "sample: V=%d above %d", V, kMaxSampleV);
  if (stride < V || stride > (1LL << 40)) return fail(GDN_ERR_INVALID_ARG, "sample: stride %lld below V=%d, or above 2^40", stride, V);
  return GDN_OK;
}

// What both calls share; the optional arrays may be NULL, never misaligned.
int fill_sample(SampleParams &p, int B, int T, int V, const gdn_bf16 *logits, long long stride, const uint8_t *active,
                const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                const float *u, int32_t *token, float *logp) {
  GDN_NEED_PTR(logits, 2);
  GDN_NEED_PTR(u, 4);
  const void *all[] = {temperature, top_k, top_p, min_p, token, logp};
  for (const void *q : all)
    if (!aligned(q, 4)) return fail(GDN_ERR_MISALIGNED, "sample: an array is not 4-byte aligned");
  p.logits = logits, p.stride = stride, p.active = active;
  p.temperature = temperature, p.top_k = top_k, p.top_p = top_p, p.min_p = min_p;
  p.u = u, p.token = token, p.logp = logp;
  p.B = B, p.T = T, p.V = V;
  return GDN_OK;
}

}  // namespace

__attribute__((visibility("default"))) int gdn_sample(int B, int V, const gdn_bf16 *logits, long long stride,
                                                      const uint8_t *active, const float *temperature,
                                                      const int32_t *top_k, const float *top_p, const float *min_p,
                                                      const float *u, int32_t *token, float *logp, void *stream) {
  NvtxRange range("gdn_sample");
  int rc = check_sample(B, 1, V, stride);
  if (rc) return rc;
  if (B == 0) return ok();
  GDN_NEED_PTR(token, 4);
  SampleParams p{};
  if ((rc = fill_sample(p, B, 1, V, logits, stride, active, temperature, top_k, top_p, min_p, u, token, logp))) return rc;
  cudaError_t e = launch_sample(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_sample launch");
  return ok();
}

__attribute__((visibility("default"))) size_t gdn_accept_sampled_workspace_bytes(int B, int T, int V) {
  if (check_sample(B, T, V, V) != GDN_OK) return 0;
  return accept_sampled_workspace_bytes(B, T);
}

__attribute__((visibility("default"))) int gdn_accept_sampled(
    int B, int T, int V, const gdn_bf16 *logits, long long stride, const int32_t *draft, const uint8_t *active,
    const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
    int32_t *keep, int32_t *next, int32_t *token, float *logp, void *ws, size_t ws_bytes, void *stream) {
  NvtxRange range("gdn_accept_sampled");
  int rc = check_sample(B, T, V, stride);
  if (rc) return rc;
  if (B == 0) return ok();
  GDN_NEED_PTR(draft, 4);
  GDN_NEED_PTR(keep, 4);
  GDN_NEED_PTR(next, 4);
  GDN_NEED_PTR(ws, 256);
  SampleParams p{};
  if ((rc = fill_sample(p, B, T, V, logits, stride, active, temperature, top_k, top_p, min_p, u, token, logp))) return rc;
  const size_t need = accept_sampled_workspace_bytes(B, T);
  if (ws_bytes < need)
    return fail(GDN_ERR_WORKSPACE, "sampled acceptance workspace has %zu bytes, needs %zu", ws_bytes, need);
  // what a row's last position compares with the drafts, and the drafts
  const size_t rows = size_t(B) * 4;
  if ((rc = check_apart("gdn_accept_sampled", {{"draft", draft, rows * T, false}, {"keep", keep, rows, true}, {"next", next, rows, true},
                                               {"token", token, rows * T, true}, {"ws", ws, need, true}})))
    return rc;
  p.draft = draft, p.keep = keep, p.next = next;
  p.ws_token = static_cast<int32_t *>(ws);
  p.ws_count = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + align256(size_t(B) * T * sizeof(int32_t)));
  cudaError_t e = launch_sample(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_accept_sampled launch");
  return ok();
}

// ---- paged 4-bit key/value cache ---------------------------------------------
namespace {

constexpr int kMaxCacheTokens = 1 << 24;  // tokens of one call

int check_kv4(const gdn_kv4_dims *d) {
  if (!d) return fail(GDN_ERR_INVALID_ARG, "dims is NULL");
  if (d->B < 0 || d->B > 65535) return fail(GDN_ERR_UNSUPPORTED, "B=%d outside [0, 65535]", d->B);
  if (d->H_kv < 1 || d->H_q < 1 || d->H_q % d->H_kv != 0 || d->H_q / d->H_kv > 64 || d->H_q > 65535)
    return fail(GDN_ERR_UNSUPPORTED, "need H_q (%d) a multiple of H_kv (%d), at most 64 times it and at most 65535",
                d->H_q, d->H_kv);
  if (d->d != 64 && d->d != 128 && d->d != 256)
    return fail(GDN_ERR_UNSUPPORTED, "need d in {64, 128, 256} (got %d)", d->d);
  if (d->page != 16 && d->page != 32 && d->page != 64)
    return fail(GDN_ERR_UNSUPPORTED, "need page in {16, 32, 64} (got %d)", d->page);
  if (d->max_pages < 1 || d->max_pages > (1 << 20))
    return fail(GDN_ERR_UNSUPPORTED, "max_pages=%d outside [1, 2^20]", d->max_pages);
  if (d->n_pages < 1 || (long long)d->n_pages * d->page >= (1LL << 31))
    return fail(GDN_ERR_UNSUPPORTED, "need n_pages (%d) >= 1 and n_pages * page < 2^31", d->n_pages);
  return GDN_OK;
}

int check_tokens(int N) {
  if (N < 0 || N > kMaxCacheTokens) return fail(GDN_ERR_UNSUPPORTED, "N=%d outside [0, %d]", N, kMaxCacheTokens);
  return GDN_OK;
}

int log2_page(const gdn_kv4_dims *d) { return d->page == 16 ? 4 : d->page == 32 ? 5 : 6; }

Kv4Geom geom_of(const gdn_kv4_dims *d) {
  return Kv4Geom{d->B, d->H_q, d->H_kv, d->d, log2_page(d), d->max_pages, d->n_pages};
}

}  // namespace

__attribute__((visibility("default"))) size_t gdn_kv4_page_bytes(const gdn_kv4_dims *dims) {
  if (check_kv4(dims) != GDN_OK) return 0;
  return size_t(dims->H_kv) * kv4_record_bytes(dims->d, dims->page);
}

namespace {

// Both forms of the plan; `shared`: with holder counts.
int plan_call(const char *name, const gdn_kv4_dims *dims, int T, int N, const int32_t *lens, const int32_t *add,
              const uint8_t *active, int32_t *held, int32_t *table, int32_t *free_list, int32_t *free_count,
              bool shared, int32_t *refs, int32_t *q_start, int32_t *q_count, int32_t *kv_len, int32_t *slots,
              int32_t *positions, void *stream) {
  NvtxRange range(name);
  int rc = check_kv4(dims);
  if (rc) return rc;
  if ((rc = check_tokens(N))) return rc;
  if (T < 0 || (T > 0 && (long long)dims->B * T > N))
    return fail(GDN_ERR_INVALID_ARG, "plan: need T >= 0 and, where T > 0, N (%d) >= B * T (%d * %d)", N, dims->B, T);
  if (shared && (long long)dims->B * dims->max_pages >= (1LL << 31))
    return fail(GDN_ERR_UNSUPPORTED, "need B * max_pages (%d * %d) < 2^31", dims->B, dims->max_pages);
  if (dims->B == 0) return ok();
  GDN_NEED_PTR(lens, 4);
  GDN_NEED_PTR(add, 4);
  GDN_NEED_PTR(active, 1);
  GDN_NEED_PTR(held, 4);
  GDN_NEED_PTR(table, 4);
  GDN_NEED_PTR(free_list, 4);
  GDN_NEED_PTR(free_count, 4);
  if (shared) GDN_NEED_PTR(refs, 4);
  GDN_NEED_PTR(q_start, 4);
  GDN_NEED_PTR(q_count, 4);
  GDN_NEED_PTR(kv_len, 4);
  if (N > 0) {
    GDN_NEED_PTR(slots, 4);
    GDN_NEED_PTR(positions, 4);
  }
  // slots follow from the lengths after kv_len is written
  const size_t rows = size_t(dims->B) * 4;
  if (shared && (rc = check_apart(name, {{"lens", lens, rows, false}, {"kv_len", kv_len, rows, true}}))) return rc;
  KvPlanParams p{};
  p.lens = lens, p.add = add, p.active = active;
  p.held = held, p.table = table, p.free_list = free_list, p.free_count = free_count, p.refs = refs;
  p.q_start = q_start, p.q_count = q_count, p.kv_len = kv_len, p.slots = slots, p.positions = positions;
  p.B = dims->B, p.T = T, p.N = N;
  p.log2P = log2_page(dims), p.max_pages = dims->max_pages, p.n_pages = dims->n_pages;
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = launch_kv_plan(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  return ok();
}

}  // namespace

__attribute__((visibility("default"))) int gdn_kv_plan(const gdn_kv4_dims *dims, int T, int N, const int32_t *lens,
                                                       const int32_t *add, const uint8_t *active, int32_t *held,
                                                       int32_t *table, int32_t *free_list, int32_t *free_count,
                                                       int32_t *q_start, int32_t *q_count, int32_t *kv_len,
                                                       int32_t *slots, int32_t *positions, void *stream) {
  return plan_call("gdn_kv_plan", dims, T, N, lens, add, active, held, table, free_list, free_count, false, nullptr,
                   q_start, q_count, kv_len, slots, positions, stream);
}

__attribute__((visibility("default"))) int gdn_kv_plan_shared(
    const gdn_kv4_dims *dims, int T, int N, const int32_t *lens, const int32_t *add, const uint8_t *active,
    int32_t *held, int32_t *table, int32_t *free_list, int32_t *free_count, int32_t *refs, int32_t *q_start,
    int32_t *q_count, int32_t *kv_len, int32_t *slots, int32_t *positions, void *stream) {
  return plan_call("gdn_kv_plan_shared", dims, T, N, lens, add, active, held, table, free_list, free_count, true, refs,
                   q_start, q_count, kv_len, slots, positions, stream);
}

__attribute__((visibility("default"))) int gdn_kv_fork(const gdn_kv4_dims *dims, int n, const int32_t *src_rows,
                                                       const int32_t *dst_rows, const int32_t *lens, int32_t *held,
                                                       int32_t *table, int32_t *free_list, int32_t *free_count,
                                                       int32_t *refs, int32_t *copy_src, int32_t *copy_dst,
                                                       void *stream) {
  NvtxRange range("gdn_kv_fork");
  int rc = check_kv4(dims);
  if (rc) return rc;
  if (n < 0 || n > kMaxForks) return fail(GDN_ERR_UNSUPPORTED, "fork: n=%d outside [0, %d]", n, kMaxForks);
  if (n == 0) return ok();
  GDN_NEED_PTR(src_rows, 4);
  GDN_NEED_PTR(dst_rows, 4);
  GDN_NEED_PTR(lens, 4);
  GDN_NEED_PTR(held, 4);
  GDN_NEED_PTR(table, 4);
  GDN_NEED_PTR(free_list, 4);
  GDN_NEED_PTR(free_count, 4);
  GDN_NEED_PTR(refs, 4);
  GDN_NEED_PTR(copy_src, 4);
  GDN_NEED_PTR(copy_dst, 4);
  // what is written before the pairs' rows are read for the last time, and all else
  const size_t pairs = size_t(n) * 4, pages = size_t(dims->n_pages) * 4, rows = size_t(dims->B) * 4;
  if ((rc = check_apart("gdn_kv_fork", {{"src_rows", src_rows, pairs, false}, {"dst_rows", dst_rows, pairs, false}, {"lens", lens, pairs, false},
                                        {"held", held, rows, true}, {"table", table, rows * dims->max_pages, true}, {"free_list", free_list, pages, false},
                                        {"free_count", free_count, 4, true}, {"refs", refs, pages, true}, {"copy_src", copy_src, pairs, true},
                                        {"copy_dst", copy_dst, pairs, true}})))
    return rc;
  KvForkParams p{};
  p.src_rows = src_rows, p.dst_rows = dst_rows, p.lens = lens, p.held = held, p.table = table;
  p.free_list = free_list, p.free_count = free_count, p.refs = refs, p.copy_src = copy_src, p.copy_dst = copy_dst;
  p.n = n, p.B = dims->B, p.log2P = log2_page(dims), p.max_pages = dims->max_pages, p.n_pages = dims->n_pages;
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = launch_kv_fork(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_kv_fork launch");
  return ok();
}

__attribute__((visibility("default"))) int gdn_kv_compact(
    const gdn_kv4_dims *dims, const int32_t *held, const int32_t *table, const int32_t *refs, int32_t *new_table,
    int32_t *new_refs, int32_t *new_free_list, int32_t *new_free_count, int32_t *page_map, int32_t *copy_src,
    int32_t *copy_dst, int32_t *copy_count, void *stream) {
  NvtxRange range("gdn_kv_compact");
  int rc = check_kv4(dims);
  if (rc) return rc;
  if (dims->B > 0) {
    GDN_NEED_PTR(held, 4);
    GDN_NEED_PTR(table, 4);
    GDN_NEED_PTR(new_table, 4);
  }
  GDN_NEED_PTR(refs, 4);
  GDN_NEED_PTR(new_refs, 4);
  GDN_NEED_PTR(new_free_list, 4);
  GDN_NEED_PTR(new_free_count, 4);
  GDN_NEED_PTR(page_map, 4);
  GDN_NEED_PTR(copy_src, 4);
  GDN_NEED_PTR(copy_dst, 4);
  GDN_NEED_PTR(copy_count, 4);
  // in place, or apart
  const size_t pages = size_t(dims->n_pages) * 4, rows = size_t(dims->B) * 4, cells = rows * dims->max_pages;
  const size_t moves = size_t(dims->n_pages > 1 ? dims->n_pages / 2 : 1) * 4;
  const bool same_table = new_table == table, same_refs = new_refs == refs;
  if ((rc = check_apart("gdn_kv_compact", {{"held", held, rows, false}, {"table", table, cells, same_table}, {"refs", refs, pages, same_refs},
                                           {"new_table", same_table ? nullptr : new_table, cells, true}, {"new_refs", same_refs ? nullptr : new_refs, pages, true},
                                           {"new_free_list", new_free_list, pages, true}, {"new_free_count", new_free_count, 4, true},
                                           {"page_map", page_map, pages, true}, {"copy_src", copy_src, moves, true}, {"copy_dst", copy_dst, moves, true},
                                           {"copy_count", copy_count, 4, true}})))
    return rc;
  KvCompactParams p{};
  p.held = held, p.table = table, p.refs = refs, p.new_table = new_table, p.new_refs = new_refs;
  p.new_free_list = new_free_list, p.new_free_count = new_free_count, p.page_map = page_map;
  p.copy_src = copy_src, p.copy_dst = copy_dst, p.copy_count = copy_count;
  p.B = dims->B, p.max_pages = dims->max_pages, p.n_pages = dims->n_pages;
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = launch_kv_compact(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_kv_compact launch");
  return ok();
}

__attribute__((visibility("default"))) int gdn_kv_copy_pages(const gdn_kv4_dims *dims, int n_layers,
                                                             void *const *pages, int n, const int32_t *src,
                                                             const int32_t *dst, const int32_t *count, void *stream) {
  NvtxRange range("gdn_kv_copy_pages");
  int rc = check_kv4(dims);
  if (rc) return rc;
  if (n_layers < 1 || n_layers > kMaxCopyLayers)
    return fail(GDN_ERR_INVALID_ARG, "n_layers=%d outside [1, %d]", n_layers, kMaxCopyLayers);
  if (n < 0) return fail(GDN_ERR_INVALID_ARG, "copy_pages: n=%d", n);
  if (!pages) return fail(GDN_ERR_INVALID_ARG, "pages is NULL");
  KvCopyParams p{};
  for (int l = 0; l < n_layers; ++l) {
    if (!pages[l]) return fail(GDN_ERR_INVALID_ARG, "layer %d: NULL pages", l);
    if (!aligned(pages[l], 16)) return fail(GDN_ERR_MISALIGNED, "layer %d: pages not 16-byte aligned", l);
    p.pages[l] = static_cast<uint8_t *>(pages[l]);
  }
  if (n == 0) return ok();
  GDN_NEED_PTR(src, 4);
  GDN_NEED_PTR(dst, 4);
  if (!aligned(count, 4)) return fail(GDN_ERR_MISALIGNED, "count is not 4-byte aligned");
  p.src = src, p.dst = dst, p.count = count;
  p.n = n, p.n_layers = n_layers, p.n_pages = dims->n_pages;
  p.page_bytes = dims->H_kv * kv4_record_bytes(dims->d, dims->page);
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = launch_kv_copy(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_kv_copy_pages launch");
  return ok();
}

__attribute__((visibility("default"))) int gdn_kv4_append(
    const gdn_kv4_dims *dims, int N, const gdn_bf16 *q, long long q_stride, const gdn_bf16 *k, long long k_stride,
    const gdn_bf16 *v, long long v_stride, const int32_t *positions, int n_axes, const float *rope, int max_pos,
    int rot, const uint8_t *axis, int style, const int32_t *slots, void *pages, gdn_bf16 *q_out, void *stream) {
  NvtxRange range("gdn_kv4_append");
  int rc = check_kv4(dims);
  if (rc) return rc;
  if ((rc = check_tokens(N))) return rc;
  if (rot < 0 || rot > dims->d || rot % 16 != 0)
    return fail(GDN_ERR_UNSUPPORTED, "append: need rot (%d) a multiple of 16 in [0, d]", rot);
  if (style != GDN_ROPE_HALF && style != GDN_ROPE_PAIRS)
    return fail(GDN_ERR_INVALID_ARG, "append: style must be GDN_ROPE_HALF or GDN_ROPE_PAIRS (got %d)", style);
  const long long wq = (long long)dims->H_q * dims->d, wk = (long long)dims->H_kv * dims->d;
  if (q_stride < wq || k_stride < wk || v_stride < wk || q_stride % 8 || k_stride % 8 || v_stride % 8)
    return fail(GDN_ERR_INVALID_ARG,
                "append: token strides (%lld, %lld, %lld) must be multiples of 8 and at least heads * d", q_stride,
                k_stride, v_stride);
  if (N == 0) return ok();
  GDN_NEED_PTR(q, 16);
  GDN_NEED_PTR(k, 16);
  GDN_NEED_PTR(v, 16);
  GDN_NEED_PTR(slots, 4);
  GDN_NEED_PTR(pages, 16);
  GDN_NEED_PTR(q_out, 16);
  Kv4AppendParams p{};
  if (rot > 0) {
    GDN_NEED_PTR(positions, 4);
    GDN_NEED_PTR(rope, 8);
    if (!axis) return fail(GDN_ERR_INVALID_ARG, "axis is NULL");
    if (n_axes < 1 || max_pos < 1)
      return fail(GDN_ERR_INVALID_ARG, "append: n_axes=%d and max_pos=%d must be positive", n_axes, max_pos);
    for (int i = 0; i < rot / 2; ++i) {
      if (axis[i] >= n_axes)
        return fail(GDN_ERR_INVALID_ARG, "append: axis[%d]=%d outside [0, %d)", i, int(axis[i]), n_axes);
      p.axis[i] = axis[i];
    }
  }
  p.q = q, p.k = k, p.v = v, p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
  p.positions = positions, p.rope = reinterpret_cast<const float2 *>(rope), p.slots = slots;
  p.pages = static_cast<uint8_t *>(pages), p.q_out = q_out;
  p.N = N, p.H_q = dims->H_q, p.H_kv = dims->H_kv, p.rot = rot, p.max_pos = max_pos, p.n_axes = n_axes;
  p.pairs = style == GDN_ROPE_PAIRS;
  p.log2P = log2_page(dims), p.n_pages = dims->n_pages;
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = launch_kv4_append(p, dims->d, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_kv4_append launch");
  return ok();
}

__attribute__((visibility("default"))) int gdn_kv4_read(const gdn_kv4_dims *dims, int N, const int32_t *slots,
                                                        const void *pages, gdn_bf16 *k, gdn_bf16 *v, void *stream) {
  NvtxRange range("gdn_kv4_read");
  int rc = check_kv4(dims);
  if (rc) return rc;
  if ((rc = check_tokens(N))) return rc;
  if (N == 0) return ok();
  GDN_NEED_PTR(slots, 4);
  GDN_NEED_PTR(pages, 16);
  GDN_NEED_PTR(k, 16);
  GDN_NEED_PTR(v, 16);
  Kv4ReadParams p{};
  p.slots = slots, p.pages = static_cast<const uint8_t *>(pages), p.k = k, p.v = v;
  p.N = N, p.H_kv = dims->H_kv, p.log2P = log2_page(dims), p.n_pages = dims->n_pages;
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = launch_kv4_read(p, dims->d, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_kv4_read launch");
  return ok();
}

__attribute__((visibility("default"))) size_t gdn_kv4_attend_workspace_bytes(const gdn_kv4_dims *dims, int N,
                                                                             int max_q) {
  if (check_kv4(dims) != GDN_OK || check_tokens(N) != GDN_OK || max_q < 1 || max_q > kMaxPrefillLen) return 0;
  return kv4_attend_workspace_bytes(geom_of(dims), N, max_q);
}

namespace {

int attend(const gdn_kv4_dims *dims, int N, int max_q, const gdn_bf16 *q, const void *pages, const int32_t *table,
           const int32_t *q_start, const int32_t *q_count, const int32_t *kv_len, float scale, gdn_bf16 *out, void *ws,
           size_t ws_bytes, void *stream, uint32_t wait_limit = kWaitLimit, uint32_t test_hold = 0) {
  int rc = check_kv4(dims);
  if (rc) return rc;
  if ((rc = check_tokens(N))) return rc;
  if (max_q < 1 || max_q > kMaxPrefillLen)
    return fail(GDN_ERR_UNSUPPORTED, "attend: max_q=%d outside [1, %d]", max_q, kMaxPrefillLen);
  if (!std::isfinite(scale)) return fail(GDN_ERR_INVALID_ARG, "attend: scale must be finite");
  if (dims->B == 0 || N == 0) return ok();
  GDN_NEED_PTR(q, 16);
  GDN_NEED_PTR(pages, 16);
  GDN_NEED_PTR(table, 4);
  GDN_NEED_PTR(q_start, 4);
  GDN_NEED_PTR(q_count, 4);
  GDN_NEED_PTR(kv_len, 4);
  GDN_NEED_PTR(out, 16);
  GDN_NEED_PTR(ws, 256);
  const size_t need = kv4_attend_workspace_bytes(geom_of(dims), N, max_q);
  if (ws_bytes < need) return fail(GDN_ERR_WORKSPACE, "attend workspace has %zu bytes, needs %zu", ws_bytes, need);
  Kv4AttendParams p{};
  p.q = q, p.pages = static_cast<const uint8_t *>(pages), p.table = table;
  p.q_start = q_start, p.q_count = q_count, p.kv_len = kv_len, p.out = out, p.ws = ws;
  p.scale = scale, p.N = N, p.max_q = max_q, p.g = geom_of(dims);
  p.wait_limit = wait_limit, p.test_hold = test_hold;
  p.status = status_word_address();
  if (!p.status) return fail(GDN_ERR_CUDA, "cannot resolve the device status word");
  cudaError_t e = launch_kv4_attend(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gdn_kv4_attend launch");
  return ok();
}

}  // namespace

__attribute__((visibility("default"))) int gdn_kv4_attend(
    const gdn_kv4_dims *dims, int N, int max_q, const gdn_bf16 *q, const void *pages, const int32_t *table,
    const int32_t *q_start, const int32_t *q_count, const int32_t *kv_len, float scale, gdn_bf16 *out, void *ws,
    size_t ws_bytes, void *stream) {
  NvtxRange range("gdn_kv4_attend");
  return attend(dims, N, max_q, q, pages, table, q_start, q_count, kv_len, scale, out, ws, ws_bytes, stream);
}

__attribute__((visibility("default"))) int gdn_test_kv4_attend_timeout(
    const gdn_kv4_dims *dims, int N, int max_q, const gdn_bf16 *q, const void *pages, const int32_t *table,
    const int32_t *q_start, const int32_t *q_count, const int32_t *kv_len, float scale, gdn_bf16 *out, void *ws,
    size_t ws_bytes, uint32_t wait_limit, void *stream) {
  NvtxRange range("gdn_test_kv4_attend_timeout");
  if (wait_limit < 1) return fail(GDN_ERR_INVALID_ARG, "gdn_test_kv4_attend_timeout: wait_limit must be >= 1");
  return attend(dims, N, max_q, q, pages, table, q_start, q_count, kv_len, scale, out, ws, ws_bytes, stream, wait_limit, 1);
}

// ---- verify without caller-provided workspace ---------------------------------
// Scratch for gdn_conv_verify_noalloc: one layer's verify captures.  It lives
// in the library's own device memory, so every GPU that loads the library
// holds these bytes until the process exits.  Host code may not use the name
// `g_noalloc_ws` as an address (on the host it is only a stand-in for the
// device symbol); the device address comes from cudaGetSymbolAddress.
static __device__ __align__(256) unsigned char g_noalloc_ws[GDN_NOALLOC_WS_BYTES];

namespace {

std::mutex g_noalloc_lock;
void *g_noalloc_ptr[64] = {nullptr};  // device address of g_noalloc_ws, per device

// Look up (once per device, with that device current) where the scratch
// array lives on the current device.
int noalloc_scratch(void **ptr) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "gdn_conv_verify_noalloc: cudaGetDevice");
  if (dev < 0 || dev >= 64) return fail(GDN_ERR_UNSUPPORTED, "device index %d above 63", dev);
  std::lock_guard<std::mutex> lock(g_noalloc_lock);
  if (!g_noalloc_ptr[dev]) {
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_ws);
    if (e != cudaSuccess || !p) return cuda_fail(e, "gdn_conv_verify_noalloc: cudaGetSymbolAddress");
    g_noalloc_ptr[dev] = p;
  }
  *ptr = g_noalloc_ptr[dev];
  return GDN_OK;
}

}  // namespace

__attribute__((visibility("default"))) int gdn_conv_verify_noalloc(
    const gdn_dims *dims, int mode, const gdn_bf16 *x, const gdn_bf16 *conv_w, const float *g,
    const float *beta, const float *state, gdn_bf16 *ring, const int32_t *offsets,
    const uint8_t *active, gdn_bf16 *out, void **layer_ws_used, void *stream) {
  int rc = check_dims(dims);
  if (rc) return rc;
  if ((rc = check_mode(mode & 0xff))) return rc;
  if ((mode & 0xff) == GDN_COMMIT_DEFERRED)
    return fail(GDN_ERR_INVALID_ARG,
                "gdn_conv_verify_noalloc: DEFERRED mode needs a workspace that persists per layer");
  const size_t need = layer_ws_bytes(dims, mode & 0xff);
  if (need > GDN_NOALLOC_WS_BYTES)
    return fail(GDN_ERR_WORKSPACE,
                "gdn_conv_verify_noalloc: this shape and mode need %zu bytes of scratch, the library's "
                "built-in scratch holds %zu; use gdn_conv_verify with a caller-allocated workspace",
                need, size_t(GDN_NOALLOC_WS_BYTES));
  void *ws = nullptr;
  if ((rc = noalloc_scratch(&ws))) return rc;
  rc = gdn_conv_verify(dims, mode, x, conv_w, g, beta, state, ring, offsets, active, out, ws,
                       GDN_NOALLOC_WS_BYTES, stream);
  if (rc == GDN_OK && layer_ws_used) *layer_ws_used = ws;
  return rc;
}

}  // extern "C"
