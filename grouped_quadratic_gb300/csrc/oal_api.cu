// oal_api.cu -- the extern "C" entry points of liboal.so (include/oal.h):
// argument validation, workspace sizing, dispatch to the kernels, error
// reporting.  No allocation happens here; all memory is the caller's.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

#include "gated.cuh"
#include "paged.cuh"

namespace oal {
oal_status launch_expand_coeffs(const float *L, const int32_t *group, int Hq, int G,
                                float eps, int packed, float *a, float *b, float *C,
                                cudaStream_t stream);
size_t simt_prefill_workspace_bytes(int B, int Hkv, int T, int packed, int chunk);
oal_status launch_prefill_simt(const void *Q, const void *K, const void *V, int is_bf16,
                               int B, int Hq, int Hkv, int T, const float *L,
                               const int32_t *group, int G, float eps, const float *a,
                               const float *b, const float *C, int packed, float *state,
                               int cont, void *Y, int chunk, void *ws, cudaStream_t stream);
size_t tc_prefill_workspace_bytes(int B, int Hq, int Hkv, int T, int chunk);
void set_intra_heads(int heads);
oal_status launch_prefill_tc(const void *Q, const void *K, const void *V, int B, int Hq,
                             int Hkv, int T, const float *L, const int32_t *group, int G,
                             float eps, const float *a, const float *b, const float *C,
                             int packed, float *state, int cont, void *Y, int chunk, void *ws,
                             cudaStream_t stream);
size_t decode_workspace_bytes(int B, int Hkv, int packed);
int decode_max_rho();
oal_status launch_decode(const void *q, const void *k, const void *v, int is_bf16, int B,
                         int Hq, int Hkv, const float *a, const float *b, const float *C,
                         int packed, float *state, void *y, void *ws, cudaStream_t stream);

size_t backward_workspace_bytes(int B, int Hq, int Hkv, int T);
oal_status launch_backward(const void *Q, const void *K, const void *V, const void *dY, int is_bf16,
                           int B, int Hq, int Hkv, int T, const float *L, const int32_t *group,
                           int G, float eps, float *dQ, float *dK, float *dV, float *dL, void *ws,
                           cudaStream_t stream);

size_t contrib_workspace_bytes(int P, int Hq, int Hkv, int T);
oal_status launch_contrib(const void *Q, const void *K, int is_bf16, int P, int Hq, int Hkv,
                          int T, const int32_t *lengths, float *chi, void *ws,
                          cudaStream_t stream);
oal_status group_dims_host(const float *chi_p, int P, int d, const int32_t *boot_idx,
                           int nboot, double alpha, double tau, double gamma, int g_min,
                           double eps, int32_t *group, int *G);

oal_status launch_gated_prefill_simt(const GatedArgs &p, cudaStream_t stream);
oal_status launch_gated_prefill_tc(const GatedArgs &p, cudaStream_t stream);
oal_status launch_gated_backward_simt(const GatedArgs &p, cudaStream_t stream);
oal_status launch_gated_backward_tc(const GatedArgs &p, cudaStream_t stream);
oal_status launch_gated_decode(const void *q, const void *k, const void *v, int is_bf16,
                               const float *g, int B, int Hq, int Hkv, float scale,
                               const int32_t *slots, int n_slots, float *state, void *y,
                               cudaStream_t stream);
oal_status launch_state_remap(void *pool, size_t slot_bytes, int n, const int32_t *map,
                              cudaStream_t stream);

oal_status launch_rope(const RopeArgs &p, int is_bf16, int form, const char *name,
                       cudaStream_t stream);
size_t paged_workspace_bytes(PagedArgs p, int is_bf16);
oal_status launch_paged(PagedArgs p, int is_bf16, void *ws, cudaStream_t stream);

// Device control block (one per device the library runs on): the status
// word kernels record errors in; then, for tests of the failure path, the
// kernel whose UMMA issuer is to wait on a barrier nothing arrives on
// (0 = none), and the limit of the bounded waits in SM cycles (0 = the
// built-in limit).
struct DeviceControl {
  int status;
  int starve;
  unsigned long long wait_limit;
};
__device__ DeviceControl g_control;
}  // namespace oal

static thread_local char t_msg[512] = "";

oal_status oal_fail(oal_status st, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_msg, sizeof t_msg, fmt, ap);
  va_end(ap);
  return st;
}

oal_status oal_check_launch(const char *what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return oal_fail(OAL_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return OAL_OK;
}

// ---- launch accounting and the timing hook
#include <atomic>
static std::atomic<unsigned long long> g_launches{0};
static thread_local cudaEvent_t *t_events = nullptr;
static thread_local int t_nevents = 0;
static thread_local int t_call_launches = 0;
static thread_local const char *t_call_names[32];

void oal_begin_call(cudaStream_t stream) {
  t_call_launches = 0;
  if (t_events && t_nevents > 0) cudaEventRecord(t_events[0], stream);
}

oal_status oal_after_launch(const char *name, cudaStream_t stream) {
  const oal_status st = oal_check_launch(name);
  if (st != OAL_OK) return st;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  const int k = ++t_call_launches;
  if (k <= 32) t_call_names[k - 1] = name;
  if (t_events && k < t_nevents) cudaEventRecord(t_events[k], stream);
  return OAL_OK;
}

#include <mutex>
static std::mutex g_control_mutex;
static int *g_control_addr[oal::kMaxDevices] = {nullptr};

int *oal_device_status_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  if (dev < 0 || dev >= oal::kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_control_mutex);
  if (!g_control_addr[dev]) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, oal::g_control) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    g_control_addr[dev] = &static_cast<oal::DeviceControl *>(p)->status;
  }
  return g_control_addr[dev];
}

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

oal_status check_ptr(const void *p, const char *name) {
  if (!p) return oal_fail(OAL_ERR_INVALID_ARG, "%s is null", name);
  if (!aligned16(p)) return oal_fail(OAL_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return OAL_OK;
}

oal_status check_common(int B, int Hq, int Hkv, int d, int dv, oal_dtype dtype,
                        oal_state_layout layout) {
  if (B < 0 || Hq <= 0 || Hkv <= 0)
    return oal_fail(OAL_ERR_INVALID_ARG, "bad sizes B=%d Hq=%d Hkv=%d", B, Hq, Hkv);
  if (Hq % Hkv != 0)
    return oal_fail(OAL_ERR_INVALID_ARG, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
  if (dtype != OAL_F32 && dtype != OAL_BF16)
    return oal_fail(OAL_ERR_INVALID_ARG, "bad dtype %d", (int)dtype);
  if (layout != OAL_STATE_FULL && layout != OAL_STATE_PACKED)
    return oal_fail(OAL_ERR_INVALID_ARG, "bad state layout %d", (int)layout);
  if (d != oal::kD || dv != oal::kDv)
    return oal_fail(OAL_ERR_UNSUPPORTED, "only d = dv = 64 is supported (d=%d dv=%d)", d, dv);
  return OAL_OK;
}

#define OAL_TRY(x)                        \
  do {                                    \
    const oal_status _s = (x);            \
    if (_s != OAL_OK) return _s;          \
  } while (0)

}  // namespace

extern "C" {

const char *oal_version(void) { return "0.1.0"; }

uint64_t oal_launch_counter(void) { return g_launches.load(std::memory_order_relaxed); }

oal_status oal_set_launch_events(cudaEvent_t *events, int n) {
  if (n < 0) return oal_fail(OAL_ERR_INVALID_ARG, "n=%d", n);
  t_events = (events && n > 0) ? events : nullptr;
  t_nevents = t_events ? n : 0;
  return OAL_OK;
}

int oal_last_call_launches(void) { return t_call_launches; }

const char *oal_last_call_launch_name(int k) {
  if (k < 0 || k >= t_call_launches || k >= 32) return "";
  return t_call_names[k];
}

const char *oal_last_error(void) { return t_msg; }

size_t oal_state_rows(int d, oal_state_layout layout) {
  if (d <= 0) return 0;
  const size_t dd = (size_t)d;
  if (layout == OAL_STATE_FULL) return 1 + dd + dd * dd;
  if (layout == OAL_STATE_PACKED) return 1 + dd + dd * (dd + 1) / 2;
  return 0;
}

size_t oal_state_elems(int d, int dv, oal_state_layout layout) {
  if (dv <= 0) return 0;
  return oal_state_rows(d, layout) * (size_t)(dv + 1);
}

size_t oal_coeff_table_elems(int d, oal_state_layout layout) {
  if (d <= 0) return 0;
  if (layout == OAL_STATE_FULL) return (size_t)d * d;
  if (layout == OAL_STATE_PACKED) return (size_t)d * (d + 1) / 2;
  return 0;
}

oal_status oal_expand_coeffs(const float *L, const int32_t *group, int Hq, int G, int d,
                             float eps, oal_state_layout layout, float *a, float *b,
                             float *C, cudaStream_t stream) {
  t_msg[0] = 0;
  if (Hq <= 0) return oal_fail(OAL_ERR_INVALID_ARG, "Hq=%d", Hq);
  if (layout != OAL_STATE_FULL && layout != OAL_STATE_PACKED)
    return oal_fail(OAL_ERR_INVALID_ARG, "bad state layout %d", (int)layout);
  if (d != oal::kD) return oal_fail(OAL_ERR_UNSUPPORTED, "only d = 64 is supported (d=%d)", d);
  if (G < 1 || G > oal::kMaxG)
    return oal_fail(OAL_ERR_UNSUPPORTED, "G=%d outside 1..%d", G, oal::kMaxG);
  if (!(eps > 0.f)) return oal_fail(OAL_ERR_INVALID_ARG, "eps must be > 0 (got %g)", eps);
  OAL_TRY(check_ptr(L, "L"));
  OAL_TRY(check_ptr(group, "group"));
  OAL_TRY(check_ptr(a, "a"));
  OAL_TRY(check_ptr(b, "b"));
  OAL_TRY(check_ptr(C, "C"));
  oal_begin_call(stream);
  return oal::launch_expand_coeffs(L, group, Hq, G, eps, layout == OAL_STATE_PACKED, a, b,
                                   C, stream);
}

static int default_chunk(oal_dtype dtype) { return dtype == OAL_BF16 ? 128 : 64; }

// bf16 inputs run on the tensor cores (tcgen05) at every chunk size; fp32
// inputs run the fp32 CUDA-core kernels.
static bool use_tc(oal_dtype dtype) { return dtype == OAL_BF16; }

size_t oal_prefill_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int dv,
                                   oal_dtype dtype, oal_state_layout layout, int chunk) {
  if (check_common(B, Hq, Hkv, d, dv, dtype, layout) != OAL_OK || T < 0) return 0;
  if (chunk == 0) chunk = default_chunk(dtype);
  if (chunk != 64 && chunk != 128 && chunk != 256) return 0;
  if (T == 0 || B == 0) return 256;
  if (use_tc(dtype)) return oal::tc_prefill_workspace_bytes(B, Hq, Hkv, T, chunk);
  return oal::simt_prefill_workspace_bytes(B, Hkv, T, layout == OAL_STATE_PACKED, chunk);
}

oal_status oal_prefill(const void *Q, const void *K, const void *V, oal_dtype dtype, int B,
                       int Hq, int Hkv, int T, int d, int dv, const float *L,
                       const int32_t *group, int G, float eps, const float *a,
                       const float *b, const float *C, oal_state_layout layout,
                       float *state, int continue_from_state, void *Y, int chunk,
                       void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  t_msg[0] = 0;
  OAL_TRY(check_common(B, Hq, Hkv, d, dv, dtype, layout));
  if (T < 0) return oal_fail(OAL_ERR_INVALID_ARG, "T=%d", T);
  if (G < 1 || G > oal::kMaxG)
    return oal_fail(OAL_ERR_UNSUPPORTED, "G=%d outside 1..%d", G, oal::kMaxG);
  if (!(eps > 0.f)) return oal_fail(OAL_ERR_INVALID_ARG, "eps must be > 0 (got %g)", eps);
  if (chunk == 0) chunk = default_chunk(dtype);
  if (chunk != 64 && chunk != 128 && chunk != 256)
    return oal_fail(OAL_ERR_INVALID_ARG, "chunk=%d (allowed: 0, 64, 128, 256)", chunk);
  t_call_launches = 0;
  if (B == 0) return OAL_OK;
  OAL_TRY(check_ptr(state, "state"));
  const int packed = layout == OAL_STATE_PACKED;
  if (T == 0) {
    if (!continue_from_state) {
      const size_t bytes = (size_t)B * Hkv * oal_state_elems(d, dv, layout) * sizeof(float);
      if (cudaMemsetAsync(state, 0, bytes, stream) != cudaSuccess)
        return oal_check_launch("state reset");
    }
    return OAL_OK;
  }
  OAL_TRY(check_ptr(Q, "Q"));
  OAL_TRY(check_ptr(K, "K"));
  OAL_TRY(check_ptr(V, "V"));
  OAL_TRY(check_ptr(Y, "Y"));
  OAL_TRY(check_ptr(L, "L"));
  OAL_TRY(check_ptr(group, "group"));
  OAL_TRY(check_ptr(a, "a"));
  OAL_TRY(check_ptr(b, "b"));
  OAL_TRY(check_ptr(C, "C"));
  OAL_TRY(check_ptr(workspace, "workspace"));
  if (((uintptr_t)workspace & 255u) != 0)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  const size_t need =
      oal_prefill_workspace_bytes(B, Hq, Hkv, T, d, dv, dtype, layout, chunk);
  if (workspace_bytes < need)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes",
                    workspace_bytes, need);
  if ((long long)T * Hq * B > (1LL << 40))
    return oal_fail(OAL_ERR_UNSUPPORTED, "problem too large");
  oal_begin_call(stream);
  if (use_tc(dtype))
    return oal::launch_prefill_tc(Q, K, V, B, Hq, Hkv, T, L, group, G, eps, a, b, C, packed,
                                  state, continue_from_state != 0, Y, chunk, workspace, stream);
  return oal::launch_prefill_simt(Q, K, V, dtype == OAL_BF16, B, Hq, Hkv, T, L, group, G,
                                  eps, a, b, C, packed, state, continue_from_state != 0,
                                  Y, chunk, workspace, stream);
}

size_t oal_prefill_backward_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int dv) {
  if (check_common(B, Hq, Hkv, d, dv, OAL_F32, OAL_STATE_FULL) != OAL_OK || T < 0) return 0;
  if (B == 0 || T == 0) return 256;
  return oal::backward_workspace_bytes(B, Hq, Hkv, T);
}

oal_status oal_prefill_backward(const void *Q, const void *K, const void *V, const void *dY,
                                oal_dtype dtype, int B, int Hq, int Hkv, int T, int d, int dv,
                                const float *L, const int32_t *group, int G, float eps, float *dQ,
                                float *dK, float *dV, float *dL, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream) {
  t_msg[0] = 0;
  OAL_TRY(check_common(B, Hq, Hkv, d, dv, dtype, OAL_STATE_FULL));
  if (T < 0) return oal_fail(OAL_ERR_INVALID_ARG, "T=%d", T);
  if (G < 1 || G > oal::kMaxG)
    return oal_fail(OAL_ERR_UNSUPPORTED, "G=%d outside 1..%d", G, oal::kMaxG);
  if (!(eps > 0.f)) return oal_fail(OAL_ERR_INVALID_ARG, "eps must be > 0 (got %g)", eps);
  OAL_TRY(check_ptr(L, "L"));
  OAL_TRY(check_ptr(group, "group"));
  OAL_TRY(check_ptr(dL, "dL"));
  t_call_launches = 0;
  if (B == 0 || T == 0) {   // no pairs: every gradient is zero (dQ, dK, dV are empty)
    const size_t bytes = (size_t)Hq * (G + 1) * (G + 1) * sizeof(float);
    if (cudaMemsetAsync(dL, 0, bytes, stream) != cudaSuccess) return oal_check_launch("dL reset");
    return OAL_OK;
  }
  OAL_TRY(check_ptr(Q, "Q"));
  OAL_TRY(check_ptr(K, "K"));
  OAL_TRY(check_ptr(V, "V"));
  OAL_TRY(check_ptr(dY, "dY"));
  OAL_TRY(check_ptr(dQ, "dQ"));
  OAL_TRY(check_ptr(dK, "dK"));
  OAL_TRY(check_ptr(dV, "dV"));
  OAL_TRY(check_ptr(workspace, "workspace"));
  if (((uintptr_t)workspace & 255u) != 0)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  const size_t need = oal_prefill_backward_workspace_bytes(B, Hq, Hkv, T, d, dv);
  if (workspace_bytes < need)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes",
                    workspace_bytes, need);
  oal_begin_call(stream);
  return oal::launch_backward(Q, K, V, dY, dtype == OAL_BF16, B, Hq, Hkv, T, L, group, G, eps, dQ,
                              dK, dV, dL, workspace, stream);
}

size_t oal_decode_workspace_bytes(int B, int Hq, int Hkv, int d, int dv,
                                  oal_state_layout layout) {
  if (check_common(B, Hq, Hkv, d, dv, OAL_F32, layout) != OAL_OK) return 0;
  if (B == 0) return 256;
  return oal::decode_workspace_bytes(B, Hkv, layout == OAL_STATE_PACKED);
}

oal_status oal_decode_step(const void *q, const void *k, const void *v, oal_dtype dtype,
                           int B, int Hq, int Hkv, int d, int dv, const float *a,
                           const float *b, const float *C, oal_state_layout layout,
                           float *state, void *y, void *workspace, size_t workspace_bytes,
                           cudaStream_t stream) {
  t_msg[0] = 0;
  OAL_TRY(check_common(B, Hq, Hkv, d, dv, dtype, layout));
  if (Hq / Hkv > oal::decode_max_rho())
    return oal_fail(OAL_ERR_UNSUPPORTED, "Hq/Hkv=%d exceeds %d", Hq / Hkv,
                    oal::decode_max_rho());
  if (B == 0) return OAL_OK;
  OAL_TRY(check_ptr(q, "q"));
  OAL_TRY(check_ptr(k, "k"));
  OAL_TRY(check_ptr(v, "v"));
  OAL_TRY(check_ptr(y, "y"));
  OAL_TRY(check_ptr(a, "a"));
  OAL_TRY(check_ptr(b, "b"));
  OAL_TRY(check_ptr(C, "C"));
  OAL_TRY(check_ptr(state, "state"));
  OAL_TRY(check_ptr(workspace, "workspace"));
  if (((uintptr_t)workspace & 255u) != 0)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  const size_t need = oal_decode_workspace_bytes(B, Hq, Hkv, d, dv, layout);
  if (workspace_bytes < need)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes",
                    workspace_bytes, need);
  oal_begin_call(stream);
  return oal::launch_decode(q, k, v, dtype == OAL_BF16, B, Hq, Hkv, a, b, C,
                            layout == OAL_STATE_PACKED, state, y, workspace, stream);
}

size_t oal_contribution_workspace_bytes(int P, int Hq, int Hkv, int T, int d) {
  if (P < 0 || Hq <= 0 || Hkv <= 0 || T < 0 || d != oal::kD) return 0;
  return std::max<size_t>(256, oal::contrib_workspace_bytes(P, Hq, Hkv, T));
}

oal_status oal_contribution_scores(const void *Q, const void *K, oal_dtype dtype, int P,
                                   int Hq, int Hkv, int T, int d, const int32_t *lengths,
                                   float *chi, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  t_msg[0] = 0;
  OAL_TRY(check_common(P, Hq, Hkv, d, d, dtype, OAL_STATE_FULL));
  if (T < 0) return oal_fail(OAL_ERR_INVALID_ARG, "bad T=%d", T);
  if (P == 0) return OAL_OK;
  if (P > 65535) return oal_fail(OAL_ERR_UNSUPPORTED, "P=%d above 65535", P);
  OAL_TRY(check_ptr(chi, "chi"));
  OAL_TRY(check_ptr(workspace, "workspace"));
  if (T > 0) {
    OAL_TRY(check_ptr(Q, "Q"));
    OAL_TRY(check_ptr(K, "K"));
    if ((T + 127) / 128 > 65535) return oal_fail(OAL_ERR_UNSUPPORTED, "T=%d too long", T);
  }
  if (lengths) OAL_TRY(check_ptr(lengths, "lengths"));
  if (((uintptr_t)workspace & 255u) != 0)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  const size_t need = oal_contribution_workspace_bytes(P, Hq, Hkv, T, d);
  if (workspace_bytes < need)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes",
                    workspace_bytes, need);
  oal_begin_call(stream);
  return oal::launch_contrib(Q, K, dtype == OAL_BF16, P, Hq, Hkv, T, lengths, chi, workspace,
                             stream);
}

oal_status oal_group_dims(const float *chi_p, int P, int d, const int32_t *boot_idx, int nboot,
                          double alpha, double tau, double gamma, int g_min, double eps,
                          int32_t *group, int *G) {
  t_msg[0] = 0;
  if (!chi_p || !boot_idx || !group || !G)
    return oal_fail(OAL_ERR_INVALID_ARG, "null pointer");
  if (P < 1 || d < 2 || nboot < 1)
    return oal_fail(OAL_ERR_INVALID_ARG, "bad sizes P=%d d=%d nboot=%d", P, d, nboot);
  if (!(alpha > 0.0 && alpha <= 1.0) || !(eps > 0.0) || !(tau > 0.0) || !(gamma >= 0.0) ||
      g_min < 1)
    return oal_fail(OAL_ERR_INVALID_ARG, "bad parameters alpha=%g tau=%g gamma=%g g_min=%d "
                    "eps=%g", alpha, tau, gamma, g_min, eps);
  for (size_t i = 0; i < (size_t)nboot * P; ++i)
    if (boot_idx[i] < 0 || boot_idx[i] >= P)
      return oal_fail(OAL_ERR_INVALID_ARG, "bootstrap index %d outside 0..%d", boot_idx[i],
                      P - 1);
  for (size_t i = 0; i < (size_t)P * d; ++i)
    if (!isfinite(chi_p[i]) || chi_p[i] < 0.f)
      return oal_fail(OAL_ERR_INVALID_ARG, "score %zu is negative or not finite", i);
  return oal::group_dims_host(chi_p, P, d, boot_idx, nboot, alpha, tau, gamma, g_min, eps,
                              group, G);
}

// ---- gated linear recurrence

static oal_status check_gated(int B, int Hq, int Hkv, int T, int d, int dv, oal_dtype dtype,
                              float scale) {
  OAL_TRY(check_common(B, Hq, Hkv, d, dv, dtype, OAL_STATE_FULL));
  if (T < 0) return oal_fail(OAL_ERR_INVALID_ARG, "T=%d", T);
  if (!isfinite(scale)) return oal_fail(OAL_ERR_INVALID_ARG, "scale=%g", scale);
  if (T > 1 << 30 ||
      (long long)B * Hkv * ((T + oal::kGC - 1) / oal::kGC + 1) > 0x3fffffffLL ||
      (long long)B * Hq > 0x7fffffffLL / 64)
    return oal_fail(OAL_ERR_UNSUPPORTED, "problem too large");
  return OAL_OK;
}

static oal_status check_workspace(const void *workspace, size_t bytes, size_t need) {
  OAL_TRY(check_ptr(workspace, "workspace"));
  if (((uintptr_t)workspace & 255u) != 0)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  if (bytes < need)
    return oal_fail(OAL_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", bytes, need);
  return OAL_OK;
}

// The workspace: per (batch, KV head) and segment one state, (backward) one
// state gradient, and one decay.
static size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
static size_t gated_states_bytes(int B, int Hkv, int nseg) {
  return (size_t)B * Hkv * nseg * oal::kGS * sizeof(float);
}

size_t oal_gated_prefill_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int dv,
                                         oal_dtype dtype) {
  if (check_gated(B, Hq, Hkv, T, d, dv, dtype, 1.f) != OAL_OK) return 0;
  if (B == 0 || T == 0) return 256;
  const int chunks = oal::gated_prefill_segment(B, Hkv, T);
  const int nseg = oal::gated_segments(T, chunks);
  return gated_states_bytes(B, Hkv, nseg) + round256((size_t)B * Hkv * nseg * sizeof(oal::GateDecay));
}

oal_status oal_gated_prefill(const void *Q, const void *K, const void *V, oal_dtype dtype,
                             const float *g, int B, int Hq, int Hkv, int T, int d, int dv,
                             float scale, const int32_t *lengths, float *state,
                             int continue_from_state, void *Y, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
  t_msg[0] = 0;
  OAL_TRY(check_gated(B, Hq, Hkv, T, d, dv, dtype, scale));
  t_call_launches = 0;
  if (B == 0) return OAL_OK;
  OAL_TRY(check_ptr(state, "state"));
  if (T == 0) {
    if (!continue_from_state &&
        cudaMemsetAsync(state, 0, gated_states_bytes(B, Hkv, 1), stream) != cudaSuccess)
      return oal_check_launch("state reset");
    return OAL_OK;
  }
  OAL_TRY(check_ptr(Q, "Q"));
  OAL_TRY(check_ptr(K, "K"));
  OAL_TRY(check_ptr(V, "V"));
  OAL_TRY(check_ptr(g, "g"));
  OAL_TRY(check_ptr(Y, "Y"));
  if (lengths) OAL_TRY(check_ptr(lengths, "lengths"));
  OAL_TRY(check_workspace(workspace, workspace_bytes,
                          oal_gated_prefill_workspace_bytes(B, Hq, Hkv, T, d, dv, dtype)));
  oal::GatedArgs p = {};
  p.Q = Q, p.K = K, p.V = V, p.g = g, p.Y = Y;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.T = T, p.scale = scale, p.lengths = lengths;
  p.state_in = continue_from_state ? state : nullptr;
  p.state_out = state;
  p.seg_chunks = oal::gated_prefill_segment(B, Hkv, T);
  p.nseg = oal::gated_segments(T, p.seg_chunks);
  p.seg_state = static_cast<float *>(workspace);
  p.seg_decay = reinterpret_cast<oal::GateDecay *>(static_cast<char *>(workspace) +
                                                   gated_states_bytes(B, Hkv, p.nseg));
  p.status = oal_device_status_word();
  if (!p.status) return oal_fail(OAL_ERR_CUDA, "no device status word");
  oal_begin_call(stream);
  if (dtype == OAL_BF16) return oal::launch_gated_prefill_tc(p, stream);
  return oal::launch_gated_prefill_simt(p, stream);
}

size_t oal_gated_backward_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int dv,
                                          oal_dtype dtype) {
  if (check_gated(B, Hq, Hkv, T, d, dv, dtype, 1.f) != OAL_OK) return 0;
  if (B == 0 || T == 0) return 256;
  const int nseg = oal::gated_segments(T, 1);   // a segment is a chunk
  return 2 * gated_states_bytes(B, Hkv, nseg) +
         round256((size_t)B * Hkv * nseg * sizeof(oal::GateDecay));
}

oal_status oal_gated_backward(const void *Q, const void *K, const void *V, oal_dtype dtype,
                              const float *g, const void *dY, int B, int Hq, int Hkv, int T,
                              int d, int dv, float scale, const int32_t *lengths,
                              const float *state0, const float *dstate, void *dQ, void *dK,
                              void *dV, float *dg, float *dstate0, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  t_msg[0] = 0;
  OAL_TRY(check_gated(B, Hq, Hkv, T, d, dv, dtype, scale));
  t_call_launches = 0;
  if (B == 0) return OAL_OK;
  if (state0) OAL_TRY(check_ptr(state0, "state0"));
  if (dstate) OAL_TRY(check_ptr(dstate, "dstate"));
  if (dstate0) OAL_TRY(check_ptr(dstate0, "dstate0"));
  if (T == 0) {   // the state passes through
    if (!dstate0) return OAL_OK;
    const size_t bytes = gated_states_bytes(B, Hkv, 1);
    const cudaError_t e = dstate ? cudaMemcpyAsync(dstate0, dstate, bytes, cudaMemcpyDeviceToDevice, stream)
                                 : cudaMemsetAsync(dstate0, 0, bytes, stream);
    return e == cudaSuccess ? OAL_OK : oal_check_launch("dstate0");
  }
  OAL_TRY(check_ptr(Q, "Q"));
  OAL_TRY(check_ptr(K, "K"));
  OAL_TRY(check_ptr(V, "V"));
  OAL_TRY(check_ptr(g, "g"));
  OAL_TRY(check_ptr(dY, "dY"));
  OAL_TRY(check_ptr(dQ, "dQ"));
  OAL_TRY(check_ptr(dK, "dK"));
  OAL_TRY(check_ptr(dV, "dV"));
  OAL_TRY(check_ptr(dg, "dg"));
  if (lengths) OAL_TRY(check_ptr(lengths, "lengths"));
  OAL_TRY(check_workspace(workspace, workspace_bytes,
                          oal_gated_backward_workspace_bytes(B, Hq, Hkv, T, d, dv, dtype)));
  oal::GatedArgs p = {};
  p.Q = Q, p.K = K, p.V = V, p.g = g, p.dY = dY;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.T = T, p.scale = scale, p.lengths = lengths;
  p.state_in = state0, p.dstate = dstate, p.dstate0 = dstate0;
  p.dQ = dQ, p.dK = dK, p.dV = dV, p.dg = dg;
  p.seg_chunks = 1;
  p.nseg = oal::gated_segments(T, p.seg_chunks);
  const size_t states = gated_states_bytes(B, Hkv, p.nseg);
  p.seg_state = static_cast<float *>(workspace);
  p.seg_grad = reinterpret_cast<float *>(static_cast<char *>(workspace) + states);
  p.seg_decay = reinterpret_cast<oal::GateDecay *>(static_cast<char *>(workspace) + 2 * states);
  p.status = oal_device_status_word();
  if (!p.status) return oal_fail(OAL_ERR_CUDA, "no device status word");
  oal_begin_call(stream);
  if (dtype == OAL_BF16) return oal::launch_gated_backward_tc(p, stream);
  return oal::launch_gated_backward_simt(p, stream);
}

oal_status oal_gated_decode_step(const void *q, const void *k, const void *v, oal_dtype dtype,
                                 const float *g, int B, int Hq, int Hkv, int d, int dv,
                                 float scale, const int32_t *slots, int n_slots, float *state,
                                 void *y, cudaStream_t stream) {
  t_msg[0] = 0;
  OAL_TRY(check_gated(B, Hq, Hkv, 1, d, dv, dtype, scale));
  if (n_slots < 0 || (!slots && n_slots < B))
    return oal_fail(OAL_ERR_INVALID_ARG, "n_slots=%d for %d sequences", n_slots, B);
  t_call_launches = 0;
  if (B == 0) return OAL_OK;
  OAL_TRY(check_ptr(q, "q"));
  OAL_TRY(check_ptr(k, "k"));
  OAL_TRY(check_ptr(v, "v"));
  OAL_TRY(check_ptr(g, "g"));
  OAL_TRY(check_ptr(y, "y"));
  if (slots) OAL_TRY(check_ptr(slots, "slots"));
  if (n_slots > 0) OAL_TRY(check_ptr(state, "state"));
  oal_begin_call(stream);
  return oal::launch_gated_decode(q, k, v, dtype == OAL_BF16, g, B, Hq, Hkv, scale, slots,
                                  n_slots, state, y, stream);
}

oal_status oal_state_remap(void *pool, size_t slot_bytes, int n_slots, const int32_t *map,
                           cudaStream_t stream) {
  t_msg[0] = 0;
  if (n_slots < 0) return oal_fail(OAL_ERR_INVALID_ARG, "n_slots=%d", n_slots);
  if (n_slots > OAL_REMAP_MAX_SLOTS)
    return oal_fail(OAL_ERR_UNSUPPORTED, "n_slots=%d above %d", n_slots, OAL_REMAP_MAX_SLOTS);
  t_call_launches = 0;
  if (n_slots == 0 || slot_bytes == 0) return OAL_OK;
  if (slot_bytes > ((size_t)1 << 46) / (size_t)n_slots)
    return oal_fail(OAL_ERR_UNSUPPORTED, "pool too large");
  OAL_TRY(check_ptr(pool, "pool"));
  OAL_TRY(check_ptr(map, "map"));
  oal_begin_call(stream);
  return oal::launch_state_remap(pool, slot_bytes, n_slots, map, stream);
}

// ---- rotary positions, the paged cache, attention over it

oal_status oal_rope_plan(const double *freq, const int32_t *axes, int64_t *plan) {
  t_msg[0] = 0;
  if (!freq || !plan) return oal_fail(OAL_ERR_INVALID_ARG, "freq or plan is null");
  for (int r = 0; r < oal::kD / 2; ++r) {
    if (!isfinite(freq[r])) return oal_fail(OAL_ERR_INVALID_ARG, "freq[%d]=%g", r, freq[r]);
    if (axes && axes[r] < 0) return oal_fail(OAL_ERR_INVALID_ARG, "axes[%d]=%d", r, axes[r]);
    // freq / 2 pi as a sum of two doubles, without its whole turns, in units of 2^-64
    const double inv = 0x1.45f306dc9c883p-3, rest = -0x1.6b01ec5417056p-57;   // 1 / (2 pi)
    const double f = fabs(freq[r]), hi = f * inv, lo = fma(f, inv, -hi) + f * rest;
    const uint64_t turns = (uint64_t)((hi - floor(hi)) * 0x1p64) +
                           (uint64_t)(int64_t)llrint((lo - floor(lo + 0.5)) * 0x1p63) * 2;
    plan[r] = (int64_t)(freq[r] < 0.0 ? 0 - turns : turns);
    plan[oal::kD / 2 + r] = axes ? axes[r] : 0;
  }
  return OAL_OK;
}

// Sizes, positions and lengths of a call that turns rows; strides of its tensors.
static oal_status rope_args(oal::RopeArgs &p, oal_dtype dtype, const void *const *x, int tensors,
                            const int64_t *strides, int B, int Hq, int Hkv, int T, int d,
                            const int64_t *plan, oal_rope_form form, const int32_t *positions,
                            int n_axes, const int32_t *past, const int32_t *lengths) {
  static const char *const names[3] = {"Q", "K", "V"};
  if (B < 0 || T < 0 || (x[0] && Hq <= 0) || (x[1] && Hkv <= 0))
    return oal_fail(OAL_ERR_INVALID_ARG, "bad sizes B=%d Hq=%d Hkv=%d T=%d", B, Hq, Hkv, T);
  if (dtype != OAL_F32 && dtype != OAL_BF16)
    return oal_fail(OAL_ERR_INVALID_ARG, "bad dtype %d", (int)dtype);
  if (form != OAL_ROPE_HALVES && form != OAL_ROPE_PAIRS)
    return oal_fail(OAL_ERR_INVALID_ARG, "bad form %d", (int)form);
  if (d != oal::kD) return oal_fail(OAL_ERR_UNSUPPORTED, "only d = 64 is supported (d=%d)", d);
  if ((long long)B * T > 1LL << 31 || (long long)Hq + 2LL * Hkv > 1 << 16)
    return oal_fail(OAL_ERR_UNSUPPORTED, "problem too large");
  if (positions && n_axes < 1) return oal_fail(OAL_ERR_INVALID_ARG, "n_axes=%d", n_axes);
  const int heads[3] = {Hq, Hkv, Hkv};
  oal::RowStrides *to[3] = {&p.q, &p.k, &p.v};
  const int unit = dtype == OAL_BF16 ? 8 : 4;
  for (int i = 0; i < tensors; ++i) {
    *to[i] = {(long long)heads[i] * T * 64, (long long)T * 64, 64};
    if (!x[i] || !strides) continue;
    *to[i] = {strides[3 * i], strides[3 * i + 1], strides[3 * i + 2]};
    for (int e = 0; e < 3; ++e)
      if (strides[3 * i + e] % unit != 0 || strides[3 * i + e] < 0)
        return oal_fail(OAL_ERR_INVALID_ARG, "stride %lld of %s is negative or no multiple of 16 bytes",
                        (long long)strides[3 * i + e], names[i]);
  }
  p.Q = x[0], p.K = x[1], p.V = tensors > 2 ? x[2] : nullptr;
  p.B = B, p.Hq = x[0] ? Hq : 0, p.Hkv = x[1] ? Hkv : 0, p.T = T;
  p.turns = reinterpret_cast<const unsigned long long *>(plan);
  p.axes = plan ? reinterpret_cast<const long long *>(plan) + oal::kD / 2 : nullptr;
  p.positions = positions, p.n_axes = n_axes, p.past = past, p.lengths = lengths;
  return OAL_OK;
}

oal_status oal_rope(const void *Q, const void *K, oal_dtype dtype, const int64_t *strides, int B,
                    int Hq, int Hkv, int T, int d, const int64_t *plan, oal_rope_form form,
                    const int32_t *positions, int n_axes, const int32_t *past,
                    const int32_t *lengths, int inverse, void *Yq, void *Yk, cudaStream_t stream) {
  t_msg[0] = 0;
  oal::RopeArgs p = {};
  const void *const x[2] = {Q, K};
  OAL_TRY(rope_args(p, dtype, x, 2, strides, B, Hq, Hkv, T, d, plan, form, positions, n_axes, past, lengths));
  t_call_launches = 0;
  if (B == 0 || T == 0) return OAL_OK;
  OAL_TRY(check_ptr(Q, "Q"));
  OAL_TRY(check_ptr(Yq, "Yq"));
  if (K) OAL_TRY(check_ptr(K, "K"));
  if (K) OAL_TRY(check_ptr(Yk, "Yk"));
  OAL_TRY(check_ptr(plan, "plan"));
  if (positions) OAL_TRY(check_ptr(positions, "positions"));
  if (past) OAL_TRY(check_ptr(past, "past"));
  if (lengths) OAL_TRY(check_ptr(lengths, "lengths"));
  p.Yq = Yq, p.Yk = Yk, p.inverse = inverse != 0;
  p.status = oal_device_status_word();
  if (!p.status) return oal_fail(OAL_ERR_CUDA, "no device status word");
  oal_begin_call(stream);
  return oal::launch_rope(p, dtype == OAL_BF16, form, "rope_kernel", stream);
}

static oal_status check_pages(oal_dtype dtype, int Hkv, int n_pages, int page_size,
                              int64_t page_stride, int max_pages, int *shift) {
  if (n_pages < 0 || max_pages < 0)
    return oal_fail(OAL_ERR_INVALID_ARG, "n_pages=%d max_pages=%d", n_pages, max_pages);
  if (page_size < 1 || (page_size & (page_size - 1)) != 0)
    return oal_fail(OAL_ERR_INVALID_ARG, "page_size=%d is not a power of two", page_size);
  if (page_size < 16 || page_size > 65536 || (long long)page_size * max_pages > 1LL << 30)
    return oal_fail(OAL_ERR_UNSUPPORTED, "page_size=%d, max_pages=%d", page_size, max_pages);
  if (page_stride < (int64_t)Hkv * page_size * oal::kD || page_stride % (dtype == OAL_BF16 ? 8 : 4) != 0 ||
      page_stride > 1LL << 38)
    return oal_fail(OAL_ERR_INVALID_ARG, "page_stride=%lld", (long long)page_stride);
  *shift = 0;
  while (1 << *shift < page_size) ++*shift;
  return OAL_OK;
}

oal_status oal_page_append(const void *Q, const void *K, const void *V, oal_dtype dtype,
                           const int64_t *strides, int B, int Hq, int Hkv, int T, int d, int dv,
                           const int64_t *plan, oal_rope_form form, const int32_t *positions,
                           int n_axes, const int32_t *past, const int32_t *lengths, void *Kp,
                           void *Vp, int n_pages, int page_size, int64_t page_stride,
                           const int32_t *table, int max_pages, void *Yq, cudaStream_t stream) {
  t_msg[0] = 0;
  oal::RopeArgs p = {};
  const void *const x[3] = {Q, K, V};
  if (dv != oal::kDv) return oal_fail(OAL_ERR_UNSUPPORTED, "only dv = 64 is supported (dv=%d)", dv);
  if (Hkv <= 0) return oal_fail(OAL_ERR_INVALID_ARG, "Hkv=%d", Hkv);
  OAL_TRY(rope_args(p, dtype, x, 3, strides, B, Hq, Hkv, T, d, plan, form, positions, n_axes, past, lengths));
  OAL_TRY(check_pages(dtype, Hkv, n_pages, page_size, page_stride, max_pages, &p.page_shift));
  if (!plan && Q) return oal_fail(OAL_ERR_INVALID_ARG, "Q without a plan");
  t_call_launches = 0;
  if (B == 0 || T == 0) return OAL_OK;
  if (Q) OAL_TRY(check_ptr(Q, "Q"));
  if (Q) OAL_TRY(check_ptr(Yq, "Yq"));
  OAL_TRY(check_ptr(K, "K"));
  OAL_TRY(check_ptr(V, "V"));
  if (plan) OAL_TRY(check_ptr(plan, "plan"));
  if (positions) OAL_TRY(check_ptr(positions, "positions"));
  OAL_TRY(check_ptr(past, "past"));
  if (lengths) OAL_TRY(check_ptr(lengths, "lengths"));
  OAL_TRY(check_ptr(Kp, "Kp"));
  OAL_TRY(check_ptr(Vp, "Vp"));
  OAL_TRY(check_ptr(table, "table"));
  p.Yq = Yq, p.Kp = Kp, p.Vp = Vp;
  p.n_pages = n_pages, p.max_pages = max_pages, p.page_stride = page_stride, p.table = table;
  p.status = oal_device_status_word();
  if (!p.status) return oal_fail(OAL_ERR_CUDA, "no device status word");
  oal_begin_call(stream);
  return oal::launch_rope(p, dtype == OAL_BF16, form, "page_append_kernel", stream);
}

static oal_status check_paged(oal::PagedArgs &p, int B, int Hq, int Hkv, int T, int d, int dv,
                              oal_dtype dtype, int n_pages, int page_size, int64_t page_stride,
                              int max_pages) {
  OAL_TRY(check_common(B, Hq, Hkv, d, dv, dtype, OAL_STATE_FULL));
  if (T < 0) return oal_fail(OAL_ERR_INVALID_ARG, "T=%d", T);
  OAL_TRY(check_pages(dtype, Hkv, n_pages, page_size, page_stride, max_pages, &p.page_shift));
  const int rho = Hq / Hkv;
  if (rho > 128 || (long long)B * Hkv > 65535 || (long long)T * rho > 1LL << 28 ||
      (long long)B * Hkv * T > 1LL << 31)
    return oal_fail(OAL_ERR_UNSUPPORTED, "problem too large");
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.T = T, p.rho = rho;
  p.n_pages = n_pages, p.max_pages = max_pages, p.page_stride = page_stride;
  return OAL_OK;
}

size_t oal_paged_attention_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int dv,
                                           oal_dtype dtype, int page_size, int max_pages) {
  oal::PagedArgs p = {};
  const int64_t stride = (int64_t)Hkv * page_size * d;
  if (check_paged(p, B, Hq, Hkv, T, d, dv, dtype, 0, page_size, stride, max_pages) != OAL_OK) return 0;
  if (B == 0 || T == 0) return 256;
  return oal::paged_workspace_bytes(p, dtype == OAL_BF16);
}

oal_status oal_paged_attention(const void *Q, oal_dtype dtype, int B, int Hq, int Hkv, int T,
                               int d, int dv, const void *Kp, const void *Vp, int n_pages,
                               int page_size, int64_t page_stride, const int32_t *table,
                               int max_pages, const int32_t *past, const int32_t *lengths,
                               float scale, float cap, int window, const float *slopes,
                               const int32_t *prefix, const int32_t *first, void *Y,
                               void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  t_msg[0] = 0;
  oal::PagedArgs p = {};
  OAL_TRY(check_paged(p, B, Hq, Hkv, T, d, dv, dtype, n_pages, page_size, page_stride, max_pages));
  if (!(scale > 0.f) || !isfinite(scale)) return oal_fail(OAL_ERR_INVALID_ARG, "scale=%g", scale);
  if (!(cap >= 0.f) || !isfinite(cap) || (cap > 0.f && !isfinite(4.f * scale / cap)))
    return oal_fail(OAL_ERR_INVALID_ARG, "cap=%g", cap);
  if (window < 0) return oal_fail(OAL_ERR_INVALID_ARG, "window=%d", window);
  t_call_launches = 0;
  if (B == 0 || T == 0) return OAL_OK;
  OAL_TRY(check_ptr(Q, "Q"));
  OAL_TRY(check_ptr(Kp, "Kp"));
  OAL_TRY(check_ptr(Vp, "Vp"));
  OAL_TRY(check_ptr(table, "table"));
  OAL_TRY(check_ptr(past, "past"));
  OAL_TRY(check_ptr(Y, "Y"));
  if (lengths) OAL_TRY(check_ptr(lengths, "lengths"));
  if (slopes) OAL_TRY(check_ptr(slopes, "slopes"));
  if (prefix) OAL_TRY(check_ptr(prefix, "prefix"));
  if (first) OAL_TRY(check_ptr(first, "first"));
  const size_t need = oal::paged_workspace_bytes(p, dtype == OAL_BF16);
  if (workspace || need > 256) OAL_TRY(check_workspace(workspace, workspace_bytes, need));
  p.Q = Q, p.Kp = Kp, p.Vp = Vp, p.Y = Y, p.table = table, p.past = past, p.lengths = lengths;
  p.scale = scale, p.cap = cap, p.window = window;
  p.slopes = slopes, p.prefix = prefix, p.first = first;
  p.status = oal_device_status_word();
  if (!p.status) return oal_fail(OAL_ERR_CUDA, "no device status word");
  oal_begin_call(stream);
  return oal::launch_paged(p, dtype == OAL_BF16, workspace, stream);
}

oal_status oal_debug_wait_test(uint64_t wait_limit_cycles, int starve) {
  t_msg[0] = 0;
  if (starve < 0 || starve > 3) return oal_fail(OAL_ERR_INVALID_ARG, "starve=%d", starve);
  int *w = oal_device_status_word();
  if (!w) return oal_fail(OAL_ERR_CUDA, "device control block unavailable");
  oal::DeviceControl c;
  cudaError_t e = cudaMemcpy(&c, w, sizeof c, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) {
    c.starve = starve;
    c.wait_limit = wait_limit_cycles;
    e = cudaMemcpy(w, &c, sizeof c, cudaMemcpyHostToDevice);
  }
  if (e != cudaSuccess)
    return oal_fail(OAL_ERR_CUDA, "setting the wait test: %s", cudaGetErrorString(e));
  return OAL_OK;
}

oal_status oal_debug_intra_heads(int heads) {
  t_msg[0] = 0;
  if (heads < 0 || heads > 2) return oal_fail(OAL_ERR_INVALID_ARG, "heads=%d", heads);
  oal::set_intra_heads(heads);
  return OAL_OK;
}

oal_status oal_sync_status(cudaStream_t stream) {
  t_msg[0] = 0;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess)
    return oal_fail(OAL_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
  int *w = oal_device_status_word();
  if (!w) return oal_fail(OAL_ERR_CUDA, "status word unavailable");
  int v = 0;
  e = cudaMemcpy(&v, w, sizeof v, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return oal_fail(OAL_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
  if (v != 0) {
    const int zero = 0;
    cudaMemcpy(w, &zero, sizeof zero, cudaMemcpyHostToDevice);
    const char *what = v == OAL_ERR_INVALID_ARG ? "a group id outside 1..G, a "
                                                  "sequence length outside 0..T, a "
                                                  "slot out of range or taken twice, or a "
                                                  "page or an axis out of range"
                       : v == OAL_ERR_TIMEOUT   ? "a device-side wait timed out"
                                                : "device error";
    return oal_fail((oal_status)v, "device status %d: %s", v, what);
  }
  return OAL_OK;
}

}  // extern "C"
