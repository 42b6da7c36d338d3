// Exported C entry points of libgdn: host-side argument validation, then the
// launchers.  Nothing is launched unless every check passes.
#include <hip/hip_runtime.h>

#include "launch.h"

using namespace gdn;

namespace {

constexpr int64_t kMaxTokens = 0x7fffffffLL;  // cu_seqlens is int32

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t esize(gdn_dtype d) { return d == GDN_FP32 ? 4 : 2; }
bool dtype_ok(gdn_dtype d) { return d == GDN_BF16 || d == GDN_FP32 || d == GDN_FP16; }

gdn_status check_shape(const gdn_shape* s) {
  if (!s) return GDN_ERR_INVALID_ARG;
  if (s->n_seq < 1 || s->total_tokens < 0 || s->total_tokens > kMaxTokens || s->hk < 1 ||
      s->hv < 1 || s->dk < 1 || s->dv < 1 || !dtype_ok(s->dtype))
    return GDN_ERR_INVALID_ARG;
  if (s->hv % s->hk != 0) return GDN_ERR_INVALID_ARG;
  if (s->dk != s->dv || (s->dk != 32 && s->dk != 128)) return GDN_ERR_UNSUPPORTED;
  if (s->conv_k != 4 || s->chunk != CHUNK) return GDN_ERR_UNSUPPORTED;
  if (s->hv > 256 || s->n_seq > 65535) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int64_t channels(const gdn_shape* s) { return 2LL * s->hk * s->dk + (int64_t)s->hv * s->dv; }

gdn_status check_ld(int64_t ld, int64_t min_cols) {
  if (ld < min_cols) return GDN_ERR_INVALID_ARG;
  if (ld % 8) return GDN_ERR_ALIGNMENT;
  return GDN_OK;
}

gdn_status check_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
  }
  return GDN_OK;
}

gdn_status chunk_supported(const gdn_shape* s) {
  // fp32 storage is supported at head dim 32 (the fp32 workload); bf16 and fp16 at 32 and 128
  if (s->dtype == GDN_FP32 && s->dk != 32) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status launched(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

#define GDN_TRY(x)                   \
  do {                               \
    gdn_status _st = (x);            \
    if (_st != GDN_OK) return _st;   \
  } while (0)

}  // namespace

extern "C" {

const char* gdn_status_string(gdn_status s) {
  switch (s) {
    case GDN_OK: return "ok";
    case GDN_ERR_INVALID_ARG: return "invalid argument";
    case GDN_ERR_UNSUPPORTED: return "unsupported configuration";
    case GDN_ERR_ALIGNMENT: return "pointer or row stride not 16-byte aligned";
    case GDN_ERR_WORKSPACE: return "workspace missing or too small";
    case GDN_ERR_LAUNCH: return "kernel launch failed";
  }
  return "unknown status";
}

gdn_status gdn_conv_fwd(const gdn_shape* s, const void* x, int64_t ldx, const float* w,
                        const int32_t* cu, int l2norm_qk, float l2_eps, void* y, int64_t ldy,
                        void* stream) {
  GDN_TRY(check_shape(s));
  GDN_TRY(check_ptrs({x, w, cu, y}));
  GDN_TRY(check_ld(ldx, channels(s)));
  GDN_TRY(check_ld(ldy, channels(s)));
  if (!(l2_eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  return launched(launch_conv_fwd(*s, x, ldx, w, cu, l2norm_qk != 0, l2_eps, y, ldy, nullptr,
                                  nullptr, (hipStream_t)stream));
}

size_t gdn_conv_bwd_workspace(const gdn_shape* s) {
  if (check_shape(s) != GDN_OK) return 0;
  return sizeof(float) * (size_t)conv_partials(s->total_tokens, conv_tt(s->total_tokens, channels(s))) *
         (size_t)channels(s) * 4;
}

gdn_status gdn_conv_bwd(const gdn_shape* s, const void* x, int64_t ldx, const float* w,
                        const int32_t* cu, int l2norm_qk, float l2_eps, const void* dy,
                        int64_t lddy, void* dx, int64_t lddx, float* dw, void* ws,
                        size_t ws_bytes, void* stream) {
  GDN_TRY(check_shape(s));
  GDN_TRY(check_ptrs({x, w, cu, dy, dx, dw}));
  GDN_TRY(check_ld(ldx, channels(s)));
  GDN_TRY(check_ld(lddy, channels(s)));
  GDN_TRY(check_ld(lddx, channels(s)));
  if (!(l2_eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_conv_bwd_workspace(s);
  if (need && (!ws || ws_bytes < need || !aligned16(ws))) return GDN_ERR_WORKSPACE;
  return launched(launch_conv_bwd(*s, x, ldx, w, cu, l2norm_qk != 0, l2_eps, dy, lddy, dx, lddx,
                                  dw, (float*)ws, nullptr, nullptr, nullptr, (hipStream_t)stream));
}

gdn_status gdn_conv_fwd_state(const gdn_shape* s, const void* x, int64_t ldx, const float* w,
                              const int32_t* cu, int l2norm_qk, float l2_eps,
                              const void* conv_state_in, void* y, int64_t ldy,
                              void* conv_state_out, void* stream) {
  GDN_TRY(check_shape(s));
  GDN_TRY(check_ptrs({x, w, cu, y}));
  GDN_TRY(check_ld(ldx, channels(s)));
  GDN_TRY(check_ld(ldy, channels(s)));
  if ((conv_state_in && !aligned16(conv_state_in)) || (conv_state_out && !aligned16(conv_state_out)))
    return GDN_ERR_ALIGNMENT;
  if (!(l2_eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  return launched(launch_conv_fwd(*s, x, ldx, w, cu, l2norm_qk != 0, l2_eps, y, ldy, conv_state_in,
                                  conv_state_out, (hipStream_t)stream));
}

gdn_status gdn_conv_bwd_state(const gdn_shape* s, const void* x, int64_t ldx, const float* w,
                              const int32_t* cu, int l2norm_qk, float l2_eps,
                              const void* conv_state_in, const void* dy, int64_t lddy,
                              const void* d_conv_state_out, void* dx, int64_t lddx, float* dw,
                              void* d_conv_state_in, void* ws, size_t ws_bytes, void* stream) {
  GDN_TRY(check_shape(s));
  GDN_TRY(check_ptrs({x, w, cu, dy, dx, dw}));
  GDN_TRY(check_ld(ldx, channels(s)));
  GDN_TRY(check_ld(lddy, channels(s)));
  GDN_TRY(check_ld(lddx, channels(s)));
  for (const void* p : {conv_state_in, d_conv_state_out, (const void*)d_conv_state_in})
    if (p && !aligned16(p)) return GDN_ERR_ALIGNMENT;
  if (!(l2_eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_conv_bwd_workspace(s);
  if (need && (!ws || ws_bytes < need || !aligned16(ws))) return GDN_ERR_WORKSPACE;
  return launched(launch_conv_bwd(*s, x, ldx, w, cu, l2norm_qk != 0, l2_eps, dy, lddy, dx, lddx,
                                  dw, (float*)ws, conv_state_in, d_conv_state_out, d_conv_state_in,
                                  (hipStream_t)stream));
}

gdn_status gdn_conv_bwd_noalloc(const gdn_shape* s, const void* x, int64_t ldx, const float* w,
                                const int32_t* cu, int l2norm_qk, float l2_eps, const void* dy,
                                int64_t lddy, void* dx, int64_t lddx, float* dw, void* stream) {
  GDN_TRY(check_shape(s));
  GDN_TRY(check_ptrs({x, w, cu, dy, dx, dw}));
  GDN_TRY(check_ld(ldx, channels(s)));
  GDN_TRY(check_ld(lddy, channels(s)));
  GDN_TRY(check_ld(lddx, channels(s)));
  if (!(l2_eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (gdn_conv_bwd_workspace(s) > CONV_BWD_NOALLOC_MAX_BYTES) return GDN_ERR_WORKSPACE;
  return launched(launch_conv_bwd_noalloc(*s, x, ldx, w, cu, l2norm_qk != 0, l2_eps, dy, lddy,
                                          dx, lddx, dw, (hipStream_t)stream));
}

gdn_status gdn_gate_fwd(const gdn_shape* s, const void* a, const void* b, const float* A_log,
                        const float* dt_bias, float* g, float* beta, void* stream) {
  GDN_TRY(check_shape(s));
  if (!a || !b || !A_log || !dt_bias || !g || !beta) return GDN_ERR_INVALID_ARG;
  return launched(launch_gate_fwd(*s, a, b, A_log, dt_bias, g, beta, (hipStream_t)stream));
}

size_t gdn_gate_bwd_workspace(const gdn_shape* s) {
  if (check_shape(s) != GDN_OK) return 0;
  return sizeof(float) * (size_t)gate_partials(s->total_tokens) * 2 * (size_t)s->hv;
}

gdn_status gdn_gate_bwd(const gdn_shape* s, const void* a, const void* b, const float* A_log,
                        const float* dt_bias, const float* dg, const float* dbeta, void* da,
                        void* db, float* dA_log, float* ddt_bias, void* ws, size_t ws_bytes,
                        void* stream) {
  GDN_TRY(check_shape(s));
  if (!a || !b || !A_log || !dt_bias || !dg || !dbeta || !da || !db || !dA_log || !ddt_bias)
    return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_gate_bwd_workspace(s);
  if (need && (!ws || ws_bytes < need || !aligned16(ws))) return GDN_ERR_WORKSPACE;
  return launched(launch_gate_bwd(*s, a, b, A_log, dt_bias, dg, dbeta, da, db, dA_log, ddt_bias,
                                  (float*)ws, (hipStream_t)stream));
}

size_t gdn_chunk_fwd_workspace(const gdn_shape* s) {
  if (check_shape(s) != GDN_OK) return 0;
  return chunk_fwd_ws_bytes(*s);
}

size_t gdn_chunk_bwd_workspace(const gdn_shape* s) {
  if (check_shape(s) != GDN_OK) return 0;
  return chunk_bwd_ws_bytes(*s);
}

gdn_status gdn_chunk_fwd(const gdn_shape* s, const void* q, const void* k, const void* v,
                         int64_t ldq, int64_t ldk, int64_t ldv, const float* g,
                         const float* beta, float scale, const float* S0, float* S_final,
                         const int32_t* cu, void* o, void* ws, size_t ws_bytes, void* stream) {
  GDN_TRY(check_shape(s));
  GDN_TRY(chunk_supported(s));
  GDN_TRY(check_ptrs({q, k, v, o, ws}));
  if (!g || !beta || !cu) return GDN_ERR_INVALID_ARG;
  if ((S0 && !aligned16(S0)) || (S_final && !aligned16(S_final))) return GDN_ERR_ALIGNMENT;
  GDN_TRY(check_ld(ldq, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(ldk, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(ldv, (int64_t)s->hv * s->dv));
  if (ws_bytes < chunk_fwd_ws_bytes(*s)) return GDN_ERR_WORKSPACE;
  return launched(launch_chunk_fwd(*s, q, k, v, ldq, ldk, ldv, g, beta, scale, S0, S_final, cu, o,
                                   ws, (hipStream_t)stream));
}

gdn_status gdn_chunk_bwd(const gdn_shape* s, const void* q, const void* k, const void* v,
                         int64_t ldq, int64_t ldk, int64_t ldv, const float* g,
                         const float* beta, float scale, const float* S0, const int32_t* cu,
                         const void* dout, const float* dS_final, void* dq, void* dk, void* dv,
                         int64_t lddq, int64_t lddk, int64_t lddv, float* dg, float* dbeta,
                         float* dS0, void* ws, size_t ws_bytes, void* stream) {
  GDN_TRY(check_shape(s));
  GDN_TRY(chunk_supported(s));
  GDN_TRY(check_ptrs({q, k, v, dout, dq, dk, dv, ws}));
  if (!g || !beta || !cu || !dg || !dbeta) return GDN_ERR_INVALID_ARG;
  if ((S0 && !aligned16(S0)) || (dS_final && !aligned16(dS_final)) || (dS0 && !aligned16(dS0)))
    return GDN_ERR_ALIGNMENT;
  GDN_TRY(check_ld(ldq, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(ldk, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(ldv, (int64_t)s->hv * s->dv));
  GDN_TRY(check_ld(lddq, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(lddk, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(lddv, (int64_t)s->hv * s->dv));
  if (ws_bytes < chunk_bwd_ws_bytes(*s)) return GDN_ERR_WORKSPACE;
  return launched(launch_chunk_bwd(*s, q, k, v, ldq, ldk, ldv, g, beta, scale, S0, cu, dout,
                                   dS_final, dq, dk, dv, lddq, lddk, lddv, dg, dbeta, dS0, ws,
                                   (hipStream_t)stream));
}

// ---- chunk phases -----------------------------------------------------------
namespace {
gdn_status check_chunk_common(const gdn_shape* s, const void* q, const void* k, int64_t ldq,
                              int64_t ldk, const void* cu, const void* ws, size_t ws_bytes,
                              size_t need) {
  GDN_TRY(check_shape(s));
  GDN_TRY(chunk_supported(s));
  GDN_TRY(check_ptrs({q, k, ws}));
  if (!cu) return GDN_ERR_INVALID_ARG;
  GDN_TRY(check_ld(ldq, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(ldk, (int64_t)s->hk * s->dk));
  if (ws_bytes < need) return GDN_ERR_WORKSPACE;
  return GDN_OK;
}
}  // namespace

gdn_status gdn_chunk_prepare(const gdn_shape* s, const void* q, const void* k, int64_t ldq,
                             int64_t ldk, const float* g, const float* beta, float scale,
                             const int32_t* cu, void* ws, size_t ws_bytes, void* stream) {
  GDN_TRY(check_chunk_common(s, q, k, ldq, ldk, cu, ws, ws_bytes,
                             s ? chunk_fwd_ws_bytes(*s) : 0));
  if (!g || !beta) return GDN_ERR_INVALID_ARG;
  return launched(launch_chunk_prepare(*s, q, k, ldq, ldk, g, beta, scale, cu, ws, false,
                                       (hipStream_t)stream));
}

gdn_status gdn_chunk_prepare_bwd(const gdn_shape* s, const void* q, const void* k, int64_t ldq,
                                 int64_t ldk, const float* g, const float* beta, float scale,
                                 const int32_t* cu, void* ws, size_t ws_bytes, void* stream) {
  GDN_TRY(check_chunk_common(s, q, k, ldq, ldk, cu, ws, ws_bytes,
                             s ? chunk_bwd_ws_bytes(*s) : 0));
  if (!g || !beta) return GDN_ERR_INVALID_ARG;
  return launched(launch_chunk_prepare(*s, q, k, ldq, ldk, g, beta, scale, cu, ws, true,
                                       (hipStream_t)stream));
}

gdn_status gdn_chunk_fwd_states(const gdn_shape* s, const void* q, const void* k, const void* v,
                                int64_t ldq, int64_t ldk, int64_t ldv, float scale,
                                const float* S0, float* S_final, const int32_t* cu, void* o,
                                void* ws, size_t ws_bytes, void* stream) {
  GDN_TRY(check_chunk_common(s, q, k, ldq, ldk, cu, ws, ws_bytes,
                             s ? chunk_fwd_ws_bytes(*s) : 0));
  GDN_TRY(check_ptrs({v, o}));
  GDN_TRY(check_ld(ldv, (int64_t)s->hv * s->dv));
  if ((S0 && !aligned16(S0)) || (S_final && !aligned16(S_final))) return GDN_ERR_ALIGNMENT;
  return launched(launch_chunk_fwd_states(*s, q, k, v, ldq, ldk, ldv, scale, S0, S_final, cu, o,
                                          ws, (hipStream_t)stream));
}

gdn_status gdn_chunk_fwd_states_save(const gdn_shape* s, const void* q, const void* k,
                                     const void* v, int64_t ldq, int64_t ldk, int64_t ldv,
                                     float scale, const float* S0, float* S_final,
                                     const int32_t* cu, void* o, void* ws, size_t ws_bytes,
                                     void* stream) {
  GDN_TRY(check_chunk_common(s, q, k, ldq, ldk, cu, ws, ws_bytes,
                             s ? chunk_bwd_ws_bytes(*s) : 0));
  GDN_TRY(check_ptrs({v, o}));
  GDN_TRY(check_ld(ldv, (int64_t)s->hv * s->dv));
  if ((S0 && !aligned16(S0)) || (S_final && !aligned16(S_final))) return GDN_ERR_ALIGNMENT;
  return launched(launch_chunk_fwd_states_save(*s, q, k, v, ldq, ldk, ldv, scale, S0, S_final, cu,
                                               o, ws, (hipStream_t)stream));
}

gdn_status gdn_chunk_bwd_states(const gdn_shape* s, const void* q, const void* k, const void* v,
                                int64_t ldq, int64_t ldk, int64_t ldv, float scale,
                                const float* S0, const int32_t* cu, void* ws, size_t ws_bytes,
                                void* stream) {
  GDN_TRY(check_chunk_common(s, q, k, ldq, ldk, cu, ws, ws_bytes,
                             s ? chunk_bwd_ws_bytes(*s) : 0));
  GDN_TRY(check_ptrs({v}));
  GDN_TRY(check_ld(ldv, (int64_t)s->hv * s->dv));
  if (S0 && !aligned16(S0)) return GDN_ERR_ALIGNMENT;
  return launched(launch_chunk_bwd_states(*s, q, k, v, ldq, ldk, ldv, scale, S0, cu, ws,
                                          (hipStream_t)stream));
}

gdn_status gdn_chunk_bwd_reverse(const gdn_shape* s, const void* q, const void* k, int64_t ldq,
                                 int64_t ldk, float scale, const int32_t* cu, const void* dout,
                                 const float* dS_final, void* dv, int64_t lddv, float* dS0,
                                 void* ws, size_t ws_bytes, void* stream) {
  GDN_TRY(check_chunk_common(s, q, k, ldq, ldk, cu, ws, ws_bytes,
                             s ? chunk_bwd_ws_bytes(*s) : 0));
  GDN_TRY(check_ptrs({dout, dv}));
  GDN_TRY(check_ld(lddv, (int64_t)s->hv * s->dv));
  if ((dS_final && !aligned16(dS_final)) || (dS0 && !aligned16(dS0))) return GDN_ERR_ALIGNMENT;
  return launched(launch_chunk_bwd_reverse(*s, q, k, ldq, ldk, scale, cu, dout, dS_final, dv, lddv,
                                           dS0, ws, (hipStream_t)stream));
}

gdn_status gdn_chunk_bwd_grads(const gdn_shape* s, const void* q, const void* k, int64_t ldq,
                               int64_t ldk, const float* beta, float scale, const int32_t* cu,
                               const void* dout, const void* dv, int64_t lddv, void* dq, void* dk,
                               int64_t lddq, int64_t lddk, float* dg, float* dbeta, void* ws,
                               size_t ws_bytes, void* stream) {
  GDN_TRY(check_chunk_common(s, q, k, ldq, ldk, cu, ws, ws_bytes,
                             s ? chunk_bwd_ws_bytes(*s) : 0));
  GDN_TRY(check_ptrs({dout, dv, dq, dk}));
  if (!beta || !dg || !dbeta) return GDN_ERR_INVALID_ARG;
  GDN_TRY(check_ld(lddv, (int64_t)s->hv * s->dv));
  GDN_TRY(check_ld(lddq, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(lddk, (int64_t)s->hk * s->dk));
  return launched(launch_chunk_bwd_grads(*s, q, k, ldq, ldk, beta, scale, cu, dout, dv, lddv, dq,
                                         dk, lddq, lddk, dg, dbeta, ws, (hipStream_t)stream));
}

gdn_status gdn_gated_norm_fwd(int64_t rows, int32_t dv, gdn_dtype dt, const void* o, const void* z,
                              const float* w, float eps, gdn_act act, void* y, void* stream) {
  if (rows < 0 || !dtype_ok(dt) || (act != GDN_ACT_SILU && act != GDN_ACT_SIGMOID))
    return GDN_ERR_INVALID_ARG;
  if (dv != 32 && dv != 128) return GDN_ERR_UNSUPPORTED;
  GDN_TRY(check_ptrs({o, z, w, y}));
  if (!(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  return launched(launch_norm_fwd(rows, dv, dt, o, z, w, eps, (int)act, y, (hipStream_t)stream));
}

size_t gdn_gated_norm_bwd_workspace(int64_t rows, int32_t dv) {
  if (rows < 0 || (dv != 32 && dv != 128)) return 0;
  return sizeof(float) * (size_t)norm_blocks(rows, dv) * (size_t)dv;
}

gdn_status gdn_gated_norm_bwd(int64_t rows, int32_t dv, gdn_dtype dt, const void* o, const void* z,
                              const float* w, float eps, gdn_act act, const void* dy, void* dout,
                              void* dz, float* dw, void* ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || !dtype_ok(dt) || (act != GDN_ACT_SILU && act != GDN_ACT_SIGMOID))
    return GDN_ERR_INVALID_ARG;
  if (dv != 32 && dv != 128) return GDN_ERR_UNSUPPORTED;
  GDN_TRY(check_ptrs({o, z, w, dy, dout, dz, dw}));
  if (!(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_gated_norm_bwd_workspace(rows, dv);
  if (!ws || ws_bytes < need || !aligned16(ws)) return GDN_ERR_WORKSPACE;
  return launched(launch_norm_bwd(rows, dv, dt, o, z, w, eps, (int)act, dy, dout, dz, dw,
                                  (float*)ws, (hipStream_t)stream));
}

gdn_status gdn_check_cu_seqlens(const gdn_shape* s, const int32_t* cu, int32_t* violations,
                                void* stream) {
  GDN_TRY(check_shape(s));
  if (!cu || !violations) return GDN_ERR_INVALID_ARG;
  if (((uintptr_t)violations & 3u) != 0) return GDN_ERR_ALIGNMENT;
  return launched(gdn::launch_check_cu(*s, cu, violations, (hipStream_t)stream));
}

}  // extern "C"

namespace {

gdn_status check_cache(const gdn_shape* s, const gdn_cache* c, bool conv) {
  if (!c || !c->S || c->n_slots < 1) return GDN_ERR_INVALID_ARG;
  if (c->S_stride < (int64_t)s->hv * s->dv * s->dk) return GDN_ERR_INVALID_ARG;
  if (!aligned16(c->S) || c->S_stride % 4) return GDN_ERR_ALIGNMENT;
  if (conv) {
    if (!c->conv || c->conv_stride < 3 * channels(s)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(c->conv) || c->conv_stride * (int64_t)esize(s->dtype) % 16)
      return GDN_ERR_ALIGNMENT;
  }
  return GDN_OK;
}

// base of rows of bytes: every slot starts at a multiple of 16 bytes
gdn_status check_slot_rows(const void* base, int64_t stride, int64_t bytes, int32_t n) {
  if (!base || n < 1 || bytes < 0 || stride < bytes) return GDN_ERR_INVALID_ARG;
  if (!aligned16(base) || stride % 16 || bytes % 16) return GDN_ERR_ALIGNMENT;
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_recurrent_fwd(const gdn_shape* s, const void* q, const void* k, const void* v,
                             int64_t ldq, int64_t ldk, int64_t ldv, const float* g,
                             const float* beta, float scale, const gdn_cache* cache,
                             const int32_t* slot_in, const int32_t* slot_out,
                             const int32_t* slot_tok, const int32_t* cu, void* o, void* stream) {
  GDN_TRY(check_shape(s));
  GDN_TRY(check_cache(s, cache, false));
  if (!cu) return GDN_ERR_INVALID_ARG;
  if (s->total_tokens > 0) {   // no tokens: states pass through, token tensors may be null
    GDN_TRY(check_ptrs({q, k, v, o}));
    if (!g || !beta) return GDN_ERR_INVALID_ARG;
  }
  GDN_TRY(check_ld(ldq, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(ldk, (int64_t)s->hk * s->dk));
  GDN_TRY(check_ld(ldv, (int64_t)s->hv * s->dv));
  StepArgs a = {};
  a.q = q; a.k = k; a.v = v; a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
  a.g = g; a.beta = beta; a.scale = scale; a.cache = *cache;
  a.slot_in = slot_in; a.slot_out = slot_out; a.slot_tok = slot_tok; a.cu = cu; a.out = o;
  return launched(launch_recurrent(*s, a, (hipStream_t)stream));
}

gdn_status gdn_step_fwd(const gdn_shape* s, const void* x, int64_t ldx, const float* w_conv,
                        const void* a, int64_t lda, const void* b, int64_t ldb,
                        const float* A_log, const float* dt_bias, const void* z, int64_t ldz,
                        const float* w_norm, float scale, float l2_eps, float norm_eps,
                        gdn_act act, const gdn_cache* cache, const int32_t* slot_in,
                        const int32_t* slot_out, const int32_t* slot_tok, const int32_t* cu,
                        void* out, void* stream) {
  GDN_TRY(check_shape(s));
  GDN_TRY(check_cache(s, cache, true));
  GDN_TRY(check_ptrs({w_conv, w_norm}));
  if (!A_log || !dt_bias || !cu) return GDN_ERR_INVALID_ARG;
  if (s->total_tokens > 0) {
    GDN_TRY(check_ptrs({x, z, out}));
    if (!a || !b) return GDN_ERR_INVALID_ARG;
  }
  if (act != GDN_ACT_SILU && act != GDN_ACT_SIGMOID) return GDN_ERR_INVALID_ARG;
  if (!(l2_eps >= 0.f) || !(norm_eps >= 0.f) || lda < s->hv || ldb < s->hv)
    return GDN_ERR_INVALID_ARG;
  GDN_TRY(check_ld(ldx, channels(s)));
  GDN_TRY(check_ld(ldz, (int64_t)s->hv * s->dv));
  StepArgs p = {};
  p.x = x; p.ldx = ldx; p.w_conv = w_conv; p.a = a; p.lda = lda; p.b = b; p.ldb = ldb;
  p.A_log = A_log; p.dt_bias = dt_bias; p.z = z; p.ldz = ldz; p.w_norm = w_norm;
  p.scale = scale; p.l2_eps = l2_eps; p.norm_eps = norm_eps; p.act = (int)act; p.cache = *cache;
  p.slot_in = slot_in; p.slot_out = slot_out; p.slot_tok = slot_tok; p.cu = cu; p.out = out;
  return launched(launch_step(*s, p, (hipStream_t)stream));
}

gdn_status gdn_check_slots(const gdn_shape* s, int32_t n_slots, const int32_t* slot_in,
                           const int32_t* slot_out, const int32_t* slot_tok, const int32_t* cu,
                           int32_t* violations, void* stream) {
  GDN_TRY(check_shape(s));
  if (n_slots < 1 || !cu || !violations) return GDN_ERR_INVALID_ARG;
  if (((uintptr_t)violations & 3u) != 0) return GDN_ERR_ALIGNMENT;
  return launched(launch_check_slots(*s, n_slots, slot_in, slot_out, slot_tok, cu, violations,
                                     (hipStream_t)stream));
}

gdn_status gdn_cache_copy(const void* src, int64_t src_stride, int32_t n_src,
                          const int32_t* src_idx, void* dst, int64_t dst_stride, int32_t n_dst,
                          const int32_t* dst_idx, int64_t bytes, int32_t n, void* stream) {
  if (n < 0) return GDN_ERR_INVALID_ARG;
  GDN_TRY(check_slot_rows(src, src_stride, bytes, n_src));
  GDN_TRY(check_slot_rows(dst, dst_stride, bytes, n_dst));
  return launched(launch_cache_copy(src, src_stride, n_src, src_idx, dst, dst_stride, n_dst,
                                    dst_idx, bytes, n, (hipStream_t)stream));
}

size_t gdn_cache_workspace(int32_t n_slots) { return n_slots < 1 ? 0 : cache_ws_bytes(n_slots); }

gdn_status gdn_cache_fork(void* base, int64_t stride, int32_t n_slots, int32_t* refs,
                          const int32_t* src, int32_t n, int32_t* dst, void* ws, size_t ws_bytes,
                          void* stream) {
  if (n < 0) return GDN_ERR_INVALID_ARG;
  if (stride < 16) return GDN_ERR_INVALID_ARG;   // slots of nothing: no move to launch
  GDN_TRY(check_slot_rows(base, stride, stride, n_slots));
  if (!refs || (n > 0 && (!src || !dst))) return GDN_ERR_INVALID_ARG;
  if (!ws || ws_bytes < cache_ws_bytes(n_slots) || !aligned16(ws)) return GDN_ERR_WORKSPACE;
  return launched(launch_cache_fork(base, stride, n_slots, refs, src, n, dst, ws,
                                    (hipStream_t)stream));
}

gdn_status gdn_cache_retain(int32_t* refs, int32_t n_slots, const int32_t* slots, int32_t n,
                            void* stream) {
  if (!refs || n_slots < 1 || n < 0 || (n > 0 && !slots)) return GDN_ERR_INVALID_ARG;
  return launched(launch_cache_count(refs, n_slots, slots, n, 1, (hipStream_t)stream));
}

gdn_status gdn_cache_release(int32_t* refs, int32_t n_slots, const int32_t* slots, int32_t n,
                             void* stream) {
  if (!refs || n_slots < 1 || n < 0 || (n > 0 && !slots)) return GDN_ERR_INVALID_ARG;
  return launched(launch_cache_count(refs, n_slots, slots, n, -1, (hipStream_t)stream));
}

gdn_status gdn_cache_compact(void* base, int64_t stride, int32_t n_slots, int32_t* refs,
                             int32_t* remap, int32_t* table, int32_t n_table, void* ws,
                             size_t ws_bytes, void* stream) {
  if (n_table < 0) return GDN_ERR_INVALID_ARG;
  if (stride < 16) return GDN_ERR_INVALID_ARG;   // slots of nothing: no move to launch
  GDN_TRY(check_slot_rows(base, stride, stride, n_slots));
  if (!refs || !remap || (n_table > 0 && !table)) return GDN_ERR_INVALID_ARG;
  if (!ws || ws_bytes < cache_ws_bytes(n_slots) || !aligned16(ws)) return GDN_ERR_WORKSPACE;
  return launched(launch_cache_compact(base, stride, n_slots, refs, remap, table, n_table, ws,
                                       (hipStream_t)stream));
}

// ---------------------------------------------------------------- around the core
static gdn_status add_norm_shape(int64_t rows, int32_t n, gdn_dtype dtype, gdn_dtype res_dtype, float eps) {
  if (rows < 0 || n < 1 || !dtype_ok(dtype) || !dtype_ok(res_dtype) || !(eps >= 0.f))
    return GDN_ERR_INVALID_ARG;
  if (res_dtype != dtype && res_dtype != GDN_FP32) return GDN_ERR_UNSUPPORTED;
  if (n % 8 || n > ADD_NORM_MAX) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// a matrix of rows that may be absent
static gdn_status check_rows(const void* p, int64_t ld, int64_t cols) {
  if (!p) return GDN_OK;
  if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
  return check_ld(ld, cols);
}

static gdn_status add_norm_fwd(int64_t rows, int32_t n, gdn_dtype dtype, gdn_dtype res_dtype, const void* x,
                               int64_t ldx, const void* res, int64_t ldr, const float* w, float eps, void* h,
                               int64_t ldh, void* y, int64_t ldy, uint8_t* scale, int64_t lds, void* stream) {
  GDN_TRY(add_norm_shape(rows, n, dtype, res_dtype, eps));
  GDN_TRY(check_ptrs({w}));
  if (rows == 0) return GDN_OK;
  GDN_TRY(check_ptrs({x, y}));
  GDN_TRY(check_ld(ldx, n));
  GDN_TRY(check_rows(res, ldr, n));
  GDN_TRY(check_rows(h, ldh, n));
  GDN_TRY(check_ld(ldy, n));
  AddNormArgs a = {};
  a.rows = rows; a.n = n; a.dtype = dtype; a.res_dtype = res_dtype; a.x = x; a.res = res; a.w = w;
  a.eps = eps; a.h = h; a.y = y; a.scale = scale; a.ldx = ldx; a.ldr = ldr; a.ldh = ldh; a.ldy = ldy;
  a.lds = lds;
  return launched(launch_add_norm_fwd(a, (hipStream_t)stream));
}

gdn_status gdn_add_norm_fwd(int64_t rows, int32_t n, gdn_dtype dtype, gdn_dtype res_dtype, const void* x,
                            int64_t ldx, const void* res, int64_t ldr, const float* w, float eps, void* h,
                            int64_t ldh, void* y, int64_t ldy, void* stream) {
  return add_norm_fwd(rows, n, dtype, res_dtype, x, ldx, res, ldr, w, eps, h, ldh, y, ldy, nullptr, 0, stream);
}

gdn_status gdn_add_norm_fwd_mx8(int64_t rows, int32_t n, gdn_dtype dtype, gdn_dtype res_dtype, const void* x,
                                int64_t ldx, const void* res, int64_t ldr, const float* w, float eps, void* h,
                                int64_t ldh, void* q, int64_t ldq, uint8_t* scale, int64_t lds, void* stream) {
  GDN_TRY(add_norm_shape(rows, n, dtype, res_dtype, eps));
  if (n % 32) return GDN_ERR_UNSUPPORTED;
  if (rows > 0 && (!scale || lds < n / 32)) return GDN_ERR_INVALID_ARG;
  if (rows > 0 && ldq % 16) return GDN_ERR_ALIGNMENT;
  return add_norm_fwd(rows, n, dtype, res_dtype, x, ldx, res, ldr, w, eps, h, ldh, q, ldq, scale, lds, stream);
}

size_t gdn_add_norm_bwd_workspace(int64_t rows, int32_t n) {
  if (rows < 0 || n < 1 || n > ADD_NORM_MAX) return 0;
  return sizeof(float) * (size_t)add_norm_blocks(rows, n) * (size_t)n;
}

gdn_status gdn_add_norm_bwd(int64_t rows, int32_t n, gdn_dtype dtype, gdn_dtype res_dtype, const void* h,
                            int64_t ldh, const float* w, float eps, const void* dy, int64_t lddy, const void* dh,
                            int64_t lddh, void* dx, int64_t lddx, void* dres, int64_t lddr, float* dw, void* ws,
                            size_t ws_bytes, void* stream) {
  GDN_TRY(add_norm_shape(rows, n, dtype, res_dtype, eps));
  GDN_TRY(check_ptrs({w}));
  if (rows > 0) {
    GDN_TRY(check_ptrs({h, dy}));
    if (!dx && !dres && !dw) return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_ld(ldh, n));
    GDN_TRY(check_ld(lddy, n));
    GDN_TRY(check_rows(dh, lddh, n));
    GDN_TRY(check_rows(dx, lddx, n));
    GDN_TRY(check_rows(dres, lddr, n));
  }
  if (dw && !aligned16(dw)) return GDN_ERR_ALIGNMENT;
  const size_t need = dw ? gdn_add_norm_bwd_workspace(rows, n) : 0;
  if (need && (!ws || ws_bytes < need || !aligned16(ws))) return GDN_ERR_WORKSPACE;
  AddNormBwdArgs a = {};
  a.rows = rows; a.n = n; a.dtype = dtype; a.res_dtype = res_dtype; a.h = h; a.dy = dy; a.dh = dh; a.w = w;
  a.eps = eps; a.dx = dx; a.dres = dres; a.dw = dw; a.partials = dw ? (float*)ws : nullptr;
  a.ldh = ldh; a.lddy = lddy; a.lddh = lddh; a.lddx = lddx; a.lddr = lddr;
  return launched(launch_add_norm_bwd(a, (hipStream_t)stream));
}

static gdn_status check_w4(int32_t n, int32_t k) {
  if (n < 1 || k < 1) return GDN_ERR_INVALID_ARG;
  // groups of 32 inputs; fewer than 2^24 tiles of 16 x 512 weights
  if (k % 32 || n > (1 << 22) || k > (1 << 20) || (int64_t)((n + 15) / 16) * ((k + 511) / 512) >= (1LL << 24))
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

static gdn_status check_packed(int32_t n, int32_t k, const void* packed, size_t bytes) {
  GDN_TRY(check_w4(n, k));
  GDN_TRY(check_ptrs({packed}));
  return bytes < w4_bytes(n, k) ? GDN_ERR_INVALID_ARG : GDN_OK;
}

size_t gdn_w4_bytes(int32_t n, int32_t k) { return check_w4(n, k) == GDN_OK ? w4_bytes(n, k) : 0; }

gdn_status gdn_w4_pack(int32_t n, int32_t k, gdn_dtype dtype, const void* w, int64_t ldw, void* packed,
                       size_t bytes, void* stream) {
  if (!dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
  GDN_TRY(check_packed(n, k, packed, bytes));
  GDN_TRY(check_ptrs({w}));
  GDN_TRY(check_ld(ldw, k));
  return launched(launch_w4_pack(dtype, w, ldw, n, k, packed, (hipStream_t)stream));
}

gdn_status gdn_w4_arrange(int32_t n, int32_t k, const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                          int64_t lds, void* packed, size_t bytes, void* stream) {
  GDN_TRY(check_packed(n, k, packed, bytes));
  GDN_TRY(check_ptrs({codes}));
  if (!scales || ldc < k / 2 || lds < k / 32) return GDN_ERR_INVALID_ARG;
  if (ldc % 16) return GDN_ERR_ALIGNMENT;
  return launched(launch_w4_arrange(codes, ldc, scales, lds, n, k, packed, (hipStream_t)stream));
}

gdn_status gdn_w4_unpack(int32_t n, int32_t k, const void* packed, size_t bytes, gdn_dtype dtype, void* w,
                         int64_t ldw, void* stream) {
  if (!dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
  GDN_TRY(check_packed(n, k, packed, bytes));
  GDN_TRY(check_ptrs({w}));
  GDN_TRY(check_ld(ldw, k));
  return launched(launch_w4_unpack(dtype, packed, n, k, w, ldw, (hipStream_t)stream));
}

gdn_status gdn_w4_fwd(int64_t rows, int32_t n, int32_t k, gdn_dtype dtype, const void* x, int64_t ldx,
                      const void* packed, size_t bytes, void* y, int64_t ldy, void* stream) {
  if (rows < 0 || !dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
  GDN_TRY(check_packed(n, k, packed, bytes));
  if (rows == 0) return GDN_OK;
  GDN_TRY(check_ptrs({x, y}));
  GDN_TRY(check_ld(ldx, k));
  GDN_TRY(check_ld(ldy, n));
  W4Args a = {};
  a.rows = rows; a.n = n; a.k = k; a.x = x; a.ldx = ldx; a.packed = packed;
  a.scales_at = w4_scales_at(n, k); a.y = y; a.ldy = ldy;
  return launched(launch_w4(a, dtype, (hipStream_t)stream));
}

gdn_status gdn_w4_fwd_mx8(int64_t rows, int32_t n, int32_t k, const void* q, int64_t ldq, const uint8_t* scale,
                          int64_t lds, const void* packed, size_t bytes, gdn_dtype dtype, void* y, int64_t ldy,
                          void* stream) {
  if (rows < 0 || !dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
  GDN_TRY(check_packed(n, k, packed, bytes));
  if (rows == 0) return GDN_OK;
  GDN_TRY(check_ptrs({q, y}));
  if (!scale || ldq < k || lds < k / 32) return GDN_ERR_INVALID_ARG;
  if (ldq % 16) return GDN_ERR_ALIGNMENT;
  GDN_TRY(check_ld(ldy, n));
  W4Args a = {};
  a.rows = rows; a.n = n; a.k = k; a.x = q; a.ldx = ldq; a.xs = scale; a.ldxs = lds; a.packed = packed;
  a.scales_at = w4_scales_at(n, k); a.y = y; a.ldy = ldy;
  return launched(launch_w4(a, dtype, (hipStream_t)stream));
}

}  // extern "C"
