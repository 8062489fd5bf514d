// C ABI of linear attention with a decay for each head: argument validation and
// dispatch.  Nothing here allocates or synchronises.
#include <math.h>

#include "falcon.h"
#include "falcon_block.h"
#include "falcon_check.h"

namespace {

using namespace falcon;

// Most heads of one call (B H): every grid then fits its 32 bits.
constexpr int64_t kMaxHeads = int64_t(1) << 21;
// Longest row: offsets within a chunk then fit 32 bits.
constexpr int64_t kMaxRow = int64_t(1) << 22;

bool width_ok(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Elements from one sequence, head and token to the next.
HeadSteps steps(bool heads, int64_t row, int64_t H, int64_t T, int64_t d) {
  if (heads) return {H * T * d, T * d, d};
  return {T * row, d, row};
}

falcon_status check_linear(const falcon_linear_problem* p, bool step, LinearArgs* a) {
  if (!p) return FALCON_ERR_NULL;
  const int T = step ? 1 : p->T;
  if (p->B < 0 || p->H < 0 || T < 0 || !width_ok(p->dk) || !width_ok(p->dv)) return FALCON_ERR_SHAPE;
  const int64_t heads = int64_t(p->B) * p->H, rows = int64_t(p->B) * T;
  if (heads > kMaxHeads || rows > kMaxTokens || elems(heads, int64_t(T) + 2 * p->dk, 128) < 0) return FALCON_ERR_SHAPE;
  const int64_t dk = int64_t(p->H) * p->dk, dv = int64_t(p->H) * p->dv;
  const bool qk_heads = !step && p->qk_heads, v_heads = !step && p->v_heads, o_heads = !step && p->o_heads;
  if ((!qk_heads && (p->q_row > kMaxRow || p->k_row > kMaxRow)) || (!v_heads && p->v_row > kMaxRow) || (!o_heads && dv > kMaxRow))
    return FALCON_ERR_SHAPE;
  if (!qk_heads && (!rows_ok(rows, p->q_row, dk) || !rows_ok(rows, p->k_row, dk))) return FALCON_ERR_SHAPE;
  if (!v_heads && !rows_ok(rows, p->v_row, dv)) return FALCON_ERR_SHAPE;
  if (!dtype_ok(p->io_dtype)) return FALCON_ERR_DTYPE;
  if (!isfinite(p->scale)) return FALCON_ERR_VALUE;
  const int64_t piece = 16 / dtype_bytes(p->io_dtype);
  if (!qk_heads && (p->q_row % piece || p->k_row % piece)) return FALCON_ERR_ALIGN;
  if (!v_heads && p->v_row % piece) return FALCON_ERR_ALIGN;
  *a = LinearArgs{};
  a->B = p->B; a->H = p->H; a->T = T; a->dk = p->dk; a->dv = p->dv;
  a->bf16 = p->io_dtype == FALCON_BF16;
  a->scale = p->scale;
  a->zero_behind = p->zero_behind != 0;
  a->q_at = steps(qk_heads, p->q_row, p->H, T, p->dk);
  a->k_at = steps(qk_heads, p->k_row, p->H, T, p->dk);
  a->v_at = steps(v_heads, p->v_row, p->H, T, p->dv);
  a->o_at = steps(o_heads, dv, p->H, T, p->dv);
  a->dqk_at = steps(qk_heads, dk, p->H, T, p->dk);
  a->dv_at = steps(v_heads, dv, p->H, T, p->dv);
  return FALCON_OK;
}

// Bytes from the first to the last element of an input.
int64_t input_bytes(const HeadSteps& at, const LinearArgs& a, int64_t d, int64_t es) {
  if (int64_t(a.B) * a.H * a.T == 0) return 0;
  return ((a.B - 1) * at.b + (a.H - 1) * at.h + (a.T - 1) * at.t + d) * es;
}

}  // namespace

extern "C" {

size_t falcon_linear_workspace_bytes(const falcon_linear_problem* p) {
  LinearArgs a;
  if (check_linear(p, false, &a) != FALCON_OK) return static_cast<size_t>(-1);
  return linear_workspace_bytes(a);
}

falcon_status falcon_linear_fwd(const falcon_linear_problem* p, const void* q, const void* k, const void* v,
                                const float* log_decay, const float* S0, const int32_t* lengths, void* o, float* S_T,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  LinearArgs a;
  falcon_status s = check_linear(p, false, &a);
  if (s != FALCON_OK) return s;
  const int64_t heads = int64_t(a.B) * a.H, n = heads * a.T, ns = heads * a.dk * a.dv, es = dtype_bytes(p->io_dtype);
  if (heads == 0 || (n == 0 && (!S_T || S_T == S0))) return FALCON_OK;
  if (n > 0 && (!q || !k || !v || !log_decay || !o)) return FALCON_ERR_NULL;
  if (!all_aligned({q, k, v, log_decay, S0, lengths, o, S_T})) return FALCON_ERR_ALIGN;
  const size_t need = linear_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return FALCON_ERR_ALIGN;
  const Range ws{need > 0 ? workspace : nullptr, static_cast<int64_t>(need)};
  if (any_overlap({{o, n * a.dv * es}, {S_T, ns * 4}, ws},
                  {{q, input_bytes(a.q_at, a, a.dk, es)}, {k, input_bytes(a.k_at, a, a.dk, es)},
                   {v, input_bytes(a.v_at, a, a.dv, es)}, {log_decay, int64_t(a.H) * 4},
                   {S0 == S_T ? nullptr : S0, ns * 4}, {lengths, int64_t(a.B) * 4}}) ||
      overlap({o, n * a.dv * es}, {S0, ns * 4}) || overlap(ws, {S0, ns * 4}))
    return FALCON_ERR_ALIAS;
  a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.S0 = S0; a.lengths = lengths;
  a.o = o; a.S_T = S_T;
  a.workspace = static_cast<float*>(workspace);
  (void)hipGetLastError();
  return finish(launch_linear_fwd(a, stream));
}

falcon_status falcon_linear_step(const falcon_linear_problem* p, const void* q, const void* k, const void* v,
                                 const float* log_decay, float* S, const uint8_t* is_first, void* o, hipStream_t stream) {
  LinearArgs a;
  falcon_status s = check_linear(p, true, &a);
  if (s != FALCON_OK) return s;
  const int64_t heads = int64_t(a.B) * a.H, ns = heads * a.dk * a.dv, es = dtype_bytes(p->io_dtype);
  if (heads == 0) return FALCON_OK;
  if (!q || !k || !v || !log_decay || !S || !o) return FALCON_ERR_NULL;
  if (!all_aligned({q, k, v, log_decay, S, o})) return FALCON_ERR_ALIGN;
  if (any_overlap({{o, heads * a.dv * es}, {S, ns * 4}},
                  {{q, input_bytes(a.q_at, a, a.dk, es)}, {k, input_bytes(a.k_at, a, a.dk, es)},
                   {v, input_bytes(a.v_at, a, a.dv, es)}, {log_decay, int64_t(a.H) * 4}, {is_first, a.B}}))
    return FALCON_ERR_ALIAS;
  a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.S = S; a.is_first = is_first; a.o = o;
  (void)hipGetLastError();
  return finish(launch_linear_step(a, stream));
}

size_t falcon_linear_bwd_workspace_bytes(const falcon_linear_problem* p) {
  LinearArgs a;
  if (check_linear(p, false, &a) != FALCON_OK) return static_cast<size_t>(-1);
  return linear_bwd_workspace_bytes(a);
}

falcon_status falcon_linear_bwd(const falcon_linear_problem* p, const void* q, const void* k, const void* v,
                                const float* log_decay, const float* S0, const int32_t* lengths, const void* dO,
                                const float* dS_T, float* dq, float* dk, float* dv, float* dlog_decay, float* dS0,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  LinearArgs a;
  falcon_status s = check_linear(p, false, &a);
  if (s != FALCON_OK) return s;
  const int64_t heads = int64_t(a.B) * a.H, n = heads * a.T, ns = heads * a.dk * a.dv, es = dtype_bytes(p->io_dtype);
  if (a.H == 0 || (heads == 0 && !dlog_decay)) return FALCON_OK;
  if (heads > 0 && !log_decay) return FALCON_ERR_NULL;
  if (n > 0 && (!q || !k || !v || !dO || !dq || !dk || !dv)) return FALCON_ERR_NULL;
  if (!all_aligned({q, k, v, log_decay, S0, lengths, dO, dS_T, dq, dk, dv, dlog_decay, dS0})) return FALCON_ERR_ALIGN;
  const size_t need = linear_bwd_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return FALCON_ERR_ALIGN;
  const Range ws{need > 0 ? workspace : nullptr, static_cast<int64_t>(need)};
  if (any_overlap({{dq, n * a.dk * 4}, {dk, n * a.dk * 4}, {dv, n * a.dv * 4}, {dlog_decay, int64_t(a.H) * 4}, {dS0, ns * 4}, ws},
                  {{q, input_bytes(a.q_at, a, a.dk, es)}, {k, input_bytes(a.k_at, a, a.dk, es)},
                   {v, input_bytes(a.v_at, a, a.dv, es)}, {log_decay, int64_t(a.H) * 4}, {S0, ns * 4},
                   {lengths, int64_t(a.B) * 4}, {dO, n * a.dv * es}, {dS_T, ns * 4}}))
    return FALCON_ERR_ALIAS;
  a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.S0 = S0; a.lengths = lengths;
  a.dO = dO; a.dS_T = dS_T;
  a.dq = dq; a.dk_out = dk; a.dv_out = dv; a.dlog_decay = dlog_decay; a.dS0 = dS0;
  a.workspace = static_cast<float*>(workspace);
  (void)hipGetLastError();
  return finish(launch_linear_bwd(a, stream));
}

}  // extern "C"
