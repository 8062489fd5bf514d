// C ABI of the operators around the recurrence: argument validation and
// dispatch.  Nothing here allocates or synchronises.
#include <math.h>

#include "falcon.h"
#include "falcon_block.h"
#include "falcon_check.h"

namespace {

using falcon::aligned16;
using falcon::all_aligned;
using falcon::any_overlap;
using falcon::ConvArgs;
using falcon::dtype_bytes;
using falcon::dtype_ok;
using falcon::elems;
using falcon::finish;
using falcon::kMaxTokens;
using falcon::NormArgs;
using falcon::overlap;
using falcon::Range;
using falcon::rows_bytes;
using falcon::rows_ok;
using falcon::ScanArgs;

// Longest row of the scan's inputs: 64 rows of float32 stay within 2^30 bytes.
constexpr int64_t kMaxScanRow = int64_t(1) << 22;

// ---- convolution ---------------------------------------------------------------
falcon_status check_conv(const falcon_conv_problem* p, bool step, ConvArgs* a) {
  if (!p) return FALCON_ERR_NULL;
  const int T = step ? 1 : p->T;
  if (p->B < 0 || T < 0 || p->C < 0 || p->W < 2 || p->W > 4) return FALCON_ERR_SHAPE;
  if (elems(p->B, int64_t(T) + 4, int64_t(p->C) + 8) < 0 || int64_t(p->B) * T > kMaxTokens) return FALCON_ERR_SHAPE;
  if (!rows_ok(int64_t(p->B) * T, p->x_row, p->C)) return FALCON_ERR_SHAPE;
  if (step && int64_t(p->B) * p->C > (int64_t(1) << 31)) return FALCON_ERR_SHAPE;
  if (!dtype_ok(p->io_dtype)) return FALCON_ERR_DTYPE;
  if (p->activation != FALCON_ACT_NONE && p->activation != FALCON_ACT_SILU) return FALCON_ERR_VALUE;
  *a = ConvArgs{};
  a->B = p->B; a->T = T; a->C = p->C; a->W = p->W;
  a->bf16 = p->io_dtype == FALCON_BF16;
  a->act = p->activation;
  a->x_row = p->x_row;
  return FALCON_OK;
}

// ---- group norm ------------------------------------------------------------------
falcon_status check_norm(const falcon_norm_problem* p, NormArgs* a) {
  if (!p) return FALCON_ERR_NULL;
  if (p->B < 0 || p->T < 0 || p->G < 0 || p->d < 1 || p->d > 4096) return FALCON_ERR_SHAPE;
  const int64_t C = int64_t(p->G) * p->d;
  if (C > (int64_t(1) << 30) || elems(p->B, p->T, C) < 0 || int64_t(p->B) * p->T > kMaxTokens) return FALCON_ERR_SHAPE;
  if (!p->x_heads && !rows_ok(int64_t(p->B) * p->T, p->x_row, C)) return FALCON_ERR_SHAPE;
  if (!dtype_ok(p->io_dtype)) return FALCON_ERR_DTYPE;
  if (p->activation < FALCON_ACT_NONE || p->activation > FALCON_ACT_ELU1) return FALCON_ERR_VALUE;
  if (!isfinite(p->eps) || p->eps < 0.0f || !isfinite(p->scale)) return FALCON_ERR_VALUE;
  *a = NormArgs{};
  a->B = p->B; a->T = p->T; a->G = p->G; a->d = p->d;
  a->bf16 = p->io_dtype == FALCON_BF16;
  a->act = p->activation;
  a->center = p->center != 0;
  a->x_heads = p->x_heads != 0;
  a->y_heads = p->y_heads != 0;
  a->eps = p->eps; a->scale = p->scale;
  a->x_row = p->x_heads ? C : p->x_row;
  return FALCON_OK;
}

// ---- selective scan ----------------------------------------------------------------
falcon_status check_scan(const falcon_scan_problem* p, bool step, bool gate, ScanArgs* a) {
  if (!p) return FALCON_ERR_NULL;
  const int T = step ? 1 : p->T;
  if (p->B < 0 || T < 0 || p->D < 0 || p->G < 1) return FALCON_ERR_SHAPE;
  if (p->N != 8 && p->N != 16 && p->N != 32 && p->N != 64) return FALCON_ERR_SHAPE;
  if (p->D % p->G != 0) return FALCON_ERR_SHAPE;
  const int64_t rows = int64_t(p->B) * T, GN = int64_t(p->G) * p->N;
  if (rows > kMaxTokens || elems(p->B, int64_t(T) + 1, int64_t(p->D) * p->N) < 0) return FALCON_ERR_SHAPE;
  const int64_t steps[] = {p->x_row, p->dt_row, gate ? p->z_row : p->D, p->b_row, p->c_row};
  for (int i = 0; i < 5; ++i)
    if (!rows_ok(rows, steps[i], i < 3 ? p->D : GN) || steps[i] > kMaxScanRow) return FALCON_ERR_SHAPE;
  if (step && int64_t(p->B) * p->D > (int64_t(1) << 27)) return FALCON_ERR_SHAPE;
  if (!dtype_ok(p->io_dtype)) return FALCON_ERR_DTYPE;
  *a = ScanArgs{};
  a->B = p->B; a->T = T; a->D = p->D; a->N = p->N; a->G = p->G;
  a->bf16 = p->io_dtype == FALCON_BF16;
  a->softplus = p->softplus != 0;
  a->x_row = p->x_row; a->dt_row = p->dt_row; a->z_row = p->z_row;
  a->b_row = p->b_row; a->c_row = p->c_row;
  a->spin_limit = falcon::wait_limit();
  return FALCON_OK;
}

}  // namespace

extern "C" {

falcon_status falcon_conv_fwd(const falcon_conv_problem* p, const void* x, const float* weight,
                              const float* bias, const void* state, const int32_t* lengths,
                              void* y, void* state_out, hipStream_t stream) {
  ConvArgs a;
  falcon_status s = check_conv(p, false, &a);
  if (s != FALCON_OK) return s;
  const int64_t n = int64_t(a.B) * a.T * a.C, ns = int64_t(a.B) * (a.W - 1) * a.C, es = dtype_bytes(p->io_dtype);
  if (int64_t(a.B) * a.C == 0 || (n == 0 && !state_out)) return FALCON_OK;
  if (!weight || (n > 0 && (!x || !y))) return FALCON_ERR_NULL;
  if (!all_aligned({x, weight, bias, state, lengths, y, state_out})) return FALCON_ERR_ALIGN;
  if (any_overlap({{y, n * es}, {state_out, ns * es}},
                  {{x, rows_bytes(int64_t(a.B) * a.T, a.x_row, a.C, es)}, {weight, int64_t(a.C) * a.W * 4},
                   {bias, int64_t(a.C) * 4}, {state, ns * es}, {lengths, int64_t(a.B) * 4}}))
    return FALCON_ERR_ALIAS;
  a.x = x; a.weight = weight; a.bias = bias; a.state = state; a.lengths = lengths;
  a.y = y; a.state_out = state_out;
  (void)hipGetLastError();
  return finish(falcon::launch_conv_fwd(a, stream));
}

falcon_status falcon_conv_step(const falcon_conv_problem* p, const void* x, const float* weight,
                               const float* bias, void* state, const uint8_t* is_first, void* y,
                               hipStream_t stream) {
  ConvArgs a;
  falcon_status s = check_conv(p, true, &a);
  if (s != FALCON_OK) return s;
  const int64_t n = int64_t(a.B) * a.C, es = dtype_bytes(p->io_dtype);
  if (n == 0) return FALCON_OK;
  if (!x || !weight || !state || !y) return FALCON_ERR_NULL;
  if (!all_aligned({x, weight, bias, state, y})) return FALCON_ERR_ALIGN;
  if (any_overlap({{y, n * es}, {state, n * (a.W - 1) * es}},
                  {{x, rows_bytes(a.B, a.x_row, a.C, es)}, {weight, int64_t(a.C) * a.W * 4},
                   {bias, int64_t(a.C) * 4}, {is_first, a.B}}))
    return FALCON_ERR_ALIAS;
  a.x = x; a.weight = weight; a.bias = bias; a.step_state = state; a.is_first = is_first; a.y = y;
  (void)hipGetLastError();
  return finish(falcon::launch_conv_step(a, stream));
}

size_t falcon_conv_bwd_workspace_bytes(const falcon_conv_problem* p) {
  ConvArgs a;
  if (check_conv(p, false, &a) != FALCON_OK) return static_cast<size_t>(-1);
  return falcon::conv_bwd_workspace_bytes(a);
}

falcon_status falcon_conv_bwd(const falcon_conv_problem* p, const void* x, const float* weight,
                              const float* bias, const void* state, const int32_t* lengths,
                              const void* dy, int32_t dy_dtype, const float* dstate_out, float* dx,
                              float* dweight, float* dbias, float* dstate, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  ConvArgs a;
  falcon_status s = check_conv(p, false, &a);
  if (s != FALCON_OK) return s;
  if (!dtype_ok(dy_dtype)) return FALCON_ERR_DTYPE;
  const int64_t n = int64_t(a.B) * a.T * a.C, ns = int64_t(a.B) * (a.W - 1) * a.C, es = dtype_bytes(p->io_dtype);
  if (a.C == 0) return FALCON_OK;
  if (!weight || !dweight || (n > 0 && (!x || !dy || !dx))) return FALCON_ERR_NULL;
  if (!all_aligned({x, weight, bias, state, lengths, dy, dstate_out, dx, dweight, dbias, dstate}))
    return FALCON_ERR_ALIGN;
  const size_t need = falcon::conv_bwd_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return FALCON_ERR_ALIGN;
  const Range ws{need > 0 ? workspace : nullptr, static_cast<int64_t>(need)};
  if (any_overlap({{dx, n * 4}, {dweight, int64_t(a.C) * a.W * 4}, {dbias, int64_t(a.C) * 4}, {dstate, ns * 4}, ws},
                  {{x, rows_bytes(int64_t(a.B) * a.T, a.x_row, a.C, es)}, {weight, int64_t(a.C) * a.W * 4},
                   {bias, int64_t(a.C) * 4}, {state, ns * es}, {lengths, int64_t(a.B) * 4},
                   {dy, n * dtype_bytes(dy_dtype)}, {dstate_out, ns * 4}}))
    return FALCON_ERR_ALIAS;
  a.x = x; a.weight = weight; a.bias = bias; a.state = state; a.lengths = lengths;
  a.dy = dy; a.dy_bf16 = dy_dtype == FALCON_BF16; a.dstate_out = dstate_out;
  a.dx = dx; a.dweight = dweight; a.dbias = dbias; a.dstate = dstate;
  a.workspace = static_cast<float*>(workspace);
  (void)hipGetLastError();
  return finish(falcon::launch_conv_bwd(a, stream));
}

falcon_status falcon_norm_fwd(const falcon_norm_problem* p, const void* x, const float* weight,
                              const float* bias, void* y, hipStream_t stream) {
  NormArgs a;
  falcon_status s = check_norm(p, &a);
  if (s != FALCON_OK) return s;
  const int64_t C = int64_t(a.G) * a.d, n = int64_t(a.B) * a.T * C, es = dtype_bytes(p->io_dtype);
  if (n == 0) return FALCON_OK;
  if (!x || !y) return FALCON_ERR_NULL;
  if (!all_aligned({x, weight, bias, y})) return FALCON_ERR_ALIGN;
  if (any_overlap({{y, n * es}}, {{x, rows_bytes(int64_t(a.B) * a.T, a.x_row, C, es)}, {weight, C * 4}, {bias, C * 4}}))
    return FALCON_ERR_ALIAS;
  a.x = x; a.weight = weight; a.bias = bias; a.y = y;
  (void)hipGetLastError();
  return finish(falcon::launch_norm_fwd(a, stream));
}

size_t falcon_norm_bwd_workspace_bytes(const falcon_norm_problem* p) {
  NormArgs a;
  if (check_norm(p, &a) != FALCON_OK) return static_cast<size_t>(-1);
  return falcon::norm_bwd_workspace_bytes(a);
}

falcon_status falcon_norm_bwd(const falcon_norm_problem* p, const void* x, const float* weight,
                              const float* bias, const void* dy, int32_t dy_dtype, float* dx,
                              float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  NormArgs a;
  falcon_status s = check_norm(p, &a);
  if (s != FALCON_OK) return s;
  if (!dtype_ok(dy_dtype)) return FALCON_ERR_DTYPE;
  const int64_t C = int64_t(a.G) * a.d, n = int64_t(a.B) * a.T * C, es = dtype_bytes(p->io_dtype);
  if (C == 0) return FALCON_OK;
  if (n > 0 && (!x || !dy || !dx)) return FALCON_ERR_NULL;
  if (!all_aligned({x, weight, bias, dy, dx, dweight, dbias})) return FALCON_ERR_ALIGN;
  const size_t need = falcon::norm_bwd_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return FALCON_ERR_ALIGN;
  const Range ws{need > 0 ? workspace : nullptr, static_cast<int64_t>(need)};
  if (any_overlap({{dx, n * 4}, {dweight, C * 4}, {dbias, C * 4}, ws},
                  {{x, rows_bytes(int64_t(a.B) * a.T, a.x_row, C, es)}, {weight, C * 4}, {bias, C * 4},
                   {dy, n * dtype_bytes(dy_dtype)}}))
    return FALCON_ERR_ALIAS;
  a.x = x; a.weight = weight; a.bias = bias;
  a.dy = dy; a.dy_bf16 = dy_dtype == FALCON_BF16;
  a.dx = dx; a.dweight = dweight; a.dbias = dbias;
  a.workspace = static_cast<float*>(workspace);
  (void)hipGetLastError();
  return finish(falcon::launch_norm_bwd(a, stream));
}

size_t falcon_scan_workspace_bytes(const falcon_scan_problem* p) {
  ScanArgs a;
  if (check_scan(p, false, false, &a) != FALCON_OK) return static_cast<size_t>(-1);
  return falcon::scan_workspace_bytes(a);
}

falcon_status falcon_scan_fwd(const falcon_scan_problem* p, const void* x, const void* dt,
                              const float* A, const void* Bm, const void* Cm, const float* Dskip,
                              const float* dt_bias, const void* z, const float* S0,
                              const int32_t* lengths, void* y, float* S_T, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  ScanArgs a;
  falcon_status s = check_scan(p, false, z != nullptr, &a);
  if (s != FALCON_OK) return s;
  const int64_t rows = int64_t(a.B) * a.T, n = rows * a.D, ns = int64_t(a.B) * a.D * a.N, GN = int64_t(a.G) * a.N;
  const int64_t es = dtype_bytes(p->io_dtype);
  if (ns == 0 || (n == 0 && (!S_T || S_T == S0))) return FALCON_OK;
  if (n > 0 && (!x || !dt || !A || !Bm || !Cm || !y)) return FALCON_ERR_NULL;
  if (!all_aligned({x, dt, A, Bm, Cm, Dskip, dt_bias, z, S0, lengths, y, S_T})) return FALCON_ERR_ALIGN;
  const size_t need = falcon::scan_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return FALCON_ERR_ALIGN;
  const Range ws{need > 0 ? workspace : nullptr, static_cast<int64_t>(need)};
  if (any_overlap({{y, n * es}, {S_T, ns * 4}, ws},
                  {{x, rows_bytes(rows, a.x_row, a.D, es)}, {dt, rows_bytes(rows, a.dt_row, a.D, es)},
                   {A, int64_t(a.D) * a.N * 4}, {Bm, rows_bytes(rows, a.b_row, GN, es)},
                   {Cm, rows_bytes(rows, a.c_row, GN, es)}, {Dskip, int64_t(a.D) * 4}, {dt_bias, int64_t(a.D) * 4},
                   {z, z ? rows_bytes(rows, a.z_row, a.D, es) : 0}, {S0 == S_T ? nullptr : S0, ns * 4},
                   {lengths, int64_t(a.B) * 4}}) ||
      overlap({y, n * es}, {S0, ns * 4}) || overlap(ws, {S0, ns * 4}))
    return FALCON_ERR_ALIAS;
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.dt_bias = dt_bias; a.z = z;
  a.S0 = S0; a.lengths = lengths; a.y = y; a.S_T = S_T;
  a.workspace = static_cast<float*>(workspace);
  (void)hipGetLastError();
  return finish(falcon::launch_scan_fwd(a, stream));
}

falcon_status falcon_scan_step(const falcon_scan_problem* p, const void* x, const void* dt,
                               const float* A, const void* Bm, const void* Cm, const float* Dskip,
                               const float* dt_bias, const void* z, float* S, const uint8_t* is_first,
                               void* y, hipStream_t stream) {
  ScanArgs a;
  falcon_status s = check_scan(p, true, z != nullptr, &a);
  if (s != FALCON_OK) return s;
  const int64_t n = int64_t(a.B) * a.D, GN = int64_t(a.G) * a.N, es = dtype_bytes(p->io_dtype);
  if (n == 0) return FALCON_OK;
  if (!x || !dt || !A || !Bm || !Cm || !S || !y) return FALCON_ERR_NULL;
  if (!all_aligned({x, dt, A, Bm, Cm, Dskip, dt_bias, z, S, y})) return FALCON_ERR_ALIGN;
  if (any_overlap({{y, n * es}, {S, n * a.N * 4}},
                  {{x, rows_bytes(a.B, a.x_row, a.D, es)}, {dt, rows_bytes(a.B, a.dt_row, a.D, es)},
                   {A, int64_t(a.D) * a.N * 4}, {Bm, rows_bytes(a.B, a.b_row, GN, es)},
                   {Cm, rows_bytes(a.B, a.c_row, GN, es)}, {Dskip, int64_t(a.D) * 4}, {dt_bias, int64_t(a.D) * 4},
                   {z, z ? rows_bytes(a.B, a.z_row, a.D, es) : 0}, {is_first, a.B}}))
    return FALCON_ERR_ALIAS;
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.dt_bias = dt_bias; a.z = z;
  a.S = S; a.is_first = is_first; a.y = y;
  (void)hipGetLastError();
  return finish(falcon::launch_scan_step(a, stream));
}

size_t falcon_scan_bwd_workspace_bytes(const falcon_scan_problem* p) {
  ScanArgs a;
  if (check_scan(p, false, false, &a) != FALCON_OK) return static_cast<size_t>(-1);
  return falcon::scan_bwd_workspace_bytes(a);
}

falcon_status falcon_scan_bwd(const falcon_scan_problem* p, const void* x, const void* dt,
                              const float* A, const void* Bm, const void* Cm, const float* Dskip,
                              const float* dt_bias, const void* z, const float* S0,
                              const int32_t* lengths, const void* dy, int32_t dy_dtype,
                              const float* dS_T, float* dx, float* ddt, float* dz, float* dA,
                              float* dB, float* dC, float* dD, float* ddt_bias, float* dS0,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  ScanArgs a;
  falcon_status s = check_scan(p, false, z != nullptr, &a);
  if (s != FALCON_OK) return s;
  if (!dtype_ok(dy_dtype)) return FALCON_ERR_DTYPE;
  const int64_t rows = int64_t(a.B) * a.T, n = rows * a.D, ns = int64_t(a.B) * a.D * a.N, GN = int64_t(a.G) * a.N;
  const int64_t es = dtype_bytes(p->io_dtype), nd = int64_t(a.D) * 4;
  if (!z) dz = nullptr;
  if (a.D == 0) {
    // no channel: nothing but dB and dC, which sum over none
    const int64_t nb = rows * GN;
    if (nb > 0 && (!dB || !dC)) return FALCON_ERR_NULL;
    if (!all_aligned({dB, dC})) return FALCON_ERR_ALIGN;
    if (nb > 0 && overlap({dB, nb * 4}, {dC, nb * 4})) return FALCON_ERR_ALIAS;
    (void)hipGetLastError();
    hipError_t e = nb > 0 ? falcon::launch_sum_parts({nullptr, 0, 2 * nb, 2 * nb, {dB, dC, nullptr}, {nb, 2 * nb}}, stream) : hipSuccess;
    return finish(e);
  }
  if (!A || !dA || (n > 0 && (!x || !dt || !Bm || !Cm || !dy || !dx || !ddt || !dB || !dC || (z && !dz))))
    return FALCON_ERR_NULL;
  if (!all_aligned({x, dt, A, Bm, Cm, Dskip, dt_bias, z, S0, lengths, dy, dS_T, dx, ddt, dz, dA, dB, dC, dD, ddt_bias, dS0}))
    return FALCON_ERR_ALIGN;
  const size_t need = falcon::scan_bwd_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return FALCON_ERR_ALIGN;
  const Range ws{need > 0 ? workspace : nullptr, static_cast<int64_t>(need)};
  if (any_overlap({{dx, n * 4}, {ddt, n * 4}, {dz, n * 4}, {dA, nd * a.N}, {dB, rows * GN * 4}, {dC, rows * GN * 4},
                   {dD, nd}, {ddt_bias, nd}, {dS0, ns * 4}, ws},
                  {{x, rows_bytes(rows, a.x_row, a.D, es)}, {dt, rows_bytes(rows, a.dt_row, a.D, es)},
                   {A, nd * a.N}, {Bm, rows_bytes(rows, a.b_row, GN, es)}, {Cm, rows_bytes(rows, a.c_row, GN, es)},
                   {Dskip, nd}, {dt_bias, nd}, {z, z ? rows_bytes(rows, a.z_row, a.D, es) : 0}, {S0, ns * 4},
                   {lengths, int64_t(a.B) * 4}, {dy, n * dtype_bytes(dy_dtype)}, {dS_T, ns * 4}}))
    return FALCON_ERR_ALIAS;
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.dt_bias = dt_bias; a.z = z;
  a.S0 = S0; a.lengths = lengths;
  a.dy = dy; a.dy_bf16 = dy_dtype == FALCON_BF16; a.dS_T = dS_T;
  a.dx = dx; a.ddt = ddt; a.dz = dz; a.dA = dA; a.dB = dB; a.dC = dC; a.dD = dD; a.ddt_bias = ddt_bias; a.dS0 = dS0;
  a.workspace = static_cast<float*>(workspace);
  (void)hipGetLastError();
  return finish(falcon::launch_scan_bwd(a, stream));
}

}  // extern "C"
