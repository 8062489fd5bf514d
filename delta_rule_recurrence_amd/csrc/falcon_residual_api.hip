// C ABI of the residual update between two blocks: argument validation and dispatch.
// Nothing here allocates or synchronises.
#include <math.h>

#include "falcon.h"
#include "falcon_block.h"
#include "falcon_check.h"

namespace {

using namespace falcon;

constexpr int64_t kMaxChannels = 8192;

int64_t steps_of_row(int64_t C) { return (C + 31) / 32; }

// `y_rows`, `gate_rows`: whether there are rows of y and of a gate, not their 8 bits.
falcon_status check_residual(const falcon_residual_problem* p, bool y_rows, bool gate_rows, ResidualArgs* a) {
  if (!p) return FALCON_ERR_NULL;
  if (p->B < 0 || p->T < 0 || p->G < 1 || p->d < 1) return FALCON_ERR_SHAPE;
  const int64_t C = int64_t(p->G) * p->d, tokens = int64_t(p->B) * p->T;
  if (C > kMaxChannels || tokens > kMaxTokens || elems(tokens, C) < 0) return FALCON_ERR_SHAPE;
  if ((y_rows && !rows_ok(tokens, p->y_row, C)) || (gate_rows && !rows_ok(tokens, p->gate_row, C))) return FALCON_ERR_SHAPE;
  if (!dtype_ok(p->io_dtype) || !dtype_ok(p->stream_dtype)) return FALCON_ERR_DTYPE;
  if (p->activation != FALCON_ACT_NONE && p->activation != FALCON_ACT_SILU && p->activation != FALCON_ACT_SIGMOID)
    return FALCON_ERR_VALUE;
  if (!isfinite(p->eps) || p->eps < 0.0f) return FALCON_ERR_VALUE;
  *a = ResidualArgs{};
  a->B = p->B; a->T = p->T; a->G = p->G; a->d = p->d;
  a->bf16 = p->io_dtype == FALCON_BF16;
  a->stream_bf16 = p->stream_dtype == FALCON_BF16;
  a->act = p->activation;
  a->post = p->post_norm != 0;
  a->pre = p->pre_norm != 0;
  a->eps = p->eps;
  a->zero_behind = p->zero_behind != 0;
  a->y_row = p->y_row; a->gate_row = p->gate_row;
  return FALCON_OK;
}

}  // namespace

extern "C" {

falcon_status falcon_residual_fwd(const falcon_residual_problem* p, const void* y, const void* gate, const void* h,
                                  const float* post_weight, const float* alpha, const float* pre_weight,
                                  const int32_t* lengths, void* h_out, void* n, const falcon_saved* saved,
                                  hipStream_t stream) {
  ResidualArgs a;
  falcon_status s = check_residual(p, true, gate != nullptr, &a);
  if (s != FALCON_OK) return s;
  const int64_t C = int64_t(a.G) * a.d, tokens = int64_t(a.B) * a.T, es = dtype_bytes(p->io_dtype), hs = dtype_bytes(p->stream_dtype);
  if (tokens == 0) return FALCON_OK;
  if (!y || !h_out || (a.pre && !n)) return FALCON_ERR_NULL;
  if (!a.pre) n = nullptr;
  falcon_saved to{};
  if (saved) {
    to = *saved;
    if (!gate) to.gate_codes = nullptr, to.gate_steps = nullptr;
    if (!to.y_codes || !to.y_steps || (gate && (!to.gate_codes || !to.gate_steps))) return FALCON_ERR_NULL;
  }
  if (!all_aligned({y, gate, h, post_weight, alpha, pre_weight, lengths, h_out, n, to.y_codes, to.y_steps, to.gate_codes, to.gate_steps}))
    return FALCON_ERR_ALIGN;
  const int64_t steps = tokens * steps_of_row(C);
  if (any_overlap({{h_out, tokens * C * hs}, {n, tokens * C * es}, {to.y_codes, tokens * C}, {to.y_steps, steps},
                   {to.gate_codes, tokens * C}, {to.gate_steps, steps}},
                  {{y, rows_bytes(tokens, a.y_row, C, es)}, {gate, gate ? rows_bytes(tokens, a.gate_row, C, es) : 0},
                   {h == h_out ? nullptr : h, tokens * C * hs}, {post_weight, C * 4}, {alpha, C * 4}, {pre_weight, C * 4},
                   {lengths, int64_t(a.B) * 4}}) ||
      (h == h_out && any_overlap({{n, tokens * C * es}}, {{h, tokens * C * hs}})))
    return FALCON_ERR_ALIAS;
  a.y = y; a.gate = gate; a.h = h;
  a.post_weight = post_weight; a.alpha = alpha; a.pre_weight = pre_weight;
  a.lengths = lengths;
  a.h_out = h_out; a.n = n;
  a.save = saved != nullptr;
  a.y_codes = to.y_codes; a.y_steps = to.y_steps; a.gate_codes = to.gate_codes; a.gate_steps = to.gate_steps;
  (void)hipGetLastError();
  return finish(launch_residual_fwd(a, stream));
}

size_t falcon_residual_bwd_workspace_bytes(const falcon_residual_problem* p) {
  ResidualArgs a;
  if (check_residual(p, false, false, &a) != FALCON_OK) return static_cast<size_t>(-1);
  return residual_bwd_workspace_bytes(a);
}

falcon_status falcon_residual_bwd(const falcon_residual_problem* p, const void* y, const void* gate, const falcon_saved* saved,
                                  const void* h_out, const float* post_weight, const float* alpha, const float* pre_weight,
                                  const int32_t* lengths, const void* dh_out, int32_t dh_out_dtype, const void* dn,
                                  int32_t dn_dtype, float* dy, float* dgate, float* dh, float* dalpha, float* dpost_weight,
                                  float* dpre_weight, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  ResidualArgs a;
  falcon_status s = check_residual(p, !saved, !saved && gate, &a);
  if (s != FALCON_OK) return s;
  if (!dtype_ok(dh_out_dtype) || !dtype_ok(dn_dtype)) return FALCON_ERR_DTYPE;
  const int64_t C = int64_t(a.G) * a.d, tokens = int64_t(a.B) * a.T, es = dtype_bytes(p->io_dtype), hs = dtype_bytes(p->stream_dtype);
  falcon_saved from{};
  if (saved) {
    if (y || gate) return FALCON_ERR_VALUE;
    from = *saved;
  }
  const bool gated = saved ? from.gate_codes != nullptr : gate != nullptr;
  if (!gated) dgate = nullptr, from.gate_steps = nullptr;
  if (!a.pre) h_out = dn = nullptr, dpre_weight = nullptr;
  if (!a.post) dpost_weight = nullptr;
  if (tokens > 0) {
    if ((saved ? !from.y_codes || !from.y_steps || (gated && !from.gate_steps) : !y) || !dy || (gated && !dgate) ||
        (a.pre && (!h_out || !dn)))
      return FALCON_ERR_NULL;
  }
  if (!all_aligned({y, gate, h_out, post_weight, alpha, pre_weight, lengths, dh_out, dn, from.y_codes, from.y_steps, from.gate_codes,
                    from.gate_steps, dy, dgate, dh, dalpha, dpost_weight, dpre_weight}))
    return FALCON_ERR_ALIGN;
  const size_t need = residual_bwd_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FALCON_ERR_WORKSPACE;
  if (workspace && !aligned16(workspace)) return FALCON_ERR_ALIGN;
  const Range ws{need > 0 ? workspace : nullptr, static_cast<int64_t>(need)};
  const int64_t grad = tokens * C * 4, steps = tokens * steps_of_row(C), dhs = tokens * C * dtype_bytes(dh_out_dtype);
  const bool in_place = dh && dh == dh_out && dh_out_dtype == FALCON_F32;
  if (any_overlap({{dy, grad}, {dgate, grad}, {dh, grad}, {dalpha, C * 4}, {dpost_weight, C * 4}, {dpre_weight, C * 4}, ws},
                  {{y, y ? rows_bytes(tokens, a.y_row, C, es) : 0}, {gate, gate ? rows_bytes(tokens, a.gate_row, C, es) : 0},
                   {from.y_codes, tokens * C}, {from.y_steps, steps}, {from.gate_codes, tokens * C}, {from.gate_steps, steps},
                   {h_out, tokens * C * hs}, {post_weight, C * 4}, {alpha, C * 4}, {pre_weight, C * 4},
                   {lengths, int64_t(a.B) * 4}, {in_place ? nullptr : dh_out, dhs}, {dn, tokens * C * dtype_bytes(dn_dtype)}}))
    return FALCON_ERR_ALIAS;
  a.y = y; a.gate = gate;
  a.save = saved != nullptr;
  a.y_codes = from.y_codes; a.y_steps = from.y_steps; a.gate_codes = from.gate_codes; a.gate_steps = from.gate_steps;
  a.h_out = const_cast<void*>(h_out);
  a.post_weight = post_weight; a.alpha = alpha; a.pre_weight = pre_weight;
  a.lengths = lengths;
  a.dh_out = dh_out; a.dh_out_bf16 = dh_out_dtype == FALCON_BF16;
  a.dn = dn; a.dn_bf16 = dn_dtype == FALCON_BF16;
  a.dy = dy; a.dgate = dgate; a.dh = dh;
  a.dalpha = dalpha; a.dpost_weight = dpost_weight; a.dpre_weight = dpre_weight;
  a.workspace = static_cast<float*>(workspace);
  (void)hipGetLastError();
  return finish(launch_residual_bwd(a, stream));
}

}  // extern "C"
