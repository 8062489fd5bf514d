// Host-side launch interface of the operators around the recurrence (short
// convolution, group norm, selective scan, linear attention, residual update).  Arguments reaching the launchers
// have been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace falcon {

enum Activation : int { kActNone = 0, kActSilu = 1, kActElu1 = 2, kActSigmoid = 3 };

struct ConvArgs {
  int B, T, C, W;
  bool bf16;
  int act;
  int64_t x_row;
  const void* x;
  const float* weight;
  const float* bias;       // may be null
  const void* state;       // may be null (zero rows)
  const int32_t* lengths;  // may be null (all T)
  void* y;
  void* state_out;         // may be null
  // backward
  const void* dy;
  bool dy_bf16;
  const float* dstate_out;  // may be null
  float* dx;
  float* dweight;
  float* dbias;            // may be null
  float* dstate;           // may be null
  float* workspace;
  // single token
  void* step_state;
  const uint8_t* is_first;  // may be null
};

// Polls a bounded wait makes before giving up (falcon_set_wait_limit).
int wait_limit();

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t st);
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t st);
size_t conv_bwd_workspace_bytes(const ConvArgs& a);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t st);

struct NormArgs {
  int B, T, G, d;
  bool bf16;
  int act;
  bool center, x_heads, y_heads;
  float eps, scale;
  int64_t x_row;
  const void* x;
  const float* weight;     // may be null (one)
  const float* bias;       // may be null
  void* y;
  const void* dy;
  bool dy_bf16;
  float* dx;
  float* dweight;          // may be null
  float* dbias;            // may be null
  float* workspace;
};

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st);
size_t norm_bwd_workspace_bytes(const NormArgs& a);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st);

struct ScanArgs {
  int B, T, D, N, G;
  bool bf16, softplus;
  int64_t x_row, dt_row, z_row, b_row, c_row;
  const void* x;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dskip;      // may be null
  const float* dt_bias;    // may be null
  const void* z;           // may be null (no gate)
  const float* S0;         // may be null (zero)
  const int32_t* lengths;  // may be null
  void* y;
  float* S_T;              // may be null; may be S0
  float* workspace;
  int spin_limit;          // polls before a wait between waves gives up
  // single token
  float* S;
  const uint8_t* is_first;
  // backward
  const void* dy;
  bool dy_bf16;
  const float* dS_T;       // may be null
  float* dx;
  float* ddt;
  float* dz;               // null without a gate
  float* dA;
  float* dB;
  float* dC;
  float* dD;               // may be null
  float* ddt_bias;         // may be null
  float* dS0;              // may be null
};

size_t scan_workspace_bytes(const ScanArgs& a);
hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t st);
hipError_t launch_scan_step(const ScanArgs& a, hipStream_t st);
size_t scan_bwd_workspace_bytes(const ScanArgs& a);
hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t st);

// Elements from one sequence, head and token of a tensor to the next.
struct HeadSteps {
  int64_t b, h, t;
};

struct LinearArgs {
  int B, H, T, dk, dv;
  bool bf16;
  float scale;
  HeadSteps q_at, k_at, v_at, o_at;   // o_at: of o or dO; gradients lie as their inputs, dense
  HeadSteps dqk_at, dv_at;
  bool zero_behind;
  const void* q;
  const void* k;
  const void* v;
  const float* log_decay;
  const float* S0;         // may be null (zero)
  const int32_t* lengths;  // may be null
  void* o;
  float* S_T;              // may be null; may be S0
  float* workspace;
  // single token
  float* S;
  const uint8_t* is_first;  // may be null
  // backward
  const void* dO;
  const float* dS_T;       // may be null
  float* dq;
  float* dk_out;
  float* dv_out;
  float* dS0;              // may be null
  float* dlog_decay;       // may be null
};

size_t linear_workspace_bytes(const LinearArgs& a);
hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_step(const LinearArgs& a, hipStream_t st);
size_t linear_bwd_workspace_bytes(const LinearArgs& a);
hipError_t launch_linear_bwd(const LinearArgs& a, hipStream_t st);

// One launch over every tile of every head: see falcon_linear_kernel.h.
struct LinearSweep {
  const void* q;           // null without outputs
  const void* k;
  const void* v;
  void* out;               // null: the tiles' sums into their slots
  HeadSteps q_at, k_at, v_at, out_at;
  const float* log_decay;
  const int32_t* lengths;  // may be null
  const float* start;      // the state before the first chunk where there are no slots; may be null (zero)
  float* last;             // the state behind the last chunk, of one tile a head; may be null
  float* slots;            // [heads][slots_each] states, tile t's at slot0 + t; may be null
  int64_t slots_each;
  int slot0;
  int64_t heads;
  int H, T, dv, tiles, chunks;   // chunks: of a tile
  int sf, sc;              // a state's element (f, c) lies at f sf + c sc
  float read, write;       // factors of what is read and of what is written
  bool rev, bf16;
  bool clear;              // zeros in the output rows behind the sequences' ends
};
// Every tile's part of the decays' gradient: see falcon_linear_decay.h.
struct LinearDecays {
  const void* q;
  const void* k;
  const void* v;
  const void* dO;
  HeadSteps q_at, k_at, v_at, o_at;
  const float* log_decay;
  const int32_t* lengths;  // may be null
  const float* S;          // [heads][s_each] states: tile t's at t, the one that enters it; may be null (zero)
  const float* R;          // [heads][r_each] adjoints: tile t's at t, from behind it; may be null (zero)
  int64_t s_each, r_each;
  float* parts;            // [B][tiles][H]
  int64_t heads;
  int H, T, dv, tiles, chunks;   // chunks: of a tile
  float read;              // factor of what is read
  bool bf16;
};

// What the tiles of one or two sweeps of the same sizes add to a state; the outputs of one;
// the gradients' sweeps, dv's first; the decays' gradient.  By the width of the (first sweep's)
// keys.
#define FALCON_LINEAR_OF(DK)                                                                                          \
  hipError_t launch_linear_sums_##DK(const LinearSweep& s, const LinearSweep* second, hipStream_t st);                \
  hipError_t launch_linear_outputs_##DK(const LinearSweep& s, hipStream_t st);                                        \
  hipError_t launch_linear_gradients_##DK(const LinearSweep& dv, const LinearSweep& dk, const LinearSweep& dq, hipStream_t st); \
  hipError_t launch_linear_decays_##DK(const LinearDecays& a, hipStream_t st);
FALCON_LINEAR_OF(16)
FALCON_LINEAR_OF(32)
FALCON_LINEAR_OF(64)
FALCON_LINEAR_OF(128)
#undef FALCON_LINEAR_OF

struct ResidualArgs {
  int B, T, G, d;
  bool zero_behind;
  bool bf16, stream_bf16;
  int act;
  bool post, pre;
  float eps;
  int64_t y_row, gate_row;
  const void* y;              // null in a backward pass from 8 bits
  const void* gate;           // may be null
  const void* h;              // may be null (zero)
  const float* post_weight;   // may be null (one)
  const float* alpha;         // may be null (one)
  const float* pre_weight;    // may be null (one)
  const int32_t* lengths;     // may be null
  void* h_out;
  void* n;                    // null without the second norm
  bool save;                  // 8 bits: written by the forward, read by the backward
  int8_t* y_codes;
  uint8_t* y_steps;
  int8_t* gate_codes;         // null without a gate
  uint8_t* gate_steps;
  // backward
  const void* dh_out;         // may be null (zero)
  const void* dn;
  bool dh_out_bf16, dn_bf16;
  float* dy;
  float* dgate;               // null without a gate
  float* dh;                  // may be null
  float* dalpha;              // may be null
  float* dpost_weight;        // may be null
  float* dpre_weight;         // may be null
  float* workspace;
};

hipError_t launch_residual_fwd(const ResidualArgs& a, hipStream_t st);
size_t residual_bwd_workspace_bytes(const ResidualArgs& a);
hipError_t launch_residual_bwd(const ResidualArgs& a, hipStream_t st);

// Columns of `parts` rows of n partial sums, `row` floats from one to the next, summed
// in a fixed order: column i goes to out[0][i] below ends[0], to out[1][i - ends[0]] below ends[1], else to
// out[2][i - ends[1]]; a null output is skipped.
struct PartSums {
  const float* in;
  int64_t parts, n, row;
  float* out[3];
  int64_t ends[2];
};
hipError_t launch_sum_parts(const PartSums& s, hipStream_t st);

}  // namespace falcon
