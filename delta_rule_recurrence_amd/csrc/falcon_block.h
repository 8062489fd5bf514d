// Host-side launch interface of the operators around the recurrence (short
// convolution, group norm, selective scan).  Arguments reaching the launchers
// have been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace falcon {

enum Activation : int { kActNone = 0, kActSilu = 1, kActElu1 = 2 };

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
