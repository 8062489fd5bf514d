// Short causal depthwise convolution with an activation (gfx950): whole
// prompts, single tokens and gradients.
//
//   p_t = bias + sum_{j < W} w_j x_{t - (W - 1) + j},   y_t = f(p_t)
//
// Every form is bound by its bytes (a few flops an element).  A thread owns V
// adjacent channels (16 bytes, or one where rows are not multiples of that)
// and a run of tokens; the last W rows slide through its registers, so each
// row is read once, and W - 1 again at the start of a run.  Measured (W = 4, bf16):
// prompts of 8 x 2048 x 2304 29 us where the tensors are still in the last-level
// cache (a copy of them 22), 42 where they are not (the copy 30), 3.6 TB/s: rows
// read again miss L2 (89 MB read for 75).  Their gradients 92 us and 5 for the sums
// of the taps (3.9 TB/s: reads of two types and float32 writes).  One token of
// 512 x 4608 10 us (3.7 TB/s): a thread loads 160 bytes of taps and bias for 128 of
// data, at addresses 128 bytes apart.

#include <algorithm>
#include <type_traits>

#include "falcon_block_device.h"
#include "falcon_launch.h"

namespace falcon {

namespace {

// The taps and biases of V channels; in wide accesses for V = 4, 8 (c a multiple of
// V, so V W floats start on a multiple of 16 bytes).
template <int W, int V>
__device__ __forceinline__ void load_taps(const float* weight, const float* bias, int c, float (&w)[W][V], float (&b)[V]) {
  float all[V * W];
  if constexpr (V > 1) {
    load_vec<float, V * W>(weight + int64_t(c) * W, all);
  } else {
#pragma unroll
    for (int j = 0; j < W; ++j) all[j] = weight[int64_t(c) * W + j];
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][v] = all[v * W + j];
  if (bias) {
    load_vec<float, V>(bias + c, b);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = 0.0f;
  }
}

// Row u of sequence b in the order "W - 1 rows of the state, then x": the
// state's for u < W - 1 (zero without one), else x's row u - (W - 1).
template <typename IO, int W, int V>
__device__ __forceinline__ void load_row(const IO* x, int64_t x_row, const IO* state, int64_t b, int T, int C, int c, int u,
                                         float (&r)[V]) {
  if (u < W - 1) {
    if (state) {
      load_vec<IO, V>(state + (b * (W - 1) + u) * C + c, r);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) r[v] = 0.0f;
    }
  } else {
    load_vec<IO, V>(x + (b * T + (u - (W - 1))) * x_row + c, r);
  }
}

// ---- prompts --------------------------------------------------------------------
template <typename IO, int W, int V, int ACT>
__global__ __launch_bounds__(256) void conv_fwd_kernel(const IO* __restrict__ x, int64_t x_row, const float* __restrict__ weight,
                                                       const float* __restrict__ bias, const IO* __restrict__ state,
                                                       const int32_t* __restrict__ lengths, IO* __restrict__ y,
                                                       IO* __restrict__ state_out, int B, int T, int C, int nvec, int run,
                                                       int nrun) {
  const int64_t id = by_xcd(blockIdx.x, gridDim.x) * 256 + threadIdx.x;
  if (id >= int64_t(B) * nrun * nvec) return;
  const int c = int(id % nvec) * V;
  const int64_t br = id / nvec;
  const int64_t b = br / nrun;
  const int t0 = int(br % nrun) * run;
  const int len = tokens_of(lengths, int(b), T);

  if (t0 == 0 && state_out) {
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      float r[V];
      load_row<IO, W, V>(x, x_row, state, b, T, C, c, len + i, r);
      store_vec<IO, V>(state_out + (b * (W - 1) + i) * C + c, r);
    }
  }
  const int t1 = min(t0 + run, len);
  if (t0 >= t1) return;
  float w[W][V], bs[V], win[W][V];
  load_taps<W, V>(weight, bias, c, w, bs);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_row<IO, W, V>(x, x_row, state, b, T, C, c, t0 + j, win[j]);
  const IO* px = x + (b * T + t0) * x_row + c;
  IO* py = y + (b * T + t0) * C + c;
#pragma unroll 4
  for (int t = t0; t < t1; ++t, px += x_row, py += C) {
    load_vec<IO, V>(px, win[W - 1]);
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float p = bs[v];
#pragma unroll
      for (int j = 0; j < W; ++j) p = __builtin_fmaf(w[j][v], win[j][v], p);
      out[v] = act_f32<ACT>(p);
    }
    store_vec<IO, V>(py, out);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) win[j][v] = win[j + 1][v];
  }
}

// ---- one token -------------------------------------------------------------------
template <typename IO, int W, int V, int ACT>
__global__ __launch_bounds__(256) void conv_step_kernel(const IO* __restrict__ x, int64_t x_row, const float* __restrict__ weight,
                                                        const float* __restrict__ bias, IO* __restrict__ state,
                                                        const uint8_t* __restrict__ is_first, IO* __restrict__ y, int B, int C,
                                                        int nvec) {
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (id >= int64_t(B) * nvec) return;
  const int c = int(id % nvec) * V;
  const int64_t b = id / nvec;
  float w[W][V], bs[V], win[W][V], out[V];
  const bool fresh = is_first && is_first[b];
  IO* ps = state + b * (W - 1) * C + c;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_vec<IO, V>(ps + int64_t(j) * C, win[j]);
  load_vec<IO, V>(x + b * x_row + c, win[W - 1]);
  load_taps<W, V>(weight, bias, c, w, bs);
  if (fresh) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) win[j][v] = 0.0f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float p = bs[v];
#pragma unroll
    for (int j = 0; j < W; ++j) p = __builtin_fmaf(w[j][v], win[j][v], p);
    out[v] = act_f32<ACT>(p);
  }
  store_vec<IO, V>(y + b * C + c, out);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_vec<IO, V>(ps + int64_t(j) * C, win[j + 1]);
}

// ---- gradients --------------------------------------------------------------------
// dp_t = dy_t f'(p_t);  dx_s = sum_j w_j dp_{s + W - 1 - j} (+ dstate_out where
// row s is one of the last W - 1);  dw_j = sum_t dp_t x_{t - (W - 1) + j}.
// Rows s < 0 are the carried state's.  A run recomputes p and dp of the W - 1
// tokens behind it.  A workgroup's 256 threads are `lanes` threads side by side
// in channels times 256 / lanes runs; their sums for the taps and the bias meet
// in LDS in a fixed order and leave as one row of partial sums.
constexpr int kBwdThreads = 256;
// Tokens loaded at once, a step ahead of their work, and tokens of a run (at 8 x 2048
// x 2304, W = 4, us: 2 ahead 97, 4 ahead 101, 1 ahead 114; runs of 16 95, of 64 91,
// but half the workgroups where there are few).
constexpr int kBwdAhead = 2, kBwdRun = 32;

template <typename IO, typename DY, int W, int V, int ACT>
__global__ __launch_bounds__(kBwdThreads) void conv_bwd_kernel(const IO* __restrict__ x, int64_t x_row, const float* __restrict__ weight,
                                                               const float* __restrict__ bias, const IO* __restrict__ state,
                                                               const int32_t* __restrict__ lengths, const DY* __restrict__ dy,
                                                               const float* __restrict__ dstate_out, float* __restrict__ dx,
                                                               float* __restrict__ dstate, float* __restrict__ parts, int B, int T,
                                                               int C, int nvec, int lanes, int run, int nrun, int64_t cblocks) {
  extern __shared__ float sums[];   // [runs of the workgroup][W + 1][lanes * V]
  const int64_t block = by_xcd(blockIdx.x, gridDim.x), rblock = block / cblocks;
  const int cblock = int(block % cblocks);
  const int runs = kBwdThreads / lanes;
  const int lane = threadIdx.x % lanes, mine = threadIdx.x / lanes;
  const int vec = cblock * lanes + lane;
  const int64_t br = rblock * runs + mine;
  const bool on = vec < nvec && br < int64_t(B) * nrun;
  const int c = vec * V;
  float dw[W][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][v] = 0.0f;
  }
  if (on) {
    const int64_t b = br / nrun;
    const int t0 = int(br % nrun) * run;
    const int len = tokens_of(lengths, int(b), T);
    const int t1 = min(t0 + run, T);          // rows of dx that are this run's: [t0, t1), and dstate's for the first
    float w[W][V], bs[V], win[W][V], dp[W][V];  // dp[j]: the slope of token t - (W - 1) + j
    load_taps<W, V>(weight, bias, c, w, bs);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) dp[j][v] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) win[j][v] = 0.0f;
    if (t0 < len) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) load_row<IO, W, V>(x, x_row, state, b, T, C, c, t0 + j, win[j]);
    }
    // kBwdAhead tokens' rows, loaded while the ones before are worked on
    float x_next[kBwdAhead][V], dy_next[kBwdAhead][V];
    auto load = [&](int tb) {
      if (tb >= len) return;
#pragma unroll
      for (int k = 0; k < kBwdAhead; ++k) {
        const int64_t token = b * T + min(tb + k, len - 1);
        load_vec<IO, V>(x + token * x_row + c, x_next[k]);
        load_vec<DY, V>(dy + token * C + c, dy_next[k]);
      }
    };
    // dx of row s = t - (W - 1), or of that row of the state; the first run's rows
    // before the first token are the state's, a later run's belong to the run before it.
    // Taps of tokens that there are, s + j for j = 0 .. W - 1, and no others: zero in
    // their place would be NaN times a tap that is not finite.
    auto back = [&](int t, auto all_there) __attribute__((always_inline)) {
      const int s = t - (W - 1);
      float out[V];
      const int i = s - (len - (W - 1));
      if (!all_there() && dstate_out && i >= 0 && i < W - 1) {
        load_vec<float, V>(dstate_out + (b * (W - 1) + i) * C + c, out);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (all_there() || (s + j >= 0 && s + j < len))
#pragma unroll
          for (int v = 0; v < V; ++v) out[v] = __builtin_fmaf(w[W - 1 - j][v], dp[j][v], out[v]);
      float* to = s >= 0 ? dx + (b * T + s) * C + c : dstate + (b * (W - 1) + t) * C + c;
      store_vec<float, V>(to, out);
    };
    // kBwdAhead tokens from tb.  INSIDE: all of them this run's and before the
    // sequence's end; else sums take those that are, again without products with zero.
    auto tokens = [&](int tb, auto inside) __attribute__((always_inline)) {
      float xs[kBwdAhead][V], gs[kBwdAhead][V];
#pragma unroll
      for (int k = 0; k < kBwdAhead; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool live = inside() || tb + k < len;
          xs[k][v] = live ? x_next[k][v] : 0.0f;
          gs[k][v] = live ? dy_next[k][v] : 0.0f;
        }
      if (tb + kBwdAhead < t1 + W - 1) load(tb + kBwdAhead);
#pragma unroll
      for (int k = 0; k < kBwdAhead; ++k) {
        const int t = tb + k;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          win[W - 1][v] = xs[k][v];
          float p = bs[v];
#pragma unroll
          for (int j = 0; j < W; ++j) p = __builtin_fmaf(w[j][v], win[j][v], p);
          dp[W - 1][v] = inside() || t < len ? gs[k][v] * act_slope_f32<ACT>(p) : 0.0f;
        }
        if (inside() || t < min(t1, len)) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            db[v] += dp[W - 1][v];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][v] = __builtin_fmaf(dp[W - 1][v], win[j][v], dw[j][v]);
          }
        }
        const int s = t - (W - 1);
        if (inside()) {
          if (s >= t0) {
            back(t, std::true_type{});
          } else if (t0 == 0 && dstate) {
            back(t, std::false_type{});
          }
        } else if (t < t1 + W - 1 && (s >= t0 || (t0 == 0 && dstate))) {
          back(t, std::false_type{});
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            win[j][v] = win[j + 1][v];
            dp[j][v] = dp[j + 1][v];
          }
      }
    };
    load(t0);
    int tb = t0;
    for (; tb + kBwdAhead <= min(t1, len); tb += kBwdAhead) tokens(tb, std::true_type{});
    for (; tb < t1 + W - 1; tb += kBwdAhead) tokens(tb, std::false_type{});
  }
  // the workgroup's sums, run by run
  const int width = lanes * V;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int j = 0; j < W; ++j) sums[(mine * (W + 1) + j) * width + lane * V + v] = dw[j][v];
    sums[(mine * (W + 1) + W) * width + lane * V + v] = db[v];
  }
  __syncthreads();
  // one row of partial sums: [C][W] of the taps, then [C] of the bias
  float* row = parts + rblock * int64_t(C) * (W + 1);
  for (int i = threadIdx.x; i < (W + 1) * width; i += kBwdThreads) {
    const int j = i / width, cc = cblock * width + i % width;
    if (cc >= C) continue;
    float s = 0.0f;
    for (int r = 0; r < runs; ++r) s += sums[(r * (W + 1)) * width + i];
    if (j < W) {
      row[int64_t(cc) * W + j] = s;
    } else {
      row[int64_t(C) * W + cc] = s;
    }
  }
}

// Elements a thread owns: 16 bytes' worth where every row starts on a multiple
// of 16 bytes, else one.
bool rows_wide(const ConvArgs& a, int v) { return a.C % v == 0 && a.x_row % v == 0; }

// Workgroups of 256 threads in one launch (a grid has 32 bits of threads).
constexpr int64_t kMaxGrid = (int64_t(1) << 24) - 1;

struct ConvBwdShape {
  int v, nvec, lanes, run, nrun;
  int64_t cblocks, rblocks;
};
ConvBwdShape conv_bwd_shape(const ConvArgs& a) {
  ConvBwdShape s{};
  s.v = rows_wide(a, 4) ? 4 : 1;
  s.nvec = (a.C + s.v - 1) / s.v;
  s.lanes = 1;
  while (s.lanes < 64 && s.lanes < s.nvec) s.lanes *= 2;
  s.cblocks = (s.nvec + s.lanes - 1) / s.lanes;
  s.run = kBwdRun;
  s.nrun = std::max(1, (a.T + s.run - 1) / s.run);
  const int runs = kBwdThreads / s.lanes;
  s.rblocks = (int64_t(a.B) * s.nrun + runs - 1) / runs;
  return s;
}

template <typename IO, int W, int V, int ACT>
hipError_t conv_fwd_typed(const ConvArgs& a, hipStream_t st) {
  const int64_t nvec = (int64_t(a.C) + V - 1) / V;
  const auto runs_of = [&](int64_t run) { return std::max<int64_t>(1, (a.T + run - 1) / run); };
  // runs of 32 tokens, or fewer where those would not fill the card (16 at 8 x 2048 x
  // 2304, bf16: three rows in sixteen are read twice), or more where a grid would
  // not hold them
  int64_t run = 32;
  while (run > 1 && a.B * runs_of(run) * nvec < 256 * 16 * 64) run /= 2;
  while (run < a.T && a.B * runs_of(run) * nvec > kMaxGrid * 256) run *= 2;
  const int64_t nrun = runs_of(run);
  // as many sequences at once as a grid holds: one at least, since nvec < 2^31
  const int64_t each = std::min<int64_t>(a.B, kMaxGrid * 256 / (nrun * nvec));
  for (int64_t b = 0; b < a.B; b += each) {
    const int64_t n = std::min(each, a.B - b), rows = b * a.T, kept = b * (W - 1) * a.C;
    const IO* state = static_cast<const IO*>(a.state);
    IO* state_out = static_cast<IO*>(a.state_out);
    conv_fwd_kernel<IO, W, V, ACT><<<dim3(unsigned((n * nrun * nvec + 255) / 256)), dim3(256), 0, st>>>(
        static_cast<const IO*>(a.x) + rows * a.x_row, a.x_row, a.weight, a.bias, state ? state + kept : nullptr,
        a.lengths ? a.lengths + b : nullptr, static_cast<IO*>(a.y) + rows * a.C, state_out ? state_out + kept : nullptr, int(n), a.T,
        a.C, int(nvec), int(run), int(nrun));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename IO, int W, int V, int ACT>
hipError_t conv_step_typed(const ConvArgs& a, hipStream_t st) {
  const int nvec = (a.C + V - 1) / V;
  const int64_t blocks = (int64_t(a.B) * nvec + 255) / 256;
  if (blocks > kMaxGrid) return hipErrorInvalidValue;
  conv_step_kernel<IO, W, V, ACT><<<dim3(unsigned(blocks)), dim3(256), 0, st>>>(
      static_cast<const IO*>(a.x), a.x_row, a.weight, a.bias, static_cast<IO*>(a.step_state), a.is_first, static_cast<IO*>(a.y),
      a.B, a.C, nvec);
  return hipGetLastError();
}

template <typename IO, typename DY, int W, int V, int ACT>
hipError_t conv_bwd_typed(const ConvArgs& a, const ConvBwdShape& s, hipStream_t st) {
  const int64_t blocks = s.rblocks * s.cblocks;
  if (blocks > kMaxGrid) return hipErrorInvalidValue;
  const size_t lds = size_t(kBwdThreads) * V * (W + 1) * sizeof(float);
  conv_bwd_kernel<IO, DY, W, V, ACT><<<dim3(unsigned(blocks)), dim3(kBwdThreads), lds, st>>>(
      static_cast<const IO*>(a.x), a.x_row, a.weight, a.bias, static_cast<const IO*>(a.state), a.lengths,
      static_cast<const DY*>(a.dy), a.dstate_out, a.dx, a.dstate, a.workspace, a.B, a.T, a.C, s.nvec, s.lanes, s.run, s.nrun,
      s.cblocks);
  return hipGetLastError();
}

// The kernels by activation, taps, type and width of access.
enum class Form { kFwd, kStep };
template <Form F, typename IO, int W, int V>
hipError_t by_act(const ConvArgs& a, hipStream_t st) {
  if constexpr (F == Form::kFwd) {
    return a.act == kActSilu ? conv_fwd_typed<IO, W, V, kActSilu>(a, st) : conv_fwd_typed<IO, W, V, kActNone>(a, st);
  } else {
    return a.act == kActSilu ? conv_step_typed<IO, W, V, kActSilu>(a, st) : conv_step_typed<IO, W, V, kActNone>(a, st);
  }
}
template <Form F, typename IO, int V>
hipError_t by_width(const ConvArgs& a, hipStream_t st) {
  switch (a.W) {
    case 2: return by_act<F, IO, 2, V>(a, st);
    case 3: return by_act<F, IO, 3, V>(a, st);
    default: return by_act<F, IO, 4, V>(a, st);
  }
}
template <Form F>
hipError_t by_type(const ConvArgs& a, hipStream_t st) {
  if (a.bf16) return rows_wide(a, 8) ? by_width<F, bf16_t, 8>(a, st) : by_width<F, bf16_t, 1>(a, st);
  return rows_wide(a, 4) ? by_width<F, float, 4>(a, st) : by_width<F, float, 1>(a, st);
}

template <typename IO, typename DY, int V>
hipError_t bwd_by_width(const ConvArgs& a, const ConvBwdShape& s, hipStream_t st) {
  const bool silu = a.act == kActSilu;
  switch (a.W) {
    case 2: return silu ? conv_bwd_typed<IO, DY, 2, V, kActSilu>(a, s, st) : conv_bwd_typed<IO, DY, 2, V, kActNone>(a, s, st);
    case 3: return silu ? conv_bwd_typed<IO, DY, 3, V, kActSilu>(a, s, st) : conv_bwd_typed<IO, DY, 3, V, kActNone>(a, s, st);
    default: return silu ? conv_bwd_typed<IO, DY, 4, V, kActSilu>(a, s, st) : conv_bwd_typed<IO, DY, 4, V, kActNone>(a, s, st);
  }
}
template <typename IO, typename DY>
hipError_t bwd_by_vec(const ConvArgs& a, const ConvBwdShape& s, hipStream_t st) {
  return s.v == 4 ? bwd_by_width<IO, DY, 4>(a, s, st) : bwd_by_width<IO, DY, 1>(a, s, st);
}

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t st) { return by_type<Form::kFwd>(a, st); }
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t st) { return by_type<Form::kStep>(a, st); }

size_t conv_bwd_workspace_bytes(const ConvArgs& a) {
  return size_t(conv_bwd_shape(a).rblocks) * size_t(a.C) * (a.W + 1) * sizeof(float);
}

hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t st) {
  const ConvBwdShape s = conv_bwd_shape(a);
  hipError_t e = hipSuccess;
  if (s.rblocks * s.cblocks > 0) {
    if (a.bf16)
      e = a.dy_bf16 ? bwd_by_vec<bf16_t, bf16_t>(a, s, st) : bwd_by_vec<bf16_t, float>(a, s, st);
    else
      e = a.dy_bf16 ? bwd_by_vec<float, bf16_t>(a, s, st) : bwd_by_vec<float, float>(a, s, st);
  }
  if (e != hipSuccess) return e;
  const int64_t taps = int64_t(a.C) * a.W;
  return launch_sum_parts({a.workspace, s.rblocks, taps + a.C, taps + a.C, {a.dweight, a.dbias, nullptr}, {taps, taps + a.C}}, st);
}

}  // namespace falcon
