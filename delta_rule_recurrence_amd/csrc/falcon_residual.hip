// The residual update of a block (gfx950): norm of the block's output by groups, gate,
// scale, sum with the stream, norm of the stream for the next block; its gradients;
// and the output and gate kept in 8 bits between the two.
//
//   yhat = y / rms_group(y),  z = post_weight yhat  (or y),  f = act(gate)  (or 1)
//   h' = h + alpha f z,       n = pre_weight h' / rms(h')
//
//   D  = dh' + r (t - hhat mean(t hhat)),  t = pre_weight dn,  r = 1 / rms(h')
//   dh = D,  dgate = D alpha z act'(gate),  dy = r_y (s - yhat mean(s yhat)),  s = D alpha f post_weight
//   dalpha = post_weight A,  dpost_weight = alpha A,  A = sum D f yhat;  dpre_weight = sum dn hhat
//
// Bound by bytes: every tensor is read or written once.  A row of C channels is held by
// 64 to 512 threads, up to two pieces of 8 channels each, from its loads to its stores;
// a thread keeps its channels' weights and walks over rows.  Sums of squares are made in
// double, so that no row of float32 numbers leaves their range.  A group's sum is a sum
// over lanes where a group is 1, 2, 4, ... 64 pieces of 8, else it goes through LDS; a
// whole row's over the row's waves.
//
// In 8 bits, 32 adjacent channels of a row share a step, the smallest power of two of which
// 127 reach the largest of them: a value is off by at most half a step, 2^-7 of the
// largest, and dividing by and multiplying with the step is exact.

#include <algorithm>

#include "falcon_block_device.h"
#include "falcon_launch.h"

namespace falcon {

namespace {

constexpr int kPiece = 8;
constexpr int kBlock = 32;        // channels of one step
constexpr int kRowsEach = 64;     // rows whose parts of the parameters' gradients one thread sums: float32 sums stay short

// How rows and groups lie on threads.
struct Shape {
  int threads_row, nc, rows_block;   // threads of a row, pieces of a thread, rows of a workgroup at a time
  int64_t blocks;
  int rows_each;                     // rows a thread walks over
  int group_lanes;                   // lanes of a group; 0: through LDS; -1: the group is the row
  size_t lds;
};

// ---- rows; their types are met at run time (a uniform branch a tensor) ---------------
// WIDE: pieces of 8 adjacent channels, one wide access each; else neighbours go to
// neighbouring lanes, element by element.
template <int NC, bool WIDE, int TPR>
struct Lane {
  int t, C;
  __device__ __forceinline__ int channel(int k, int i) const { return WIDE ? (k * TPR + t) * kPiece + i : (k * kPiece + i) * TPR + t; }
};

template <int NC, bool WIDE, int TPR, typename E>
__device__ __forceinline__ void load_typed(const E* p, const Lane<NC, WIDE, TPR>& at, float missing, float (&v)[NC][kPiece]) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[k][i] = missing;
      const int c = at.channel(k, 0);
      if (c < at.C) load_vec<E, kPiece>(p + c, v[k]);
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const int c = at.channel(k, i);
        v[k][i] = c < at.C ? io<E>::load(p, c) : missing;
      }
    }
  }
}
// Row `row` of `step` elements; `on` false: not read, zeros.
template <int NC, bool WIDE, int TPR>
__device__ __forceinline__ void load_row(const void* p, bool bf16, int64_t at_row, const Lane<NC, WIDE, TPR>& at, bool on, float (&v)[NC][kPiece]) {
  if (on && p) {
    if (bf16) {
      load_typed<NC, WIDE, TPR>(static_cast<const bf16_t*>(p) + at_row, at, 0.0f, v);
    } else {
      load_typed<NC, WIDE, TPR>(static_cast<const float*>(p) + at_row, at, 0.0f, v);
    }
  } else {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[k][i] = 0.0f;
  }
}
template <int NC, bool WIDE, int TPR, typename E>
__device__ __forceinline__ void store_typed(E* p, const Lane<NC, WIDE, TPR>& at, const float (&v)[NC][kPiece]) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    if constexpr (WIDE) {
      const int c = at.channel(k, 0);
      if (c < at.C) store_vec<E, kPiece>(p + c, v[k]);
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const int c = at.channel(k, i);
        if (c < at.C) io<E>::store(p, c, v[k][i]);
      }
    }
  }
}
template <int NC, bool WIDE, int TPR>
__device__ __forceinline__ void store_row(void* p, bool bf16, int64_t at_row, const Lane<NC, WIDE, TPR>& at, const float (&v)[NC][kPiece]) {
  if (bf16) {
    store_typed<NC, WIDE, TPR>(static_cast<bf16_t*>(p) + at_row, at, v);
  } else {
    store_typed<NC, WIDE, TPR>(static_cast<float*>(p) + at_row, at, v);
  }
}
template <int NC, bool WIDE, int TPR>
__device__ __forceinline__ void load_params(const float* p, float missing, const Lane<NC, WIDE, TPR>& at, float (&v)[NC][kPiece]) {
  if (p) {
    load_typed<NC, WIDE, TPR>(p, at, missing, v);
  } else {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[k][i] = missing;
  }
}

// ---- 8 bits ---------------------------------------------------------------------------
// A step's byte is its float32 exponent field; 255, whose step is infinite, with codes of
// zero stands for channels that were not all finite: they come back as NaN.
__device__ __forceinline__ float step_of(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ uint32_t step_byte(uint32_t largest) {
  if (largest >= 0x7f800000u) return 255;
  // largest = 1.m 2^E fits 127 steps of 2^(E - 6) = 1.984375 2^E, or of twice that
  const int b = int(largest >> 23) - 6 + ((largest & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return uint32_t(max(b, 1));
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int m = 1; m < LANES; m *= 2) v = max(v, uint32_t(__shfl_xor(int(v), m)));
  return v;
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <int NC, bool WIDE, int TPR>
__device__ __forceinline__ void pack_row(int8_t* codes, uint8_t* steps, const Lane<NC, WIDE, TPR>& at, bool on, const float (&v)[NC][kPiece]) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    if constexpr (WIDE) {
      uint32_t largest = 0;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) largest = max(largest, magnitude(v[k][i]));
      const uint32_t byte = step_byte(lanes_max<kBlock / kPiece>(largest));
      const float inverse = byte == 255 ? 0.0f : step_of(254 - byte);
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const int code = byte == 255 ? 0 : int(__builtin_rintf(v[k][i] * inverse));
        w[i / 4] |= (uint32_t(code) & 255u) << (8 * (i % 4));
      }
      const int c = at.channel(k, 0);
      if (on && c < at.C) {
        *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0], w[1]);
        if (c % kBlock == 0) steps[c / kBlock] = uint8_t(byte);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const uint32_t byte = step_byte(lanes_max<kBlock>(magnitude(v[k][i])));
        const int c = at.channel(k, i);
        if (on && c < at.C) {
          codes[c] = byte == 255 ? int8_t(0) : int8_t(int(__builtin_rintf(v[k][i] * step_of(254 - byte))));
          if (c % kBlock == 0) steps[c / kBlock] = uint8_t(byte);
        }
      }
    }
  }
}
template <int NC, bool WIDE, int TPR>
__device__ __forceinline__ void unpack_row(const int8_t* codes, const uint8_t* steps, const Lane<NC, WIDE, TPR>& at, bool on, float (&v)[NC][kPiece]) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[k][i] = 0.0f;
    if constexpr (WIDE) {
      const int c = at.channel(k, 0);
      if (on && c < at.C) {
        const uint2 w = *reinterpret_cast<const uint2*>(codes + c);
        const float step = step_of(steps[c / kBlock]);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) v[k][i] = float(int8_t((i < 4 ? w.x : w.y) >> (8 * (i % 4)))) * step;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const int c = at.channel(k, i);
        if (on && c < at.C) v[k][i] = float(codes[c]) * step_of(steps[c / kBlock]);
      }
    }
  }
}

// ---- sums --------------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ double dpp_plus(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(u)), CTRL, 0xf, 0xf, true));
  const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(uint32_t(u >> 32)), CTRL, 0xf, 0xf, true));
  return v + __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
// Sum over aligned groups of `lanes` lanes (a power of two up to 64, the same for the
// whole wave, which must be active), in every lane.
__device__ __forceinline__ double lanes_sum(double v, int lanes) {
  if (lanes >= 2) v = dpp_plus<0xb1>(v);
  if (lanes >= 4) v = dpp_plus<0x4e>(v);
  if (lanes >= 8) v = dpp_plus<0x141>(v);
  if (lanes >= 16) v = dpp_plus<0x140>(v);
  if (lanes >= 32) v += __shfl_xor(v, 16);
  if (lanes >= 64) v += __shfl_xor(v, 32);
  return v;
}

// 1 / sqrt(m) as two factors, the first a power of two, so that x times the first does
// not overflow where the product with both does not (m from squares of any float32).
struct Inverse {
  float power, rest;
  __device__ __forceinline__ float times(float x) const { return x * power * rest; }
  __device__ __forceinline__ float whole() const { return power * rest; }
};
__device__ __forceinline__ Inverse inverse_root(double m) {
  int e = __builtin_amdgcn_frexp_exp(m);              // m = f 2^e, f in [1/2, 1); 0 for 0, infinity and NaN
  e += e & 1;                                         // an even one: f in [1/4, 1)
  const float f = float(__builtin_amdgcn_ldexp(m, -e));
  const int half = -e / 2, first = min(half, 120);
  return {__builtin_amdgcn_ldexpf(1.0f, first), __builtin_amdgcn_ldexpf(__builtin_amdgcn_rsqf(f), half - first)};
}

// The sums of one row over its groups.  `mine`: this thread's part, of each of its
// pieces (WIDE) or channels.  The result is in place: each piece's (channel's) group's sum.
// Every thread of the workgroup takes part.
template <int NC, bool WIDE, int TPR>
struct Sums {
  static constexpr int kParts = WIDE ? 1 : kPiece;
  static constexpr int kWaves = TPR / 64;
  double* lds;            // of this row: [3 slots][2 turns][2 sums][kWaves], then [items + G] where groups go through it
  int lanes, G, d;        // Shape::group_lanes

  // One sum over the row, or two at once.  Rounds with the same `slot` must have another barrier
  // between them; `turn` alternates.
  template <bool BOTH>
  __device__ __forceinline__ void row(double& a, double& b, int slot, int turn, const Lane<NC, WIDE, TPR>& at) const {
    a = lanes_sum(a, 64);
    if constexpr (BOTH) b = lanes_sum(b, 64);
    if constexpr (kWaves > 1) {
      double* const mine = lds + (slot * 2 + turn) * 2 * kWaves;
      const int w = at.t / 64;
      if (at.t % 64 == 0) {
        mine[w] = a;
        if constexpr (BOTH) mine[kWaves + w] = b;
      }
      __syncthreads();
      a = b = 0.0;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        a += mine[k];
        if constexpr (BOTH) b += mine[kWaves + k];
      }
    }
  }
  __device__ __forceinline__ void groups(double (&part)[NC][kParts], int slot, int turn, const Lane<NC, WIDE, TPR>& at) const {
    if (lanes < 0) {
      double all = 0.0, none = 0.0;
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kParts; ++i) all += part[k][i];
      row<false>(all, none, slot, turn, at);
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kParts; ++i) part[k][i] = all;
    } else if (WIDE && lanes > 0) {
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kParts; ++i) part[k][i] = lanes_sum(part[k][i], lanes);
    } else {
      constexpr int kUnit = WIDE ? kPiece : 1;
      const int items = at.C / kUnit, each = d / kUnit;
      double* const item = lds + 12 * kWaves;
      double* const sum = item + items;
      __syncthreads();    // the last round's sums have been read
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const int c = at.channel(k, i);
          if (c < at.C) item[c / kUnit] = part[k][i];
        }
      __syncthreads();
      // a wave a group at a time
      for (int g = at.t / 64; g < G; g += kWaves) {
        double s = 0.0;
        for (int j = at.t % 64; j < each; j += 64) s += item[g * each + j];
        s = lanes_sum(s, 64);
        if (at.t % 64 == 0) sum[g] = s;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const int c = at.channel(k, i);
          part[k][i] = c < at.C ? sum[c / d] : 0.0;
        }
    }
  }
};

// f(k, i) for every channel of a thread, with the activation's number as a constant.
template <int NC, typename F>
__device__ __forceinline__ void each_channel(int act, F f) {
  auto all = [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) f(k, i, kind);
  };
  if (act == kActSilu) {
    all(std::integral_constant<int, kActSilu>{});
  } else if (act == kActSigmoid) {
    all(std::integral_constant<int, kActSigmoid>{});
  } else {
    all(std::integral_constant<int, kActNone>{});
  }
}

// Which row of which sequence, and whether it is there.
struct RowAt {
  int64_t row;
  bool inside, live;      // of the call; before its sequence's end
};
__device__ __forceinline__ RowAt row_at(int64_t row, const ResidualArgs& a) {
  RowAt r{row, row < int64_t(a.B) * a.T, false};
  if (r.inside) {
    r.live = true;
    if (a.lengths) {
      const int b = int(uint32_t(row) / uint32_t(a.T));
      r.live = int(row - int64_t(b) * a.T) < tokens_of(a.lengths, b, a.T);
    }
  }
  return r;
}

template <int TPR>
constexpr int threads_of() {
  return TPR < 256 ? 256 : TPR;
}

template <int TPR, int NC, bool WIDE>
__global__ __launch_bounds__(threads_of<TPR>()) void residual_fwd_kernel(ResidualArgs a, int rows_each, int group_lanes) {
  constexpr int kRows = threads_of<TPR>() / TPR;
  using At = Lane<NC, WIDE, TPR>;
  using S = Sums<NC, WIDE, TPR>;
  extern __shared__ double lds[];
  const int C = a.G * a.d;
  const At at{int(threadIdx.x) % TPR, C};
  const int mine = int(threadIdx.x) / TPR;
  const int row_lds = S::kWaves * 12 + (group_lanes == 0 ? C / (WIDE ? kPiece : 1) + a.G : 0);
  const S sums{lds + mine * row_lds, group_lanes, a.G, a.d};
  const double inv_d = 1.0 / a.d, inv_C = 1.0 / C;
  float aw[NC][kPiece], wn[NC][kPiece];
  load_params<NC, WIDE, TPR>(a.alpha, 1.0f, at, aw);
  load_params<NC, WIDE, TPR>(a.post ? a.post_weight : nullptr, 1.0f, at, wn);
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int i = 0; i < kPiece; ++i) aw[k][i] *= wn[k][i];
  load_params<NC, WIDE, TPR>(a.pre_weight, 1.0f, at, wn);
  const int64_t first = int64_t(blockIdx.x) * rows_each * kRows;
  for (int it = 0; it < rows_each; ++it) {
    const RowAt r = row_at(first + int64_t(it) * kRows + mine, a);
    float y[NC][kPiece], h[NC][kPiece];
    load_row<NC, WIDE, TPR>(a.y, a.bf16, r.row * a.y_row, at, r.live, y);
    load_row<NC, WIDE, TPR>(a.h, a.stream_bf16, r.row * C, at, r.live, h);
    float u[NC][kPiece];
    if (a.gate) load_row<NC, WIDE, TPR>(a.gate, a.bf16, r.row * a.gate_row, at, r.live, u);
    if (a.save) {
      const int64_t blocks = (C + kBlock - 1) / kBlock;
      pack_row<NC, WIDE, TPR>(a.y_codes + r.row * C, a.y_steps + r.row * blocks, at, r.live, y);
      if (a.gate) pack_row<NC, WIDE, TPR>(a.gate_codes + r.row * C, a.gate_steps + r.row * blocks, at, r.live, u);
    }
    if (a.post) {
      double part[NC][S::kParts];
#pragma unroll
      for (int k = 0; k < NC; ++k) {
#pragma unroll
        for (int i = 0; i < S::kParts; ++i) part[k][i] = 0.0;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) part[k][WIDE ? 0 : i] = __builtin_fma(double(y[k][i]), double(y[k][i]), part[k][WIDE ? 0 : i]);
      }
      sums.groups(part, 0, it & 1, at);
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        Inverse inv;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          if (!WIDE || i == 0) inv = inverse_root(__builtin_fma(part[k][WIDE ? 0 : i], inv_d, double(a.eps)));
          y[k][i] = inv.times(y[k][i]);
        }
      }
    }
    if (a.gate) {
      each_channel<NC>(a.act, [&](int k, int i, auto kind) { y[k][i] *= act_f32<kind()>(u[k][i]); });
    }
    double squares = 0.0, none = 0.0;
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        h[k][i] = __builtin_fmaf(aw[k][i], y[k][i], h[k][i]);
        const double x = at.channel(k, i) < C ? double(h[k][i]) : 0.0;
        squares = __builtin_fma(x, x, squares);
      }
    if (r.live) store_row<NC, WIDE, TPR>(a.h_out, a.stream_bf16, r.row * C, at, h);
    if (a.pre) {
      sums.template row<false>(squares, none, 1, it & 1, at);
      const Inverse inv = inverse_root(__builtin_fma(squares, inv_C, double(a.eps)));
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) h[k][i] = inv.times(h[k][i]) * wn[k][i];
      if (r.live) store_row<NC, WIDE, TPR>(a.n, a.bf16, r.row * C, at, h);
    }
  }
}

template <int TPR, int NC, bool WIDE>
__global__ __launch_bounds__(threads_of<TPR>()) void residual_bwd_kernel(ResidualArgs a, int rows_each, int group_lanes, float* parts) {
  constexpr int kThreads = threads_of<TPR>(), kRows = kThreads / TPR;
  using At = Lane<NC, WIDE, TPR>;
  using S = Sums<NC, WIDE, TPR>;
  extern __shared__ double lds[];
  const int C = a.G * a.d;
  const At at{int(threadIdx.x) % TPR, C};
  const int mine = int(threadIdx.x) / TPR;
  const int row_lds = S::kWaves * 12 + (group_lanes == 0 ? C / (WIDE ? kPiece : 1) + a.G : 0);
  const S sums{lds + mine * row_lds, group_lanes, a.G, a.d};
  const double inv_d = 1.0 / a.d, inv_C = 1.0 / C;
  float aw[NC][kPiece], wn[NC][kPiece], A[NC][kPiece], N[NC][kPiece];
  load_params<NC, WIDE, TPR>(a.alpha, 1.0f, at, aw);
  load_params<NC, WIDE, TPR>(a.post ? a.post_weight : nullptr, 1.0f, at, wn);
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      aw[k][i] *= wn[k][i];
      A[k][i] = N[k][i] = 0.0f;
    }
  load_params<NC, WIDE, TPR>(a.pre_weight, 1.0f, at, wn);
  const int64_t blocks = (C + kBlock - 1) / kBlock;
  const int64_t first = int64_t(blockIdx.x) * rows_each * kRows;
  for (int it = 0; it < rows_each; ++it) {
    const RowAt r = row_at(first + int64_t(it) * kRows + mine, a);
    float y[NC][kPiece], u[NC][kPiece], D[NC][kPiece];
    if (a.save) {
      unpack_row<NC, WIDE, TPR>(a.y_codes + r.row * C, a.y_steps + r.row * blocks, at, r.live, y);
      if (a.gate_codes) unpack_row<NC, WIDE, TPR>(a.gate_codes + r.row * C, a.gate_steps + r.row * blocks, at, r.live, u);
    } else {
      load_row<NC, WIDE, TPR>(a.y, a.bf16, r.row * a.y_row, at, r.live, y);
      if (a.gate) load_row<NC, WIDE, TPR>(a.gate, a.bf16, r.row * a.gate_row, at, r.live, u);
    }
    load_row<NC, WIDE, TPR>(a.dh_out, a.dh_out_bf16, r.row * C, at, r.live, D);
    if (a.pre) {
      float h[NC][kPiece], t[NC][kPiece];
      load_row<NC, WIDE, TPR>(a.h_out, a.stream_bf16, r.row * C, at, r.live, h);
      load_row<NC, WIDE, TPR>(a.dn, a.dn_bf16, r.row * C, at, r.live, t);
      double squares = 0.0, dots = 0.0;
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          const double x = double(h[k][i]);
          squares = __builtin_fma(x, x, squares);
          dots = __builtin_fma(x, double(t[k][i] * wn[k][i]), dots);
        }
      sums.template row<true>(squares, dots, 0, it & 1, at);
      // (a row that is not there is zero throughout, whatever eps)
      const Inverse inv = inverse_root(r.live ? __builtin_fma(squares, inv_C, double(a.eps)) : 1.0);
      const float mean = float(dots * inv_C * double(inv.power) * double(inv.rest)), whole = inv.whole();
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          const float hhat = inv.times(h[k][i]);
          N[k][i] = __builtin_fmaf(t[k][i], hhat, N[k][i]);
          D[k][i] = __builtin_fmaf(whole, __builtin_fmaf(-hhat, mean, t[k][i] * wn[k][i]), D[k][i]);
        }
    }
    if (a.dh && r.inside) store_row<NC, WIDE, TPR>(a.dh, false, r.row * C, at, D);
    // D becomes D f, and dgate is made next to it
    Inverse inv[NC][S::kParts];
    if (a.post) {
      double part[NC][S::kParts];
#pragma unroll
      for (int k = 0; k < NC; ++k) {
#pragma unroll
        for (int i = 0; i < S::kParts; ++i) part[k][i] = 0.0;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) part[k][WIDE ? 0 : i] = __builtin_fma(double(y[k][i]), double(y[k][i]), part[k][WIDE ? 0 : i]);
      }
      sums.groups(part, 1, it & 1, at);
#pragma unroll
      for (int k = 0; k < NC; ++k) {
#pragma unroll
        for (int i = 0; i < S::kParts; ++i) inv[k][i] = inverse_root(r.live ? __builtin_fma(part[k][i], inv_d, double(a.eps)) : 1.0);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) y[k][i] = inv[k][WIDE ? 0 : i].times(y[k][i]);
      }
    }
    if (a.dgate) {
      each_channel<NC>(a.act, [&](int k, int i, auto kind) {
        const float x = u[k][i];
        u[k][i] = D[k][i] * aw[k][i] * y[k][i] * act_slope_f32<kind()>(x);
        D[k][i] *= act_f32<kind()>(x);
      });
      if (r.inside) store_row<NC, WIDE, TPR>(a.dgate, false, r.row * C, at, u);
    }
    double part[NC][S::kParts];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
#pragma unroll
      for (int i = 0; i < S::kParts; ++i) part[k][i] = 0.0;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        A[k][i] = __builtin_fmaf(D[k][i], y[k][i], A[k][i]);
        D[k][i] *= aw[k][i];
        part[k][WIDE ? 0 : i] = __builtin_fma(double(D[k][i]), double(y[k][i]), part[k][WIDE ? 0 : i]);
      }
    }
    if (a.post) {
      sums.groups(part, 2, it & 1, at);
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          const Inverse& v = inv[k][WIDE ? 0 : i];
          D[k][i] = v.whole() * __builtin_fmaf(-y[k][i], float(part[k][WIDE ? 0 : i] * inv_d), D[k][i]);
        }
    }
    if (r.inside) store_row<NC, WIDE, TPR>(a.dy, false, r.row * C, at, D);
  }
  if (!parts) return;
  // the workgroup's sums over its rows, in a fixed order: one row of partial sums, [C]
  // each of alpha, post_weight and pre_weight
  float* const out = parts + int64_t(blockIdx.x) * 3 * C;
  float* const shared = reinterpret_cast<float*>(lds);   // [kThreads][kPiece]
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPiece; ++i) shared[threadIdx.x * kPiece + i] = which ? N[k][i] : A[k][i];
      __syncthreads();
      if (mine == 0) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          const int c = at.channel(k, i);
          if (c < C) {
            double s = 0.0;
            for (int m = 0; m < kRows; ++m) s += shared[(m * TPR + at.t) * kPiece + i];
            if (which) {
              out[2 * C + c] = float(s);
            } else {
              out[c] = float(s * (a.post && a.post_weight ? a.post_weight[c] : 1.0f));
              out[C + c] = float(s * (a.alpha ? a.alpha[c] : 1.0f));
            }
          }
        }
      }
    }
  }
}

bool wide(const ResidualArgs& a) {
  const int64_t C = int64_t(a.G) * a.d;
  return C % kPiece == 0 && (!a.post || a.d % kPiece == 0) && (!a.y || a.y_row % kPiece == 0) && (!a.gate || a.gate_row % kPiece == 0);
}

Shape shape_of(const ResidualArgs& a, bool bwd) {
  Shape s{};
  const int C = a.G * a.d;
  s.nc = C <= 512 ? 1 : 2;
  s.threads_row = 64;
  while (s.threads_row * s.nc * kPiece < C) s.threads_row *= 2;
  s.rows_block = std::max(1, 256 / s.threads_row);
  const int64_t rows = int64_t(a.B) * a.T;
  const int64_t most = bwd ? 1024 : 2048;
  const int64_t each = std::max<int64_t>(1, (rows + most * s.rows_block - 1) / (most * s.rows_block));
  s.rows_each = int(bwd ? std::min<int64_t>(each, kRowsEach) : each);
  s.blocks = (rows + int64_t(s.rows_each) * s.rows_block - 1) / (int64_t(s.rows_each) * s.rows_block);
  const bool w = wide(a);
  const int lanes = a.d / kPiece;
  s.group_lanes = a.G == 1 || !a.post ? -1 : w && lanes <= 64 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  const size_t row = size_t(s.threads_row / 64) * 12 + (s.group_lanes == 0 ? size_t(w ? C / kPiece : C) + a.G : 0);
  s.lds = s.rows_block * row * sizeof(double);
  if (bwd) s.lds = std::max(s.lds, size_t(s.rows_block) * s.threads_row * kPiece * sizeof(float));
  return s;
}

// Calls go(threads of a row, pieces, wide) with compile-time values.
template <typename Go>
hipError_t by_shape(const ResidualArgs& a, const Shape& s, Go go) {
  using std::integral_constant;
  auto by_wide = [&](auto tpr, auto nc) { return wide(a) ? go(tpr, nc, std::true_type{}) : go(tpr, nc, std::false_type{}); };
  const integral_constant<int, 2> two{};
  if (s.nc == 1) return by_wide(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  switch (s.threads_row) {
    case 64: return by_wide(integral_constant<int, 64>{}, two);
    case 128: return by_wide(integral_constant<int, 128>{}, two);
    case 256: return by_wide(integral_constant<int, 256>{}, two);
    default: return by_wide(integral_constant<int, 512>{}, two);
  }
}

template <typename Kernel>
hipError_t allow_lds(Kernel kernel, size_t lds) {
  if (lds <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
}

}  // namespace

hipError_t launch_residual_fwd(const ResidualArgs& a, hipStream_t st) {
  const Shape s = shape_of(a, false);
  return by_shape(a, s, [&](auto tpr, auto nc, auto w) {
    auto* const kernel = residual_fwd_kernel<tpr(), nc(), w()>;
    const hipError_t e = allow_lds(kernel, s.lds);
    if (e != hipSuccess) return e;
    kernel<<<dim3(unsigned(s.blocks)), dim3(threads_of<tpr()>()), s.lds, st>>>(a, s.rows_each, s.group_lanes);
    return hipGetLastError();
  });
}

size_t residual_bwd_workspace_bytes(const ResidualArgs& a) {
  return size_t(shape_of(a, true).blocks) * 3 * size_t(a.G) * a.d * sizeof(float);
}

hipError_t launch_residual_bwd(const ResidualArgs& a, hipStream_t st) {
  const Shape s = shape_of(a, true);
  const bool params = a.dalpha || a.dpost_weight || a.dpre_weight;
  if (s.blocks > 0) {
    const hipError_t e = by_shape(a, s, [&](auto tpr, auto nc, auto w) {
      auto* const kernel = residual_bwd_kernel<tpr(), nc(), w()>;
      const hipError_t e = allow_lds(kernel, s.lds);
      if (e != hipSuccess) return e;
      kernel<<<dim3(unsigned(s.blocks)), dim3(threads_of<tpr()>()), s.lds, st>>>(a, s.rows_each, s.group_lanes, params ? a.workspace : nullptr);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (!params) return hipSuccess;
  const int64_t C = int64_t(a.G) * a.d;
  return launch_sum_parts({a.workspace, s.blocks, 3 * C, 3 * C, {a.dalpha, a.dpost_weight, a.dpre_weight}, {C, 2 * C}}, st);
}

}  // namespace falcon
