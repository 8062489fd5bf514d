// Selective state space scan (gfx950): prompts, single tokens and gradients.
//
//   delta_t = softplus(dt_t + bias),  S_t = exp(delta_t A) S_{t-1} + delta_t x_t B_t,
//   read_t = <C_t, S_t> + D x_t,      y_t = read_t silu(z_t)
//
// and backwards, with q_t = dy_t silu(z_t) and G_t the gradient of S_t:
//
//   G_t = q_t C_t + exp(delta_{t+1} A) G_{t+1},   m_t = G_t exp(delta_t A) S_{t-1},
//   dC_t = sum_c q_t S_t,   dB_t = sum_c G_t delta_t x_t,   u_t = <G_t, B_t>,
//   ddelta_t = <A, m_t> + u_t x_t,   dA = sum_t m_t delta_t,   dx_t = u_t delta_t + D q_t.
//

#include <algorithm>
#include <type_traits>

#include "falcon_block_device.h"
#include "falcon_launch.h"

namespace falcon {

namespace {

constexpr int kLanes = 64;

struct ScanDims {
  int B, T, D, G, Dg, tiles;   // Dg channels a group, in `tiles` waves of 64
  int64_t x_row, dt_row, z_row, b_row, c_row;
};

template <typename IO>
struct ScanIn {
  const IO* x;
  const IO* dt;
  const float* A;
  const IO* Bm;
  const IO* Cm;
  const float* Dskip;
  const float* dt_bias;
  const IO* z;
  const float* S0;
  const int32_t* lengths;
};

// The wave's sequence, group and this lane's channel (clamped where the group
// ends inside the wave; such lanes compute on a valid channel and store nothing).
struct Place {
  int b, g, c;
  bool on;
};
__device__ __forceinline__ Place place_of(const ScanDims& d, int64_t wave) {
  const int64_t per = int64_t(d.G) * d.tiles;
  Place p;
  p.b = int(wave / per);
  const int r = int(wave % per);
  p.g = r / d.tiles;
  const int c = (r % d.tiles) * kLanes + int(threadIdx.x % kLanes);
  p.on = c < d.Dg;
  p.c = p.g * d.Dg + min(c, d.Dg - 1);
  return p;
}

template <int N>
__device__ __forceinline__ void load_state(const float* p, float (&s)[N]) {
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    const float4 v = reinterpret_cast<const float4*>(p)[k];
    s[4 * k] = v.x; s[4 * k + 1] = v.y; s[4 * k + 2] = v.z; s[4 * k + 3] = v.w;
  }
}
template <int N>
__device__ __forceinline__ void store_state(float* p, const float (&s)[N]) {
#pragma unroll
  for (int k = 0; k < N / 4; ++k)
    reinterpret_cast<float4*>(p)[k] = make_float4(s[4 * k], s[4 * k + 1], s[4 * k + 2], s[4 * k + 3]);
}

template <bool SOFTPLUS>
__device__ __forceinline__ float step_of(float v) { return SOFTPLUS ? softplus_f32(v) : v; }

// ---- prompts ----------------------------------------------------------------------
// A lane owns four states of one channel: N / 4 lanes a channel, 256 / N channels
// a wave.  A workgroup's kFwdWaves waves take sixteen tokens in turn.  What does
// not need the state (step sizes, gates, decays, B and C) a wave works out ahead;
// then it takes the state from the wave before, runs its sixteen steps, hands the
// state on and makes the reads, while the next wave is at its steps.  So a
// channel's tokens keep several waves busy with no operation done twice.
// Bound by the vector units: an exp2 (8 cycles a wave) and its argument, the
// product u B and a multiply-add for the state and one for the read (4 each).
// What a token and a channel need once is worked out by one lane of a quad for
// every fourth token and handed round by quad permutes.
constexpr int kTok = 16;

template <int N>
struct Lanes {
  static constexpr int kPer = N / 4;                    // lanes a channel
  static constexpr int kChannels = 64 / kPer;           // channels a wave
  static constexpr int kQuad = kPer < 4 ? kPer : 4;     // lanes that share the tokens' work
  static constexpr int kRegs = kTok / kQuad;            // tokens a lane works out
};

// Value of lane J of this lane's group of Q (2 or 4) lanes.
template <int Q, int J>
__device__ __forceinline__ float from_lane(float v) {
  constexpr int kCtrl = Q == 4 ? J * 0x55 : (J | (J << 2) | ((2 + J) << 4) | ((2 + J) << 6));
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, false));
}

// Sixteen (or fewer) rows of one tensor as a buffer: an access behind its rows
// reads zero or is dropped, so no address is clamped, and a lane's offsets are
// the same 32-bit numbers at every step.  Rows have at most 2^24 elements.
template <typename E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const E* p, int64_t row, int64_t token, int rows) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(p + token * row), 0, max(rows, 0) * int(row) * int(sizeof(E)), 0x00020000);
}
// Loads leave the bits as they are, so that nothing waits for them before their
// use; widen() then gives the value.
template <typename E> struct bits_of { using type = uint32_t; };
template <> struct bits_of<bf16_t> { using type = uint16_t; };
template <typename E>
using bits_t = typename bits_of<E>::type;
template <typename E>
__device__ __forceinline__ bits_t<E> load_bits(__amdgpu_buffer_rsrc_t r, int offset) {
  if constexpr (sizeof(E) == 2) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, offset, 0, 0);
  } else {
    return __builtin_amdgcn_raw_buffer_load_b32(r, offset, 0, 0);
  }
}
__device__ __forceinline__ float widen(uint16_t bits) { return bf16_to_f32(bits); }
__device__ __forceinline__ float widen(uint32_t bits) { return __uint_as_float(bits); }
// v, or zero: by its bits, so that the compiler makes no branch of it.
__device__ __forceinline__ float kept(float v, bool keep) { return __uint_as_float(__float_as_uint(v) & (keep ? 0xffffffffu : 0u)); }
template <typename E>
__device__ __forceinline__ void store_one(__amdgpu_buffer_rsrc_t r, int offset, float v) {
  if constexpr (sizeof(E) == 2) {
    __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v), r, offset, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, offset, 0, 0);
  }
}
// Four consecutive elements, bf16 ones as two words: one access where `wide`,
// else one each (and a wait, to pair them: rows of such widths are rare).
template <typename E>
constexpr int kFourWords = sizeof(E) == 2 ? 2 : 4;
template <typename E>
__device__ __forceinline__ void load_four_bits(__amdgpu_buffer_rsrc_t r, int offset, bool wide, uint32_t (&v)[kFourWords<E>]) {
  if constexpr (sizeof(E) == 2) {
    if (wide) {
      const auto w = __builtin_amdgcn_raw_buffer_load_b64(r, offset, 0, 0);
      v[0] = w[0];
      v[1] = w[1];
    } else {
      v[0] = load_bits<E>(r, offset) | (uint32_t(load_bits<E>(r, offset + 2)) << 16);
      v[1] = load_bits<E>(r, offset + 4) | (uint32_t(load_bits<E>(r, offset + 6)) << 16);
    }
  } else if (wide) {
    const auto w = __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load_bits<E>(r, offset + 4 * i);
  }
}
template <typename E>
__device__ __forceinline__ float4 widen_four(const uint32_t (&v)[kFourWords<E>]) {
  if constexpr (sizeof(E) == 2) {
    return make_float4(__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u), __uint_as_float(v[1] << 16),
                       __uint_as_float(v[1] & 0xffff0000u));
  } else {
    return make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
  }
}
constexpr int kNowhere = 0x7ffffff0;   // an offset behind every buffer

// A lane's byte offsets into sixteen rows: its tokens' rows of the tensors a
// channel wide, and its fours of B and C.
template <typename IO, int N>
struct Offsets {
  using L = Lanes<N>;
  static constexpr int kUnits = (kTok * L::kPer + 63) / 64;   // fours of B (and C) a lane loads
  int x, dt, z, b[kUnits], c[kUnits];
  __device__ __forceinline__ Offsets(const ScanDims& d, int g, int c_) {
    const int lane = threadIdx.x % 64, j = lane % L::kQuad;
    x = (j * int(d.x_row) + c_) * int(sizeof(IO));
    dt = (j * int(d.dt_row) + c_) * int(sizeof(IO));
    z = (j * int(d.z_row) + c_) * int(sizeof(IO));
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int unit = u * 64 + lane, token = unit / L::kPer, at = g * N + 4 * (unit % L::kPer);
      b[u] = unit < kTok * L::kPer ? (token * int(d.b_row) + at) * int(sizeof(IO)) : kNowhere;
      c[u] = unit < kTok * L::kPer ? (token * int(d.c_row) + at) * int(sizeof(IO)) : kNowhere;
    }
  }
};

// The bits of a wave's sixteen tokens' inputs, loaded a turn ahead; zero behind
// the sequence's end.
template <typename IO, int N>
struct Tokens {
  bits_t<IO> x[Lanes<N>::kRegs], dt[Lanes<N>::kRegs], z[Lanes<N>::kRegs];
  uint32_t b[Offsets<IO, N>::kUnits][kFourWords<IO>], c[Offsets<IO, N>::kUnits][kFourWords<IO>];
};
template <typename IO, int N>
__device__ __forceinline__ void load_tokens(const ScanDims& d, const ScanIn<IO>& in, int64_t b, int t0, int len, bool wide,
                                            const Offsets<IO, N>& o, Tokens<IO, N>& k) {
  using L = Lanes<N>;
  const int64_t token = b * d.T + t0;
  const int rows = min(len - t0, kTok);
  const auto rx = rows_at(in.x, d.x_row, token, rows), rdt = rows_at(in.dt, d.dt_row, token, rows);
#pragma unroll
  for (int i = 0; i < L::kRegs; ++i) {
    k.x[i] = load_bits<IO>(rx, o.x + i * L::kQuad * int(d.x_row) * int(sizeof(IO)));
    k.dt[i] = load_bits<IO>(rdt, o.dt + i * L::kQuad * int(d.dt_row) * int(sizeof(IO)));
  }
  if (in.z) {
    const auto rz = rows_at(in.z, d.z_row, token, rows);
#pragma unroll
    for (int i = 0; i < L::kRegs; ++i) k.z[i] = load_bits<IO>(rz, o.z + i * L::kQuad * int(d.z_row) * int(sizeof(IO)));
  }
  const auto rb = rows_at(in.Bm, d.b_row, token, rows), rc = rows_at(in.Cm, d.c_row, token, rows);
#pragma unroll
  for (int u = 0; u < Offsets<IO, N>::kUnits; ++u) {
    load_four_bits<IO>(rb, o.b[u], wide, k.b[u]);
    load_four_bits<IO>(rc, o.c[u], wide, k.c[u]);
  }
}

// B and C of the wave's tokens to its part of LDS, [kTok][N] each.
template <typename IO, int N>
__device__ __forceinline__ void stage_shared(const Tokens<IO, N>& k, float* Bs, float* Cs) {
  const int lane = threadIdx.x % 64;
#pragma unroll
  for (int u = 0; u < Offsets<IO, N>::kUnits; ++u) {
    const int unit = u * 64 + lane;
    if (kTok * N / 4 % 64 == 0 || unit < kTok * N / 4) {
      *reinterpret_cast<float4*>(Bs + 4 * unit) = widen_four<IO>(k.b[u]);
      *reinterpret_cast<float4*>(Cs + 4 * unit) = widen_four<IO>(k.c[u]);
    }
  }
}

__device__ __forceinline__ void four(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}

// A lane's fours of rows 4 k .. 4 k + 3 of a [kTok][N] array.
template <int N>
__device__ __forceinline__ void four_rows(const float* p, int k, float (&v)[4][4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) four(p + (4 * k + r) * N, v[r]);
}

// f(t, row) for t = 0 .. 15 in order, `row` this lane's four of row t of the
// [kTok][N] array p; the rows come four at a time, four ahead, the first of
// them already in `first`.
template <int N, int K = 0, typename F>
__device__ __forceinline__ void each_row(const float* p, float (&first)[4][4], F f) {
  float ahead[4][4];
  if constexpr (K + 1 < kTok / 4) four_rows<N>(p, K + 1, ahead);
  __builtin_amdgcn_sched_barrier(0);
  f(std::integral_constant<int, 4 * K>{}, first[0]);
  f(std::integral_constant<int, 4 * K + 1>{}, first[1]);
  f(std::integral_constant<int, 4 * K + 2>{}, first[2]);
  f(std::integral_constant<int, 4 * K + 3>{}, first[3]);
  if constexpr (K + 1 < kTok / 4) each_row<N, K + 1>(p, ahead, f);
}

// f(t, j, i) for t = 0 .. 15 in order, with t = kQuad i + j known at compile time.
template <int Q, int I = 0, typename F>
__device__ __forceinline__ void each_token(F f) {
  if constexpr (I < kTok) {
    f(std::integral_constant<int, I>{}, std::integral_constant<int, I % Q>{}, std::integral_constant<int, I / Q>{});
    if constexpr (I % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    each_token<Q, I + 1>(f);
  }
}

// Workgroups b, b + 8, b + 16, ... run on one XCD: neighbours in channels, which
// share cache lines of every row, follow one another there.
__device__ __forceinline__ int64_t by_xcd(int64_t block, int64_t blocks) {
  const int64_t each = blocks / 8, more = blocks % 8, x = block % 8;
  return x * each + min(x, more) + block / 8;
}

constexpr int kFwdWaves = 4;

// A turn of a wave: token block `turn` may start once *at has reached it.  False
// if that did not happen within `limit` polls (then the caller poisons its
// results; see falcon_set_wait_limit).
__device__ __forceinline__ bool wait_turn(const int* at, int turn, int limit) {
  for (int polls = 0; __hip_atomic_load(at, __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP) < turn; ++polls) {
    if (polls >= limit) return false;
  }
  return true;
}

template <typename IO, int N, bool SOFTPLUS>
__global__ __launch_bounds__(64 * kFwdWaves, N == 16 || N == 32 ? 3 : 2) void scan_fwd_kernel(
    ScanDims d, ScanIn<IO> in, bool wide, IO* __restrict__ y, float* __restrict__ S_T, int limit) {
  using L = Lanes<N>;
  __shared__ float shared[kFwdWaves][2][kTok * N];      // B, C of a wave's tokens
  __shared__ float4 passed[64];                         // the state on its way to the next wave
  __shared__ int turns;                                 // token blocks whose steps are done
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int64_t id = by_xcd(blockIdx.x, gridDim.x);
  const int tile = int(id % d.tiles), g = int(id / d.tiles % d.G);
  const int64_t b = id / (int64_t(d.tiles) * d.G);
  const int in_group = tile * L::kChannels + lane / L::kPer;
  const bool on = in_group < d.Dg;
  const int c = g * d.Dg + min(in_group, d.Dg - 1), s = lane % L::kPer, j = lane % L::kQuad;
  const int len = tokens_of(in.lengths, int(b), d.T);
  const int64_t at = (b * d.D + c) * N + 4 * s;
  float h[4] = {0.0f, 0.0f, 0.0f, 0.0f}, A2[4];
  if (in.S0 && wave == 0) four(in.S0 + at, h);
  four(in.A + int64_t(c) * N + 4 * s, A2);
#pragma unroll
  for (int n = 0; n < 4; ++n) A2[n] *= kLog2e;
  const float skip = in.Dskip ? in.Dskip[c] : 0.0f, bias = in.dt_bias ? in.dt_bias[c] : 0.0f;
  float* Bs = shared[wave][0];
  float* Cs = shared[wave][1];
  const Offsets<IO, N> offsets(d, g, c);
  const int y_at = on && s < L::kQuad ? (j * d.D + c) * int(sizeof(IO)) : kNowhere;

  Tokens<IO, N> next;
  if (wave * kTok < len) load_tokens<IO, N>(d, in, b, wave * kTok, len, wide, offsets, next);
  if (threadIdx.x == 0) turns = 0;
  __syncthreads();
  for (int turn = wave; turn * kTok < len; turn += kFwdWaves) {
    const int t0 = turn * kTok;
    float delta[L::kRegs], x[L::kRegs], gate[L::kRegs], u[L::kRegs];
    stage_shared<IO, N>(next, Bs, Cs);
#pragma unroll
    for (int i = 0; i < L::kRegs; ++i) {
      const bool live = t0 + L::kQuad * i + j < len;
      x[i] = widen(next.x[i]);
      delta[i] = kept(step_of<SOFTPLUS>(widen(next.dt[i]) + bias), live);
      u[i] = delta[i] * x[i];
      gate[i] = in.z ? act_f32<kActSilu>(widen(next.z[i])) : 1.0f;
    }
    if (t0 + kFwdWaves * kTok < len) load_tokens<IO, N>(d, in, b, t0 + kFwdWaves * kTok, len, wide, offsets, next);
    // the decays
    float v[kTok][4];
    each_token<L::kQuad>([&](auto t, auto jj, auto i) {
      const float dt = from_lane<L::kQuad, jj()>(delta[i()]);
#pragma unroll
      for (int n = 0; n < 4; ++n) v[t()][n] = __builtin_amdgcn_exp2f(dt * A2[n]);
    });
    __builtin_amdgcn_wave_barrier();
    float rows[4][4];
    four_rows<N>(Bs + 4 * s, 0, rows);
    // the steps, each decay giving way to its state
    if (turn > 0) {
      const bool came = wait_turn(&turns, turn, limit);
      four(reinterpret_cast<const float*>(&passed[lane]), h);
      if (!came) h[0] = h[1] = h[2] = h[3] = __builtin_nanf("");
    }
    __builtin_amdgcn_s_setprio(2);
    each_row<N>(Bs + 4 * s, rows, [&](auto t, const float (&bt)[4]) {
      const float ut = from_lane<L::kQuad, t() % L::kQuad>(u[t() / L::kQuad]);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        h[n] = __builtin_fmaf(v[t()][n], h[n], ut * bt[n]);
        v[t()][n] = h[n];
      }
    });
    passed[lane] = make_float4(h[0], h[1], h[2], h[3]);
    if (lane == 0) __hip_atomic_store(&turns, turn + 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_WORKGROUP);
    __builtin_amdgcn_s_setprio(0);
    // the reads
    float read[L::kRegs];
    four_rows<N>(Cs + 4 * s, 0, rows);
    each_row<N>(Cs + 4 * s, rows, [&](auto t, const float (&ct)[4]) {
      constexpr int jj = t() % L::kQuad;
      float r = ct[0] * v[t()][0];
#pragma unroll
      for (int n = 1; n < 4; ++n) r = __builtin_fmaf(ct[n], v[t()][n], r);
      r = lanes_sum<L::kPer>(r);
      read[t() / L::kQuad] = jj == 0 || j == jj ? r : read[t() / L::kQuad];
    });
    const auto ry = rows_at(y, d.D, b * d.T + t0, min(len - t0, kTok));
#pragma unroll
    for (int i = 0; i < L::kRegs; ++i)
      store_one<IO>(ry, y_at == kNowhere ? kNowhere : y_at + i * L::kQuad * d.D * int(sizeof(IO)),
                    __builtin_fmaf(skip, x[i], read[i]) * gate[i]);
    __builtin_amdgcn_wave_barrier();
  }
  // the wave that ran the last tokens (wave 0 where there are none) has the end
  const int last = len > 0 ? (len - 1) / kTok % kFwdWaves : 0;
  if (S_T && wave == last && on) *reinterpret_cast<float4*>(S_T + at) = make_float4(h[0], h[1], h[2], h[3]);
}

// Every state, one token after another: [B, T, D, N], for the gradients.
template <typename IO, int N, bool SOFTPLUS>
__global__ __launch_bounds__(64) void scan_states_kernel(ScanDims d, ScanIn<IO> in, float* states) {
  const Place p = place_of(d, blockIdx.x);
  const int len = tokens_of(in.lengths, p.b, d.T);
  const int64_t at = (int64_t(p.b) * d.D + p.c) * N;
  float S[N], A2[N];
  load_state<N>(in.A + int64_t(p.c) * N, A2);
#pragma unroll
  for (int n = 0; n < N; ++n) A2[n] *= kLog2e;
  if (in.S0) {
    load_state<N>(in.S0 + at, S);
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) S[n] = 0.0f;
  }
  const float bias = in.dt_bias ? in.dt_bias[p.c] : 0.0f;
  for (int t = 0; t < len; ++t) {
    const int64_t token = int64_t(p.b) * d.T + t;
    const float x = io<IO>::load(in.x, token * d.x_row + p.c);
    const float delta = step_of<SOFTPLUS>(io<IO>::load(in.dt, token * d.dt_row + p.c) + bias);
    const IO* pb = in.Bm + token * d.b_row + p.g * N;
    const float u = delta * x;
#pragma unroll
    for (int n = 0; n < N; ++n) S[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A2[n]), S[n], u * io<IO>::load(pb, n));
    if (p.on) store_state<N>(states + (token * d.D + p.c) * N, S);
  }
}

// ---- one token --------------------------------------------------------------------
template <typename IO, int N, bool SOFTPLUS>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanDims d, ScanIn<IO> in, float* S_io, const uint8_t* is_first, IO* y) {
  constexpr int kPer = N / 4;   // lanes of four states each share a channel
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t want = id / kPer;
  const int q = int(id % kPer);
  const int64_t cell = min(want, int64_t(d.B) * d.D - 1);
  const int64_t b = cell / d.D;
  const int c = int(cell - b * d.D), g = c / d.Dg;
  float S[4], A2[4];
  load_state<4>(S_io + cell * N + 4 * q, S);
  load_state<4>(in.A + int64_t(c) * N + 4 * q, A2);
  if (is_first && is_first[b]) {
#pragma unroll
    for (int n = 0; n < 4; ++n) S[n] = 0.0f;
  }
  const float x = io<IO>::load(in.x, b * d.x_row + c);
  const float delta = step_of<SOFTPLUS>(io<IO>::load(in.dt, b * d.dt_row + c) + (in.dt_bias ? in.dt_bias[c] : 0.0f));
  const IO* pb = in.Bm + b * d.b_row + g * N + 4 * q;
  const IO* pc = in.Cm + b * d.c_row + g * N + 4 * q;
  float read = 0.0f;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    S[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * (A2[n] * kLog2e)), S[n], delta * x * io<IO>::load(pb, n));
    read = __builtin_fmaf(io<IO>::load(pc, n), S[n], read);
  }
  read = lanes_sum<kPer>(read);
  if (want < int64_t(d.B) * d.D) {
    store_state<4>(S_io + cell * N + 4 * q, S);
    if (q == 0) {
      read = __builtin_fmaf(in.Dskip ? in.Dskip[c] : 0.0f, x, read);
      if (in.z) read *= act_f32<kActSilu>(io<IO>::load(in.z, b * d.z_row + c));
      io<IO>::store(y, b * d.D + c, read);
    }
  }
}

// ---- gradients ----------------------------------------------------------------------
// One wave a sequence and 64 channels, from the last token to the first, with
// every state from scan_fwd_kernel.  What sums over channels (dB, dC) leaves as
// one row a wave, what sums over sequences (dA, dD, ddt_bias) as one a sequence.
template <typename IO, typename DY, int N, bool SOFTPLUS>
__global__ __launch_bounds__(64) void scan_bwd_kernel(ScanDims d, ScanIn<IO> in, const DY* dy, const float* dS_T, const float* states,
                                                      float* dx, float* ddt, float* dz, float* dS0, float* bc_parts, float* par_parts) {
  const Place p = place_of(d, blockIdx.x);
  const int len = tokens_of(in.lengths, p.b, d.T);
  const int tile = int(blockIdx.x % d.tiles);
  const int64_t at = (int64_t(p.b) * d.D + p.c) * N;
  const int lane = threadIdx.x;
  float A[N], G[N], dA[N];
  load_state<N>(in.A + int64_t(p.c) * N, A);
#pragma unroll
  for (int n = 0; n < N; ++n) G[n] = dA[n] = 0.0f;
  if (dS_T) load_state<N>(dS_T + at, G);
  const float skip = in.Dskip ? in.Dskip[p.c] : 0.0f, bias = in.dt_bias ? in.dt_bias[p.c] : 0.0f;
  float dskip = 0.0f, dbias = 0.0f;
  const float live = p.on ? 1.0f : 0.0f;
  for (int t = d.T - 1; t >= 0; --t) {
    const int64_t token = int64_t(p.b) * d.T + t;
    float* part = bc_parts + ((token * d.G + p.g) * d.tiles + tile) * 2 * N;
    if (t >= len) {
      if (p.on) {
        dx[token * d.D + p.c] = 0.0f;
        ddt[token * d.D + p.c] = 0.0f;
        if (dz) dz[token * d.D + p.c] = 0.0f;
      }
      if (lane < 2 * N) part[lane] = 0.0f;
      if (2 * N > kLanes && lane + kLanes < 2 * N) part[lane + kLanes] = 0.0f;
      continue;
    }
    const float x = io<IO>::load(in.x, token * d.x_row + p.c);
    const float raw = io<IO>::load(in.dt, token * d.dt_row + p.c) + bias;
    const float delta = step_of<SOFTPLUS>(raw);
    const float up = io<DY>::load(dy, token * d.D + p.c);
    const IO* pb = in.Bm + token * d.b_row + p.g * N;
    const IO* pc = in.Cm + token * d.c_row + p.g * N;
    const float z = in.z ? io<IO>::load(in.z, token * d.z_row + p.c) : 0.0f;
    const float q = in.z ? up * act_f32<kActSilu>(z) : up;
    float S[N], P[N];
    load_state<N>(states + (token * d.D + p.c) * N, S);
    if (t > 0) {
      load_state<N>(states + ((token - 1) * d.D + p.c) * N, P);
    } else if (in.S0) {
      load_state<N>(in.S0 + at, P);
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) P[n] = 0.0f;
    }
    float read = skip * x, u = 0.0f, turn = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float bn = io<IO>::load(pb, n), cn = io<IO>::load(pc, n);
      read = __builtin_fmaf(cn, S[n], read);
      G[n] = __builtin_fmaf(q, cn, G[n]);
      u = __builtin_fmaf(G[n], bn, u);
      const float db = lanes_sum<kLanes>(live * G[n] * delta * x), dc = lanes_sum<kLanes>(live * q * S[n]);
      if (lane == 0) {
        part[n] = db;
        part[N + n] = dc;
      }
      G[n] *= __builtin_amdgcn_exp2f(delta * (A[n] * kLog2e));
      const float m = G[n] * P[n];
      turn = __builtin_fmaf(A[n], m, turn);
      dA[n] = __builtin_fmaf(m, delta, dA[n]);
    }
    const float dd = (turn + u * x) * (SOFTPLUS ? sigmoid_f32(raw) : 1.0f);
    dskip = __builtin_fmaf(q, x, dskip);
    dbias += dd;
    if (p.on) {
      dx[token * d.D + p.c] = __builtin_fmaf(u, delta, skip * q);
      ddt[token * d.D + p.c] = dd;
      if (dz) dz[token * d.D + p.c] = up * read * act_slope_f32<kActSilu>(z);
    }
  }
  if (p.on) {
    if (dS0) store_state<N>(dS0 + at, G);
    // a sequence's row: [D, N] of dA, [D] of dD, [D] of ddt_bias
    float* row = par_parts + int64_t(p.b) * d.D * (N + 2);
    store_state<N>(row + int64_t(p.c) * N, dA);
    row[int64_t(d.D) * N + p.c] = dskip;
    row[int64_t(d.D) * (N + 1) + p.c] = dbias;
  }
}

// dB, dC of every token and group from its waves' rows.
__global__ __launch_bounds__(256) void scan_bc_kernel(const float* __restrict__ parts, int tiles, int N, int64_t n, float* __restrict__ dB,
                                                      float* __restrict__ dC) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
    const int64_t tg = i / (2 * N);
    const int k = int(i % (2 * N));
    float s = 0.0f;
    for (int j = 0; j < tiles; ++j) s += parts[(tg * tiles + j) * 2 * N + k];
    if (k < N) {
      dB[tg * N + k] = s;
    } else {
      dC[tg * N + k - N] = s;
    }
  }
}

// dA, dD and ddt_bias from the sequences' rows.
__global__ __launch_bounds__(256) void scan_params_kernel(const float* __restrict__ parts, int rows, int D, int N, float* __restrict__ dA,
                                                          float* __restrict__ dD, float* __restrict__ ddt_bias) {
  const int64_t n = int64_t(D) * (N + 2);
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
    double s = 0.0;
    for (int r = 0; r < rows; ++r) s += parts[r * n + i];
    if (i < int64_t(D) * N) {
      dA[i] = float(s);
    } else if (i < int64_t(D) * (N + 1)) {
      if (dD) dD[i - int64_t(D) * N] = float(s);
    } else if (ddt_bias) {
      ddt_bias[i - int64_t(D) * (N + 1)] = float(s);
    }
  }
}

ScanDims dims_of(const ScanArgs& a) {
  ScanDims d{};
  d.B = a.B; d.T = a.T; d.D = a.D; d.G = a.G;
  d.Dg = a.D / a.G;
  d.tiles = (d.Dg + kLanes - 1) / kLanes;
  d.x_row = a.x_row; d.dt_row = a.dt_row; d.z_row = a.z_row; d.b_row = a.b_row; d.c_row = a.c_row;
  return d;
}

template <typename IO>
ScanIn<IO> inputs_of(const ScanArgs& a) {
  return {static_cast<const IO*>(a.x), static_cast<const IO*>(a.dt), a.A, static_cast<const IO*>(a.Bm), static_cast<const IO*>(a.Cm),
          a.Dskip, a.dt_bias, static_cast<const IO*>(a.z), a.S0, a.lengths};
}

constexpr int64_t kMaxGrid = (int64_t(1) << 24) - 1;

// Fours of B and C lie on multiples of a four's size.
bool fours_wide(const ScanArgs& a) { return a.b_row % 4 == 0 && a.c_row % 4 == 0; }

template <typename IO, int N, bool SP>
hipError_t fwd_typed(const ScanArgs& a, hipStream_t st) {
  ScanDims d = dims_of(a);
  d.tiles = (d.Dg + Lanes<N>::kChannels - 1) / Lanes<N>::kChannels;
  const int64_t blocks = int64_t(a.B) * a.G * d.tiles;
  if (blocks > kMaxGrid) return hipErrorInvalidValue;
  scan_fwd_kernel<IO, N, SP><<<dim3(unsigned(blocks)), dim3(64 * kFwdWaves), 0, st>>>(d, inputs_of<IO>(a), fours_wide(a),
                                                                                     static_cast<IO*>(a.y), a.S_T, a.spin_limit);
  return hipGetLastError();
}

template <typename IO, int N, bool SP>
hipError_t step_typed(const ScanArgs& a, hipStream_t st) {
  const int64_t blocks = (int64_t(a.B) * a.D * (N / 4) + 255) / 256;
  if (blocks > kMaxGrid) return hipErrorInvalidValue;
  scan_step_kernel<IO, N, SP><<<dim3(unsigned(blocks)), dim3(256), 0, st>>>(dims_of(a), inputs_of<IO>(a), a.S, a.is_first,
                                                                           static_cast<IO*>(a.y));
  return hipGetLastError();
}

int64_t states_floats(const ScanArgs& a) { return int64_t(a.B) * a.T * a.D * a.N; }
int64_t bc_floats(const ScanArgs& a) { return int64_t(a.B) * a.T * a.G * dims_of(a).tiles * 2 * a.N; }
int64_t params_floats(const ScanArgs& a) { return int64_t(a.B) * a.D * (a.N + 2); }

template <typename IO, typename DY, int N, bool SP>
hipError_t bwd_typed(const ScanArgs& a, hipStream_t st) {
  const ScanDims d = dims_of(a);
  const int64_t waves = int64_t(a.B) * a.G * d.tiles;
  float* states = a.workspace;
  float* bc = states + states_floats(a);
  float* par = bc + bc_floats(a);
  hipError_t e = hipSuccess;
  if (waves > kMaxGrid) return hipErrorInvalidValue;
  if (waves > 0) {
    scan_states_kernel<IO, N, SP><<<dim3(unsigned(waves)), dim3(64), 0, st>>>(d, inputs_of<IO>(a), states);
    scan_bwd_kernel<IO, DY, N, SP><<<dim3(unsigned(waves)), dim3(64), 0, st>>>(d, inputs_of<IO>(a), static_cast<const DY*>(a.dy), a.dS_T,
                                                                              states, a.dx, a.ddt, a.dz, a.dS0, bc, par);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  const int64_t n = int64_t(a.B) * a.T * a.G * 2 * N;
  if (n > 0) {
    scan_bc_kernel<<<dim3(unsigned(std::min<int64_t>((n + 255) / 256, 1 << 16))), dim3(256), 0, st>>>(bc, d.tiles, N, n, a.dB, a.dC);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  scan_params_kernel<<<dim3(unsigned(std::min<int64_t>((int64_t(a.D) * (N + 2) + 255) / 256, 1 << 16))), dim3(256), 0, st>>>(
      par, a.B, a.D, N, a.dA, a.dD, a.ddt_bias);
  return hipGetLastError();
}

// Calls go(N, softplus) with compile-time values.
template <typename Go>
hipError_t by_size(const ScanArgs& a, Go go) {
  auto sp = [&](auto n) { return a.softplus ? go(n, std::true_type{}) : go(n, std::false_type{}); };
  switch (a.N) {
    case 8: return sp(std::integral_constant<int, 8>{});
    case 16: return sp(std::integral_constant<int, 16>{});
    case 32: return sp(std::integral_constant<int, 32>{});
    default: return sp(std::integral_constant<int, 64>{});
  }
}

}  // namespace

size_t scan_workspace_bytes(const ScanArgs&) { return 0; }

hipError_t launch_scan_fwd(const ScanArgs& a, hipStream_t st) {
  if (a.T == 0) return launch_state_copy(a.S0, a.S_T, int64_t(a.B) * a.D * a.N, st);
  return by_size(a, [&](auto n, auto sp) {
    return a.bf16 ? fwd_typed<bf16_t, n(), sp()>(a, st) : fwd_typed<float, n(), sp()>(a, st);
  });
}

hipError_t launch_scan_step(const ScanArgs& a, hipStream_t st) {
  return by_size(a, [&](auto n, auto sp) {
    return a.bf16 ? step_typed<bf16_t, n(), sp()>(a, st) : step_typed<float, n(), sp()>(a, st);
  });
}

size_t scan_bwd_workspace_bytes(const ScanArgs& a) {
  return size_t(states_floats(a) + bc_floats(a) + params_floats(a)) * sizeof(float);
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t st) {
  return by_size(a, [&](auto n, auto sp) {
    if (a.bf16) return a.dy_bf16 ? bwd_typed<bf16_t, bf16_t, n(), sp()>(a, st) : bwd_typed<bf16_t, float, n(), sp()>(a, st);
    return a.dy_bf16 ? bwd_typed<float, bf16_t, n(), sp()>(a, st) : bwd_typed<float, float, n(), sp()>(a, st);
  });
}

}  // namespace falcon
