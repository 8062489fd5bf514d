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

struct ScanDims {
  int B, T, D, G, Dg, tiles;   // Dg channels a group, in `tiles` waves of 256 / N
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

// ---- chunks --------------------------------------------------------------------------
// A span of tokens cut into chunks, worked on at once: scan_ends_kernel gives each
// chunk's map S -> exp(A sum delta) S + E (and, for the gradients, the map
// G -> exp(A sum delta) G + R from the chunk's end to its start, R = sum_t
// exp(A sum_{s <= t} delta_s) q_t C_t); scan_carry_kernel runs through the chunks
// and leaves, in their places, the state that enters each chunk and the gradient
// that enters it from behind.
struct Chunks {
  int tokens, count;      // tokens of a chunk (a multiple of kTok), chunks of a sequence
  float* sums;            // [B, count, D]     sum of delta
  float* E;               // [B, count, D, N]  E, then the state before the chunk
  float* R;               // [B, count, D, N]  R, then the gradient behind it (gradients only)
  // the maps up to each of the chunk's later sixteens (gradients only)
  int subs;               // tokens / kTok - 1
  float* sub_sums;        // [B, count, subs, D]
  float* sub_E;           // [B, count, subs, D, N]
};

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
// every fourth token and handed round by quad permutes.  8 x 2048 x 1536, N = 16:
// 112 us, the vector units busy 81 % of the time (of 127 us under the profiler); two
// scans a wave from zero and from the joined states (no waiting, every product twice)
// took 176, and decays that the compiler had let sink below the wait 130.
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

template <int CTRL>
__device__ __forceinline__ float dpp_of(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// v[t] of every lane summed over a channel's lanes, for the group's Q tokens t: the
// lane of token j gets the sum of v[j].  Each step halves what a lane carries.
template <int N>
__device__ __forceinline__ float own_sum(const float (&v)[Lanes<N>::kQuad], int j) {
  const bool odd = j & 1, far = j & 2;
  float s = (odd ? v[1] : v[0]) + dpp_of<0xb1>(odd ? v[0] : v[1]);        // quad_perm [1, 0, 3, 2]
  if constexpr (Lanes<N>::kQuad == 4) {
    const float s2 = (odd ? v[3] : v[2]) + dpp_of<0xb1>(odd ? v[2] : v[3]);
    s = (far ? s2 : s) + dpp_of<0x4e>(far ? s : s2);                      // quad_perm [2, 3, 0, 1]
  }
  // the other quads' lanes of the same token: the mirror inside 8 lanes with the
  // quads' order put right again, or rotations of the row of 16
  if constexpr (Lanes<N>::kPer == 8) s += dpp_of<0x1b>(dpp_of<0x141>(s));  // row_half_mirror, quad_perm [3, 2, 1, 0]
  if constexpr (Lanes<N>::kPer == 16) {
    s = dpp_plus<0x124>(s);                                               // row_ror 4
    s = dpp_plus<0x128>(s);                                               // row_ror 8
  }
  return s;
}

// Some rows of one tensor as a buffer: an access behind them reads zero or is
// dropped, so no address is clamped, and a lane's offsets are the same 32-bit
// numbers at every step.  The rows together have less than 2^30 bytes (sixteen of
// at most 2^22 elements, or a chunk's few rows of states).
template <typename E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const E* p, int64_t row, int64_t token, int rows) {
  const int bytes = __builtin_amdgcn_readfirstlane(max(rows, 0)) * int(row) * int(sizeof(E));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(p + token * row), 0, bytes, 0x00020000);
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
// An offset behind every buffer, also with 2^30 added (offsets are unsigned).
constexpr int kNowhere = 0x7ffffff0;

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

// B and C of the wave's tokens to its part of LDS, [kTok][N] each (and zeros up to
// a whole wave's fours).
template <int N>
constexpr int kShared = kTok * N < 256 ? 256 : kTok * N;
template <typename IO, int N>
__device__ __forceinline__ void stage_shared(const Tokens<IO, N>& k, float* Bs, float* Cs) {
  const int lane = threadIdx.x % 64;
#pragma unroll
  for (int u = 0; u < Offsets<IO, N>::kUnits; ++u) {
    const int unit = u * 64 + lane;
    *reinterpret_cast<float4*>(Bs + 4 * unit) = widen_four<IO>(k.b[u]);
    *reinterpret_cast<float4*>(Cs + 4 * unit) = widen_four<IO>(k.c[u]);
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

constexpr int kFwdWaves = 4;

// Where a lane stands in the channels of a wave, tile `tile` of group g.
template <int N>
struct Cell {
  int c, s, j;        // channel, four of its states, token of the quad
  bool on;
  __device__ __forceinline__ Cell(const ScanDims& d, int g, int tile, int lane = threadIdx.x % 64) {
    using L = Lanes<N>;
    const int in_group = tile * L::kChannels + lane / L::kPer;
    on = in_group < d.Dg;
    c = g * d.Dg + min(in_group, d.Dg - 1);
    s = lane % L::kPer;
    j = lane % L::kQuad;
  }
};
// The lane, worked out anew: what follows from it is not kept in registers till here.
__device__ __forceinline__ int lane_again() {
  int lane = threadIdx.x % 64;
  asm volatile("" : "+v"(lane));
  return lane;
}

// Turns.  *done counts the token blocks whose steps are through; a wave waits for it
// to reach its own block's number, up to `limit` polls (falcon_set_wait_limit).  A
// wave that gives up goes on, as the waves behind it do, with a state that is none,
// and marks the workgroup's tokens as lost: run_alone then makes them good.
__device__ __forceinline__ void wait_turn(const int* done, int turn, int limit, int* lost) {
  for (int polls = 0; __hip_atomic_load(done, __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP) < turn; ++polls) {
    if (polls >= limit) {
      *lost = 1;
      break;
    }
    __builtin_amdgcn_s_sleep(1);
  }
}

// Lost tokens, [first, len) of sequence b for a wave's channels: a wave by itself runs
// them one after another from the state `before` them, with the operations, orders and
// roundings of the turns, so the results are the same bit for bit.  Leaves the state.
template <typename IO, int N, bool SOFTPLUS>
__device__ __forceinline__ void run_alone(const ScanDims& d, const ScanIn<IO>& in, int64_t b, int g, int tile, int first, int len,
                                          const float* before, IO* y, float (&h)[4]) {
  using L = Lanes<N>;
  const Cell<N> cell(d, g, tile, lane_again());
  const int c = cell.c, s = cell.s;
  float A2[4];
  h[0] = h[1] = h[2] = h[3] = 0.0f;
  if (before) four(before + int64_t(c) * N + 4 * s, h);
  four(in.A + int64_t(c) * N + 4 * s, A2);
#pragma unroll
  for (int n = 0; n < 4; ++n) A2[n] *= kLog2e;
  const float skip = in.Dskip ? in.Dskip[c] : 0.0f, bias = in.dt_bias ? in.dt_bias[c] : 0.0f;
  for (int t = first; t < len; ++t) {
    const int64_t token = b * d.T + t;
    const float x = io<IO>::load(in.x, token * d.x_row + c);
    const float delta = step_of<SOFTPLUS>(io<IO>::load(in.dt, token * d.dt_row + c) + bias), u = delta * x;
    const float gate = in.z ? act_f32<kActSilu>(io<IO>::load(in.z, token * d.z_row + c)) : 1.0f;
    const IO* pb = in.Bm + token * d.b_row + int64_t(g) * N + 4 * s;
    const IO* pc = in.Cm + token * d.c_row + int64_t(g) * N + 4 * s;
    float read = 0.0f, group[L::kQuad];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A2[n]), h[n], u * io<IO>::load(pb, n));
      const float ct = io<IO>::load(pc, n);
      read = n == 0 ? ct * h[n] : __builtin_fmaf(ct, h[n], read);
    }
#pragma unroll
    for (int q = 0; q < L::kQuad; ++q) group[q] = read;
    read = own_sum<N>(group, cell.j);
    if (cell.on && s == 0) io<IO>::store(y, token * d.D + c, __builtin_fmaf(skip, x, read) * gate);
  }
}

// (Three waves a SIMD keep 1 to 6 registers in memory with N = 32, none with 16.)
template <typename IO, int N, bool SOFTPLUS>
__global__ __launch_bounds__(64 * kFwdWaves, N == 16 || N == 32 ? 3 : 2) void scan_fwd_kernel(
    ScanDims d, ScanIn<IO> in, bool wide, Chunks k, IO* __restrict__ y, float* __restrict__ S_T, int limit) {
  using L = Lanes<N>;
  __shared__ float shared[kFwdWaves][2][kShared<N>];      // B, C of a wave's tokens
  __shared__ float4 passed[64];                         // the state on its way to the next wave
  __shared__ int turns, lost;                           // token blocks whose steps are done; whether a wait gave up
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int64_t id = by_xcd(blockIdx.x, gridDim.x);
  const int tile = int(id % d.tiles), g = int(id / d.tiles % d.G);
  const int64_t bc = id / (int64_t(d.tiles) * d.G), b = bc / k.count;   // b count + chunk
  const Cell<N> here(d, g, tile);
  const int c = here.c, s = here.s, j = here.j;
  const int whole = __builtin_amdgcn_readfirstlane(tokens_of(in.lengths, int(b), d.T));
  const int first = int(bc % k.count) * k.tokens, len = min(first + k.tokens, whole);   // this chunk: [first, len)
  float h[4] = {0.0f, 0.0f, 0.0f, 0.0f}, A2[4];
  if (wave == 0) {
    if (k.E) {
      four(k.E + (bc * d.D + c) * N + 4 * s, h);
    } else if (in.S0) {
      four(in.S0 + (b * d.D + c) * N + 4 * s, h);
    }
  }
  four(in.A + int64_t(c) * N + 4 * s, A2);
#pragma unroll
  for (int n = 0; n < 4; ++n) A2[n] *= kLog2e;
  const float skip = in.Dskip ? in.Dskip[c] : 0.0f, bias = in.dt_bias ? in.dt_bias[c] : 0.0f;
  float* Bs = shared[wave][0];
  float* Cs = shared[wave][1];
  const Offsets<IO, N> offsets(d, g, c);
  const uint32_t y_at = here.on && s < L::kQuad ? (j * d.D + c) * int(sizeof(IO)) : kNowhere;

  Tokens<IO, N> next;
  if (first + wave * kTok < len) load_tokens<IO, N>(d, in, b, first + wave * kTok, len, wide, offsets, next);
  if (threadIdx.x == 0) turns = lost = 0;
  __syncthreads();
  for (int turn = wave; first + turn * kTok < len; turn += kFwdWaves) {
    const int t0 = first + turn * kTok;
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
    // (kept from sinking below the wait)
#pragma unroll
    for (int t = 0; t < kTok; ++t)
#pragma unroll
      for (int n = 0; n < 4; ++n) asm volatile("" : "+v"(v[t][n]));
    __builtin_amdgcn_wave_barrier();
    float rows[4][4];
    four_rows<N>(Bs + 4 * s, 0, rows);
    // the steps, each decay giving way to its state
    if (turn > 0) {
      wait_turn(&turns, turn, limit, &lost);
      four(reinterpret_cast<const float*>(&passed[lane]), h);
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
    float read[L::kRegs], group[L::kQuad];
    four_rows<N>(Cs + 4 * s, 0, rows);
    each_row<N>(Cs + 4 * s, rows, [&](auto t, const float (&ct)[4]) {
      constexpr int jj = t() % L::kQuad;
      group[jj] = ct[0] * v[t()][0];
#pragma unroll
      for (int n = 1; n < 4; ++n) group[jj] = __builtin_fmaf(ct[n], v[t()][n], group[jj]);
      if constexpr (jj == L::kQuad - 1) read[t() / L::kQuad] = own_sum<N>(group, j);
    });
    const auto ry = rows_at(y, d.D, b * d.T + t0, min(len - t0, kTok));
#pragma unroll
    for (int i = 0; i < L::kRegs; ++i)
      store_one<IO>(ry, y_at + uint32_t(i * L::kQuad) * d.D * sizeof(IO),
                    __builtin_fmaf(skip, x[i], read[i]) * gate[i]);
    __builtin_amdgcn_wave_barrier();
  }
  // the end is with the wave that ran the last tokens (wave 0 of the first chunk
  // where there are none)
  bool holds = whole > 0 ? len == whole && first < whole && wave == (whole - 1 - first) / kTok % kFwdWaves : first == 0 && wave == 0;
  __syncthreads();
  if (__builtin_amdgcn_readfirstlane(lost)) {
    // the first wave runs the chunk again, behind the others' stores of y
    __threadfence();
    __syncthreads();
    if (wave > 0) return;
    holds = len == whole;
    run_alone<IO, N, SOFTPLUS>(d, in, b, g, tile, first, len, k.E ? k.E + bc * d.D * N : in.S0 ? in.S0 + b * d.D * N : nullptr, y, h);
  }
  const Cell<N> cell(d, g, tile, lane_again());
  if (S_T && holds && cell.on)
    *reinterpret_cast<float4*>(S_T + (b * d.D + cell.c) * N + 4 * cell.s) = make_float4(h[0], h[1], h[2], h[3]);
}

// ---- one token --------------------------------------------------------------------
// N / 4 lanes a channel, four states each: bound by the states, read and written once.
// 512 x 1536, N = 16: 20 us, 5.3 TB/s, what a copy reaches.
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

// dy of either type: bits as loaded, shifted into place where it is bf16.
struct Incoming {
  const void* dy;
  bool bf16;
};
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const Incoming& in, int64_t row, int64_t token, int rows) {
  return in.bf16 ? rows_at(static_cast<const bf16_t*>(in.dy), row, token, rows) : rows_at(static_cast<const float*>(in.dy), row, token, rows);
}
__device__ __forceinline__ float widen(const Incoming& in, uint32_t bits) { return __uint_as_float(in.bf16 ? bits << 16 : bits); }

constexpr int kEndsWaves = 4;

// A map after another.  From nothing it leaves its own part alone: where states grow
// (delta A > 0) its factor may overflow.
__device__ __forceinline__ float carried(float factor, float from, float own) {
  return from == 0.0f ? own : __builtin_fmaf(factor, from, own);
}

// For the gradients one wave a chunk and 256 / N channels, four neighbouring tiles of
// channels a workgroup.  For the forward, whose chunks are few and long, a
// workgroup's four waves take a quarter of one chunk each and join their maps (one
// wave a chunk left the card half empty: 63 us of 1 x 16384 x 768's 125).
template <typename IO, int N, bool SOFTPLUS, bool GRAD>
__global__ __launch_bounds__(64 * kEndsWaves) void scan_ends_kernel(ScanDims d, ScanIn<IO> in, bool wide, Incoming up, Chunks k,
                                                                    int64_t waves) {
  using L = Lanes<N>;
  __shared__ float shared[kEndsWaves][2][kShared<N>];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t id = GRAD ? by_xcd(blockIdx.x, gridDim.x) * kEndsWaves + wave : by_xcd(blockIdx.x, gridDim.x);
  if (id >= waves) return;
  const int tile = int(id % d.tiles), g = int(id / d.tiles % d.G);
  const int64_t bc = id / (int64_t(d.tiles) * d.G);     // b count + chunk
  const int64_t b = bc / k.count;
  const int part = GRAD ? k.tokens : k.tokens / kEndsWaves;
  const int first = int(bc % k.count) * k.tokens + (GRAD ? 0 : wave * part);
  const Cell<N> cell(d, g, tile);
  const int len = __builtin_amdgcn_readfirstlane(tokens_of(in.lengths, int(b), d.T)), end = min(first + part, len);
  float A2[4], E[4] = {0.0f, 0.0f, 0.0f, 0.0f}, R[4] = {0.0f, 0.0f, 0.0f, 0.0f}, P[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sum = 0.0f;
  four(in.A + int64_t(cell.c) * N + 4 * cell.s, A2);
#pragma unroll
  for (int n = 0; n < 4; ++n) A2[n] *= kLog2e;
  const float bias = in.dt_bias ? in.dt_bias[cell.c] : 0.0f;
  float* Bs = shared[wave][0];
  float* Cs = shared[wave][1];
  const Offsets<IO, N> offsets(d, g, cell.c);
  const int up_size = up.bf16 ? 2 : 4, up_at = (cell.j * d.D + cell.c) * up_size;
  Tokens<IO, N> next;
  uint32_t up_next[L::kRegs] = {};
  auto load = [&](int t0) {
    load_tokens<IO, N>(d, in, b, t0, end, wide, offsets, next);
    if constexpr (GRAD) {
      const auto r = rows_at(up, d.D, b * d.T + t0, min(end - t0, kTok));
      if (up.bf16) {
#pragma unroll
        for (int i = 0; i < L::kRegs; ++i) up_next[i] = load_bits<bf16_t>(r, up_at + i * L::kQuad * d.D * 2);
      } else {
#pragma unroll
        for (int i = 0; i < L::kRegs; ++i) up_next[i] = load_bits<float>(r, up_at + i * L::kQuad * d.D * 4);
      }
    }
  };
  // the map of the chunk's tokens before t0 (stores by offset: no branch around the
  // lane moves)
  const auto sub_E = rows_at(k.sub_E, int64_t(d.D) * N, bc * k.subs, GRAD ? k.subs : 0);
  const auto sub_sums = rows_at(k.sub_sums, d.D, bc * k.subs, GRAD ? k.subs : 0);
  const uint32_t E_at = cell.on ? (cell.c * N + 4 * cell.s) * 4 : kNowhere, sum_at = cell.on && cell.s == 0 ? cell.c * 4 : kNowhere;
  auto sub_map = [&](int t0) {
    const uint32_t row = (t0 - first) / kTok - 1;
    const auto bits = [](float v) { return __float_as_uint(v); };
    typedef uint32_t four_words __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(four_words{bits(E[0]), bits(E[1]), bits(E[2]), bits(E[3])}, sub_E, E_at + row * d.D * N * 4, 0, 0);
    store_one<float>(sub_sums, sum_at + row * d.D * 4, lanes_sum<L::kQuad>(sum));
  };
  if (first < end) load(first);
  int t0 = first;
  for (; t0 < end; t0 += kTok) {
    float delta[L::kRegs], u[L::kRegs], q[L::kRegs];
    stage_shared<IO, N>(next, Bs, Cs);
#pragma unroll
    for (int i = 0; i < L::kRegs; ++i) {
      delta[i] = kept(step_of<SOFTPLUS>(widen(next.dt[i]) + bias), t0 + L::kQuad * i + cell.j < end);
      u[i] = delta[i] * widen(next.x[i]);
      if constexpr (GRAD) {
        q[i] = widen(up, up_next[i]);
        if (in.z) q[i] *= act_f32<kActSilu>(widen(next.z[i]));
      }
    }
    if (t0 + kTok < end) load(t0 + kTok);
    if constexpr (GRAD) {
      if (t0 > first) sub_map(t0);
    }
#pragma unroll
    for (int i = 0; i < L::kRegs; ++i) sum += delta[i];
    __builtin_amdgcn_wave_barrier();
    each_token<L::kQuad>([&](auto t, auto jj, auto i) {
      const float dt = from_lane<L::kQuad, jj()>(delta[i()]), ut = from_lane<L::kQuad, jj()>(u[i()]);
      float bt[4], a[4];
      four(Bs + t() * N + 4 * cell.s, bt);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        a[n] = __builtin_amdgcn_exp2f(dt * A2[n]);
        E[n] = __builtin_fmaf(a[n], E[n], ut * bt[n]);
      }
      if constexpr (GRAD) {
        const float qt = from_lane<L::kQuad, jj()>(q[i()]);
        float ct[4];
        four(Cs + t() * N + 4 * cell.s, ct);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          P[n] *= a[n];
          R[n] = __builtin_fmaf(P[n], qt * ct[n], R[n]);
        }
      }
    });
    __builtin_amdgcn_wave_barrier();
  }
  if constexpr (GRAD) {
    // sixteens that the sequence does not reach
    for (t0 = max(t0, first + kTok); t0 < first + k.tokens; t0 += kTok) sub_map(t0);
  }
  sum = lanes_sum<L::kQuad>(sum);
  if constexpr (!GRAD) {
    __shared__ float4 E_of[kEndsWaves][64];
    __shared__ float sum_of[kEndsWaves][64];
    const int lane = threadIdx.x % 64;
    E_of[wave][lane] = make_float4(E[0], E[1], E[2], E[3]);
    sum_of[wave][lane] = sum;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < kEndsWaves; ++w) {
      float own[4];
      four(reinterpret_cast<const float*>(&E_of[w][lane]), own);
      const float s = sum_of[w][lane];
#pragma unroll
      for (int n = 0; n < 4; ++n) E[n] = carried(__builtin_amdgcn_exp2f(s * A2[n]), E[n], own[n]);
      sum += s;
    }
  }
  if (cell.on) {
    const int64_t at = (bc * d.D + cell.c) * N + 4 * cell.s;
    *reinterpret_cast<float4*>(k.E + at) = make_float4(E[0], E[1], E[2], E[3]);
    if constexpr (GRAD) *reinterpret_cast<float4*>(k.R + at) = make_float4(R[0], R[1], R[2], R[3]);
    if (cell.s == 0) k.sums[bc * d.D + cell.c] = sum;
  }
}

// One thread a state.  Loads run kAhead chunks in front.
constexpr int kAhead = 8;
template <bool GRAD>
__global__ __launch_bounds__(256) void scan_carry_kernel(int D, int N, int64_t states, Chunks k, const float* __restrict__ A,
                                                         const float* __restrict__ S0, const float* __restrict__ dS_T,
                                                         float* __restrict__ dS0) {
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (id >= states) return;
  const int64_t DN = int64_t(D) * N, b = id / DN, dn = id - b * DN;
  const int c = int(dn / N);
  const float A2 = A[dn] * kLog2e;
  const int64_t first = b * k.count;
  float H = S0 ? S0[id] : 0.0f;
  for (int k0 = 0; k0 < k.count; k0 += kAhead) {
    float sum[kAhead], E[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = first + min(k0 + i, k.count - 1);
      sum[i] = k.sums[at * D + c];
      E[i] = k.E[at * DN + dn];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (k0 + i < k.count) {
        k.E[(first + k0 + i) * DN + dn] = H;
        H = carried(__builtin_amdgcn_exp2f(A2 * sum[i]), H, E[i]);
      }
  }
  if constexpr (GRAD) {
    float G = dS_T ? dS_T[id] : 0.0f;
    for (int k0 = k.count - 1; k0 >= 0; k0 -= kAhead) {
      float sum[kAhead], R[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t at = first + max(k0 - i, 0);
        sum[i] = k.sums[at * D + c];
        R[i] = k.R[at * DN + dn];
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (k0 - i >= 0) {
          k.R[(first + k0 - i) * DN + dn] = G;
          G = carried(__builtin_amdgcn_exp2f(A2 * sum[i]), G, R[i]);
        }
    }
    if (dS0) dS0[id] = G;
  }
}

// ---- gradients ----------------------------------------------------------------------
// A workgroup takes one chunk of one group and, four waves side by side, its
// channels, 4 x 256 / N at a time.  A wave takes the chunk's sixteens from the last
// to the first: forward from the state before them (from scan_ends_kernel's maps;
// decays and states stay in registers), then back with G.
// What sums over channels (dB, dC) is summed over the wave's lanes by lane swaps
// and over its channel tiles in LDS, over the waves at the end, in this order;
// workgroups of other channels leave rows of partial sums.  What sums over tokens
// (dA, dD, ddt_bias) leaves as one row a chunk.  8 x 2048 x 768, N = 16: maps 68 us,
// carry 14, this kernel 188, sums 10; bound by the vector units (about 100
// instructions a token and wave) at two waves a SIMD, which the 128 registers of
// decays and states allow.  (With N = 8 they do not: 41 to 57 registers a lane are
// kept in memory, and 8 x 2048 x 768 takes 256 us.)  Eights instead of sixteens
// (fewer registers, more maps) ran slower at N = 16.
constexpr int kBwdWaves = 4;
template <int N>
constexpr int kChunkTokens = N <= 16 ? 64 : 1024 / N;   // so that LDS holds the sums of 2 N a token and wave

// Sums of vb[0..3] and vc[0..3] over the wave's channels.  The lanes of a row of 16
// end with one of the four states each (row_state), a lane the sum of vb where bit
// 3 is clear and that of vc where it is set; for N = 64, whose rows hold one
// channel, vb's sum in `w` and vc's in `w2`.
template <int N>
__device__ __forceinline__ void channels_sum(const float (&vb)[4], const float (&vc)[4], bool high, float& w, float& w2) {
  auto swap32 = [](float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  auto swap16 = [](float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  w = swap16(swap32(vb[0], vb[1]), swap32(vb[2], vb[3]));
  w2 = swap16(swap32(vc[0], vc[1]), swap32(vc[2], vc[3]));
  if constexpr (Lanes<N>::kPer <= 2) {
    w = dpp_plus<0x4e>(w);     // quad_perm [2, 3, 0, 1]
    w2 = dpp_plus<0x4e>(w2);
  }
  if constexpr (Lanes<N>::kPer <= 4) {
    w = dpp_plus<0x124>(w);    // row_ror 4
    w2 = dpp_plus<0x124>(w2);
  }
  if constexpr (Lanes<N>::kPer <= 8) {
    // each half keeps one of the two and hands over its part of the other
    const float give = high ? w : w2, keep = high ? w2 : w;
    w = keep + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, give), 0x128, 0xf, 0xf, true));   // row_ror 8
  }
}
// The state of its four that a lane's row of 16 holds after channels_sum.
__device__ __forceinline__ int row_state(int lane) {
  const int r = lane / 16;
  return (r & 1) * 2 + (r >> 1);
}

// One wave's sixteen tokens of every input the gradients need, as loaded.
template <typename IO, int N>
struct BwdTokens {
  bits_t<IO> x[Lanes<N>::kRegs], dt[Lanes<N>::kRegs], z[Lanes<N>::kRegs];
  uint32_t dy[Lanes<N>::kRegs];
};

struct ScanGrads {
  float* dx;
  float* ddt;
  float* dz;
  float* bc;       // dB and dC, or rows of partial sums: [sets][B T][G][2][N]
  float* params;   // [B count] rows of params_row floats: dA, dD, ddt_bias of a chunk
};

// D (N + 2) floats, and as many more as put every row on a multiple of 16 bytes.
__host__ __device__ __forceinline__ int64_t params_row(int D, int N) { return (int64_t(D) * (N + 2) + 3) / 4 * 4; }

template <typename IO, int N, bool SOFTPLUS>
__global__ __launch_bounds__(64 * kBwdWaves, 2) void scan_bwd_kernel(ScanDims d, ScanIn<IO> in, Incoming up, Chunks k,
                                                                    ScanGrads out, int sets) {
  using L = Lanes<N>;
  constexpr int kTokens = kChunkTokens<N>, kSub = kTokens / kTok;
  __shared__ float shared[2][kTokens * N];                  // B, C of the chunk
  __shared__ float bc[kBwdWaves][kTokens][2][N];            // dB, dC
  __shared__ float4 before[kBwdWaves][kSub][64];            // the state before each sixteen
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
  const int64_t id = by_xcd(blockIdx.x, gridDim.x);
  const int set = int(id % sets), g = int(id / sets % d.G);
  const int64_t chunk = id / (int64_t(sets) * d.G), b = chunk / k.count;
  const int first = int(chunk % k.count) * kTokens;
  const int len = __builtin_amdgcn_readfirstlane(tokens_of(in.lengths, int(b), d.T));

  for (int i = threadIdx.x; i < kTokens * N; i += 64 * kBwdWaves) {
    const int t = first + i / N;
    const bool live = t < len;
    const int64_t token = b * d.T + min(t, len - 1);
    shared[0][i] = live ? io<IO>::load(in.Bm, token * d.b_row + g * N + i % N) : 0.0f;
    shared[1][i] = live ? io<IO>::load(in.Cm, token * d.c_row + g * N + i % N) : 0.0f;
  }
  for (int i = threadIdx.x; i < kBwdWaves * kTokens * 2 * N; i += 64 * kBwdWaves) (&bc[0][0][0][0])[i] = 0.0f;
  __syncthreads();

  const int groups = (d.tiles + kBwdWaves - 1) / kBwdWaves;      // of kBwdWaves tiles each
  for (int tg = set; tg < groups; tg += sets) {
    const int tile = tg * kBwdWaves + wave;
    if (tile >= d.tiles) continue;
    const Cell<N> cell(d, g, tile);
    const int s = cell.s, j = cell.j;
    const int64_t at = (chunk * d.D + cell.c) * N + 4 * s;
    float A[4], A2[4], h[4], G[4], dA[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dskip = 0.0f, dbias = 0.0f;
    four(in.A + int64_t(cell.c) * N + 4 * s, A);
    four(k.E + at, h);
    four(k.R + at, G);
#pragma unroll
    for (int n = 0; n < 4; ++n) A2[n] = A[n] * kLog2e;
    const float skip = in.Dskip ? in.Dskip[cell.c] : 0.0f, bias = in.dt_bias ? in.dt_bias[cell.c] : 0.0f;
    const int es = sizeof(IO);
    const int x_at = (j * int(d.x_row) + cell.c) * es, dt_at = (j * int(d.dt_row) + cell.c) * es, z_at = (j * int(d.z_row) + cell.c) * es;
    const int up_at = (j * d.D + cell.c) * (up.bf16 ? 2 : 4);
    const uint32_t out_at = cell.on && s < L::kQuad ? (j * d.D + cell.c) * 4 : kNowhere;
    // where this lane adds to dB (bit 3 clear) or dC, if at all
    const bool high = L::kPer <= 8 && lane & 8, adds = (lane & 7) < L::kPer;
    float* at_bc = &bc[wave][0][high ? 1 : 0][4 * s + row_state(lane)];
    BwdTokens<IO, N> next;
    auto load = [&](int m) {
      const int64_t token = b * d.T + first + m * kTok;
      const int rows = min(len - (first + m * kTok), kTok);
      const auto rx = rows_at(in.x, d.x_row, token, rows), rdt = rows_at(in.dt, d.dt_row, token, rows), ru = rows_at(up, d.D, token, rows);
#pragma unroll
      for (int i = 0; i < L::kRegs; ++i) {
        next.x[i] = load_bits<IO>(rx, x_at + i * L::kQuad * int(d.x_row) * es);
        next.dt[i] = load_bits<IO>(rdt, dt_at + i * L::kQuad * int(d.dt_row) * es);
      }
      if (up.bf16) {
#pragma unroll
        for (int i = 0; i < L::kRegs; ++i) next.dy[i] = load_bits<bf16_t>(ru, up_at + i * L::kQuad * d.D * 2);
      } else {
#pragma unroll
        for (int i = 0; i < L::kRegs; ++i) next.dy[i] = load_bits<float>(ru, up_at + i * L::kQuad * d.D * 4);
      }
      if (in.z) {
        const auto rz = rows_at(in.z, d.z_row, token, rows);
#pragma unroll
        for (int i = 0; i < L::kRegs; ++i) next.z[i] = load_bits<IO>(rz, z_at + i * L::kQuad * int(d.z_row) * es);
      }
    };

    load(kSub - 1);
    // the state before each sixteen
    before[wave][0][lane] = make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
    for (int m = 1; m < kSub; ++m) {
      const int64_t row = (chunk * k.subs + m - 1) * d.D + cell.c;
      const float sum = k.sub_sums[row];
      float E[4];
      four(k.sub_E + row * N + 4 * s, E);
      before[wave][m][lane] = make_float4(carried(__builtin_amdgcn_exp2f(sum * A2[0]), h[0], E[0]), carried(__builtin_amdgcn_exp2f(sum * A2[1]), h[1], E[1]),
                                          carried(__builtin_amdgcn_exp2f(sum * A2[2]), h[2], E[2]), carried(__builtin_amdgcn_exp2f(sum * A2[3]), h[3], E[3]));
    }

    for (int m = kSub - 1; m >= 0; --m) {
      const int t0 = first + m * kTok;
      const int64_t token = b * d.T + t0;
      float delta[L::kRegs], x[L::kRegs], u[L::kRegs], q[L::kRegs], dy[L::kRegs], z[L::kRegs], raw[L::kRegs];
#pragma unroll
      for (int i = 0; i < L::kRegs; ++i) {
        // lanes without a channel of their own add nothing: u and q zero
        x[i] = widen(next.x[i]);
        raw[i] = widen(next.dt[i]) + bias;
        delta[i] = kept(step_of<SOFTPLUS>(raw[i]), t0 + L::kQuad * i + j < len);
        u[i] = kept(delta[i] * x[i], cell.on);
        dy[i] = kept(widen(up, next.dy[i]), cell.on);
        z[i] = in.z ? widen(next.z[i]) : 0.0f;
        q[i] = in.z ? dy[i] * act_f32<kActSilu>(z[i]) : dy[i];
      }
      // forward: the decays, and the state before every token
      float a[kTok][4], prev[kTok][4];
      four(reinterpret_cast<const float*>(&before[wave][m][lane]), h);
      each_token<L::kQuad>([&](auto t, auto jj, auto i) {
        const float dt = from_lane<L::kQuad, jj()>(delta[i()]), ut = from_lane<L::kQuad, jj()>(u[i()]);
        float bt[4];
        four(&shared[0][(m * kTok + t()) * N + 4 * s], bt);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          prev[t()][n] = h[n];
          a[t()][n] = __builtin_amdgcn_exp2f(dt * A2[n]);
          h[n] = __builtin_fmaf(a[t()][n], h[n], ut * bt[n]);
        }
      });
      // back
      float du[L::kRegs], turn[L::kRegs], read[L::kRegs], sums[4], sums2[4];
      each_token<L::kQuad>([&](auto back, auto, auto) {
        constexpr int t = kTok - 1 - back(), i = t / L::kQuad, jj = t % L::kQuad;
        const float dt = from_lane<L::kQuad, jj>(delta[i]), ut = from_lane<L::kQuad, jj>(u[i]), qt = from_lane<L::kQuad, jj>(q[i]);
        float bt[4], ct[4], vb[4], vc[4], r = 0.0f, su = 0.0f, st = 0.0f;
        four(&shared[0][(m * kTok + t) * N + 4 * s], bt);
        four(&shared[1][(m * kTok + t) * N + 4 * s], ct);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float now;                                  // the state after token t
          if constexpr (t == kTok - 1) {
            now = h[n];
          } else {
            now = prev[t + 1][n];
          }
          G[n] = __builtin_fmaf(qt, ct[n], G[n]);
          r = __builtin_fmaf(ct[n], now, r);
          su = __builtin_fmaf(G[n], bt[n], su);
          vb[n] = G[n] * ut;
          vc[n] = qt * now;
          G[n] *= a[t][n];
          const float mt = G[n] * prev[t][n];
          st = __builtin_fmaf(A[n], mt, st);
          dA[n] = __builtin_fmaf(mt, dt, dA[n]);
        }
        if (t0 + t >= len) {
          // Behind the sequence's end every factor is zero, but zero times a state or a
          // gradient that is not finite is not: these tokens, the first that come by,
          // leave nothing.  (The empty asm keeps this a branch: four selects a token
          // took 6 us of 260, the branch 2.)
          asm volatile("");
          dA[0] = dA[1] = dA[2] = dA[3] = 0.0f;
        }
        channels_sum<N>(vb, vc, high, sums[t % 4], sums2[t % 4]);
        if constexpr (t % 4 == 0) {
          if (adds) {
            // read, add and write, four tokens at a time: an LDS atomic here took 80
            // cycles each, and 303 us of the whole in place of 260
            float* to = at_bc + (m * kTok + t) * 2 * N;
            float old[4], old2[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              old[k] = to[k * 2 * N];
              if constexpr (L::kPer == 16) old2[k] = to[k * 2 * N + N];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              to[k * 2 * N] = old[k] + sums[k];
              if constexpr (L::kPer == 16) to[k * 2 * N + N] = old2[k] + sums2[k];
            }
          }
        }
        // half the decays and states are done with: room for the next sixteen
        if constexpr (t == kTok / 2) {
          if (m > 0) load(m - 1);
        }
        r = lanes_sum<L::kPer>(r);
        su = lanes_sum<L::kPer>(su);
        st = lanes_sum<L::kPer>(st);
        const bool first_of_four = jj == L::kQuad - 1;
        read[i] = first_of_four || j == jj ? r : read[i];
        du[i] = first_of_four || j == jj ? su : du[i];
        turn[i] = first_of_four || j == jj ? st : turn[i];
      });
      const int all = min(d.T - t0, kTok);
      const auto rdx = rows_at(out.dx, d.D, token, all), rddt = rows_at(out.ddt, d.D, token, all);
#pragma unroll
      for (int i = 0; i < L::kRegs; ++i) {
        const uint32_t o = out_at + uint32_t(i * L::kQuad) * d.D * 4;
        const bool live = t0 + L::kQuad * i + j < len;    // (zeros behind the end, whatever the state: not products with zero)
        const float dd = kept((turn[i] + du[i] * x[i]) * (SOFTPLUS ? sigmoid_f32(raw[i]) : 1.0f), live);
        dskip = __builtin_fmaf(q[i], x[i], dskip);
        dbias += dd;
        store_one<float>(rdx, o, kept(__builtin_fmaf(du[i], delta[i], skip * q[i]), live));
        store_one<float>(rddt, o, dd);
      }
      if (out.dz) {
        const auto rdz = rows_at(out.dz, d.D, token, all);
#pragma unroll
        for (int i = 0; i < L::kRegs; ++i)
          store_one<float>(rdz, out_at + uint32_t(i * L::kQuad) * d.D * 4,
                           kept(dy[i] * __builtin_fmaf(skip, x[i], read[i]) * act_slope_f32<kActSilu>(z[i]), t0 + L::kQuad * i + j < len));
      }
    }
    dskip = lanes_sum<L::kQuad>(dskip);
    dbias = lanes_sum<L::kQuad>(dbias);
    if (cell.on) {
      float* row = out.params + chunk * params_row(d.D, N);
      *reinterpret_cast<float4*>(row + int64_t(cell.c) * N + 4 * s) = make_float4(dA[0], dA[1], dA[2], dA[3]);
      if (s == 0) {
        row[int64_t(d.D) * N + cell.c] = dskip;
        row[int64_t(d.D) * (N + 1) + cell.c] = dbias;
      }
    }
  }
  __syncthreads();
  float* rows = out.bc + int64_t(set) * d.B * d.T * d.G * 2 * N;
  for (int i = threadIdx.x; i < kTokens * 2 * N; i += 64 * kBwdWaves) {
    const int t = first + i / (2 * N);
    if (t >= d.T) break;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kBwdWaves; ++w) v += (&bc[w][0][0][0])[i];
    if (t >= len) v = 0.0f;   // (as above: not what a state that is not finite left)
    rows[((b * d.T + t) * d.G + g) * 2 * N + i % (2 * N)] = v;
  }
}

// dB, dC of every token and group from the sets' rows.
__global__ __launch_bounds__(256) void scan_bc_kernel(const float* __restrict__ parts, int sets, int N, int64_t n, float* __restrict__ dB,
                                                      float* __restrict__ dC) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
    const int64_t tg = i / (2 * N);
    const int k = int(i % (2 * N));
    float s = 0.0f;
    for (int j = 0; j < sets; ++j) s += parts[j * n + i];
    if (k < N) {
      dB[tg * N + k] = s;
    } else {
      dC[tg * N + k - N] = s;
    }
  }
}

// Channels a wave: 256 / N.
ScanDims dims_of(const ScanArgs& a) {
  ScanDims d{};
  d.B = a.B; d.T = a.T; d.D = a.D; d.G = a.G;
  d.Dg = a.D / a.G;
  d.tiles = (d.Dg + 256 / a.N - 1) / (256 / a.N);
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

// Chunks of the forward.  One where there are channels for more than kCutBelow
// workgroups or fewer than kCutFrom tokens; else enough for kCutInto workgroups.
// Cutting works out every decay twice and takes two launches more, so it pays only
// where a long chain of turns would leave most of the card idle (D = 1536, N = 16,
// us, one chunk against cut): B = 1: T = 256: 12 and 19, T = 1024: 34 and 25,
// T = 4096: 119 and 60; B = 2: T = 1024: 34 and 37, T = 4096: 120 and 110.  With
// N = 8 (48 workgroups): T = 256: 13 and 19, T = 768: 29 and 23, T = 4096: 132 and
// 48; with N = 64 (96 workgroups): T = 256: 12 and 19, T = 768: 27 and 29, T = 1024:
// 35 and 30, T = 4096: 123 and 72.  768 workgroups are one round of three a CU for
// N = 16 and 32; 1024 (1 x 16384 x 768: 126 us against 107) and 2560 (112) are not.
// N = 8 and 64 run two a CU, and yet 512 workgroups are slower there, too (T = 4096:
// 62 us against 48, and 91 against 72).
constexpr int64_t kCutBelow = 128, kCutInto = 768;
constexpr int kCutFrom = 768;
struct FwdShape {
  int tokens, count;
  int64_t sums, states;   // floats of the workspace's parts (sums padded to 16 bytes)
};
FwdShape fwd_shape(const ScanArgs& a) {
  const ScanDims d = dims_of(a);
  const int64_t blocks = int64_t(a.B) * a.G * d.tiles;
  FwdShape s{std::max(a.T, 1), 1, 0, 0};
  if (blocks == 0 || blocks > kCutBelow || a.T < kCutFrom) return s;
  constexpr int kRound = kFwdWaves * kTok;   // tokens of one turn of every wave
  const int64_t want = std::min<int64_t>((kCutInto + blocks - 1) / blocks, a.T / kRound);
  s.tokens = int(((a.T + want - 1) / want + kRound - 1) / kRound * kRound);
  s.count = (a.T + s.tokens - 1) / s.tokens;
  s.sums = (int64_t(a.B) * s.count * a.D + 3) / 4 * 4;
  s.states = int64_t(a.B) * s.count * a.D * a.N;
  return s;
}

template <typename IO, int N, bool SP>
hipError_t fwd_typed(const ScanArgs& a, hipStream_t st) {
  const ScanDims d = dims_of(a);
  const FwdShape s = fwd_shape(a);
  const int64_t blocks = int64_t(a.B) * s.count * a.G * d.tiles;
  if (blocks > kMaxGrid) return hipErrorInvalidValue;
  const ScanIn<IO> in = inputs_of<IO>(a);
  Chunks k{};
  k.tokens = s.tokens;
  k.count = s.count;
  if (s.count > 1) {
    k.E = a.workspace;
    k.sums = k.E + s.states;
    const int64_t states = int64_t(a.B) * a.D * N;
    scan_ends_kernel<IO, N, SP, false><<<dim3(unsigned(blocks)), dim3(64 * kEndsWaves), 0, st>>>(d, in, fours_wide(a),
                                                                                                          Incoming{nullptr, false}, k, blocks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    scan_carry_kernel<false><<<dim3(unsigned((states + 255) / 256)), dim3(256), 0, st>>>(a.D, N, states, k, a.A, a.S0, nullptr, nullptr);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  scan_fwd_kernel<IO, N, SP><<<dim3(unsigned(blocks)), dim3(64 * kFwdWaves), 0, st>>>(d, in, fours_wide(a), k, static_cast<IO*>(a.y), a.S_T,
                                                                                     a.spin_limit);
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

// The backward's workspace: the chunks' maps, partial sums of dB and dC, and the
// chunks' rows of parameter gradients.
struct BwdShape {
  int tokens, count, sets;
  int64_t sums, states, subs, bc, params;   // floats of each part (sums padded to 16 bytes)
};
BwdShape bwd_shape(const ScanArgs& a) {
  BwdShape s{};
  s.tokens = a.N <= 16 ? 64 : 1024 / a.N;
  s.count = (a.T + s.tokens - 1) / s.tokens;
  const int64_t chunks = int64_t(a.B) * s.count;
  const ScanDims d = dims_of(a);
  const int64_t groups = (d.tiles + kBwdWaves - 1) / kBwdWaves;
  // two workgroups a CU fill the card; more only add rows of partial sums
  s.sets = int(std::min<int64_t>(std::max<int64_t>(groups, 1), std::max<int64_t>(1, (512 + chunks * a.G - 1) / std::max<int64_t>(1, chunks * a.G))));
  s.subs = s.tokens / kTok - 1;
  s.sums = (chunks * a.D * (1 + s.subs) + 3) / 4 * 4;
  s.states = chunks * a.D * a.N;
  s.bc = int64_t(s.sets) * a.B * a.T * a.G * 2 * a.N;
  s.params = chunks * params_row(a.D, a.N);
  return s;
}

template <typename IO, int N, bool SP>
hipError_t bwd_typed(const ScanArgs& a, hipStream_t st) {
  static_assert(kChunkTokens<N> == (N <= 16 ? 64 : 1024 / N));
  const ScanDims d = dims_of(a);
  const BwdShape s = bwd_shape(a);
  Chunks k{};
  k.tokens = s.tokens;
  k.count = s.count;
  k.subs = int(s.subs);
  k.E = a.workspace;
  k.R = k.E + s.states;
  k.sub_E = k.R + s.states;
  float* bc = k.sub_E + s.states * s.subs;
  float* params = bc + s.bc;
  k.sums = params + s.params;
  const int64_t chunks = int64_t(a.B) * s.count, states = int64_t(a.B) * a.D * N;
  k.sub_sums = k.sums + chunks * a.D;
  const ScanIn<IO> in = inputs_of<IO>(a);
  const Incoming up{a.dy, a.dy_bf16};
  const int64_t waves = chunks * a.G * d.tiles, ends = (waves + kEndsWaves - 1) / kEndsWaves, blocks = chunks * a.G * s.sets;
  if (ends > kMaxGrid || blocks > kMaxGrid || (states + 255) / 256 > kMaxGrid) return hipErrorInvalidValue;
  hipError_t e = hipSuccess;
  if (ends > 0) {
    scan_ends_kernel<IO, N, SP, true><<<dim3(unsigned(ends)), dim3(64 * kEndsWaves), 0, st>>>(d, in, fours_wide(a), up, k, waves);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (states > 0) {
    scan_carry_kernel<true><<<dim3(unsigned((states + 255) / 256)), dim3(256), 0, st>>>(a.D, N, states, k, a.A, a.S0, a.dS_T, a.dS0);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (blocks > 0) {
    const ScanGrads out{a.dx, a.ddt, a.dz, bc, params};
    scan_bwd_kernel<IO, N, SP><<<dim3(unsigned(blocks)), dim3(64 * kBwdWaves), 0, st>>>(d, in, up, k, out, s.sets);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t n = int64_t(a.B) * a.T * a.G * 2 * N;
  if (n > 0) {
    scan_bc_kernel<<<dim3(unsigned(std::min<int64_t>((n + 255) / 256, 1 << 16))), dim3(256), 0, st>>>(bc, s.sets, N, n, a.dB, a.dC);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t DN = int64_t(a.D) * N;
  return launch_sum_parts({params, chunks, DN + 2 * a.D, params_row(a.D, N), {a.dA, a.dD, a.ddt_bias}, {DN, DN + a.D}}, st);
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

size_t scan_workspace_bytes(const ScanArgs& a) {
  const FwdShape s = fwd_shape(a);
  return size_t(s.states + s.sums) * sizeof(float);
}

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
  const BwdShape s = bwd_shape(a);
  return size_t((2 + s.subs) * s.states + s.bc + s.params + s.sums) * sizeof(float);
}

hipError_t launch_scan_bwd(const ScanArgs& a, hipStream_t st) {
  return by_size(a, [&](auto n, auto sp) {
    return a.bf16 ? bwd_typed<bf16_t, n(), sp()>(a, st) : bwd_typed<float, n(), sp()>(a, st);
  });
}

}  // namespace falcon
