// Group norm with an activation, a token's group of d channels at a time
// (gfx950), and its gradients.
//
//   xhat = (x - mu) r,  r = 1 / sqrt(mean((x - mu)^2) + eps),  y = scale f(w xhat + b)
//   dp = scale dy f'(p),  dh = w dp,
//   dx = r (dh - [center] mean(dh) - xhat mean(dh xhat)),  dw = sum dp xhat,  db = sum dp
//
// Bound by bytes.  LANES lanes share a group, each with NC pieces of 8 adjacent
// channels; a group stays in registers, so x is read once, and the sums over
// its lanes are lane moves.  A thread keeps its channels' weights and walks over
// tokens, the next one's loads in flight.  Measured at 8 x 2048 tokens of 12 groups
// of 64 (bf16, ELU + 1, rows to heads): 12 us, 4.3 TB/s; gradients 26 us and 5 for
// the parameters' sums (4.9 TB/s).  The index of a token in its sequence comes from a
// multiply (a 64-bit division by T a token and thread made the 12 us 29).  Groups of
// more than 2048 channels keep the gradients' sums in memory, not in registers:
// 2^18 tokens of 4096 take 12.4 ms, 2^19 of 2048 3.2.

#include <algorithm>

#include "falcon_block_device.h"
#include "falcon_launch.h"

namespace falcon {

namespace {

constexpr int kPiece = 8;   // adjacent channels of one access

// Where token b T + t, group g lies: rows at token * row + g d, heads at
// ((b G + g) T + t) d.
struct Layout {
  bool heads;
  int64_t row;
};
// n / T for n < 2^31 as a product and a shift, worked out on the host.
struct Divisor {
  uint32_t magic, shift;
};
__device__ __forceinline__ uint32_t quotient(uint32_t n, Divisor by) { return (__umulhi(n, by.magic) + n) >> by.shift; }
__device__ __forceinline__ int64_t group_at(Layout l, uint32_t token, int g, int T, Divisor by_T, int G, int d) {
  if (!l.heads) return token * l.row + int64_t(g) * d;
  const uint32_t b = quotient(token, by_T), t = token - b * uint32_t(T);
  return ((int64_t(b) * G + g) * T + t) * d;
}

// Channel i of a lane's piece k.  WIDE: pieces of 8 adjacent channels, one wide
// access each; else neighbours go to neighbouring lanes, element by element.
template <int LANES, bool WIDE>
__device__ __forceinline__ int channel(int k, int i, int l) {
  return WIDE ? (k * LANES + l) * kPiece + i : (k * kPiece + i) * LANES + l;
}
template <typename E, int LANES, int NC, bool WIDE>
__device__ __forceinline__ void load_group(const E* p, int l, int d, float (&v)[NC][kPiece]) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    if constexpr (WIDE) {
      const int e = channel<LANES, WIDE>(k, 0, l);
      if (e < d) {
        load_vec<E, kPiece>(p + e, v[k]);
      } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) v[k][i] = 0.0f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const int e = channel<LANES, WIDE>(k, i, l);
        v[k][i] = e < d ? io<E>::load(p, e) : 0.0f;
      }
    }
  }
}
template <typename E, int LANES, int NC, bool WIDE>
__device__ __forceinline__ void store_group(E* p, int l, int d, const float (&v)[NC][kPiece]) {
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    if constexpr (WIDE) {
      const int e = channel<LANES, WIDE>(k, 0, l);
      if (e < d) store_vec<E, kPiece>(p + e, v[k]);
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const int e = channel<LANES, WIDE>(k, i, l);
        if (e < d) io<E>::store(p, e, v[k][i]);
      }
    }
  }
}

// xhat in place of x; returns r.  Channels behind d hold zero before and after.
template <int LANES, int NC, bool WIDE>
__device__ __forceinline__ float normalise(float (&x)[NC][kPiece], int l, int d, float inv_d, bool center, float eps) {
  if (center) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) s += x[k][i];
    const float mu = lanes_sum<LANES>(s) * inv_d;
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) x[k][i] = channel<LANES, WIDE>(k, i, l) < d ? x[k][i] - mu : 0.0f;
  }
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int i = 0; i < kPiece; ++i) q = __builtin_fmaf(x[k][i], x[k][i], q);
  const float m = __builtin_fmaf(lanes_sum<LANES>(q), inv_d, eps);
  float r = __builtin_amdgcn_rsqf(m), scaled = 1.0f;
  // Squares that leave float32's normal numbers (values past 2^60 or, with eps = 0,
  // below 2^-63): the groups concerned once more, scaled by a power of two.  The whole
  // wave goes along, for the moves between lanes.
  if (__builtin_amdgcn_ballot_w64(!(m >= 0x1p-126f && m <= 0x1.fffffep127f))) {
    if (m < 0x1p-126f) scaled = 0x1p75f;
    if (m > 0x1.fffffep127f) scaled = 0x1p-75f;
    q = 0.0f;
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        x[k][i] *= scaled;
        q = __builtin_fmaf(x[k][i], x[k][i], q);
      }
    r = __builtin_amdgcn_rsqf(__builtin_fmaf(lanes_sum<LANES>(q), inv_d, eps * scaled * scaled));
  }
#pragma unroll
  for (int k = 0; k < NC; ++k)
#pragma unroll
    for (int i = 0; i < kPiece; ++i) x[k][i] *= r;
  return r * scaled;
}

// The weights of this lane's channels of group g; channels behind d get zero.
template <int LANES, int NC, bool WIDE>
__device__ __forceinline__ void load_params(const float* p, float missing, int g, int l, int d, float (&v)[NC][kPiece]) {
  if (p) {
    load_group<float, LANES, NC, WIDE>(p + int64_t(g) * d, l, d, v);
  } else {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[k][i] = channel<LANES, WIDE>(k, i, l) < d ? missing : 0.0f;
  }
}

// A workgroup: `cols` threads side by side (whole groups of LANES lanes) times
// `rows` tokens at a time; thread column cblock * cols + threadIdx % cols is
// group column / LANES, lane column % LANES.  Every thread of a wave runs the
// same number of tokens, those without one of their own on a valid one that
// they do not store, since lane moves need the whole wave.
struct NormShape {
  int lanes, nc, cols, rows, threads;
  int64_t cblocks, tblocks, tokens_each;
};

// The activation of a whole group, chosen once a group (a uniform branch; one
// kernel for every activation).
template <int NC, typename F>
__device__ __forceinline__ void each_act(int act, F f) {
  auto all = [&](auto kind) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) f(c, i, kind);
  };
  if (act == kActSilu) {
    all(std::integral_constant<int, kActSilu>{});
  } else if (act == kActElu1) {
    all(std::integral_constant<int, kActElu1>{});
  } else {
    all(std::integral_constant<int, kActNone>{});
  }
}

template <typename IO, int LANES, int NC, bool WIDE>
__global__ __launch_bounds__(256) void norm_fwd_kernel(const IO* __restrict__ x, Layout lx, const float* __restrict__ weight,
                                                       const float* __restrict__ bias, IO* __restrict__ y, Layout ly, uint32_t tokens,
                                                       int T, Divisor by_T, int G, int d, bool center, int act, float eps, float scale, int cols,
                                                       int rows, int64_t cblocks, int64_t tokens_each) {
  const int64_t tblock = blockIdx.x / cblocks;
  const int col = int(blockIdx.x % cblocks) * cols + int(threadIdx.x) % cols;
  const int mine = int(threadIdx.x) / cols;
  const int l = col % LANES;
  const bool on = col / LANES < G && mine < rows;
  const int g = min(col / LANES, G - 1);
  const float inv_d = 1.0f / float(d);
  float w[NC][kPiece], bs[NC][kPiece];
  load_params<LANES, NC, WIDE>(weight, 1.0f, g, l, d, w);
  load_params<LANES, NC, WIDE>(bias, 0.0f, g, l, d, bs);
  uint32_t want = uint32_t(tblock * tokens_each * rows) + mine;
  float next[NC][kPiece];
  load_group<IO, LANES, NC, WIDE>(x + group_at(lx, min(want, tokens - 1), g, T, by_T, G, d), l, d, next);
  for (int64_t k = 0; k < tokens_each; ++k, want += rows) {
    float v[NC][kPiece];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[c][i] = next[c][i];
    if (k + 1 < tokens_each)
      load_group<IO, LANES, NC, WIDE>(x + group_at(lx, min(want + rows, tokens - 1), g, T, by_T, G, d), l, d, next);
    normalise<LANES, NC, WIDE>(v, l, d, inv_d, center, eps);
    each_act<NC>(act, [&](int c, int i, auto kind) {
      v[c][i] = act_f32<kind()>(__builtin_fmaf(v[c][i], w[c][i], bs[c][i])) * scale;
    });
    if (on && want < tokens) store_group<IO, LANES, NC, WIDE>(y + group_at(ly, want, g, T, by_T, G, d), l, d, v);
  }
}

// A thread's sums of the parameters' gradients go on for kSumTokens tokens, then they
// are added to what it holds in LDS: a float32 sum of n tokens that all have one sign
// is off by up to 64 + n / 64 roundings, not n.  (In registers that would cost a
// wave a SIMD; a row of partial sums every 64 tokens took 12 % longer at 8 x 16384
// tokens of 12 x 128.)
constexpr int kSumTokens = 64;

template <typename IO, int LANES, int NC, bool WIDE>
__global__ __launch_bounds__(256) void norm_bwd_kernel(const IO* __restrict__ x, Layout lx, const float* __restrict__ weight,
                                                       const float* __restrict__ bias, const void* __restrict__ dy, bool dy_bf16, Layout ly,
                                                       float* __restrict__ dx, Layout ldx, float* __restrict__ parts, uint32_t tokens,
                                                       int T, Divisor by_T, int G, int d, bool center, int act, float eps, float scale, int cols,
                                                       int rows, int64_t cblocks, int64_t tokens_each) {
  __shared__ float sums[256 * kPiece];
  extern __shared__ float folded[];          // [2][NC kPiece][threads], where tokens_each > kSumTokens
  const bool folds = parts && tokens_each > kSumTokens;
  const int64_t tblock = blockIdx.x / cblocks;
  const int col = int(blockIdx.x % cblocks) * cols + int(threadIdx.x) % cols;
  const int mine = int(threadIdx.x) / cols;
  const int l = col % LANES;
  const bool on = col / LANES < G && mine < rows;
  const int g = min(col / LANES, G - 1);
  const float inv_d = 1.0f / float(d);
  float w[NC][kPiece], bs[NC][kPiece], dw[NC][kPiece], db[NC][kPiece];
  load_params<LANES, NC, WIDE>(weight, 1.0f, g, l, d, w);
  load_params<LANES, NC, WIDE>(bias, 0.0f, g, l, d, bs);
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < kPiece; ++i) dw[c][i] = db[c][i] = 0.0f;
  // each(f): f(this thread's place, its sum) for all of its sums
  auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        f(folded[(c * kPiece + i) * blockDim.x + threadIdx.x], dw[c][i]);
        f(folded[((NC + c) * kPiece + i) * blockDim.x + threadIdx.x], db[c][i]);
      }
  };
  if (folds) each([](float& held, float&) { held = 0.0f; });
  uint32_t want = uint32_t(tblock * tokens_each * rows) + mine;
  float x_next[NC][kPiece], dy_next[NC][kPiece];
  auto load = [&](uint32_t token) {
    load_group<IO, LANES, NC, WIDE>(x + group_at(lx, token, g, T, by_T, G, d), l, d, x_next);
    const int64_t at_y = group_at(ly, token, g, T, by_T, G, d);
    if (dy_bf16) {
      load_group<bf16_t, LANES, NC, WIDE>(static_cast<const bf16_t*>(dy) + at_y, l, d, dy_next);
    } else {
      load_group<float, LANES, NC, WIDE>(static_cast<const float*>(dy) + at_y, l, d, dy_next);
    }
  };
  load(min(want, tokens - 1));
  for (int64_t k = 0; k < tokens_each; ++k, want += rows) {
    const uint32_t token = min(want, tokens - 1);
    const bool live = on && want < tokens;
    float v[NC][kPiece], dh[NC][kPiece];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        v[c][i] = x_next[c][i];
        dh[c][i] = dy_next[c][i];
      }
    // (large groups have no registers to spare: they load as they go)
    if (NC <= 2 && k + 1 < tokens_each) load(min(want + rows, tokens - 1));
    const float r = normalise<LANES, NC, WIDE>(v, l, d, inv_d, center, eps);
    float s1 = 0.0f, s2 = 0.0f;
    each_act<NC>(act, [&](int c, int i, auto kind) {
      const float p = __builtin_fmaf(v[c][i], w[c][i], bs[c][i]);
      const float dp = live ? dh[c][i] * act_slope_f32<kind()>(p) * scale : 0.0f;
      db[c][i] += dp;
      dw[c][i] = __builtin_fmaf(dp, v[c][i], dw[c][i]);
      dh[c][i] = dp * w[c][i];
      s1 += dh[c][i];
      s2 = __builtin_fmaf(dh[c][i], v[c][i], s2);
    });
    const float m1 = center ? lanes_sum<LANES>(s1) * inv_d : 0.0f;
    const float m2 = lanes_sum<LANES>(s2) * inv_d;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[c][i] = r * (dh[c][i] - m1 - v[c][i] * m2);
    if (live) store_group<float, LANES, NC, WIDE>(dx + group_at(ldx, token, g, T, by_T, G, d), l, d, v);
    if (NC > 2 && k + 1 < tokens_each) load(min(want + rows, tokens - 1));
    if (folds && k % kSumTokens == kSumTokens - 1) {
      each([](float& held, float& sum) {
        held += sum;
        sum = 0.0f;
      });
    }
  }
  if (!parts) return;
  if (folds) each([](float& held, float& sum) { sum += held; });
  // the workgroup's sums over its rows of tokens, in a fixed order: one row of
  // partial sums, [C] of the weights and [C] of the biases
  const int64_t C = int64_t(G) * d;
  float* row = parts + tblock * 2 * C;
  for (int which = 0; which < 2; ++which) {
    for (int c = 0; c < NC; ++c) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPiece; ++i) sums[threadIdx.x * kPiece + i] = which ? db[c][i] : dw[c][i];
      __syncthreads();
      if (on && mine == 0) {
        for (int i = 0; i < kPiece; ++i) {
          const int e = channel<LANES, WIDE>(c, i, l);
          double s = 0.0;
          for (int r = 0; r < rows; ++r) s += sums[(r * cols + int(threadIdx.x)) * kPiece + i];
          if (e < d) row[which * C + int64_t(g) * d + e] = float(s);
        }
      }
    }
  }
}

// Whole pieces of 8 in wide accesses where every group starts on a multiple of
// 16 bytes in x, y and dx.
bool groups_wide(const NormArgs& a) { return a.d % kPiece == 0 && a.x_row % kPiece == 0; }

NormShape norm_shape(const NormArgs& a, bool bwd) {
  NormShape s{};
  const int pieces = (a.d + kPiece - 1) / kPiece;
  s.lanes = 1;
  while (s.lanes < 64 && s.lanes < pieces) s.lanes *= 2;
  s.nc = 1;
  while (s.nc * s.lanes < pieces) s.nc *= 2;
  const int64_t all = int64_t(a.G) * s.lanes;
  // whole rows side by side up to 256 threads, in whole groups
  s.cols = int(std::min<int64_t>(all, 256 / s.lanes * s.lanes));
  s.cblocks = (all + s.cols - 1) / s.cols;
  s.rows = std::max(1, 256 / s.cols);
  s.threads = (s.rows * s.cols + 63) / 64 * 64;
  const int64_t tokens = int64_t(a.B) * a.T;
  // Tokens a thread walks over: workgroups in whole rounds of the 256 CUs.  Forward
  // eight a CU.  The gradients' workgroups each leave a row of partial sums: two a
  // CU (8 x 2048 tokens of one group of 1024: 39 us; 54 at 2.5 a CU, 49 at four), or
  // four where they have fewer than four waves (12 groups of 64, three waves: 31 us;
  // 35 at two).
  const int64_t most = bwd ? (s.threads > 192 ? 512 : 1024) : 2048;
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((tokens + s.rows - 1) / s.rows, std::max<int64_t>(1, most / s.cblocks)));
  s.tokens_each = (tokens + blocks * s.rows - 1) / (blocks * s.rows);
  s.tblocks = s.tokens_each > 0 ? (tokens + s.tokens_each * s.rows - 1) / (s.tokens_each * s.rows) : 0;
  return s;
}

Divisor divisor(uint32_t by) {
  uint32_t shift = 0;
  while ((uint64_t(1) << shift) < by) ++shift;
  const uint64_t magic = ((uint64_t(1) << 32) * ((uint64_t(1) << shift) - by)) / by + 1;
  return {uint32_t(magic), shift};
}

Layout x_layout(const NormArgs& a) { return {a.x_heads, a.x_row}; }
Layout dense(const NormArgs& a, bool heads) { return {heads, int64_t(a.G) * a.d}; }

template <typename IO, int LANES, int NC, bool WIDE>
hipError_t norm_fwd_typed(const NormArgs& a, const NormShape& s, hipStream_t st) {
  norm_fwd_kernel<IO, LANES, NC, WIDE><<<dim3(unsigned(s.tblocks * s.cblocks)), dim3(s.threads), 0, st>>>(
      static_cast<const IO*>(a.x), x_layout(a), a.weight, a.bias, static_cast<IO*>(a.y), dense(a, a.y_heads), uint32_t(int64_t(a.B) * a.T),
      a.T, divisor(a.T), a.G, a.d, a.center, a.act, a.eps, a.scale, s.cols, s.rows, s.cblocks, s.tokens_each);
  return hipGetLastError();
}

template <typename IO, int LANES, int NC, bool WIDE>
hipError_t norm_bwd_typed(const NormArgs& a, const NormShape& s, hipStream_t st) {
  auto* const kernel = norm_bwd_kernel<IO, LANES, NC, WIDE>;
  const size_t lds = (a.dweight || a.dbias) && s.tokens_each > kSumTokens ? size_t(2) * NC * kPiece * s.threads * sizeof(float) : 0;
  if (lds > 32 * 1024) {   // with the 8 KiB of its own past what a launch may take unasked
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3(unsigned(s.tblocks * s.cblocks)), dim3(s.threads), lds, st>>>(
      static_cast<const IO*>(a.x), x_layout(a), a.weight, a.bias, a.dy, a.dy_bf16, dense(a, a.y_heads), a.dx, dense(a, a.x_heads),
      a.dweight || a.dbias ? a.workspace : nullptr, uint32_t(int64_t(a.B) * a.T), a.T, divisor(a.T), a.G, a.d, a.center, a.act, a.eps, a.scale, s.cols, s.rows,
      s.cblocks, s.tokens_each);
  return hipGetLastError();
}

// Calls go(lanes, nc, wide) with compile-time values.
template <typename Go>
hipError_t by_lanes(const NormArgs& a, const NormShape& s, Go go) {
  using std::integral_constant;
  auto wide = [&](auto lanes, auto nc) {
    return groups_wide(a) ? go(lanes, nc, std::true_type{}) : go(lanes, nc, std::false_type{});
  };
  const integral_constant<int, 1> one{};
  switch (s.lanes) {
    case 1: return wide(one, one);
    case 2: return wide(integral_constant<int, 2>{}, one);
    case 4: return wide(integral_constant<int, 4>{}, one);
    case 8: return wide(integral_constant<int, 8>{}, one);
    case 16: return wide(integral_constant<int, 16>{}, one);
    case 32: return wide(integral_constant<int, 32>{}, one);
    default: break;
  }
  const integral_constant<int, 64> all{};
  switch (s.nc) {
    case 1: return wide(all, one);
    case 2: return wide(all, integral_constant<int, 2>{});
    case 4: return wide(all, integral_constant<int, 4>{});
    default: return wide(all, integral_constant<int, 8>{});
  }
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
  const NormShape s = norm_shape(a, false);
  return by_lanes(a, s, [&](auto lanes, auto nc, auto wide) {
    return a.bf16 ? norm_fwd_typed<bf16_t, lanes(), nc(), wide()>(a, s, st) : norm_fwd_typed<float, lanes(), nc(), wide()>(a, s, st);
  });
}

size_t norm_bwd_workspace_bytes(const NormArgs& a) {
  return size_t(norm_shape(a, true).tblocks) * 2 * size_t(a.G) * a.d * sizeof(float);
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st) {
  const NormShape s = norm_shape(a, true);
  hipError_t e = hipSuccess;
  if (s.tblocks > 0) {
    e = by_lanes(a, s, [&](auto lanes, auto nc, auto wide) {
      return a.bf16 ? norm_bwd_typed<bf16_t, lanes(), nc(), wide()>(a, s, st) : norm_bwd_typed<float, lanes(), nc(), wide()>(a, s, st);
    });
  }
  if (e != hipSuccess || (!a.dweight && !a.dbias)) return e;
  const int64_t C = int64_t(a.G) * a.d;
  return launch_sum_parts({a.workspace, s.tblocks, 2 * C, 2 * C, {a.dweight, a.dbias, nullptr}, {C, 2 * C}}, st);
}

}  // namespace falcon
