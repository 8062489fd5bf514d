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
// one to sixteen waves, a piece of 8 channels a thread, from its loads to its stores; a
// thread keeps its channels' weights and walks over rows.  Sums of squares are made in
// double, so that no row of float32 numbers leaves their range.  A group's sum is a sum
// over lanes where a group is 1, 2, 4, ... 64 pieces of 8, else it goes through LDS; a
// whole row's over the row's waves.  Rows are dealt out one after the other to all
// workgroups, which so work on neighbouring memory at a time (8 x 2048 x 768 in bfloat16,
// gradients: 81 us with a run of rows a workgroup, 78 us so; 5555 x 2304: 96 and 81 us).
// Measured there: forward 34 us (176 MB, 5.2 TB/s), gradients 69 us (330 MB, 4.8 TB/s).
//
// In 8 bits, 32 adjacent channels of a row share a step, the smallest power of two of which
// 127 reach the largest of them: a value is off by at most half a step, less than 1/127 of
// the largest (but at the smallest step, 2^-126), and dividing by and multiplying with the step is exact.

#include <algorithm>

#include "falcon_block_device.h"
#include "falcon_launch.h"

namespace falcon {

namespace {

constexpr int kPiece = 8;
constexpr int kBlock = 32;        // channels of one step
// Bytes of gradients from which they are written past the last cache (256 MiB), which would
// hold little of them for their reader.
constexpr int64_t kPastCache = int64_t(128) << 20;
constexpr int kRowsEach = 64;     // rows whose parts of the parameters' gradients one thread sums: float32 sums stay short

// How rows and groups lie on threads.
struct Shape {
  int threads_row, rows_block;       // threads of a row (whole waves), rows of a workgroup at a time
  int64_t blocks;
  int rows_each;                     // rows a thread walks over
  int group_lanes;                   // lanes of a group; 0: through LDS; -1: the group is the row
  size_t lds;
};

// ---- rows; their types are met at run time (a uniform branch a tensor) ---------------
// A thread has 8 channels: a piece of 8 neighbours, read and written at once at whatever
// alignment, or, of rows shorter than that, one element after the other of those a thread
// apart.  A row's last piece may be short: its thread reads the row's last 8 channels, and
// those that are the thread's before it count as absent (rows of whole pieces by a form of
// their own: 76 us against 86 for the gradients of 16384 rows of 768).  Where groups are whole
// pieces (or the row) a piece is one part of a group's sum, else each of its channels is.
enum Form { kElements, kChannels, kRagged, kPieces };
constexpr bool by_piece(int form) { return form >= kRagged; }

template <int FORM>
struct Lane {
  int t, C, threads;      // of the row's threads
  // channels of a piece ahead of the thread's own; 8 or more behind the row's end
  __device__ __forceinline__ int skip() const { return FORM == kPieces ? (t * kPiece < C ? 0 : kPiece) : max(t * kPiece - (C - kPiece), 0); }
  __device__ __forceinline__ int channel(int i) const { return FORM == kElements ? i * threads + t : min(t * kPiece, C - kPiece) + i; }
  __device__ __forceinline__ bool has(int i) const { return FORM == kElements ? channel(i) < C : i >= skip(); }
};

// Whatever the alignment of its elements, a piece is read and written in 16 bytes.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((aligned(2))) u32x4_at2;
typedef u32x4 __attribute__((aligned(4))) u32x4_at4;
typedef u32x2 __attribute__((aligned(1))) u32x2_at1;

template <int FORM>
__device__ __forceinline__ void load_params(const float* p, float missing, const Lane<FORM>& at, float (&v)[kPiece]) {
#pragma unroll
  for (int i = 0; i < kPiece; ++i) v[i] = missing;
  if (!p) return;
  if constexpr (FORM == kElements) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] = at.has(i) ? p[at.channel(i)] : missing;
  } else {
    const u32x4_at4* q = reinterpret_cast<const u32x4_at4*>(p + at.channel(0));
    const u32x4 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] = at.has(i) ? __uint_as_float(i < 4 ? a[i] : b[i - 4]) : missing;
  }
}

// A step's byte is its float32 exponent field; 255, whose step is infinite, with codes of
// zero stands for channels that were not all finite: they come back as NaN.
__device__ __forceinline__ float step_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// A thread's channels of a row as they lie in memory: a row's loads are all under way before
// the first is waited for, which conversions right behind each would do.
template <int FORM>
struct Raw {
  static constexpr bool kPiecewise = FORM != kElements;
  uint32_t w[kPiece];                       // of a piece packed, else a channel each
  uint32_t step[kPiecewise ? 1 : kPiece];   // of 8 bits

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < (kPiecewise ? 1 : kPiece); ++i) step[i] = 0;
  }
  // Threads behind a row's end read its last piece, too: a branch around the loads would be in
  // the way of the sums over lanes behind them.
  __device__ __forceinline__ void fetch(const void* p, bool bf16, int64_t at_row, const Lane<FORM>& at) {
    if constexpr (kPiecewise) {
      if (bf16) {
        const u32x4 a = *reinterpret_cast<const u32x4_at2*>(static_cast<const bf16_t*>(p) + at_row + at.channel(0));
        w[0] = a[0], w[1] = a[1], w[2] = a[2], w[3] = a[3];
      } else {
        const u32x4_at4* q = reinterpret_cast<const u32x4_at4*>(static_cast<const float*>(p) + at_row + at.channel(0));
        const u32x4 a = q[0], b = q[1];
        w[0] = a[0], w[1] = a[1], w[2] = a[2], w[3] = a[3];
        w[4] = b[0], w[5] = b[1], w[6] = b[2], w[7] = b[3];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const int c = at.channel(i);
        if (c < at.C) w[i] = bf16 ? static_cast<const uint16_t*>(p)[at_row + c] : static_cast<const uint32_t*>(p)[at_row + c];
      }
    }
  }
  __device__ __forceinline__ void fetch8(const int8_t* codes, const uint8_t* steps, const Lane<FORM>& at) {
    if constexpr (kPiecewise) {
      const u32x2 a = *reinterpret_cast<const u32x2_at1*>(codes + at.channel(0));
      w[0] = a[0], w[1] = a[1];
      step[0] = steps[min(at.t * kPiece, at.C - 1) / kBlock];
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const int c = at.channel(i);
        if (c < at.C) w[i] = uint8_t(codes[c]), step[i] = steps[c / kBlock];
      }
    }
  }
  // (absent channels: zero)
  __device__ __forceinline__ uint32_t word(int k, const Lane<FORM>& at) const { return FORM == kPieces && at.skip() != 0 ? 0 : w[k]; }
  __device__ __forceinline__ void values(bool bf16, const Lane<FORM>& at, float (&v)[kPiece]) const {
    if (bf16) {
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
        v[i] = __uint_as_float(!kPiecewise ? w[i] << 16 : i % 2 ? word(i / 2, at) & 0xffff0000u : word(i / 2, at) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[i] = __uint_as_float(word(i, at));
    }
    none_absent(at, v);
  }
  __device__ __forceinline__ void values8(const Lane<FORM>& at, float (&v)[kPiece]) const {
    const float size = step_of(FORM == kPieces && at.skip() != 0 ? 0 : step[0]);
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
      v[i] = kPiecewise ? float(int8_t(word(i / 4, at) >> (8 * (i % 4)))) * size : float(int8_t(w[i])) * step_of(step[kPiecewise ? 0 : i]);
    none_absent(at, v);
  }
  __device__ __forceinline__ void none_absent(const Lane<FORM>& at, float (&v)[kPiece]) const {
    if constexpr (kPiecewise && FORM != kPieces) {
      int skip = at.skip();
      asm volatile("" : "+v"(skip));   // (eight comparisons made ahead would fill the scalar registers)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) v[i] = i >= skip ? v[i] : 0.0f;
    }
  }
};

// `past`: past the cache.
__device__ __forceinline__ void store_piece(float* p, const float (&v)[kPiece], bool past) {
  u32x4_at4* const q = reinterpret_cast<u32x4_at4*>(p);
  const u32x4 a = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  const u32x4 b = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
  if (past) {
    asm volatile("");   // (else both ways become one, through the cache)
    __builtin_nontemporal_store(a, q);
    __builtin_nontemporal_store(b, q + 1);
    asm volatile("");
  } else {
    q[0] = a;
    q[1] = b;
  }
}
__device__ __forceinline__ void store_piece(bf16_t* p, const float (&v)[kPiece], bool) {
  *reinterpret_cast<u32x4_at2*>(p) = u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
}
template <int FORM, typename E>
__device__ __forceinline__ void store_typed(E* p, const Lane<FORM>& at, const float (&v)[kPiece], bool past) {
  if (FORM != kElements && at.skip() == 0) {
    store_piece(p + at.channel(0), v, past);
  } else if (FORM == kElements || (FORM != kPieces && at.skip() < kPiece)) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      if (at.has(i)) io<E>::store(p, at.channel(i), v[i]);
    }
  }
}
template <int FORM>
__device__ __forceinline__ void store_row(void* p, bool bf16, int64_t at_row, const Lane<FORM>& at, const float (&v)[kPiece], bool past = false) {
  if (bf16) {
    store_typed<FORM>(static_cast<bf16_t*>(p) + at_row, at, v, past);
  } else {
    store_typed<FORM>(static_cast<float*>(p) + at_row, at, v, past);
  }
}
// ---- 8 bits ---------------------------------------------------------------------------
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

template <int FORM>
__device__ __forceinline__ void pack_row(int8_t* codes, uint8_t* steps, const Lane<FORM>& at, bool on, bool live, const float (&v)[kPiece]) {
  if constexpr (FORM != kElements) {
    uint32_t largest = 0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) largest = max(largest, magnitude(v[i]));
    const uint32_t byte = step_byte(lanes_max<kBlock / kPiece>(largest));
    const float inverse = byte == 255 ? 0.0f : step_of(254 - byte);
    u32x2 w = {0, 0};
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const int code = byte == 255 ? 0 : int(__builtin_rintf(v[i] * inverse));
      w[i / 4] |= (uint32_t(code) & 255u) << (8 * (i % 4));
    }
    if (on && at.skip() < kPiece) {
      if (FORM == kPieces || at.skip() == 0) {
        *reinterpret_cast<u32x2_at1*>(codes + at.channel(0)) = w;
      } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          if (at.has(i)) codes[at.channel(i)] = int8_t(w[i / 4] >> (8 * (i % 4)));
        }
      }
      if (at.t % (kBlock / kPiece) == 0) steps[at.t / (kBlock / kPiece)] = live ? uint8_t(byte) : 0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      const uint32_t byte = step_byte(lanes_max<kBlock>(magnitude(v[i])));
      const int c = at.channel(i);
      if (on && c < at.C) {
        codes[c] = byte == 255 ? int8_t(0) : int8_t(int(__builtin_rintf(v[i] * step_of(254 - byte))));
        if (c % kBlock == 0) steps[c / kBlock] = live ? uint8_t(byte) : 0;
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

// The sums of one row over its groups, of each thread's parts.  The result is in place: each
// part's group's sum.
// Every thread of the workgroup takes part.
template <int FORM>
struct Sums {
  static constexpr int kParts = by_piece(FORM) ? 1 : kPiece;
  double* lds;            // of this row: [3 slots][2 turns][2 sums][waves], then [items + G] where groups go through it
  int lanes, G, d, waves; // Shape::group_lanes; the row's waves

  // One sum over the row, or two at once.  Rounds with the same `slot` must have another barrier
  // between them; `turn` alternates.
  template <bool BOTH>
  __device__ __forceinline__ void row(double& a, double& b, int slot, int turn, const Lane<FORM>& at) const {
    a = lanes_sum(a, 64);
    if constexpr (BOTH) b = lanes_sum(b, 64);
    if (waves > 1) {
      double* const mine = lds + (slot * 2 + turn) * 2 * waves;
      const int w = at.t / 64;
      if (at.t % 64 == 0) {
        mine[w] = a;
        if constexpr (BOTH) mine[waves + w] = b;
      }
      __syncthreads();
      a = b = 0.0;
      for (int k = 0; k < waves; ++k) {
        a += mine[k];
        if constexpr (BOTH) b += mine[waves + k];
      }
    }
  }
  __device__ __forceinline__ void groups(double (&part)[kParts], int slot, int turn, const Lane<FORM>& at) const {
    if (lanes < 0) {
      double all = 0.0, none = 0.0;
#pragma unroll
        for (int i = 0; i < kParts; ++i) all += part[i];
      row<false>(all, none, slot, turn, at);
#pragma unroll
        for (int i = 0; i < kParts; ++i) part[i] = all;
    } else if (by_piece(FORM) && lanes > 0) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) part[i] = lanes_sum(part[i], lanes);
    } else {
      constexpr int kUnit = by_piece(FORM) ? kPiece : 1;
      const int items = at.C / kUnit, each = d / kUnit;
      double* const item = lds + 12 * waves;
      double* const sum = item + items;
      __syncthreads();    // the last round's sums have been read
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          if (at.has(i)) item[at.channel(i) / kUnit] = part[i];
        }
      __syncthreads();
      // a wave a group at a time
      for (int g = at.t / 64; g < G; g += waves) {
        double s = 0.0;
        for (int j = at.t % 64; j < each; j += 64) s += item[g * each + j];
        s = lanes_sum(s, 64);
        if (at.t % 64 == 0) sum[g] = s;
      }
      __syncthreads();
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          part[i] = at.has(i) ? sum[at.channel(i) / d] : 0.0;
        }
    }
  }
};

// f(i) for every channel of a thread, with the activation's number as a constant.
template <typename F>
__device__ __forceinline__ void each_channel(int act, F f) {
  auto all = [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) f(i, kind);
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

// Zeros behind a sequence's end, also where a weight is not finite.
__device__ __forceinline__ void none_behind(const RowAt& r, float (&v)[kPiece]) {
  if (!r.live) {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] = 0.0f;
  }
}

// A workgroup's rows: LDS of each, and which is this thread's.
template <int FORM>
struct Block {
  Lane<FORM> at;
  Sums<FORM> sums;
  int rows, mine, row_lds;   // row_lds: doubles
  __device__ __forceinline__ Block(const ResidualArgs& a, int threads_row, int group_lanes, double* lds) {
    const int C = a.G * a.d, waves = threads_row / 64;
    row_lds = waves * 12 + (group_lanes == 0 ? C / (by_piece(FORM) ? kPiece : 1) + a.G : 0);
    rows = int(blockDim.x) / threads_row;
    mine = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / threads_row);
    at = {int(threadIdx.x) - mine * threads_row, C, threads_row};
    sums = {lds + mine * row_lds, group_lanes, a.G, a.d, waves};
  }
};

template <int MOST, int FORM>
__global__ __launch_bounds__(MOST, (FORM == kElements ? 2 : 4)) void residual_fwd_kernel(ResidualArgs a, int threads_row, int rows_each, int group_lanes) {
  using S = Sums<FORM>;
  extern __shared__ double lds[];
  const int C = a.G * a.d;
  const Block<FORM> block(a, threads_row, group_lanes, lds);
  const Lane<FORM>& at = block.at;
  const S& sums = block.sums;
  const int mine = block.mine, rows = block.rows;
  const double inv_d = 1.0 / a.d, inv_C = 1.0 / C;
  float aw[kPiece], wn[kPiece];
  load_params<FORM>(a.alpha, 1.0f, at, aw);
  load_params<FORM>(a.post ? a.post_weight : nullptr, 1.0f, at, wn);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) aw[i] *= wn[i];
  load_params<FORM>(a.pre_weight, 1.0f, at, wn);
  const int64_t first = int64_t(blockIdx.x) * rows + mine, stride = int64_t(gridDim.x) * rows;
  Raw<FORM> yr, hr, ur;
  auto fetch = [&](const RowAt& r) {
    yr.clear(), hr.clear(), ur.clear();
    if (r.live) {
      yr.fetch(a.y, a.bf16, r.row * a.y_row, at);
      if (a.h) hr.fetch(a.h, a.stream_bf16, r.row * C, at);
      if (a.gate) ur.fetch(a.gate, a.bf16, r.row * a.gate_row, at);
    }
  };
  RowAt next = row_at(first, a);
  fetch(next);
  for (int it = 0; it < rows_each; ++it) {
    const RowAt r = next;
    float y[kPiece], h[kPiece], u[kPiece];
    yr.values(a.bf16, at, y);
    hr.values(a.stream_bf16, at, h);
    ur.values(a.bf16, at, u);
    if (it + 1 < rows_each) {
      next = row_at(r.row + stride, a);
      fetch(next);
    }
    if (a.save) {
      const int64_t blocks = (C + kBlock - 1) / kBlock;
      pack_row<FORM>(a.y_codes + r.row * C, a.y_steps + r.row * blocks, at, r.live || (r.inside && a.zero_behind), r.live, y);
      if (a.gate) pack_row<FORM>(a.gate_codes + r.row * C, a.gate_steps + r.row * blocks, at, r.live || (r.inside && a.zero_behind), r.live, u);
    }
    if (a.post) {
      double part[S::kParts];
#pragma unroll
      for (int i = 0; i < S::kParts; ++i) part[i] = 0.0;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) part[by_piece(FORM) ? 0 : i] = __builtin_fma(double(y[i]), double(y[i]), part[by_piece(FORM) ? 0 : i]);
      sums.groups(part, 0, it & 1, at);
      Inverse inv;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        if (!by_piece(FORM) || i == 0) inv = inverse_root(__builtin_fma(part[by_piece(FORM) ? 0 : i], inv_d, double(a.eps)));
        y[i] = inv.times(y[i]);
      }
    }
    if (a.gate) {
      each_channel(a.act, [&](int i, auto kind) { y[i] *= act_f32<kind()>(u[i]); });
    }
    double squares = 0.0, none = 0.0;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        h[i] = __builtin_fmaf(aw[i], y[i], h[i]);
        // (absent groups of zeros are not finite with eps = 0)
        const double x = (by_piece(FORM) ? at.skip() < kPiece : at.has(i)) ? double(h[i]) : 0.0;
        squares = __builtin_fma(x, x, squares);
      }
    const bool cleared = r.inside && !r.live && a.zero_behind;
    if (cleared) none_behind(r, h);
    if (r.live || cleared) store_row<FORM>(a.h_out, a.stream_bf16, r.row * C, at, h);
    if (a.pre) {
      sums.template row<false>(squares, none, 1, it & 1, at);
      const Inverse inv = inverse_root(__builtin_fma(squares, inv_C, double(a.eps)));
#pragma unroll
        for (int i = 0; i < kPiece; ++i) h[i] = inv.times(h[i]) * wn[i];
      none_behind(r, h);
      if (r.live || cleared) store_row<FORM>(a.n, a.bf16, r.row * C, at, h);
    }
  }
}

template <int MOST, int FORM>
__global__ __launch_bounds__(MOST, (by_piece(FORM) ? 4 : FORM == kChannels ? 3 : 2)) void residual_bwd_kernel(ResidualArgs a, int threads_row, int rows_each, int group_lanes, float* parts) {
  using S = Sums<FORM>;
  extern __shared__ double lds[];
  const int C = a.G * a.d;
  const Block<FORM> block(a, threads_row, group_lanes, lds);
  const Lane<FORM>& at = block.at;
  const S& sums = block.sums;
  const int mine = block.mine, rows = block.rows;
  const double inv_d = 1.0 / a.d, inv_C = 1.0 / C;
  float aw[kPiece], wn[kPiece], A[kPiece], N[kPiece];
  load_params<FORM>(a.alpha, 1.0f, at, aw);
  load_params<FORM>(a.post ? a.post_weight : nullptr, 1.0f, at, wn);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      aw[i] *= wn[i];
      A[i] = N[i] = 0.0f;
    }
  load_params<FORM>(a.pre_weight, 1.0f, at, wn);
  // Of pieces the weights wait in LDS, [4][threads of a row] of 16 bytes: their registers are
  // what four waves a SIMD lack.
  float4* const weights = reinterpret_cast<float4*>(lds + (rows * block.row_lds + 1) / 2 * 2) + at.t;
  if constexpr (by_piece(FORM)) {
    if (mine == 0) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        weights[q * threads_row] = make_float4(aw[4 * q], aw[4 * q + 1], aw[4 * q + 2], aw[4 * q + 3]);
        weights[(2 + q) * threads_row] = make_float4(wn[4 * q], wn[4 * q + 1], wn[4 * q + 2], wn[4 * q + 3]);
      }
    }
    __syncthreads();
  }
  auto weights_at = [&](int first, float (&v)[kPiece]) {
    if constexpr (by_piece(FORM)) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 x = weights[(first + q) * threads_row];
        v[4 * q] = x.x, v[4 * q + 1] = x.y, v[4 * q + 2] = x.z, v[4 * q + 3] = x.w;
      }
    }
  };
  // (with inputs from memory: gradients of 16384 rows of 768, 151 MB, 85.5 us past the cache,
  // 87.5 us through it; with the forward ahead of them, 122 and 128 us)
  const bool past_cache = int64_t(a.B) * a.T * C * (1 + (a.dgate != nullptr) + (a.dh != nullptr)) * 4 > kPastCache;
  const int64_t blocks = (C + kBlock - 1) / kBlock;
  const int64_t first = int64_t(blockIdx.x) * rows + mine, stride = int64_t(gridDim.x) * rows;
  Raw<FORM> yr, ur, Dr, hr, tr;
  const bool gated = a.gate || a.gate_codes;
  auto fetch = [&](const RowAt& r) {
    yr.clear(), ur.clear(), Dr.clear(), hr.clear(), tr.clear();
    if (r.live) {
      if (a.save) {
        yr.fetch8(a.y_codes + r.row * C, a.y_steps + r.row * blocks, at);
        if (gated) ur.fetch8(a.gate_codes + r.row * C, a.gate_steps + r.row * blocks, at);
      } else {
        yr.fetch(a.y, a.bf16, r.row * a.y_row, at);
        if (gated) ur.fetch(a.gate, a.bf16, r.row * a.gate_row, at);
      }
      if (a.pre) {
        hr.fetch(a.h_out, a.stream_bf16, r.row * C, at);
        tr.fetch(a.dn, a.dn_bf16, r.row * C, at);
      }
      if (a.dh_out) Dr.fetch(a.dh_out, a.dh_out_bf16, r.row * C, at);
    }
  };
  for (int it = 0; it < rows_each; ++it) {
    const RowAt r = row_at(first + int64_t(it) * stride, a);
    fetch(r);
    float y[kPiece], u[kPiece], D[kPiece], h[kPiece], t[kPiece];
    if (a.save) {
      yr.values8(at, y);
      ur.values8(at, u);
    } else {
      yr.values(a.bf16, at, y);
      ur.values(a.bf16, at, u);
    }
    Dr.values(a.dh_out_bf16, at, D);
    hr.values(a.stream_bf16, at, h);
    tr.values(a.dn_bf16, at, t);
    if (a.pre) {
      weights_at(2, wn);
      double squares = 0.0, dots = 0.0;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          const double x = double(h[i]);
          squares = __builtin_fma(x, x, squares);
          dots = __builtin_fma(x, double(t[i] * wn[i]), dots);
        }
      sums.template row<true>(squares, dots, 0, it & 1, at);
      // (a row that is not there is zero throughout, whatever eps)
      const Inverse inv = inverse_root(r.live ? __builtin_fma(squares, inv_C, double(a.eps)) : 1.0);
      const float mean = float(dots * inv_C * double(inv.power) * double(inv.rest)), whole = inv.whole();
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          const float hhat = inv.times(h[i]);
          N[i] = __builtin_fmaf(t[i], hhat, N[i]);
          D[i] = __builtin_fmaf(whole, __builtin_fmaf(-hhat, mean, t[i] * wn[i]), D[i]);
        }
    }
    none_behind(r, D);
    if (a.dh && r.inside) store_row<FORM>(a.dh, false, r.row * C, at, D, past_cache);
    weights_at(0, aw);
    // D becomes D f, and dgate is made next to it
    Inverse inv[S::kParts];
    if (a.post) {
      double part[S::kParts];
#pragma unroll
      for (int i = 0; i < S::kParts; ++i) part[i] = 0.0;
#pragma unroll
      for (int i = 0; i < kPiece; ++i) part[by_piece(FORM) ? 0 : i] = __builtin_fma(double(y[i]), double(y[i]), part[by_piece(FORM) ? 0 : i]);
      sums.groups(part, 1, it & 1, at);
#pragma unroll
      for (int i = 0; i < S::kParts; ++i) inv[i] = inverse_root(r.live ? __builtin_fma(part[i], inv_d, double(a.eps)) : 1.0);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) y[i] = inv[by_piece(FORM) ? 0 : i].times(y[i]);
    }
    if (a.dgate) {
      each_channel(a.act, [&](int i, auto kind) {
        const float x = u[i];
        u[i] = D[i] * aw[i] * y[i] * act_slope_f32<kind()>(x);
        D[i] *= act_f32<kind()>(x);
      });
      none_behind(r, u);
      if (r.inside) store_row<FORM>(a.dgate, false, r.row * C, at, u, past_cache);
    }
    double part[S::kParts];
#pragma unroll
    for (int i = 0; i < S::kParts; ++i) part[i] = 0.0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      A[i] = __builtin_fmaf(D[i], y[i], A[i]);
      D[i] *= aw[i];
      part[by_piece(FORM) ? 0 : i] = __builtin_fma(double(D[i]), double(y[i]), part[by_piece(FORM) ? 0 : i]);
    }
    if (a.post) {
      sums.groups(part, 2, it & 1, at);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          const Inverse& v = inv[by_piece(FORM) ? 0 : i];
          D[i] = v.whole() * __builtin_fmaf(-y[i], float(part[by_piece(FORM) ? 0 : i] * inv_d), D[i]);
        }
    }
    none_behind(r, D);
    if (r.inside) store_row<FORM>(a.dy, false, r.row * C, at, D, past_cache);
  }
  if (!parts) return;
  // the workgroup's sums over its rows, in a fixed order: one row of partial sums, [C]
  // each of alpha, post_weight and pre_weight
  float* const out = parts + int64_t(blockIdx.x) * 3 * C;
  float* const shared = reinterpret_cast<float*>(lds);   // [threads][kPiece]
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPiece; ++i) shared[threadIdx.x * kPiece + i] = which ? N[i] : A[i];
    __syncthreads();
    if (mine == 0) {
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        const int c = at.channel(i);
        if (at.has(i)) {
          double s = 0.0;
          for (int m = 0; m < rows; ++m) s += shared[(m * threads_row + at.t) * kPiece + i];
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

Form form_of(const ResidualArgs& a) {
  const int C = a.G * a.d;
  if (C < kPiece) return kElements;
  if (a.post && a.G > 1 && a.d % kPiece != 0) return kChannels;
  return C % kPiece == 0 ? kPieces : kRagged;
}

Shape shape_of(const ResidualArgs& a, bool bwd) {
  Shape s{};
  const int C = a.G * a.d;
  s.threads_row = (C + 64 * kPiece - 1) / (64 * kPiece) * 64;
  s.rows_block = std::max(1, 256 / s.threads_row);
  const int64_t rows = int64_t(a.B) * a.T;
  // as many workgroups as the CUs hold at a time, at three or four waves a SIMD: one more round of a
  // few costs what a whole one does (5555 rows of 2304, five waves each, gradients: 72 us
  // with two a CU, 96 us with three; forward 8001 rows 62 and 75 us).  Workgroups of three waves fit
  // five times: forward, 16384 rows from memory, of 1536 70.5 us and 72 with four, of 1280 60 and 64, of 1100
  // 64 and 69; but gradients of 8192 rows of 1536 76 us and 74 with four.
  const int waves = s.rows_block * s.threads_row / 64, simd = bwd && !by_piece(form_of(a)) ? 3 : 4;
  const int64_t most = 256 * (waves == 3 && !bwd ? 5 : std::max(1, simd / ((waves + 3) / 4)));
  const int64_t each = std::max<int64_t>(1, (rows + most * s.rows_block - 1) / (most * s.rows_block));
  s.rows_each = int(bwd ? std::min<int64_t>(each, kRowsEach) : each);
  s.blocks = (rows + int64_t(s.rows_each) * s.rows_block - 1) / (int64_t(s.rows_each) * s.rows_block);
  const bool pieces = by_piece(form_of(a));
  const int lanes = a.d / kPiece;
  s.group_lanes = a.G == 1 || !a.post ? -1 : pieces && lanes <= 64 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  const size_t row = size_t(s.threads_row / 64) * 12 + (s.group_lanes == 0 ? size_t(pieces ? C / kPiece : C) + a.G : 0);
  s.lds = s.rows_block * row * sizeof(double);
  if (bwd && pieces) s.lds = (s.lds + 15) / 16 * 16 + size_t(s.threads_row) * 4 * sizeof(float4);   // the weights
  if (bwd) s.lds = std::max(s.lds, size_t(s.rows_block) * s.threads_row * kPiece * sizeof(float));
  return s;
}

// Calls go(most threads, form) with compile-time values.  Four waves a SIMD, 128 registers a
// thread, is what a workgroup of 1024 threads has and what the forms of pieces are held to, so
// these come for any width at once; the gradients of channels take 167 where three waves a
// SIMD do (12 of them in memory, 56 at 128).
template <bool BWD, typename Go>
hipError_t by_shape(const ResidualArgs& a, const Shape& s, Go go) {
  using std::integral_constant;
  switch (form_of(a)) {
    case kElements: return go(integral_constant<int, 256>{}, integral_constant<int, kElements>{});
    case kChannels:
      if constexpr (BWD) {
        if (s.threads_row <= 512) return go(integral_constant<int, 512>{}, integral_constant<int, kChannels>{});
      }
      return go(integral_constant<int, 1024>{}, integral_constant<int, kChannels>{});
    case kRagged: return go(integral_constant<int, 1024>{}, integral_constant<int, kRagged>{});
    default: return go(integral_constant<int, 1024>{}, integral_constant<int, kPieces>{});
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
  return by_shape<false>(a, s, [&](auto most, auto form) {
    auto* const kernel = residual_fwd_kernel<most(), form()>;
    const hipError_t e = allow_lds(kernel, s.lds);
    if (e != hipSuccess) return e;
    kernel<<<dim3(unsigned(s.blocks)), dim3(s.threads_row * s.rows_block), s.lds, st>>>(a, s.threads_row, s.rows_each, s.group_lanes);
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
    const hipError_t e = by_shape<true>(a, s, [&](auto most, auto form) {
      auto* const kernel = residual_bwd_kernel<most(), form()>;
      const hipError_t e = allow_lds(kernel, s.lds);
      if (e != hipSuccess) return e;
      kernel<<<dim3(unsigned(s.blocks)), dim3(s.threads_row * s.rows_block), s.lds, st>>>(a, s.threads_row, s.rows_each, s.group_lanes, params ? a.workspace : nullptr);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (!params) return hipSuccess;
  const int64_t C = int64_t(a.G) * a.d;
  return launch_sum_parts({a.workspace, s.blocks, 3 * C, 3 * C, {a.dalpha, a.dpost_weight, a.dpre_weight}, {C, 2 * C}}, st);
}

}  // namespace falcon
