// Linear attention with a decay for each head, a tile of chunks a workgroup
// (gfx950, MFMA).
//
// With a = exp(log_decay) of a head and chunks of 64 tokens (n in the last one),
// token s of a chunk and the state S that enters it:
//
//   o_s   = read ( a^(s + 1) S^T q_s + write sum_(r <= s) a^(s - r) (q_s . k_r) v_r )
//   S'    = a^n S + write sum_s a^(n - 1 - s) k_s v_s^T
//
// A sweep against time (REV) starts at a sequence's end and carries the state's
// adjoint, already decayed to the token before the chunk:
//
//   o_s   = read ( a^(n - 1 - s) R^T q_s + write sum_(r >= s) a^(r - s) (q_s . k_r) v_r )
//   R'    = a^n R + write sum_s a^(s + 1) k_s v_s^T
//
// so that the three gradients are sweeps of the same kernel: dq = (dO, v, k)
// forward, dk = (v, dO, q) and dv = (k, q, dO) against time.
//
// Wave w works on the 16 tokens of row block w % 4 and, with eight waves, on every
// second block of 16 output columns.  Its scores come out of the matrix unit
// transposed (keys by queries), which is what the next product takes as its
// second operand, so they never leave the registers; keys and values lie in LDS
// as they came and are turned on the way out (transposing reads for bfloat16).
// Wave w owns columns w, w + WAVES, ... of 16 of the state, in float32
// registers, and leaves it in LDS as operand fragments for all waves.
//
// bfloat16 inputs enter the products as they are.  What is float32 (decayed
// scores, states, decayed values) enters as a sum of bfloat16 terms, which keep 8
// bits each: two for results in bfloat16 (2^-17 of the operand is lost, against
// 2^-9 in the result), three where they are float32 and for the state.  float32
// inputs use the float32 matrix instruction throughout.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "falcon_block.h"
#include "falcon_block_device.h"
#include "falcon_mfma_frag.h"

namespace falcon {
namespace linear {

using frag::bf16x8;
using frag::f32x4;
using frag::s16x4;

constexpr int kChunk = 64;

// ---- operands: eight values a lane of a 32-wide block of the summed axis ---------
struct f32x8 {
  f32x4 lo, hi;
};
template <int N>
struct Terms {
  bf16x8 t[N];
};

// The exact operand of an input, and the operand of float32 values.
template <typename IO, int TERMS>
struct Operands;
template <int TERMS>
struct Operands<bf16_t, TERMS> {
  using Exact = bf16x8;
  using Split = Terms<TERMS>;
};
template <int TERMS>
struct Operands<float, TERMS> {
  using Exact = f32x8;
  using Split = f32x8;
};

template <int N>
__device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Terms<N>& out) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    bf16x8 t;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t[e] = static_cast<__bf16>(lo[e]);
      t[e + 4] = static_cast<__bf16>(hi[e]);
      lo[e] -= static_cast<float>(t[e]);
      hi[e] -= static_cast<float>(t[e + 4]);
    }
    out.t[n] = t;
  }
}
__device__ __forceinline__ void split(f32x4 lo, f32x4 hi, f32x8& out) { out = {lo, hi}; }

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) { return frag::mfma32(a, b, c); }
template <int N>
__device__ __forceinline__ f32x4 mma(bf16x8 a, const Terms<N>& b, f32x4 c) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n) c = frag::mfma32(a, b.t[n], c);
  return c;
}
template <int N>
__device__ __forceinline__ f32x4 mma(const Terms<N>& a, bf16x8 b, f32x4 c) {
#pragma unroll
  for (int n = N - 1; n >= 0; --n) c = frag::mfma32(a.t[n], b, c);
  return c;
}
// v_mfma_f32_16x16x4_f32 sums one value of each of the four lane groups, so eight
// of them make the 32-wide block.
__device__ __forceinline__ f32x4 mma(const f32x8& a, const f32x8& b, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo[e], b.lo[e], c, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi[e], b.hi[e], c, 0, 0, 0);
  return c;
}

// ---- staged rows ------------------------------------------------------------------
// 64 rows of max(D, 32) elements (the columns behind D hold zero) and 16 bytes
// between rows, which spreads 16 rows' reads over the banks.
template <typename IO, int D>
struct Stage {
  static constexpr int kWidth = D < 32 ? 32 : D;
  static constexpr int kPitch = kWidth + 16 / int(sizeof(IO));
  static constexpr int kBytes = kChunk * kPitch * int(sizeof(IO));
};

// A row's eight values 32 b + 8 g .. + 7 of its columns.
template <int PITCH>
__device__ __forceinline__ bf16x8 row_frag(const bf16_t* rows, int row, int b, int g) {
  return *reinterpret_cast<const bf16x8*>(rows + row * PITCH + 32 * b + 8 * g);
}
template <int PITCH>
__device__ __forceinline__ f32x8 row_frag(const float* rows, int row, int b, int g) {
  const f32x4* p = reinterpret_cast<const f32x4*>(rows + row * PITCH + 32 * b + 8 * g);
  return {p[0], p[1]};
}

__device__ __forceinline__ s16x4 read_turned(const bf16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
}
// Tokens {32 m + 4 g .. + 3, 32 m + 16 + 4 g .. + 3} (the order in which stacked
// result tiles hold them) of one column a lane: column first + step (l / 4) + l % 4
// of lane l < 16 of a group.  The transposing read takes from each lane the address
// of four neighbours and gives lane l the element l % 4 of segment l / 4 of four rows.
template <int PITCH>
__device__ __forceinline__ bf16x8 turned_frag(const bf16_t* rows, int m, int first, int step, int g, int c16) {
  const bf16_t* p = rows + (32 * m + 4 * g + (c16 >> 2)) * PITCH + first + step * (c16 & 3);
  const s16x4 lo = read_turned(p), hi = read_turned(p + 16 * PITCH);
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int PITCH>
__device__ __forceinline__ f32x8 turned_frag(const float* rows, int m, int first, int step, int g, int c16) {
  const float* p = rows + (32 * m + 4 * g) * PITCH + first + step * (c16 >> 2) + (c16 & 3);
  f32x8 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v.lo[e] = p[e * PITCH];
    v.hi[e] = p[(16 + e) * PITCH];
  }
  return v;
}

__device__ __forceinline__ f32x4 widened(bf16x8 v, int half) {
  f32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = static_cast<float>(v[4 * half + e]);
  return r;
}
__device__ __forceinline__ f32x4 widened(const f32x8& v, int half) { return half ? v.hi : v.lo; }

// A chunk's rows on the way from memory to LDS, 16 bytes a thread and access.
template <typename IO, int D, int THREADS>
struct Rows {
  static constexpr int kEach = 16 / int(sizeof(IO));        // elements of an access
  static constexpr int kSegs = D / kEach;                    // accesses of a row
  static constexpr int kAll = kChunk * kSegs;
  static constexpr int kMine = (kAll + THREADS - 1) / THREADS;
  uint4 r[kMine];

  // Rows behind the chunk's n tokens are not read: their threads take the last one.
  __device__ __forceinline__ void fetch(const IO* first, int64_t t_step, int n, int tid) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int piece = tid + i * THREADS;
      const int row = min(piece / kSegs, n - 1), seg = piece % kSegs;
      r[i] = *reinterpret_cast<const uint4*>(first + row * t_step + seg * kEach);
    }
  }
  __device__ __forceinline__ void store(IO* rows, int n, int tid) const {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int piece = tid + i * THREADS;
      const int row = piece / kSegs, seg = piece % kSegs;
      if (kAll % THREADS == 0 || piece < kAll)
        *reinterpret_cast<uint4*>(rows + row * Stage<IO, D>::kPitch + seg * kEach) = row < n ? r[i] : make_uint4(0, 0, 0, 0);
    }
  }
};

// a^n, with a^0 = 1 for every a.
__device__ __forceinline__ float power(float log2_a, int n) {
  return n == 0 ? 1.0f : __builtin_amdgcn_exp2f(log2_a * float(n));
}

template <int DV>
constexpr int waves() {
  // eight where the state of 128 columns would not fit a wave's registers next to the rest
  return DV >= 128 ? 8 : 4;
}
// LDS: keys, values and, for outputs, the state as fragments.
template <typename IO, int DK, int DV, int TERMS, bool OUT>
constexpr int lds_bytes() {
  const int frags = sizeof(IO) == 2 ? TERMS * 16 : 32;
  return Stage<IO, DK>::kBytes + Stage<IO, DV>::kBytes + (OUT ? (DV / 16) * (Stage<IO, DK>::kWidth / 32) * 64 * frags : 0);
}

__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store4(bf16_t* p, f32x4 v) { frag::store_half(reinterpret_cast<uint16_t*>(p), v); }

// OUT false: only what the tile's chunks add to a state, from zero, into the tile's slot.
template <typename IO, typename O, int DK, int DV, bool OUT>
__global__ __launch_bounds__(64 * waves<DV>()) void sweep_kernel(LinearSweep s) {
  constexpr int kTerms = sizeof(O) == 2 ? 2 : 3;
  constexpr int kWaves = waves<DV>(), kThreads = 64 * kWaves, kHalves = kWaves / 4;
  constexpr int kB = Stage<IO, DK>::kWidth / 32;           // 32-wide blocks of the key axis
  constexpr int kCols = DV / 16;                           // 16-wide blocks of the value axis
  constexpr int kOwn = (kCols + kWaves - 1) / kWaves;      // of these, a wave's part of the state
  constexpr int kPk = Stage<IO, DK>::kPitch, kPv = Stage<IO, DV>::kPitch;
  using Ops = Operands<IO, kTerms>;
  using Exact = typename Ops::Exact;
  using Split = typename Ops::Split;
  using Written = typename Operands<IO, 3>::Split;

  extern __shared__ __attribute__((aligned(16))) char lds[];
  IO* const ks = reinterpret_cast<IO*>(lds);
  IO* const vs = reinterpret_cast<IO*>(lds + Stage<IO, DK>::kBytes);
  Split* const ss = reinterpret_cast<Split*>(lds + Stage<IO, DK>::kBytes + Stage<IO, DV>::kBytes);

  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, c16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rw = w & 3, half = w >> 2;
  const int64_t bh = blockIdx.x / s.tiles;
  const int tile = int(blockIdx.x % s.tiles);
  const int b = int(bh / s.H), h = int(bh % s.H);
  const int len = tokens_of(s.lengths, b, s.T);
  const int first = tile * s.chunks * kChunk;
  const int chunks = min((len - first + kChunk - 1) / kChunk, s.chunks);
  const float e = s.log_decay[h] * kLog2e;

  const IO* const K = static_cast<const IO*>(s.k) + b * s.k_at.b + h * s.k_at.h + first * s.k_at.t;
  const IO* const V = static_cast<const IO*>(s.v) + b * s.v_at.b + h * s.v_at.h + first * s.v_at.t;
  const IO* const Q = OUT ? static_cast<const IO*>(s.q) + b * s.q_at.b + h * s.q_at.h + first * s.q_at.t : nullptr;
  O* const out = OUT ? static_cast<O*>(s.out) + b * s.out_at.b + h * s.out_at.h + first * s.out_at.t : nullptr;
  float* const slot = s.slots ? s.slots + (bh * s.slots_each + s.slot0 + tile) * (DK * DV) : nullptr;

  // A state's element (f, c) at f sf + c sc.  Rows 32 b + 8 g + 4 t + r of column
  // 16 cb + c16 lie in S[.][b][t][r]: two tiles stacked are eight neighbours of the
  // key axis, as a row of queries is read.
  f32x4 S[kOwn][kB][2];
  const float* const from = OUT ? (slot ? slot : s.start ? s.start + bh * (DK * DV) : nullptr) : nullptr;
#pragma unroll
  for (int j = 0; j < kOwn; ++j)
#pragma unroll
    for (int bb = 0; bb < kB; ++bb)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        S[j][bb][t] = frag::zero4();
        const int f = 32 * bb + 8 * g + 4 * t, cb = w + j * kWaves;
        if (OUT && from && cb < kCols && f < DK)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[j][bb][t][r] = from[(f + r) * s.sf + (16 * cb + c16) * s.sc];
      }
  auto keep = [&](float* to) {
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
#pragma unroll
      for (int bb = 0; bb < kB; ++bb)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int f = 32 * bb + 8 * g + 4 * t, cb = w + j * kWaves;
          if (cb < kCols && f < DK)
#pragma unroll
            for (int r = 0; r < 4; ++r) to[(f + r) * s.sf + (16 * cb + c16) * s.sc] = S[j][bb][t][r];
        }
  };
  if (chunks <= 0) {   // nothing of the sequence is left for this tile
    if constexpr (OUT) {
      if (s.last) keep(s.last + bh * (DK * DV));
    }
    return;
  }
  // The state as the first operand S^T of the read, for every wave.
  auto publish = [&]() {
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
#pragma unroll
      for (int bb = 0; bb < kB; ++bb) {
        const int cb = w + j * kWaves;
        if (cb < kCols) {
          Split t;
          split(S[j][bb][0], S[j][bb][1], t);
          ss[(cb * kB + bb) * 64 + l] = t;
        }
      }
  };
  if constexpr (DK < 32) {
    for (int i = tid; i < kChunk * kPk; i += kThreads) ks[i] = IO{};
    __syncthreads();
  }
  // Decays between this lane's query token i = 16 rw + c16 and the keys of its score
  // rows, 16 sb + 4 g + r; of the entering state at token i; of this lane's tokens
  // 32 m + 16 u + 4 g + r at the chunk's end (a whole chunk's).
  f32x4 mask[OUT ? 4 : 1];
  const int i = 16 * rw + c16;
  if constexpr (OUT) {
#pragma unroll
    for (int sb = 0; sb < 4; ++sb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int gap = s.rev ? 16 * sb + 4 * g + r - i : i - (16 * sb + 4 * g + r);
        mask[sb][r] = gap >= 0 ? power(e, max(gap, 0)) * s.write : 0.0f;
      }
  }
  f32x4 to_end[2][2];
  auto ends = [&](int n) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 32 * m + 16 * u + 4 * g + r;
          to_end[m][u][r] = power(e, s.rev ? min(t + 1, n) : max(n - 1 - t, 0)) * s.write;
        }
  };
  ends(kChunk);

  Rows<IO, DK, kThreads> kr;
  Rows<IO, DV, kThreads> vr;
  auto chunk_at = [&](int step) { return s.rev ? chunks - 1 - step : step; };
  auto tokens_in = [&](int c) { return min(len - first - c * kChunk, kChunk); };
  {
    const int c = chunk_at(0), n = tokens_in(c);
    kr.fetch(K + int64_t(c) * kChunk * s.k_at.t, s.k_at.t, n, tid);
    vr.fetch(V + int64_t(c) * kChunk * s.v_at.t, s.v_at.t, n, tid);
  }
  for (int step = 0; step < chunks; ++step) {
    const int c = chunk_at(step), n = tokens_in(c);
    const bool more = step + 1 < chunks;
    if constexpr (OUT) publish();
    kr.store(ks, n, tid);
    vr.store(vs, n, tid);
    Exact qf[kB];
    if constexpr (OUT) {
      const IO* q = Q + (int64_t(c) * kChunk + min(i, n - 1)) * s.q_at.t;
#pragma unroll
      for (int bb = 0; bb < kB; ++bb) {
        const bool there = DK >= 32 || g < 2;
        const IO* p = q + 32 * bb + (there ? 8 * g : 0);
        if constexpr (sizeof(IO) == 2) {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          qf[bb] = __builtin_bit_cast(bf16x8, there ? v : make_uint4(0, 0, 0, 0));
        } else {
          const f32x4* p4 = reinterpret_cast<const f32x4*>(p);
          qf[bb] = {there ? p4[0] : frag::zero4(), there ? p4[1] : frag::zero4()};
        }
      }
    }
    __syncthreads();
    if (more) {
      const int next = chunk_at(step + 1), nn = tokens_in(next);
      kr.fetch(K + int64_t(next) * kChunk * s.k_at.t, s.k_at.t, nn, tid);
      vr.fetch(V + int64_t(next) * kChunk * s.v_at.t, s.v_at.t, nn, tid);
    }
    if constexpr (OUT) {
      // scores, keys by queries, decayed
      f32x4 p[4];
#pragma unroll
      for (int sb = 0; sb < 4; ++sb) {
        p[sb] = frag::zero4();
        if (s.rev ? sb >= rw : sb <= rw) {
#pragma unroll
          for (int bb = 0; bb < kB; ++bb) p[sb] = mma(row_frag<kPk>(ks, 16 * sb + c16, bb, g), qf[bb], p[sb]);
          // (a product with the mask's zero would keep what is not finite)
#pragma unroll
          for (int r = 0; r < 4; ++r) p[sb][r] = mask[sb][r] != 0.0f ? p[sb][r] * mask[sb][r] : 0.0f;
        }
      }
      Split pf[2];
      split(p[0], p[1], pf[0]);
      split(p[2], p[3], pf[1]);
      const float into = power(e, s.rev ? max(n - 1 - i, 0) : i + 1);
      const bool low = s.rev ? rw < 2 : true, high = s.rev ? true : rw >= 2;
#pragma unroll
      for (int j = 0; j < (kCols + kHalves - 1) / kHalves; ++j) {
        const int cb = j * kHalves + half;
        f32x4 o = frag::zero4();
#pragma unroll
        for (int bb = 0; bb < kB; ++bb) o = mma(ss[(cb * kB + bb) * 64 + l], qf[bb], o);
        o = o * into;
        if (low) o = mma(turned_frag<kPv>(vs, 0, 16 * cb, 4, g, c16), pf[0], o);
        if (high) o = mma(turned_frag<kPv>(vs, 1, 16 * cb, 4, g, c16), pf[1], o);
        if (i < n) store4(out + (int64_t(c) * kChunk + i) * s.out_at.t + 16 * cb + 4 * g, o * s.read);
      }
    }
    if (!OUT || more || s.last) {
      if (n < kChunk) ends(n);
      const float across = power(e, n);
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const int cb = w + j * kWaves;
        if (cb < kCols) {
          Written vf[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const Exact v = turned_frag<kPv>(vs, m, 16 * cb, 4, g, c16);
            split(widened(v, 0) * to_end[m][0], widened(v, 1) * to_end[m][1], vf[m]);
          }
#pragma unroll
          for (int bb = 0; bb < kB; ++bb)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              f32x4 acc = S[j][bb][t] * across;
#pragma unroll
              for (int m = 0; m < 2; ++m) acc = mma(turned_frag<kPk>(ks, m, 32 * bb + 4 * t, 8, g, c16), vf[m], acc);
              S[j][bb][t] = acc;
            }
        }
      }
      if (n < kChunk) ends(kChunk);   // (against time the short chunk comes first)
    }
    __syncthreads();
  }
  if constexpr (OUT) {
    if (s.last) keep(s.last + bh * (DK * DV));
  } else {
    keep(slot);
  }
}

template <typename IO, typename O, int DK, int DV, bool OUT>
hipError_t launch_sweep(const LinearSweep& s, hipStream_t st) {
  auto* const kernel = sweep_kernel<IO, O, DK, DV, OUT>;
  constexpr int lds = lds_bytes<IO, DK, DV, sizeof(O) == 2 ? 2 : 3, OUT>();
  static_assert(lds <= 160 * 1024);
  if constexpr (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3(unsigned(s.heads * s.tiles)), dim3(64 * waves<DV>()), lds, st>>>(s);
  return hipGetLastError();
}

// The sweeps of keys of DK, by value width, types and whether there are outputs.
template <int DK>
hipError_t sweep_of(const LinearSweep& s, hipStream_t st) {
  auto by_type = [&](auto dv) -> hipError_t {
    constexpr int DV = decltype(dv)::value;
    if (!s.out) return s.bf16 ? launch_sweep<bf16_t, float, DK, DV, false>(s, st) : launch_sweep<float, float, DK, DV, false>(s, st);
    if (!s.bf16) return launch_sweep<float, float, DK, DV, true>(s, st);
    return s.out_bf16 ? launch_sweep<bf16_t, bf16_t, DK, DV, true>(s, st) : launch_sweep<bf16_t, float, DK, DV, true>(s, st);
  };
  using std::integral_constant;
  switch (s.dv) {
    case 16: return by_type(integral_constant<int, 16>{});
    case 32: return by_type(integral_constant<int, 32>{});
    case 64: return by_type(integral_constant<int, 64>{});
    default: return by_type(integral_constant<int, 128>{});
  }
}

}  // namespace linear
}  // namespace falcon
