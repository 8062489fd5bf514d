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
// Wave w owns columns w, w + waves, ... of 16 of the values: the state's, in float32
// registers that are an operand of the read as they lie, and the outputs' of all 64
// tokens.  Narrow values leave waves over, which share the tokens of a column.  The
// scores of 16 tokens are made by one wave each and pass through LDS, as do the
// queries, both as operand fragments; they come out of the matrix unit transposed (keys
// by queries), which is what the next product takes as its second operand.  Keys and
// values lie in LDS as they came and are turned on the way out (transposing reads for
// bfloat16).  The rows of the next chunk are on their way while one is worked on.
//
// bfloat16 inputs enter the products as they are.  What is float32 (decayed
// scores, states, decayed values) enters as a sum of three bfloat16 terms, which keep
// 8 bits each and so all of float32's.  float32 inputs use the float32 matrix
// instruction throughout.
//
// What bounds it, at 8 x 2048 x 12 x 64 in bfloat16: sums 13 us for 63 MB and gradients 75 us for
// 330 MB, about a copy's rate; outputs of a prompt 31 us for 116 MB (3.7 TB/s), of which the third
// term of float32 operands takes 3 and values that are not finite, looked for, 2.  At 128 x 128 a
// state fills the registers of eight waves, one workgroup a CU, whose products, vector
// instructions and LDS reads follow one another (25, 35 and 26 % of the time).  The state as
// an operand from registers, where it passed through LDS before, and rows of the next chunk
// ahead: outputs (with two terms) 35 -> 29 us; factored decays, which leave registers for a third
// workgroup: 29 -> 25 us.
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
// Lanes 16 g .. 16 g + 15 hold indices {4 g .. + 3, 16 + 4 g .. + 3} of a block: what two
// stacked result tiles hold, and neighbours in LDS for the transposing reads.
struct f32x8 {
  f32x4 lo, hi;
};
constexpr int kTerms = 3;
struct Terms {
  bf16x8 t[kTerms];
};

// The exact operand of an input, and the operand of float32 values.
template <typename IO>
struct Operands;
template <>
struct Operands<bf16_t> {
  using Exact = bf16x8;
  using Split = Terms;
};
template <>
struct Operands<float> {
  using Exact = f32x8;
  using Split = f32x8;
};

// Two floats to the nearest bfloat16s, and what is lost.
__device__ __forceinline__ uint32_t split2(float& x, float& y) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const uint32_t t = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
  x -= __uint_as_float(t << 16);
  y -= __uint_as_float(t & 0xffff0000u);
  return t;
}
__device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Terms& out) {
  float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
  for (int n = 0; n < kTerms; ++n) {
    uint4 t;
    t.x = split2(v[0], v[1]);
    t.y = split2(v[2], v[3]);
    t.z = split2(v[4], v[5]);
    t.w = split2(v[6], v[7]);
    out.t[n] = __builtin_bit_cast(bf16x8, t);
  }
}
__device__ __forceinline__ void split(f32x4 lo, f32x4 hi, f32x8& out) { out = {lo, hi}; }

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) { return frag::mfma32(a, b, c); }
__device__ __forceinline__ f32x4 mma(bf16x8 a, const Terms& b, f32x4 c) {
#pragma unroll
  for (int n = kTerms - 1; n >= 0; --n) c = frag::mfma32(a, b.t[n], c);
  return c;
}
__device__ __forceinline__ f32x4 mma(const Terms& a, bf16x8 b, f32x4 c) {
#pragma unroll
  for (int n = kTerms - 1; n >= 0; --n) c = frag::mfma32(a.t[n], b, c);
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

// A row's eight values of block b of its columns.
template <int PITCH>
__device__ __forceinline__ bf16x8 row_frag(const bf16_t* rows, int row, int b, int g) {
  const s16x4* p = reinterpret_cast<const s16x4*>(rows + row * PITCH + 32 * b + 4 * g);
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(p[0], p[4], 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int PITCH>
__device__ __forceinline__ f32x8 row_frag(const float* rows, int row, int b, int g) {
  const f32x4* p = reinterpret_cast<const f32x4*>(rows + row * PITCH + 32 * b + 4 * g);
  return {p[0], p[4]};
}

__device__ __forceinline__ s16x4 read_turned(const bf16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
}
// The eight tokens of block m of column first + c16.  The transposing read takes from
// each lane the address of four neighbours and gives lane l < 16 of a group the element
// l % 4 of segment l / 4 of four rows.
template <int PITCH>
__device__ __forceinline__ bf16x8 turned_frag(const bf16_t* rows, int m, int first, int g, int c16) {
  const bf16_t* p = rows + (32 * m + 4 * g + (c16 >> 2)) * PITCH + first + 4 * (c16 & 3);
  const s16x4 lo = read_turned(p), hi = read_turned(p + 16 * PITCH);
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int PITCH>
__device__ __forceinline__ f32x8 turned_frag(const float* rows, int m, int first, int g, int c16) {
  const float* p = rows + (32 * m + 4 * g) * PITCH + first + c16;
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

// Operand fragments in LDS, 64 lanes' parts of 16 bytes next to each other.
__device__ __forceinline__ void put(char* lds, int frag, int l, bf16x8 v) { reinterpret_cast<bf16x8*>(lds)[frag * 64 + l] = v; }
__device__ __forceinline__ void get(const char* lds, int frag, int l, bf16x8& v) { v = reinterpret_cast<const bf16x8*>(lds)[frag * 64 + l]; }
__device__ __forceinline__ void put(char* lds, int frag, int l, const Terms& v) {
#pragma unroll
  for (int n = 0; n < kTerms; ++n) put(lds, frag * kTerms + n, l, v.t[n]);
}
__device__ __forceinline__ void get(const char* lds, int frag, int l, Terms& v) {
#pragma unroll
  for (int n = 0; n < kTerms; ++n) get(lds, frag * kTerms + n, l, v.t[n]);
}
__device__ __forceinline__ void put(char* lds, int frag, int l, const f32x8& v) {
  f32x4* p = reinterpret_cast<f32x4*>(lds) + frag * 128 + l;
  p[0] = v.lo;
  p[64] = v.hi;
}
__device__ __forceinline__ void get(const char* lds, int frag, int l, f32x8& v) {
  const f32x4* p = reinterpret_cast<const f32x4*>(lds) + frag * 128 + l;
  v = {p[0], p[64]};
}

// One number of a fragment that was put as float32.
template <typename IO>
__device__ __forceinline__ float got(const char* lds, int frag, int l, int e) {
  if constexpr (sizeof(IO) == 4) {
    return reinterpret_cast<const float*>(lds)[(frag * 128 + (e >> 2) * 64 + l) * 4 + (e & 3)];
  } else {
    float sum = 0.0f;
    for (int n = kTerms - 1; n >= 0; --n) sum += io<bf16_t>::load(reinterpret_cast<const bf16_t*>(lds), ((frag * kTerms + n) * 64 + l) * 8 + e);
    return sum;
  }
}

// Whether an operand holds an infinity or a NaN: an exponent of ones carries into the sign.
__device__ __forceinline__ bool not_finite(bf16x8 v) {
  const uint4 u = __builtin_bit_cast(uint4, v);
  auto carry = [](uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; };
  return ((carry(u.x) | carry(u.y) | carry(u.z) | carry(u.w)) & 0x80008000u) != 0;
}
__device__ __forceinline__ bool not_finite(const f32x8& v) {
  uint32_t all = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    all |= ((__float_as_uint(v.lo[e]) & 0x7f800000u) + 0x00800000u) | ((__float_as_uint(v.hi[e]) & 0x7f800000u) + 0x00800000u);
  return (all & 0x80000000u) != 0;
}

// Columns 8 g .. + 7 of a row, the lane's own, to where the fragment has them.
__device__ __forceinline__ void put_row(char* lds, int frag, int g, int c16, bf16x8 v) {
  uint2* p = reinterpret_cast<uint2*>(lds) + (frag * 64 + 32 * (g & 1) + c16) * 2 + (g >> 1);
  const uint4 u = __builtin_bit_cast(uint4, v);
  p[0] = make_uint2(u.x, u.y);
  p[32] = make_uint2(u.z, u.w);
}
__device__ __forceinline__ void put_row(char* lds, int frag, int g, int c16, const f32x8& v) {
  f32x4* p = reinterpret_cast<f32x4*>(lds) + frag * 128 + 64 * (g >> 1) + 32 * (g & 1) + c16;
  p[0] = v.lo;
  p[16] = v.hi;
}

// A chunk's rows on the way from memory to LDS, 16 bytes a thread and access.
template <typename IO, int D, int THREADS>
struct Rows {
  static constexpr int kEach = 16 / int(sizeof(IO));        // elements of an access
  static constexpr int kSegs = D / kEach;                    // accesses of a row
  static constexpr int kAll = kChunk * kSegs;
  static constexpr int kMine = (kAll + THREADS - 1) / THREADS;
  static_assert(THREADS % kSegs == 0);
  uint4 r[kMine];

  // The chunk's n tokens are rows `shift` on.  Threads of other rows read its first or last
  // token.  (Offsets within a chunk fit 32 bits: rows have at most 2^22 elements.)
  __device__ __forceinline__ void fetch(const IO* first, int t_step, int n, int shift, int tid) {
    const char* const p = reinterpret_cast<const char*>(first);
    const uint32_t seg = uint32_t(tid % kSegs) * 16, step = uint32_t(t_step) * uint32_t(sizeof(IO));
    if (n == kChunk && kAll % THREADS == 0) {
      const uint32_t at = uint32_t(tid / kSegs) * step + seg;
#pragma unroll
      for (int i = 0; i < kMine; ++i) r[i] = *reinterpret_cast<const uint4*>(p + int64_t(i * (THREADS / kSegs)) * step + at);
    } else {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int row = min(max(tid / kSegs + i * (THREADS / kSegs) - shift, 0), n - 1);
        r[i] = *reinterpret_cast<const uint4*>(p + (uint32_t(row) * step + seg));
      }
    }
  }
  __device__ __forceinline__ void store(IO* rows, int n, int shift, int tid) const {
    const int first = tid / kSegs, seg = tid % kSegs;
    uint4* const p = reinterpret_cast<uint4*>(rows + first * Stage<IO, D>::kPitch + seg * kEach);
    constexpr int kStep = THREADS / kSegs * Stage<IO, D>::kPitch * int(sizeof(IO)) / 16;
    if (n == kChunk && kAll % THREADS == 0) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) p[i * kStep] = r[i];
    } else {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int row = first + i * (THREADS / kSegs);
        if (kAll % THREADS == 0 || row < kChunk) p[i * kStep] = uint32_t(row - shift) < uint32_t(n) ? r[i] : make_uint4(0, 0, 0, 0);
      }
    }
  }
};

// a^n, with a^0 = 1 for every a.
__device__ __forceinline__ float power(float log2_a, int n) {
  return n == 0 ? 1.0f : __builtin_amdgcn_exp2f(log2_a * float(n));
}

// Waves of a workgroup: eight where what four hold would not fit their registers, float32
// operands of 128 columns and states of 128 x 128 (16384 x 12 in bfloat16 by two terms: outputs
// 63 us, four waves 72 us with 48 registers in memory; halves of the values apart 70 us).
template <typename IO, int DK, int DV>
constexpr int waves() {
  return (sizeof(IO) == 4 && (DK >= 128 || DV >= 128)) || (DK >= 128 && DV >= 128) ? 8 : 4;
}
// Waves of a SIMD that the registers leave room for: three (168 registers)
// where LDS has room for three workgroups.
template <typename IO, int DK, int DV>
constexpr int waves_simd() {
  return sizeof(IO) == 2 && DK <= 64 && DV <= 64 ? 3 : 2;
}
// LDS: keys, values and, for outputs, queries and scores as fragments.
template <typename IO, int DK, int DV, bool OUT>
constexpr int lds_once() {
  const int scores = 8 * 64 * (sizeof(IO) == 2 ? kTerms * 16 : 32);
  return Stage<IO, DK>::kBytes + Stage<IO, DV>::kBytes + (OUT ? kChunk * Stage<IO, DK>::kWidth * int(sizeof(IO)) + scores : 0);
}
// Two places in turn for what is read up to a chunk's end (the keys; without outputs the
// values, too) save the barrier there, where as many workgroups fit a CU all the same.
template <typename IO, int DK, int DV, bool OUT>
constexpr bool in_turn() {
  const int once = lds_once<IO, DK, DV, OUT>(), more = Stage<IO, DK>::kBytes + (OUT ? 0 : Stage<IO, DV>::kBytes);
  const int room = waves_simd<IO, DK, DV>() * 4 / waves<IO, DK, DV>(), before = 160 * 1024 / once, after = 160 * 1024 / (once + more);
  return after >= (before < room ? before : room);
}
template <typename IO, int DK, int DV, bool OUT>
constexpr int lds_bytes() {
  return lds_once<IO, DK, DV, OUT>() + (in_turn<IO, DK, DV, OUT>() ? Stage<IO, DK>::kBytes + (OUT ? 0 : Stage<IO, DV>::kBytes) : 0);
}

__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store4(bf16_t* p, f32x4 v) { frag::store_half(reinterpret_cast<uint16_t*>(p), v); }

// The tile `block` of a sweep.  OUT false: only what the tile's chunks add to a state,
// from zero, into the tile's slot.
template <typename IO, typename O, int DK, int DV, bool OUT>
__device__ __forceinline__ void sweep(const LinearSweep& s, uint32_t block, char* lds) {
  constexpr int kWaves = waves<IO, DK, DV>(), kThreads = 64 * kWaves;
  constexpr int kB = Stage<IO, DK>::kWidth / 32;           // 32-wide blocks of the key axis
  constexpr int kCols = DV / 16;                           // 16-wide blocks of the value axis
  constexpr int kOwn = kCols >= kWaves ? kCols / kWaves : 1;   // of these, a wave's
  constexpr int kShare = kCols >= kWaves ? 1 : kWaves / kCols; // waves that share a block of columns
  constexpr int kRows = kShare >= 4 ? 1 : 4 / kShare;      // blocks of 16 tokens whose outputs a wave makes
  constexpr int kPk = Stage<IO, DK>::kPitch, kPv = Stage<IO, DV>::kPitch;
  using Ops = Operands<IO>;
  using Exact = typename Ops::Exact;
  using Split = typename Ops::Split;

  // Where registers are left the reads of LDS for several products are issued ahead of the
  // first one: by itself the compiler waits for each in turn (heads of 128 x 128 by two terms: outputs
  // of a prompt 63 -> 62 us, gradients 124 -> 121 us; narrower heads have no registers left).
  constexpr bool kAhead = kWaves == 8 && sizeof(IO) == 2;
  auto issued = [&]() {
    if constexpr (kAhead) asm volatile("" ::: "memory");
  };
  constexpr bool kInTurn = in_turn<IO, DK, DV, OUT>();
  char* const second = lds + lds_once<IO, DK, DV, OUT>();
  IO* ks = reinterpret_cast<IO*>(lds);
  IO* vs = reinterpret_cast<IO*>(lds + Stage<IO, DK>::kBytes);
  char* const qs = lds + Stage<IO, DK>::kBytes + Stage<IO, DV>::kBytes;   // [4][kB] fragments
  char* const ps = qs + kChunk * Stage<IO, DK>::kWidth * int(sizeof(IO)); // [4][2] fragments

  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, c16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rw = w & 3;                                    // the block of tokens whose scores this wave makes
  const int share = kShare > 1 ? w / kCols : 0;
  auto column = [&](int j) { return kShare > 1 ? w % kCols : w + j * kWaves; };
  auto tokens = [&](int x) { return share + x * kShare; };  // block x of this wave's outputs
  const bool makes = kShare <= 4 || share < 4;

  const int64_t bh = block / uint32_t(s.tiles);
  const int tile = int(block % uint32_t(s.tiles));
  const int b = int(uint32_t(bh) / uint32_t(s.H)), h = int(uint32_t(bh) % uint32_t(s.H));
  const int len = tokens_of(s.lengths, b, s.T);
  const int first = tile * s.chunks * kChunk;
  const int chunks = min((len - first + kChunk - 1) / kChunk, s.chunks);
  const float e = s.log_decay[h] * kLog2e;

  const IO* const K = static_cast<const IO*>(s.k) + b * s.k_at.b + h * s.k_at.h + first * s.k_at.t;
  const IO* const V = static_cast<const IO*>(s.v) + b * s.v_at.b + h * s.v_at.h + first * s.v_at.t;
  const IO* const Q = OUT ? static_cast<const IO*>(s.q) + b * s.q_at.b + h * s.q_at.h + first * s.q_at.t : nullptr;
  O* const out = OUT ? static_cast<O*>(s.out) + b * s.out_at.b + h * s.out_at.h + first * s.out_at.t : nullptr;
  const int k_step = int(s.k_at.t), v_step = int(s.v_at.t), q_step = int(s.q_at.t), out_step = int(s.out_at.t);
  float* const slot = s.slots ? s.slots + (bh * s.slots_each + s.slot0 + tile) * (DK * DV) : nullptr;

  if constexpr (OUT) {
    if (s.clear) {   // the tile's rows behind the sequence's end
      constexpr int kEach = DV * int(sizeof(O)) / 16;
      const int from = max(len - first, 0), to = min(s.T - first, s.chunks * kChunk);
      for (int64_t i = tid; i < int64_t(to - from) * kEach; i += kThreads)
        *reinterpret_cast<uint4*>(out + (from + i / kEach) * s.out_at.t + i % kEach * (16 / int(sizeof(O)))) = make_uint4(0, 0, 0, 0);
    }
  }
  Rows<IO, DK, kThreads> kr;
  Rows<IO, DV, kThreads> vr;
  Exact qr[OUT ? kB : 1];
  auto chunk_at = [&](int step) { return s.rev ? chunks - 1 - step : step; };
  auto tokens_in = [&](int c) { return min(len - first - c * kChunk, kChunk); };
  // A short chunk's tokens are its last rows, or its first against time: what is written
  // decays by the row alone.
  auto shift_of = [&](int n) { return s.rev ? 0 : kChunk - n; };
  auto fetch = [&](int c) {
    const int n = tokens_in(c), shift = shift_of(n);
    kr.fetch(K + int64_t(c) * kChunk * k_step, k_step, n, shift, tid);
    vr.fetch(V + int64_t(c) * kChunk * v_step, v_step, n, shift, tid);
    if constexpr (OUT) {
      if (w < 4) {
        // columns 32 bb + 8 g .. + 7 of query row 16 rw + c16
        const bool there = DK >= 32 || g < 2;
        const char* p = reinterpret_cast<const char*>(Q + int64_t(c) * kChunk * q_step);
        const uint32_t row = uint32_t(min(max(16 * rw + c16 - shift, 0), n - 1)) * uint32_t(q_step);
#pragma unroll
        for (int bb = 0; bb < kB; ++bb) {
          const uint32_t at = (row + 32 * bb + (there ? 8 * g : 0)) * uint32_t(sizeof(IO));
          if constexpr (sizeof(IO) == 2) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + at);
            qr[bb] = __builtin_bit_cast(bf16x8, there ? v : make_uint4(0, 0, 0, 0));
          } else {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(p + at), hi = *reinterpret_cast<const f32x4*>(p + at + 16);
            qr[bb] = {there ? lo : frag::zero4(), there ? hi : frag::zero4()};
          }
        }
      }
    }
  };
  if (chunks > 0) fetch(chunk_at(0));

  // A state's element (f, c) at f sf + c sc.  Rows 32 b + 16 t + 4 g + r of column
  // 16 cb + c16 lie in S[.][b][t][r].
  f32x4 S[kOwn][kB][2];
  const float* const from = OUT ? (slot ? slot : s.start ? s.start + bh * (DK * DV) : nullptr) : nullptr;
#pragma unroll
  for (int j = 0; j < kOwn; ++j)
#pragma unroll
    for (int bb = 0; bb < kB; ++bb)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        S[j][bb][t] = frag::zero4();
        const int f = 32 * bb + 16 * t + 4 * g;
        if (OUT && from && f < DK) {
          const float* p = from + f * s.sf + (16 * column(j) + c16) * s.sc;
          if (s.sf == 1) {   // the transposed state
            S[j][bb][t] = *reinterpret_cast<const f32x4*>(p);
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[j][bb][t][r] = p[r * s.sf];
          }
        }
      }
  auto keep = [&](float* to) {
    if (share > 0) return;
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
#pragma unroll
      for (int bb = 0; bb < kB; ++bb)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int f = 32 * bb + 16 * t + 4 * g;
          if (f < DK)
#pragma unroll
            for (int r = 0; r < 4; ++r) to[(f + r) * s.sf + (16 * column(j) + c16) * s.sc] = S[j][bb][t][r];
        }
  };
  if (chunks <= 0) {   // nothing of the sequence is left for this tile
    if constexpr (OUT) {
      if (s.last) keep(s.last + bh * (DK * DV));
    }
    return;
  }
  if constexpr (DK < 32) {
    for (int i = tid; i < kChunk * kPk; i += kThreads) {
      ks[i] = IO{};
      if constexpr (kInTurn) reinterpret_cast<IO*>(second)[i] = IO{};
    }
    __syncthreads();
  }
  // Decays, as products of a factor of the four rows 4 g + r of a block of 16 and one of
  // the row r: from a key row 32 m + 16 u + 4 g + r to the chunk's end, and to this lane's
  // query row 16 rw + c16.  In the block of the queries themselves they have a mask.
  constexpr int kPairs = kWaves == 8 ? 1 : 2;              // pairs m of 16 keys that are this wave's
  auto pair = [&](int x) { return kWaves == 8 ? w >> 2 : x; };
  float by_row[4], to_end[2][2], to_query[OUT ? kPairs : 1][2];
  f32x4 own;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    by_row[r] = power(e, s.rev ? r : 3 - r);
    const int gap = s.rev ? 4 * g + r - c16 : c16 - (4 * g + r);
    own[r] = gap >= 0 ? power(e, max(gap, 0)) * s.write * s.read : 0.0f;
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = 32 * m + 16 * u + 4 * g;
      to_end[m][u] = power(e, s.rev ? row + 1 : kChunk - 4 - row) * s.write;
    }
  if constexpr (OUT) {
#pragma unroll
    for (int x = 0; x < kPairs; ++x)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 32 * pair(x) + 16 * u + 4 * g, i = 16 * rw + c16;
        to_query[x][u] = power(e, max(s.rev ? row - i : i - row - 3, 0)) * s.write * s.read;
      }
  }
  // ... and of the entering state at the rows of this wave's outputs, of whole chunks.
  float into[OUT ? kRows : 1];
  if constexpr (OUT) {
#pragma unroll
    for (int x = 0; x < kRows; ++x) into[x] = power(e, s.rev ? kChunk - 1 - (16 * tokens(x) + c16) : 16 * tokens(x) + c16 + 1) * s.read;
  }
  const float whole = power(e, kChunk);

  for (int step = 0; step < chunks; ++step) {
    const int c = chunk_at(step), n = tokens_in(c);
    const bool more = step + 1 < chunks;
    if constexpr (kInTurn) {
      ks = reinterpret_cast<IO*>(step % 2 ? second : lds);
      if constexpr (!OUT) vs = reinterpret_cast<IO*>((step % 2 ? second : lds) + Stage<IO, DK>::kBytes);
    }
    const int shift = shift_of(n);
    kr.store(ks, n, shift, tid);
    vr.store(vs, n, shift, tid);
    if constexpr (OUT) {
      if (w < 4) {
#pragma unroll
        for (int bb = 0; bb < kB; ++bb) put_row(qs, rw * kB + bb, g, c16, qr[bb]);
      }
    }
    __syncthreads();
    if (more) fetch(chunk_at(step + 1));
    Exact vf[kOwn][2];
    f32x4 o[OUT ? kRows : 1][kOwn];
    if constexpr (OUT) {
      // scores, keys by queries, decayed
      Exact qf[kB];
#pragma unroll
      for (int bb = 0; bb < kB; ++bb) get(qs, rw * kB + bb, l, qf[bb]);
#pragma unroll
      for (int x = 0; x < kPairs; ++x) {
        const int m = pair(x);
        if (!(s.rev ? m == 1 || rw < 2 : m == 0 || rw >= 2)) continue;   // all behind (before) these tokens
        f32x4 p[2];
        auto keys = [&](int u, int bb) __attribute__((always_inline)) { return row_frag<kPk>(ks, 32 * m + 16 * u + c16, bb, g); };
        Exact kf[kAhead ? 2 : 1][kB];
        if constexpr (kAhead) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int bb = 0; bb < kB; ++bb) kf[u][bb] = keys(u, bb);
          issued();
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          p[u] = frag::zero4();
#pragma unroll
          for (int bb = 0; bb < kB; ++bb) p[u] = mma(kAhead ? kf[kAhead ? u : 0][bb] : keys(u, bb), qf[bb], p[u]);
          const int block = 2 * m + u;
          if (block == rw) {
            // (a product with the mask's zero would keep what is not finite)
#pragma unroll
            for (int r = 0; r < 4; ++r) p[u][r] = own[r] != 0.0f ? p[u][r] * own[r] : 0.0f;
          } else if (s.rev ? block > rw : block < rw) {
#pragma unroll
            for (int r = 0; r < 4; ++r) p[u][r] *= to_query[x][u] * by_row[r];
          } else {
            p[u] = frag::zero4();
          }
        }
        Split pf;
        split(p[0], p[1], pf);
        put(ps, rw * 2 + m, l, pf);
      }
      // what the entering state gives
#pragma unroll
      for (int x = 0; x < kRows; ++x)
#pragma unroll
        for (int j = 0; j < kOwn; ++j) o[x][j] = frag::zero4();
      if (makes) {
        Exact q[kAhead ? 2 : 1][kRows];
        auto queries = [&](int bb, Exact (&to)[kRows]) __attribute__((always_inline)) {
#pragma unroll
          for (int x = 0; x < kRows; ++x) get(qs, tokens(x) * kB + bb, l, to[x]);
        };
        if constexpr (kAhead) queries(0, q[0]);
#pragma unroll
        for (int bb = 0; bb < kB; ++bb) {
          if constexpr (kAhead) {
            if (bb + 1 < kB) queries(bb + 1, q[(bb + 1) % 2]);
            issued();
          } else {
            queries(bb, q[0]);
          }
          Split sf[kOwn];
#pragma unroll
          for (int j = 0; j < kOwn; ++j) split(S[j][bb][0], S[j][bb][1], sf[j]);
#pragma unroll
          for (int x = 0; x < kRows; ++x)
#pragma unroll
            for (int j = 0; j < kOwn; ++j) o[x][j] = mma(sf[j], q[kAhead ? bb % 2 : 0][x], o[x][j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
#pragma unroll
      for (int m = 0; m < 2; ++m) vf[j][m] = turned_frag<kPv>(vs, m, 16 * column(j), g, c16);
    if constexpr (OUT) {
      __syncthreads();
      if (makes) {
        char* const to = reinterpret_cast<char*>(out + int64_t(c) * kChunk * out_step);
        Split pf[kAhead ? 2 : 1][2];
        // (of a pair that is all behind these tokens there are no scores, and none is used)
        auto scores = [&](int x, Split (&to)[2]) __attribute__((always_inline)) {
#pragma unroll
          for (int m = 0; m < 2; ++m) get(ps, tokens(x) * 2 + m, l, to[m]);
        };
        if constexpr (kAhead) scores(0, pf[0]);
        float noticed = 0.0f;   // NaN, once there is an output that is not finite
#pragma unroll
        for (int x = 0; x < kRows; ++x) {
          const int rb = tokens(x), i = 16 * rb + c16 - shift;
          if constexpr (kAhead) {
            if (x + 1 < kRows) scores(x + 1, pf[(x + 1) % 2]);
            issued();
          }
          const float at_row = n == kChunk ? into[x] : power(e, max(s.rev ? n - 1 - i : i + 1, 0)) * s.read;
#pragma unroll
          for (int j = 0; j < kOwn; ++j) o[x][j] = o[x][j] * at_row;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (!(s.rev ? m == 1 || rb < 2 : m == 0 || rb >= 2)) continue;
            if constexpr (!kAhead) get(ps, rb * 2 + m, l, pf[0][m]);
#pragma unroll
            for (int j = 0; j < kOwn; ++j) o[x][j] = mma(vf[j][m], pf[kAhead ? x % 2 : 0][m], o[x][j]);
          }
#pragma unroll
          for (int j = 0; j < kOwn; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) noticed = __builtin_fmaf(o[x][j][r], 0.0f, noticed);
          if (uint32_t(i) < uint32_t(n)) {
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
              store4(reinterpret_cast<O*>(to + (uint32_t(i) * uint32_t(out_step) + 16 * column(j) + 4 * g) * uint32_t(sizeof(O))), o[x][j]);
          }
        }
        // A value that is not finite times a score that the mask has made zero is not zero: the
        // columns that hold one once more, by the terms that each token has.  (Rows from memory: LDS
        // may hold the next chunk's.)  The branch costs 2 of 31 us at 8 x 2048 x 12 x 64 and 4 of 75 us
        // of the gradients by what it keeps the compiler from moving across; values cleaned
        // where they are staged, or such tiles once more behind the loop, cost more.
        if (__any(noticed != 0.0f)) {
          __threadfence();   // behind what other lanes have stored there
          const IO* const queries = Q + int64_t(c) * kChunk * q_step;
          const IO* const values = V + int64_t(c) * kChunk * v_step;
#pragma unroll
          for (int j = 0; j < kOwn; ++j) {
            int bad = not_finite(vf[j][0]) || not_finite(vf[j][1]);
            bad |= __shfl_xor(bad, 16);
            bad |= __shfl_xor(bad, 32);
            if (!__any(bad)) continue;
            const int col = 16 * column(j) + c16;
#pragma unroll 1
            for (int x = 0; x < 16 * kRows; ++x) {
              const int row = 16 * tokens(x / 16) + x % 16, i = row - shift;
              if (uint32_t(i) >= uint32_t(n)) continue;
              float sum = 0.0f;
#pragma unroll
              for (int bb = 0; bb < kB; ++bb)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                  if (32 * bb + 16 * t < DK)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                      sum = __builtin_fmaf(S[j][bb][t][r], io<IO>::load(queries, i * q_step + 32 * bb + 16 * t + 4 * g + r), sum);
              sum += __shfl_xor(sum, 16);
              sum += __shfl_xor(sum, 32);
              sum *= power(e, s.rev ? n - 1 - i : i + 1) * s.read;
#pragma unroll 1
              for (int k = s.rev ? i : 0; k < (s.rev ? n : i + 1); ++k) {
                const int key = k + shift;
                sum = __builtin_fmaf(got<IO>(ps, row / 16 * 2 + key / 32, (key & 12) * 4 + row % 16, (key & 3) + (key & 16) / 4),
                                     io<IO>::load(values, k * v_step + col), sum);
              }
              if (bad && g == 0) io<O>::store(reinterpret_cast<O*>(to), i * out_step + col, sum);
            }
          }
        }
      }
    }
    if (!OUT || more || s.last) {
      const float across = n < kChunk ? power(e, n) : whole;
      Split wf[kOwn][2];
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          f32x4 part[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            part[u] = widened(vf[j][m], u) * to_end[m][u];
#pragma unroll
            for (int r = 0; r < 4; ++r) part[u][r] *= by_row[r];
          }
          split(part[0], part[1], wf[j][m]);
        }
#pragma unroll
      for (int bb = 0; bb < kB; ++bb)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          Exact kf[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) kf[m] = turned_frag<kPk>(ks, m, 32 * bb + 16 * t, g, c16);
#pragma unroll
          for (int j = 0; j < kOwn; ++j) {
            if constexpr (sizeof(IO) == 4) {
              // A chunk's 16 products in two halves from zero, added once: each added to the state would
              // be rounded at its size.  (bfloat16's are six, and registers are short.)  One half after
              // the other, no reads for the next block ahead: 6 to 8 registers in memory at 128 x 128
              // instead of 25.
              const f32x4 first = mma(kf[0], wf[j][0], frag::zero4());
              asm volatile("" ::: "memory");
              S[j][bb][t] = S[j][bb][t] * across + (first + mma(kf[1], wf[j][1], frag::zero4()));
            } else {
              f32x4 acc = S[j][bb][t] * across;
#pragma unroll
              for (int m = 0; m < 2; ++m) acc = mma(kf[m], wf[j][m], acc);
              S[j][bb][t] = acc;
            }
          }
        }
    }
    if constexpr (!kInTurn) __syncthreads();
  }
  if constexpr (OUT) {
    if (s.last) keep(s.last + bh * (DK * DV));
  } else {
    keep(slot);
  }
}

// One sweep, or what two sweeps' tiles add, one after the other.
struct Sweeps2 {
  LinearSweep s[2];
  uint32_t blocks;     // of each
};
template <typename IO, typename O, int DK, int DV, bool OUT>
__global__ __launch_bounds__((64 * waves<IO, DK, DV>()), (waves_simd<IO, DK, DV>())) void sweep_kernel(Sweeps2 p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const uint32_t which = blockIdx.x >= p.blocks ? 1 : 0;
  sweep<IO, O, DK, DV, OUT>(p.s[which], blockIdx.x - which * p.blocks, lds);
}

// The three gradients' sweeps, dv's over keys of DK, dk's and dq's over keys of DV.  The
// three workgroups of a tile read the same rows: they lie eight apart, which is the
// same XCD, so that two of them find the rows in its L2.
struct Sweeps3 {
  LinearSweep s[3];
  uint32_t blocks;
};
template <typename IO, int DK, int DV>
__global__ __launch_bounds__((64 * waves<IO, DK, DV>()), (waves_simd<IO, DK, DV>())) void gradients_kernel(Sweeps3 p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const uint32_t which = blockIdx.x / 8 % 3, block = blockIdx.x / 24 * 8 + blockIdx.x % 8;
  if (block >= p.blocks) return;
  if constexpr (DK == DV) {
    sweep<IO, float, DK, DV, true>(p.s[which], block, lds);
  } else if (which == 0) {
    sweep<IO, float, DK, DV, true>(p.s[0], block, lds);
  } else {
    sweep<IO, float, DV, DK, true>(p.s[which], block, lds);
  }
}

template <typename Kernel, typename Args>
hipError_t launch(Kernel kernel, uint32_t blocks, int threads, int lds, const Args& args, hipStream_t st) {
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3(blocks), dim3(threads), lds, st>>>(args);
  return hipGetLastError();
}

template <typename IO, typename O, int DK, int DV, bool OUT>
hipError_t launch_sweep(const LinearSweep& s, const LinearSweep* second, hipStream_t st) {
  constexpr int lds = lds_bytes<IO, DK, DV, OUT>();
  static_assert(lds <= 160 * 1024);
  const uint32_t blocks = uint32_t(s.heads * s.tiles);
  return launch(sweep_kernel<IO, O, DK, DV, OUT>, blocks * (second ? 2 : 1), 64 * waves<IO, DK, DV>(), lds,
                Sweeps2{{s, second ? *second : s}, blocks}, st);
}

template <typename IO, int DK, int DV>
hipError_t launch_gradients(const LinearSweep& dv, const LinearSweep& dk, const LinearSweep& dq, hipStream_t st) {
  constexpr int a = lds_bytes<IO, DK, DV, true>(), b = lds_bytes<IO, DV, DK, true>(), lds = a > b ? a : b;
  static_assert(lds <= 160 * 1024);
  const uint32_t blocks = uint32_t(dv.heads * dv.tiles);
  return launch(gradients_kernel<IO, DK, DV>, (blocks + 7) / 8 * 24, 64 * waves<IO, DK, DV>(), lds, Sweeps3{{dv, dk, dq}, blocks}, st);
}

template <typename F>
hipError_t by_width(int dv, F f) {
  using std::integral_constant;
  switch (dv) {
    case 16: return f(integral_constant<int, 16>{});
    case 32: return f(integral_constant<int, 32>{});
    case 64: return f(integral_constant<int, 64>{});
    default: return f(integral_constant<int, 128>{});
  }
}

// What tiles with keys of DK add, of one or two sweeps of the same sizes; outputs of a
// prompt; the gradients.
template <int DK>
hipError_t sums_of(const LinearSweep& s, const LinearSweep* second, hipStream_t st) {
  return by_width(s.dv, [&](auto dv) {
    return s.bf16 ? launch_sweep<bf16_t, float, DK, dv(), false>(s, second, st) : launch_sweep<float, float, DK, dv(), false>(s, second, st);
  });
}
template <int DK>
hipError_t outputs_of(const LinearSweep& s, hipStream_t st) {
  return by_width(s.dv, [&](auto dv) {
    return s.bf16 ? launch_sweep<bf16_t, bf16_t, DK, dv(), true>(s, nullptr, st) : launch_sweep<float, float, DK, dv(), true>(s, nullptr, st);
  });
}
template <int DK>
hipError_t gradients_of(const LinearSweep& dv, const LinearSweep& dk, const LinearSweep& dq, hipStream_t st) {
  return by_width(dv.dv, [&](auto width) {
    return dv.bf16 ? launch_gradients<bf16_t, DK, width()>(dv, dk, dq, st) : launch_gradients<float, DK, width()>(dv, dk, dq, st);
  });
}

}  // namespace linear
}  // namespace falcon
