// The gradient of a head's log decay in linear attention, a tile of chunks a workgroup
// (gfx950, MFMA).
//
// A pair of a token r that writes and a token s that reads counts a^(s - r) (q_s . k_r)
// (dO_s . v_r), s - r times.  With the state S that enters a chunk of n tokens and D its
// derivative by the log of the decay, counted from the tile's start (where D = 0), s and r
// from 0 in the chunk:
//
//   reads  sum_s a^(s + 1) q_s^T (D + (s + 1) S) dO_s + sum_(r < s) (s - r) a^(s - r) (q_s . k_r) (dO_s . v_r)
//   S'     = a^n S + sum_r a^(n - 1 - r) k_r v_r^T
//   D'     = a^n (D + n S) + sum_r (n - 1 - r) a^(n - 1 - r) k_r v_r^T
//
// and at the tile's end <D, R>, with the adjoint R that enters it from behind.  Every term has
// been decayed as often as it counts: what a token reads of its own write, which no decay
// makes small, is in none of them, and a head's error stays that of float32 sums of its own
// terms (2e-7 to 7e-7 of the root of their squares' sum, from log_decay -0.004 to -60).
// k . dk - q . dq summed along the tokens would need one product of states a tile and no
// states in between, but there that part cancels between float32 numbers: 1e-4 of the terms
// at -1, 3e-2 at -5, 32 times the terms at -12.
//
// The reads of the state are taken as <D, A0> + <S, A1>, with A0 and A1 the sums over tokens of
// a^(s + 1) q_s dO_s^T, counted and not: four products alike, over the tokens of a chunk, whose
// results lie as S and D do.  A wave owns columns of 16 of the values, as in the sweeps;
// where there are fewer than waves, several share a column's rows.  Pairs are the product of
// two tiles of scores, 16 queries a wave.  float32 operands as sums of three bfloat16 terms or
// by the float32 matrix instruction, as in the sweeps; what adds up over a tile, in double.
//
// A chunk's rows are loaded where they are needed: workgroups that share a CU hide it better
// than loads a chunk ahead, whose registers they lack (8 x 2048 x 12 x 64 x 64 in bfloat16 36 us,
// ahead 43 us; 2 x 4096 x 12 x 128 x 128 in bfloat16 64 and 61 us; 4096 x 8 x 128 x 128 in float32 57
// and 70 us, 60 now that its chunks' sums come in halves).
#pragma once

#include "falcon_linear_kernel.h"

namespace falcon {
namespace linear {

constexpr float kLog2eRest = 1.92596299112661747e-8f;   // log2(e) less kLog2e

// a^n by a base of two float32 numbers and an exponent split into whole and fraction: what is
// lost does not grow with the exponent.
struct Base {
  float hi, lo;
  __device__ __forceinline__ explicit Base(float log_a) {
#pragma clang fp contract(off)   // (the rounded product, also where a power takes it times one)
    log_a = log_a < -1000.0f ? -1000.0f : log_a;   // (zero from the first power on)
    hi = log_a * kLog2e;
    lo = __builtin_fmaf(log_a, kLog2e, -hi) + log_a * kLog2eRest;
  }
};
__device__ __forceinline__ float power(const Base& a, int n) {
  const float whole = __builtin_rintf(a.hi * float(n));
  const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(a.hi, float(n), -whole) + a.lo * float(n));
  return __builtin_amdgcn_ldexpf(p, int(whole));
}

// Eight waves where four would own twice 32 registers of states, as in the sweeps with float32.
template <int DK, int DV>
constexpr int decay_waves() {
  return DK >= 128 || DV >= 128 ? 8 : 4;
}
template <typename IO, int DK, int DV>
constexpr int decay_lds() {
  return 2 * (Stage<IO, DK>::kBytes + Stage<IO, DV>::kBytes);
}

template <typename IO, int DK, int DV>
__global__ __launch_bounds__((64 * decay_waves<DK, DV>()), 2) void decay_kernel(LinearDecays a) {
  constexpr int kWaves = decay_waves<DK, DV>(), kThreads = 64 * kWaves;
  constexpr int kBk = Stage<IO, DK>::kWidth / 32, kBv = Stage<IO, DV>::kWidth / 32;
  constexpr int kPk = Stage<IO, DK>::kPitch, kPv = Stage<IO, DV>::kPitch;
  constexpr int kCols = DV / 16, kRowTiles = DK / 16;
  constexpr int kOwn = kCols >= kWaves ? kCols / kWaves : 1;                   // a wave's blocks of 16 columns
  constexpr int kShare = kCols >= kWaves ? 1 : kWaves / kCols;                 // waves of a block of columns
  constexpr int kMine = kRowTiles > kShare ? kRowTiles / kShare : 1;           // a wave's blocks of 16 rows of it
  constexpr int kPairs = kWaves == 8 ? 1 : 2;                                  // pairs m of 16 keys that are this wave's
  using Exact = typename Operands<IO>::Exact;
  using Split = typename Operands<IO>::Split;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ double sums[kWaves];
  IO* const ks = reinterpret_cast<IO*>(lds);
  IO* const qs = ks + kChunk * kPk;
  IO* const vs = qs + kChunk * kPk;
  IO* const os = vs + kChunk * kPv;

  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, c16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rw = w & 3;
  const int share = kShare > 1 ? w / kCols : 0;
  auto column = [&](int j) { return kShare > 1 ? w % kCols : w + j * kWaves; };
  auto row_tile = [&](int y) { return share + y * kShare; };
  const bool works = kShare <= kRowTiles || share < kRowTiles;

  const int64_t bh = blockIdx.x / uint32_t(a.tiles);
  const int tile = int(blockIdx.x % uint32_t(a.tiles));
  const int b = int(uint32_t(bh) / uint32_t(a.H)), h = int(uint32_t(bh) % uint32_t(a.H));
  const int len = tokens_of(a.lengths, b, a.T);
  const int first = tile * a.chunks * kChunk;
  const int chunks = min((len - first + kChunk - 1) / kChunk, a.chunks);
  const Base e(a.log_decay[h]);

  double pairs = 0.0, reads = 0.0, behind = 0.0;
  if (chunks > 0) {
    const IO* const K = static_cast<const IO*>(a.k) + b * a.k_at.b + h * a.k_at.h + first * a.k_at.t;
    const IO* const Q = static_cast<const IO*>(a.q) + b * a.q_at.b + h * a.q_at.h + first * a.q_at.t;
    const IO* const V = static_cast<const IO*>(a.v) + b * a.v_at.b + h * a.v_at.h + first * a.v_at.t;
    const IO* const O = static_cast<const IO*>(a.dO) + b * a.o_at.b + h * a.o_at.h + first * a.o_at.t;
    Rows<IO, DK, kThreads> kr, qr;
    Rows<IO, DV, kThreads> vr, orow;
    auto tokens_in = [&](int c) { return min(len - first - c * kChunk, kChunk); };
    // (a short chunk's tokens are its last rows, as in a sweep forward)
    auto fetch = [&](int c) {
      const int n = tokens_in(c), shift = kChunk - n;
      const int64_t t = int64_t(c) * kChunk;
      kr.fetch(K + t * a.k_at.t, int(a.k_at.t), n, shift, tid);
      qr.fetch(Q + t * a.q_at.t, int(a.q_at.t), n, shift, tid);
      vr.fetch(V + t * a.v_at.t, int(a.v_at.t), n, shift, tid);
      orow.fetch(O + t * a.o_at.t, int(a.o_at.t), n, shift, tid);
    };
    // Rows 16 row_tile(y) + 4 g + r of column 16 column(j) + c16 lie in S[j][y][r].
    f32x4 S[kOwn][kMine], D[kOwn][kMine];
    auto element = [&](int j, int y) { return (16 * row_tile(y) + 4 * g) * DV + 16 * column(j) + c16; };
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
#pragma unroll
      for (int y = 0; y < kMine; ++y) {
        S[j][y] = D[j][y] = frag::zero4();
        if (a.S && works) {
          const float* p = a.S + (bh * a.s_each + tile) * (DK * DV) + element(j, y);
#pragma unroll
          for (int r = 0; r < 4; ++r) S[j][y][r] = p[r * DV];
        }
      }
    if constexpr (DK < 32 || DV < 32) {   // the columns behind narrow rows
      for (int i = tid; i < 2 * kChunk * (kPk + kPv); i += kThreads) ks[i] = IO{};
      __syncthreads();
    }
    // Decays as in the sweeps: a factor of the four rows 4 g + r of a block of 16 and one of the row.
    auto pair = [&](int x) { return kWaves == 8 ? w >> 2 : x; };
    float down[4], up[4], to_end[2][2], to_start[2][2], to_query[kPairs][2];
    f32x4 own;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      down[r] = power(e, 3 - r);
      up[r] = power(e, r);
      const int gap = c16 - (4 * g + r);
      own[r] = gap > 0 ? power(e, max(gap, 0)) * float(gap) : 0.0f;
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 32 * m + 16 * u + 4 * g;
        to_end[m][u] = power(e, kChunk - 4 - row);
        to_start[m][u] = power(e, row + 1);
      }
#pragma unroll
    for (int x = 0; x < kPairs; ++x)
#pragma unroll
      for (int u = 0; u < 2; ++u) to_query[x][u] = power(e, max(16 * rw + c16 - (32 * pair(x) + 16 * u + 4 * g) - 3, 0));
    const float across = power(e, kChunk);

    // (reads of LDS for all products at once would, too)
    auto issued = [] { asm volatile("" ::: "memory"); };
    const float own_row = float(4 * g);
    for (int c = 0; c < chunks; ++c) {
      const int n = tokens_in(c), shift = kChunk - n;
      fetch(c);
      kr.store(ks, n, shift, tid);
      qr.store(qs, n, shift, tid);
      vr.store(vs, n, shift, tid);
      orow.store(os, n, shift, tid);
      __syncthreads();
      // (products of the factors made ahead of the loop would fill the registers)
      float base = own_row;
      asm volatile("" : "+v"(base));
#pragma unroll
      for (int r = 0; r < 4; ++r) asm volatile("" : "+v"(down[r]), "+v"(up[r]));
      // pairs inside the chunk, keys by queries
      {
        Exact qf[kBk], of[kBv];
#pragma unroll
        for (int bb = 0; bb < kBk; ++bb) qf[bb] = row_frag<kPk>(qs, 16 * rw + c16, bb, g);
#pragma unroll
        for (int bb = 0; bb < kBv; ++bb) of[bb] = row_frag<kPv>(os, 16 * rw + c16, bb, g);
#pragma unroll
        for (int x = 0; x < kPairs; ++x)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int block = 2 * pair(x) + u;
            if (block > rw) continue;   // all behind these queries
            issued();
            f32x4 p = frag::zero4(), d = frag::zero4();
#pragma unroll
            for (int bb = 0; bb < kBk; ++bb) p = mma(row_frag<kPk>(ks, 16 * block + c16, bb, g), qf[bb], p);
#pragma unroll
            for (int bb = 0; bb < kBv; ++bb) d = mma(row_frag<kPv>(vs, 16 * block + c16, bb, g), of[bb], d);
            float sum = 0.0f;
            const float gap = float(16 * (rw - block) + c16) - base;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float weight = block == rw ? own[r] : to_query[x][u] * down[r] * (gap - float(r));
              // (a product with the mask's zero would keep what is not finite)
              sum = weight != 0.0f ? __builtin_fmaf(p[r] * weight, d[r], sum) : sum;
            }
            pairs += double(sum);
          }
      }
      // Rows by columns over half of the chunk's tokens: an operand of decayed rows, and of the
      // same counted.
      auto operands = [&](const IO* rows, int m, int j, const f32x4 (&weight)[2], float first_count, float each, Split& plain,
                          Split& counted) __attribute__((always_inline)) {
        const Exact x = turned_frag<kPv>(rows, m, 16 * column(j), g, c16);
        f32x4 part[2], times[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          part[u] = widened(x, u);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            part[u][r] *= weight[u][r];
            times[u][r] = part[u][r] * (first_count + each * float(16 * u + r));
          }
        }
        split(part[0], part[1], plain);
        split(times[0], times[1], counted);
      };
      if (works) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          f32x4 weight[2];
          if (n == kChunk) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int r = 0; r < 4; ++r) weight[u][r] = to_start[m][u] * up[r];
          } else {   // (rows ahead of a short chunk's tokens are zero)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int r = 0; r < 4; ++r) weight[u][r] = power(e, max(32 * m + 16 * u + 4 * g + r + 1 - shift, 0));
          }
#pragma unroll
          for (int j = 0; j < kOwn; ++j) {
            Split plain, counted;
            operands(os, m, j, weight, base + float(32 * m + 1 - shift), 1.0f, plain, counted);
            Exact x = turned_frag<kPk>(qs, m, 16 * row_tile(0), g, c16);
#pragma unroll
            for (int y = 0; y < kMine; ++y) {
              const Exact next = turned_frag<kPk>(qs, m, 16 * row_tile(y + 1 < kMine ? y + 1 : y), g, c16);
              issued();
              float sum = 0.0f;
              const f32x4 a1 = mma(x, counted, frag::zero4());
#pragma unroll
              for (int r = 0; r < 4; ++r) sum = __builtin_fmaf(S[j][y][r], a1[r], sum);
              if (c > 0) {   // (D is zero at the tile's start)
                const f32x4 a0 = mma(x, plain, frag::zero4());
#pragma unroll
                for (int r = 0; r < 4; ++r) sum = __builtin_fmaf(D[j][y][r], a0[r], sum);
              }
              reads += double(sum);
              x = next;
            }
          }
        }
        // (also where no one reads the result: a branch around it costs copies of both states.  The
        // chunk's sums are made from zero and added once: a product added to the states would be
        // rounded at their size each time, 16 times a chunk in float32.)
        const float whole = n == kChunk ? across : power(e, n), tokens = float(n);
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          f32x4 s0[kMine], s1[kMine];
#pragma unroll
          for (int y = 0; y < kMine; ++y) s0[y] = s1[y] = frag::zero4();
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            f32x4 weight[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int r = 0; r < 4; ++r) weight[u][r] = to_end[m][u] * down[r];
            Split plain, counted;
            operands(vs, m, j, weight, float(kChunk - 1 - 32 * m) - base, -1.0f, plain, counted);
            Exact x = turned_frag<kPk>(ks, m, 16 * row_tile(0), g, c16);
#pragma unroll
            for (int y = 0; y < kMine; ++y) {
              const Exact next = turned_frag<kPk>(ks, m, 16 * row_tile(y + 1 < kMine ? y + 1 : y), g, c16);
              issued();
              if (sizeof(IO) == 2 || m == 0) {
                s0[y] = mma(x, plain, s0[y]);
                s1[y] = mma(x, counted, s1[y]);
              } else {   // (16 products in a row are rounded more than two halves)
                s0[y] = s0[y] + mma(x, plain, frag::zero4());
                s1[y] = s1[y] + mma(x, counted, frag::zero4());
              }
              x = next;
            }
          }
#pragma unroll
          for (int y = 0; y < kMine; ++y) {
            D[j][y] = (D[j][y] + S[j][y] * tokens) * whole + s1[y];
            S[j][y] = S[j][y] * whole + s0[y];
          }
        }
      }
      __syncthreads();
    }
    if (a.R && works) {
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
#pragma unroll
        for (int y = 0; y < kMine; ++y) {
          const float* p = a.R + (bh * a.r_each + tile) * (DK * DV) + element(j, y);
#pragma unroll
          for (int r = 0; r < 4; ++r) behind = __builtin_fma(double(D[j][y][r]), double(p[r * DV]), behind);
        }
    }
  }
  double sum = __builtin_fma(pairs + reads, double(a.read), behind);
#pragma unroll
  for (int m = 32; m > 0; m /= 2) sum += __shfl_xor(sum, m);
  if (l == 0) sums[w] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kWaves; ++i) sum += sums[i];
    a.parts[(int64_t(b) * a.tiles + tile) * a.H + h] = float(sum);
  }
}

template <typename IO, int DK, int DV>
hipError_t launch_decays(const LinearDecays& a, hipStream_t st) {
  constexpr int lds = decay_lds<IO, DK, DV>();
  static_assert(lds + 64 <= 160 * 1024);
  return launch(decay_kernel<IO, DK, DV>, uint32_t(a.heads * a.tiles), 64 * decay_waves<DK, DV>(), lds, a, st);
}
template <int DK>
hipError_t decays_of(const LinearDecays& a, hipStream_t st) {
  return by_width(a.dv, [&](auto dv) { return a.bf16 ? launch_decays<bf16_t, DK, dv()>(a, st) : launch_decays<float, DK, dv()>(a, st); });
}

}  // namespace linear
}  // namespace falcon
