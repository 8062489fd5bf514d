// Linear attention with a decay for each head (gfx950): how its sweeps follow one
// another, the states between tiles and single tokens.
//
//   S_t = exp(log_decay) S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t
//
// A head's tokens are cut into tiles of whole chunks.  Since a tile adds to a state
// whatever state it meets, the tiles' sums are made first, all at once; a pass over
// them, an element of the state a thread, leaves in each tile's slot the state that
// enters it; then every tile runs from there.  A head that is one tile takes the last
// step alone.

#include <algorithm>

#include "falcon_block_device.h"
#include "falcon_launch.h"
#include "falcon_linear_kernel.h"

namespace falcon {

namespace {

using linear::kChunk;
using linear::power;

// How a head's tokens are cut.
struct Tiles {
  int64_t heads;
  int chunks, tiles;   // chunks of a tile; tiles of a head
};

Tiles cut(const LinearArgs& a, bool bwd) {
  const int64_t heads = int64_t(a.B) * a.H, all = (int64_t(a.T) + kChunk - 1) / kChunk;
  // tiles of a head for three workgroups a CU, or for the two or one that wide heads leave room
  // for (kernels of a prompt together, when this was chosen: 8 x 2048 x 12 x 64, 384 tiles 60 us,
  // 768 56 us, 1536 62 us; 16384 x 12 x 128 x 128, 256 tiles 105 us, 512 113 us, 768 119 us)
  const int64_t all_tiles = a.dk * a.dv > 64 * 128 ? 256 : a.dk * a.dv > 64 * 64 ? 512 : 768;
  const int64_t want = std::max<int64_t>(1, all_tiles / std::max<int64_t>(heads, 1));   // (one more would take a round of its own)
  // A short prompt's heads take one tile each: one launch for three, and no states between
  // tiles.  us of a call / of a replay, one tile and several.  Outputs in bfloat16, 8 heads: 4 chunks
  // of 64 x 64 16/16 and 21/12, of 64 x 128 19/19 and 21/14, of 128 x 128 22/22 and 21/16 (2 chunks 14/13 and
  // 21/16); 96 heads: 4 chunks of 64 x 64 17/17 and 21/21, 8 chunks 30/30 and 25/26, of 64 x 128 34/35 and
  // 35/35, of 128 x 128 41/42 and 49/50.  float32, 8 heads: 2 chunks of 64 x 64 14/14 and 21/14, of 128 x
  // 128 31/31 and 26/25 (1 chunk 18 both); 96 heads: 4 chunks 25/26 and 26/26, of 128 x 128 59/60 and 61/61,
  // 8 chunks 47/48 and 37/38.  Gradients in bfloat16, 8 heads: 4 chunks of 64 x 64 18/15 and 24/12; 96
  // heads: 8 chunks 35/35 and 44/44, of 128 x 128 76/76 and 106/106; float32, 8 heads: 2 chunks of 128 x 128
  // 26/26 and 28/27; 96 heads: 4 chunks of 64 x 64 38/37 and 44/45.  (So a call by itself decides for few heads:
  // a replay of 4 chunks would rather have several tiles.)
  const int64_t base = a.bf16 ? 4 : 2, size = a.dk * a.dv;
  const bool twice = heads >= 64 && (bwd || !a.bf16 || size >= 64 * 128), half = heads < 64 && !bwd && size > 64 * 128;
  const int64_t few = twice ? 2 * base : half ? base / 2 : base;
  const int64_t chunks = all <= few ? std::max<int64_t>(all, 1) : std::max<int64_t>(1, (all + want - 1) / want);
  return {heads, int(chunks), int(std::max<int64_t>(1, (all + chunks - 1) / chunks))};
}

// ---- states between tiles -----------------------------------------------------------
// Slot of tile t holds what the tile adds; it gets the state that enters the tile.
// Against time the tiles follow one another from the last to the first, and the state
// that leaves the first goes to slot 0.
constexpr int kAhead = 16;   // slots in flight

struct Carry {
  float* slots;
  int64_t slots_each;
  int slot0;
  const float* start;      // may be null (zero)
  float* last;             // may be null
  bool rev;
};
struct Carries {
  Carry c[2];              // one or two of the same sizes
  const float* log_decay;
  const int32_t* lengths;
  int H, T, tiles, chunks, size;   // size: elements of a state
};

// The state passes the tiles in double: in float32 each would leave a rounding and the error of
// its decay in all states behind it (250 tiles that hardly forget: 135 units of 2^-24 against 1),
// and the decays' gradient, which adds up their products with the adjoints, would show it.  1.5 of 12 us
// at 8 x 2048 x 12 x 64, both ways.  A workgroup a head, 256 elements of its state and a carry.
// (Heads of several tiles are at most 384: more are a tile each.)
__global__ __launch_bounds__(256) void carry_kernel(Carries a) {
  const Carry c = a.c[blockIdx.z];
  const uint32_t bh = blockIdx.x;
  const int e = int(blockIdx.y * 256 + threadIdx.x);
  const int64_t at = int64_t(bh) * a.size + e;
  const int b = int(bh / uint32_t(a.H)), h = int(bh % uint32_t(a.H));
  const int len = tokens_of(a.lengths, b, a.T), tokens = a.chunks * kChunk;
  const double log2_a = double(a.log_decay[h]) * 1.4426950408889634;   // log2(e)
  double s = c.start ? c.start[at] : 0.0f;
  float* const slots = c.slots + (bh * c.slots_each + c.slot0) * a.size + e;
  const int used = min((len + tokens - 1) / tokens, a.tiles);
  const double whole = exp2(log2_a * tokens), end = exp2(log2_a * (len - (used - 1) * tokens));   // of a tile, of the last one
  for (int base = 0; base < used; base += kAhead) {
    float add[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int t = min(base + k, used - 1);
      add[k] = slots[int64_t(c.rev ? used - 1 - t : t) * a.size];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (base + k < used) {
        const int t = c.rev ? used - 1 - base - k : base + k;
        slots[int64_t(t) * a.size] = float(s);
        s = __builtin_fma(s, t == used - 1 ? end : whole, double(add[k]));
      }
    }
  }
  if (c.rev && c.slot0 > 0) slots[-int64_t(a.size)] = float(s);
  if (c.last) c.last[at] = float(s);
}

hipError_t launch_carry(const LinearArgs& l, const Tiles& t, const Carry& c, const Carry* second, hipStream_t st) {
  const int size = l.dk * l.dv;
  carry_kernel<<<dim3(unsigned(t.heads), unsigned(size / 256), second ? 2 : 1), dim3(256), 0, st>>>(
      {{c, second ? *second : c}, l.log_decay, l.lengths, l.H, l.T, t.tiles, t.chunks, size});
  return hipGetLastError();
}

#define FALCON_BY_KEYS(what, dk, ...)                         \
  ((dk) == 16   ? launch_linear_##what##_16(__VA_ARGS__)      \
   : (dk) == 32 ? launch_linear_##what##_32(__VA_ARGS__)      \
   : (dk) == 64 ? launch_linear_##what##_64(__VA_ARGS__)      \
                : launch_linear_##what##_128(__VA_ARGS__))

// What the sweeps of one call share.
LinearSweep sweep_base(const LinearArgs& a, const Tiles& t) {
  LinearSweep s{};
  s.log_decay = a.log_decay;
  s.lengths = a.lengths;
  s.heads = t.heads;
  s.H = a.H;
  s.T = a.T;
  s.tiles = t.tiles;
  s.chunks = t.chunks;
  s.bf16 = a.bf16;
  s.read = s.write = 1.0f;
  return s;
}

// ---- single tokens ---------------------------------------------------------------------
// A workgroup a head, four columns of the state and every (threads / (dv / 4))-th row a
// thread; the threads' parts of the read meet in LDS.  Bound by the state, read and
// written once (512 x 12 x 128 x 128: 162 us from memory, 5.0 TB/s).
template <typename IO>
__global__ __launch_bounds__(256) void linear_step_kernel(const IO* __restrict__ q, int64_t q_row, const IO* __restrict__ k, int64_t k_row,
                                                          const IO* __restrict__ v, int64_t v_row, const float* __restrict__ log_decay,
                                                          float* __restrict__ S, const uint8_t* __restrict__ is_first, IO* __restrict__ o,
                                                          int H, int dk, int dv, float scale) {
  __shared__ float4 parts[256];
  const int64_t bh = blockIdx.x;
  const int b = int(bh / H), h = int(bh % H);
  const int cols = dv / 4, col = threadIdx.x % cols, row0 = threadIdx.x / cols, step = blockDim.x / cols;
  const float a = is_first && is_first[b] ? 0.0f : power(log_decay[h] * kLog2e, 1);
  const bool fresh = is_first && is_first[b];
  q += b * q_row + int64_t(h) * dk;
  k += b * k_row + int64_t(h) * dk;
  float vv[4];
  load_vec<IO, 4>(v + b * v_row + int64_t(h) * dv + 4 * col, vv);
  float* const mine = S + bh * dk * dv + 4 * col;
  float4 sum = make_float4(0, 0, 0, 0);
  for (int f0 = row0; f0 < dk; f0 += 8 * step) {
    float4 s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int f = f0 + i * step;
      s[i] = make_float4(0, 0, 0, 0);
      if (f < dk && !fresh) s[i] = *reinterpret_cast<const float4*>(mine + int64_t(f) * dv);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int f = f0 + i * step;
      if (f < dk) {
        const float kf = io<IO>::load(k, f), qf = io<IO>::load(q, f);
        s[i].x = __builtin_fmaf(s[i].x, a, kf * vv[0]);
        s[i].y = __builtin_fmaf(s[i].y, a, kf * vv[1]);
        s[i].z = __builtin_fmaf(s[i].z, a, kf * vv[2]);
        s[i].w = __builtin_fmaf(s[i].w, a, kf * vv[3]);
        *reinterpret_cast<float4*>(mine + int64_t(f) * dv) = s[i];
        sum.x = __builtin_fmaf(s[i].x, qf, sum.x);
        sum.y = __builtin_fmaf(s[i].y, qf, sum.y);
        sum.z = __builtin_fmaf(s[i].z, qf, sum.z);
        sum.w = __builtin_fmaf(s[i].w, qf, sum.w);
      }
    }
  }
  parts[threadIdx.x] = sum;
  __syncthreads();
  if (int(threadIdx.x) < cols) {
    for (int r = 1; r < step; ++r) {
      const float4 p = parts[r * cols + col];
      sum.x += p.x;
      sum.y += p.y;
      sum.z += p.z;
      sum.w += p.w;
    }
    const float out[4] = {sum.x * scale, sum.y * scale, sum.z * scale, sum.w * scale};
    store_vec<IO, 4>(o + bh * dv + 4 * col, out);
  }
}

template <typename IO>
hipError_t step_of(const LinearArgs& a, hipStream_t st) {
  const int threads = std::min(256, a.dk * a.dv / 4);
  linear_step_kernel<IO><<<dim3(unsigned(int64_t(a.B) * a.H)), dim3(threads), 0, st>>>(
      static_cast<const IO*>(a.q), a.q_at.b, static_cast<const IO*>(a.k), a.k_at.b, static_cast<const IO*>(a.v), a.v_at.b,
      a.log_decay, a.S, a.is_first, static_cast<IO*>(a.o), a.H, a.dk, a.dv, a.scale);
  return hipGetLastError();
}

// ---- gradients -------------------------------------------------------------------------
// Workspace of the gradients: S slots and R slots (one more) where heads have several tiles,
// rows of partial sums of the decays' gradient.
struct BwdLayout {
  int64_t S, R, parts;   // floats
  BwdLayout(const LinearArgs& a, const Tiles& t) {
    const int64_t size = int64_t(a.dk) * a.dv;
    S = t.tiles > 1 ? t.heads * t.tiles * size : 0;
    R = t.tiles > 1 ? t.heads * (t.tiles + 1) * size : 0;
    parts = int64_t(a.B) * t.tiles * a.H;
  }
};

}  // namespace

size_t linear_workspace_bytes(const LinearArgs& a) {
  const Tiles t = cut(a, false);
  return t.tiles > 1 ? size_t(t.heads) * t.tiles * a.dk * a.dv * sizeof(float) : 0;
}

hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t st) {
  if (a.T == 0) return launch_state_copy(a.S0, a.S_T, int64_t(a.B) * a.H * a.dk * a.dv, st);
  const Tiles t = cut(a, false);
  LinearSweep s = sweep_base(a, t);
  s.k = a.k; s.v = a.v;
  s.k_at = a.k_at; s.v_at = a.v_at;
  s.dv = a.dv;
  s.sf = a.dv; s.sc = 1;
  hipError_t e = hipSuccess;
  if (t.tiles > 1) {
    s.slots = a.workspace;
    s.slots_each = t.tiles;
    e = FALCON_BY_KEYS(sums, a.dk, s, nullptr, st);
    if (e != hipSuccess) return e;
    e = launch_carry(a, t, {a.workspace, t.tiles, 0, a.S0, a.S_T, false}, nullptr, st);
    if (e != hipSuccess) return e;
  } else {
    s.start = a.S0;
    s.last = a.S_T;
  }
  s.q = a.q; s.q_at = a.q_at;
  s.out = a.o; s.out_at = a.o_at;
  s.read = a.scale;
  s.clear = a.zero_behind && a.lengths;
  return FALCON_BY_KEYS(outputs, a.dk, s, st);
}

hipError_t launch_linear_step(const LinearArgs& a, hipStream_t st) { return a.bf16 ? step_of<bf16_t>(a, st) : step_of<float>(a, st); }

size_t linear_bwd_workspace_bytes(const LinearArgs& a) {
  const BwdLayout l(a, cut(a, true));
  return size_t(l.S + l.R + l.parts) * sizeof(float);
}

hipError_t launch_linear_bwd(const LinearArgs& a, hipStream_t st) {
  const Tiles t = cut(a, true);
  const BwdLayout l(a, t);
  float* const S = a.workspace;
  float* const R = S + l.S;
  float* const parts = R + l.R;
  const int size = a.dk * a.dv;
  if (t.heads == 0) return launch_sum_parts({parts, 0, a.H, a.H, {a.dlog_decay, nullptr, nullptr}, {a.H, a.H}}, st);
#define FALCON_TRY(call)                   \
  do {                                     \
    const hipError_t e_ = (call);          \
    if (e_ != hipSuccess) return e_;       \
  } while (0)
  // what each tile adds to the state, and to its adjoint, where a head has several
  const bool several = t.tiles > 1;
  LinearSweep s = sweep_base(a, t);
  s.k = a.k; s.v = a.v;
  s.k_at = a.k_at; s.v_at = a.v_at;
  s.dv = a.dv;
  s.sf = a.dv; s.sc = 1;
  if (several) s.slots = S, s.slots_each = t.tiles;
  LinearSweep r = sweep_base(a, t);
  r.k = a.q; r.v = a.dO;
  r.k_at = a.q_at; r.v_at = a.o_at;
  r.dv = a.dv;
  r.sf = a.dv; r.sc = 1;
  if (several) r.slots = R, r.slots_each = t.tiles + 1, r.slot0 = 1;
  r.rev = true;
  s.clear = r.clear = a.lengths != nullptr;
  r.write = a.scale;
  if (several) {
    FALCON_TRY(FALCON_BY_KEYS(sums, a.dk, s, &r, st));
    const Carry back{R, t.tiles + 1, 1, a.dS_T, a.dS0, true};
    FALCON_TRY(launch_carry(a, t, {S, t.tiles, 0, a.S0, nullptr, false}, &back, st));
  } else {
    s.start = a.S0;
    r.start = a.dS_T;
  }
  // dv = (k, q, dO) against time
  LinearSweep dv = r;
  dv.q = a.k; dv.q_at = a.k_at;
  dv.out = a.dv_out; dv.out_at = a.dv_at;
  if (!several) dv.last = a.dS0;
  // dk = (v, dO, q) against time, from the transposed adjoint
  LinearSweep dk = r;
  dk.q = a.v; dk.q_at = a.v_at;
  dk.k = a.dO; dk.k_at = a.o_at;
  dk.v = a.q; dk.v_at = a.q_at;
  dk.dv = a.dk;
  dk.sf = 1; dk.sc = a.dv;
  dk.out = a.dk_out; dk.out_at = a.dqk_at;
  // dq = (dO, v, k), from the transposed state
  LinearSweep dq = s;
  dq.q = a.dO; dq.q_at = a.o_at;
  dq.k = a.v; dq.k_at = a.v_at;
  dq.v = a.k; dq.v_at = a.k_at;
  dq.dv = a.dk;
  dq.sf = 1; dq.sc = a.dv;
  dq.read = a.scale;
  dq.out = a.dq; dq.out_at = a.dqk_at;
  FALCON_TRY(FALCON_BY_KEYS(gradients, a.dk, dv, dk, dq, st));
  if (a.dlog_decay) {
    LinearDecays d{};
    d.q = a.q; d.k = a.k; d.v = a.v; d.dO = a.dO;
    d.q_at = a.q_at; d.k_at = a.k_at; d.v_at = a.v_at; d.o_at = a.o_at;
    d.log_decay = a.log_decay;
    d.lengths = a.lengths;
    d.S = several ? S : a.S0;
    d.R = several ? R + size : a.dS_T;
    d.s_each = t.tiles;
    d.r_each = several ? t.tiles + 1 : 1;
    d.parts = parts;
    d.heads = t.heads;
    d.H = a.H; d.T = a.T; d.dv = a.dv; d.tiles = t.tiles; d.chunks = t.chunks;
    d.read = a.scale;
    d.bf16 = a.bf16;
    FALCON_TRY(FALCON_BY_KEYS(decays, a.dk, d, st));
    FALCON_TRY(launch_sum_parts({parts, int64_t(a.B) * t.tiles, a.H, a.H, {a.dlog_decay, nullptr, nullptr}, {a.H, a.H}}, st));
  }
#undef FALCON_TRY
  return hipSuccess;
}

}  // namespace falcon
