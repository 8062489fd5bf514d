// Linear attention with a decay for each head (gfx950): how its sweeps follow one
// another, the states between tiles, single tokens and the decays' gradient.
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

Tiles cut(const LinearArgs& a) {
  const int64_t heads = int64_t(a.B) * a.H, all = (int64_t(a.T) + kChunk - 1) / kChunk;
  const int64_t want = std::max<int64_t>(1, (768 + heads - 1) / std::max<int64_t>(heads, 1));   // tiles of a head for three a CU
  const int64_t chunks = std::max<int64_t>(2, (all + want - 1) / want);
  return {heads, int(chunks), int(std::max<int64_t>(1, (all + chunks - 1) / chunks))};
}

// ---- states between tiles -----------------------------------------------------------
// Slot of tile t holds what the tile adds; it gets the state that enters the tile.
// Against time the tiles follow one another from the last to the first, and the state
// that leaves the first goes to slot 0.
constexpr int kAhead = 8;   // slots in flight

struct Carry {
  float* slots;
  int64_t slots_each;
  int slot0;
  const float* start;      // may be null (zero)
  float* last;             // may be null
  const float* log_decay;
  const int32_t* lengths;
  int64_t heads;
  int H, T, tiles, chunks, size;   // size: elements of a state
  bool rev;
};

__global__ __launch_bounds__(256) void carry_kernel(Carry c) {
  const int64_t each = c.size / 4;
  const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (at >= c.heads * each) return;
  const int64_t bh = at / each;
  const int64_t e = (at - bh * each) * 4;
  const int b = int(bh / c.H), h = int(bh % c.H);
  const int len = tokens_of(c.lengths, b, c.T), tokens = c.chunks * kChunk;
  const float log2_a = c.log_decay[h] * kLog2e;
  float4 s = make_float4(0, 0, 0, 0);
  if (c.start) s = *reinterpret_cast<const float4*>(c.start + bh * c.size + e);
  float* const slots = c.slots + (bh * c.slots_each + c.slot0) * c.size + e;
  const int used = min((len + tokens - 1) / tokens, c.tiles);
  const float whole = power(log2_a, tokens);
  auto slot = [&](int t) { return reinterpret_cast<float4*>(slots + int64_t(t) * c.size); };
  for (int base = 0; base < used; base += kAhead) {
    float4 add[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int t = min(base + k, used - 1);
      add[k] = *slot(c.rev ? used - 1 - t : t);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (base + k < used) {
        const int t = c.rev ? used - 1 - base - k : base + k;
        *slot(t) = s;
        const float across = t == used - 1 ? power(log2_a, len - t * tokens) : whole;
        s.x = __builtin_fmaf(s.x, across, add[k].x);
        s.y = __builtin_fmaf(s.y, across, add[k].y);
        s.z = __builtin_fmaf(s.z, across, add[k].z);
        s.w = __builtin_fmaf(s.w, across, add[k].w);
      }
    }
  }
  if (c.rev && c.slot0 > 0) *slot(-1) = s;
  if (c.last) *reinterpret_cast<float4*>(c.last + bh * c.size + e) = s;
}

hipError_t launch_carry(const Carry& c, hipStream_t st) {
  carry_kernel<<<dim3(unsigned((c.heads * (c.size / 4) + 255) / 256)), dim3(256), 0, st>>>(c);
  return hipGetLastError();
}

hipError_t launch_sweep(const LinearSweep& s, int dk, hipStream_t st) {
  switch (dk) {
    case 16: return launch_linear_sweep_16(s, st);
    case 32: return launch_linear_sweep_32(s, st);
    case 64: return launch_linear_sweep_64(s, st);
    default: return launch_linear_sweep_128(s, st);
  }
}

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
// written once.
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

// ---- the decays' gradient ------------------------------------------------------------------
// With R_t the adjoint of S_t, d log_decay = sum over t of X_t = a <S_(t-1), R_t>, and
//
//   X_(t+1) = <S_t, R_t> - q_t . dq_t = X_t + k_t . dk_t - q_t . dq_t
//
// so a tile of n tokens gives n X_1 + sum_j (n - 1 - j) (k_j . dk_j - q_j . dq_j), j from
// 0, with X_1 the product of the two states at its start.  Summed in double; a row of
// partial sums for each sequence and tile, a column for each head.
struct DecayGrad {
  const void* q;
  const void* k;
  HeadSteps q_at, k_at, d_at;
  const float* dq;
  const float* dk;
  const float* S;          // [heads][tiles] states that enter the tiles
  const float* R;          // [heads][tiles + 1]: slot t, the adjoint before tile t's first token
  const int32_t* lengths;
  float* parts;
  int H, T, d, tiles, chunks, size;
};

template <typename IO>
__global__ __launch_bounds__(256) void decay_grad_kernel(DecayGrad a) {
  __shared__ double sums[256];
  const int64_t bh = blockIdx.x / a.tiles;
  const int tile = int(blockIdx.x % a.tiles);
  const int b = int(bh / a.H), h = int(bh % a.H);
  const int first = tile * a.chunks * kChunk;
  const int n = min(tokens_of(a.lengths, b, a.T) - first, a.chunks * kChunk);
  double sum = 0.0;
  if (n > 0) {
    const float* s = a.S + (bh * a.tiles + tile) * a.size;
    const float* r = a.R + (bh * (a.tiles + 1) + tile) * a.size;
    for (int e = threadIdx.x; e < a.size; e += 256) sum += double(s[e]) * r[e];
    sum *= n;
    // d / 4 threads a token
    const int each = a.d / 4, part = threadIdx.x % each * 4;
    const int64_t at = b * a.d_at.b + h * a.d_at.h + part;
    const IO* q = static_cast<const IO*>(a.q) + b * a.q_at.b + h * a.q_at.h + part;
    const IO* k = static_cast<const IO*>(a.k) + b * a.k_at.b + h * a.k_at.h + part;
    for (int j = threadIdx.x / each; j < n; j += 256 / each) {
      const int64_t t = first + j;
      float qv[4], kv[4], dqv[4], dkv[4];
      load_vec<IO, 4>(q + t * a.q_at.t, qv);
      load_vec<IO, 4>(k + t * a.k_at.t, kv);
      load_vec<float, 4>(a.dq + at + t * a.d_at.t, dqv);
      load_vec<float, 4>(a.dk + at + t * a.d_at.t, dkv);
      double u = 0.0;
#pragma unroll
      for (int e = 0; e < 4; ++e) u += double(kv[e]) * dkv[e] - double(qv[e]) * dqv[e];
      sum += u * (n - 1 - j);
    }
  }
  sums[threadIdx.x] = sum;
  __syncthreads();
  for (int half = 128; half > 0; half /= 2) {
    if (int(threadIdx.x) < half) sums[threadIdx.x] += sums[threadIdx.x + half];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.parts[(int64_t(b) * a.tiles + tile) * a.H + h] = float(sums[0]);
}

// ---- zeros behind the sequences' ends --------------------------------------------------------
struct Tail {
  float* out;
  HeadSteps at;
  int d;
};
// A workgroup a head and a sequence's rows from its end on, all gradients.
__global__ __launch_bounds__(256) void tails_kernel(Tail x, Tail y, Tail z, const int32_t* lengths, int H, int T) {
  const int64_t bh = blockIdx.x;
  const int b = int(bh / H), h = int(bh % H);
  const int len = tokens_of(lengths, b, T);
  auto clear = [&](const Tail& p) {
    const int each = p.d / 4;
    float* out = p.out + b * p.at.b + h * p.at.h;
    for (int64_t i = threadIdx.x; i < int64_t(T - len) * each; i += 256)
      *reinterpret_cast<float4*>(out + (len + i / each) * p.at.t + i % each * 4) = make_float4(0, 0, 0, 0);
  };
  clear(x);
  clear(y);
  clear(z);
}

// Workspace of the gradients: S slots, R slots (one more), rows of partial sums.
struct BwdLayout {
  int64_t S, R, parts;   // floats
  BwdLayout(const LinearArgs& a, const Tiles& t) {
    const int64_t size = int64_t(a.dk) * a.dv;
    S = t.heads * t.tiles * size;
    R = t.heads * (t.tiles + 1) * size;
    parts = int64_t(a.B) * t.tiles * a.H;
  }
};

}  // namespace

size_t linear_workspace_bytes(const LinearArgs& a) {
  const Tiles t = cut(a);
  return t.tiles > 1 ? size_t(t.heads) * t.tiles * a.dk * a.dv * sizeof(float) : 0;
}

hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t st) {
  if (a.T == 0) return launch_state_copy(a.S0, a.S_T, int64_t(a.B) * a.H * a.dk * a.dv, st);
  const Tiles t = cut(a);
  LinearSweep s = sweep_base(a, t);
  s.k = a.k; s.v = a.v;
  s.k_at = a.k_at; s.v_at = a.v_at;
  s.dv = a.dv;
  s.sf = a.dv; s.sc = 1;
  hipError_t e = hipSuccess;
  if (t.tiles > 1) {
    s.slots = a.workspace;
    s.slots_each = t.tiles;
    e = launch_sweep(s, a.dk, st);
    if (e != hipSuccess) return e;
    const Carry c{a.workspace, t.tiles, 0, a.S0, a.S_T, a.log_decay, a.lengths, t.heads, a.H, a.T, t.tiles, t.chunks, a.dk * a.dv, false};
    e = launch_carry(c, st);
    if (e != hipSuccess) return e;
  } else {
    s.start = a.S0;
    s.last = a.S_T;
  }
  s.q = a.q; s.q_at = a.q_at;
  s.out = a.o; s.out_at = a.o_at;
  s.out_bf16 = a.bf16;
  s.read = a.scale;
  return launch_sweep(s, a.dk, st);
}

hipError_t launch_linear_step(const LinearArgs& a, hipStream_t st) { return a.bf16 ? step_of<bf16_t>(a, st) : step_of<float>(a, st); }

size_t linear_bwd_workspace_bytes(const LinearArgs& a) {
  const BwdLayout l(a, cut(a));
  return size_t(l.S + l.R + l.parts) * sizeof(float);
}

hipError_t launch_linear_bwd(const LinearArgs& a, hipStream_t st) {
  const Tiles t = cut(a);
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
  // what each tile adds to the state, and to its adjoint
  LinearSweep s = sweep_base(a, t);
  s.k = a.k; s.v = a.v;
  s.k_at = a.k_at; s.v_at = a.v_at;
  s.dv = a.dv;
  s.sf = a.dv; s.sc = 1;
  s.slots = S; s.slots_each = t.tiles;
  FALCON_TRY(launch_sweep(s, a.dk, st));
  LinearSweep r = sweep_base(a, t);
  r.k = a.q; r.v = a.dO;
  r.k_at = a.q_at; r.v_at = a.o_at;
  r.dv = a.dv;
  r.sf = a.dv; r.sc = 1;
  r.slots = R; r.slots_each = t.tiles + 1; r.slot0 = 1;
  r.rev = true;
  r.write = a.scale;
  FALCON_TRY(launch_sweep(r, a.dk, st));
  FALCON_TRY(launch_carry({S, t.tiles, 0, a.S0, nullptr, a.log_decay, a.lengths, t.heads, a.H, a.T, t.tiles, t.chunks, size, false}, st));
  FALCON_TRY(launch_carry({R, t.tiles + 1, 1, a.dS_T, a.dS0, a.log_decay, a.lengths, t.heads, a.H, a.T, t.tiles, t.chunks, size, true}, st));
  // dv = (k, q, dO) against time
  r.q = a.k; r.q_at = a.k_at;
  r.out = a.dv_out; r.out_at = a.dv_at;
  FALCON_TRY(launch_sweep(r, a.dk, st));
  // dk = (v, dO, q) against time, from the transposed adjoint
  r.q = a.v; r.q_at = a.v_at;
  r.k = a.dO; r.k_at = a.o_at;
  r.v = a.q; r.v_at = a.q_at;
  r.dv = a.dk;
  r.sf = 1; r.sc = a.dv;
  r.out = a.dk_out; r.out_at = a.dqk_at;
  FALCON_TRY(launch_sweep(r, a.dv, st));
  // dq = (dO, v, k), from the transposed state
  s.q = a.dO; s.q_at = a.o_at;
  s.k = a.v; s.k_at = a.v_at;
  s.v = a.k; s.v_at = a.k_at;
  s.dv = a.dk;
  s.sf = 1; s.sc = a.dv;
  s.read = a.scale;
  s.out = a.dq; s.out_at = a.dqk_at;
  FALCON_TRY(launch_sweep(s, a.dv, st));
  if (a.lengths) {
    tails_kernel<<<dim3(unsigned(t.heads)), dim3(256), 0, st>>>({a.dq, a.dqk_at, a.dk}, {a.dk_out, a.dqk_at, a.dk}, {a.dv_out, a.dv_at, a.dv},
                                                                a.lengths, a.H, a.T);
    FALCON_TRY(hipGetLastError());
  }
  if (a.dlog_decay) {
    const DecayGrad d{a.q, a.k, a.q_at, a.k_at, a.dqk_at, a.dq, a.dk_out, S, R, a.lengths, parts, a.H, a.T, a.dk, t.tiles, t.chunks, size};
    const dim3 grid(unsigned(t.heads * t.tiles));
    if (a.bf16) {
      decay_grad_kernel<bf16_t><<<grid, dim3(256), 0, st>>>(d);
    } else {
      decay_grad_kernel<float><<<grid, dim3(256), 0, st>>>(d);
    }
    FALCON_TRY(hipGetLastError());
    FALCON_TRY(launch_sum_parts({parts, int64_t(a.B) * t.tiles, a.H, a.H, {a.dlog_decay, nullptr, nullptr}, {a.H, a.H}}, st));
  }
#undef FALCON_TRY
  return hipSuccess;
}

}  // namespace falcon
