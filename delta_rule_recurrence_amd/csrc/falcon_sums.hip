// Sums of rows of partial sums (gfx950): the last step of the parameter
// gradients.  A workgroup sums 64 columns; its sixteen waves take every sixteenth
// row each, several loads in flight, and their sums (in double) meet in LDS in
// order, so the result does not depend on how the work ran.

#include <algorithm>

#include "falcon_block.h"

namespace falcon {

namespace {

constexpr int kSlices = 16;
constexpr int kInFlight = 8;

__global__ __launch_bounds__(64 * kSlices) void sum_parts_kernel(PartSums s) {
  __shared__ double sums[kSlices][64];
  const int lane = threadIdx.x % 64, slice = threadIdx.x / 64;
  for (int64_t c0 = int64_t(blockIdx.x) * 64; c0 < s.n; c0 += int64_t(gridDim.x) * 64) {
    const int64_t i = c0 + lane;
    double v = 0.0;
    if (i < s.n) {
      int64_t p = slice;
      for (; p + (kInFlight - 1) * kSlices < s.parts; p += kInFlight * kSlices) {
        float x[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) x[k] = s.in[(p + k * kSlices) * s.row + i];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) v += x[k];
      }
      for (; p < s.parts; p += kSlices) v += s.in[p * s.row + i];
    }
    sums[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && i < s.n) {
      double all = 0.0;
#pragma unroll
      for (int k = 0; k < kSlices; ++k) all += sums[k][lane];
      const int which = i < s.ends[0] ? 0 : i < s.ends[1] ? 1 : 2;
      float* out = s.out[which];
      if (out) out[i - (which == 0 ? 0 : s.ends[which - 1])] = float(all);
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_sum_parts(const PartSums& s, hipStream_t st) {
  const int64_t blocks = std::min<int64_t>((s.n + 63) / 64, 1 << 16);
  sum_parts_kernel<<<dim3(unsigned(blocks)), dim3(64 * kSlices), 0, st>>>(s);
  return hipGetLastError();
}

}  // namespace falcon
