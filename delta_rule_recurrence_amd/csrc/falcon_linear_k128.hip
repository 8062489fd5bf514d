// Sweeps of linear attention over keys of 128.
#include "falcon_linear_decay.h"

namespace falcon {

hipError_t launch_linear_sums_128(const LinearSweep& s, const LinearSweep* second, hipStream_t st) {
  return linear::sums_of<128>(s, second, st);
}
hipError_t launch_linear_outputs_128(const LinearSweep& s, hipStream_t st) { return linear::outputs_of<128>(s, st); }
hipError_t launch_linear_gradients_128(const LinearSweep& dv, const LinearSweep& dk, const LinearSweep& dq, hipStream_t st) {
  return linear::gradients_of<128>(dv, dk, dq, st);
}
hipError_t launch_linear_decays_128(const LinearDecays& a, hipStream_t st) { return linear::decays_of<128>(a, st); }

}  // namespace falcon
