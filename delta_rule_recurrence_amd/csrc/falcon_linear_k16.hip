// Sweeps of linear attention over keys of 16.
#include "falcon_linear_decay.h"

namespace falcon {

hipError_t launch_linear_sums_16(const LinearSweep& s, const LinearSweep* second, hipStream_t st) {
  return linear::sums_of<16>(s, second, st);
}
hipError_t launch_linear_outputs_16(const LinearSweep& s, hipStream_t st) { return linear::outputs_of<16>(s, st); }
hipError_t launch_linear_gradients_16(const LinearSweep& dv, const LinearSweep& dk, const LinearSweep& dq, hipStream_t st) {
  return linear::gradients_of<16>(dv, dk, dq, st);
}
hipError_t launch_linear_decays_16(const LinearDecays& a, hipStream_t st) { return linear::decays_of<16>(a, st); }

}  // namespace falcon
