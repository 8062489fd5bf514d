// Sweeps of linear attention over keys of 64.
#include "falcon_linear_decay.h"

namespace falcon {

hipError_t launch_linear_sums_64(const LinearSweep& s, const LinearSweep* second, hipStream_t st) {
  return linear::sums_of<64>(s, second, st);
}
hipError_t launch_linear_outputs_64(const LinearSweep& s, hipStream_t st) { return linear::outputs_of<64>(s, st); }
hipError_t launch_linear_gradients_64(const LinearSweep& dv, const LinearSweep& dk, const LinearSweep& dq, hipStream_t st) {
  return linear::gradients_of<64>(dv, dk, dq, st);
}
hipError_t launch_linear_decays_64(const LinearDecays& a, hipStream_t st) { return linear::decays_of<64>(a, st); }

}  // namespace falcon
