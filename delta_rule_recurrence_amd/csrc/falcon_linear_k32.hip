// Sweeps of linear attention over keys of 32.
#include "falcon_linear_decay.h"

namespace falcon {

hipError_t launch_linear_sums_32(const LinearSweep& s, const LinearSweep* second, hipStream_t st) {
  return linear::sums_of<32>(s, second, st);
}
hipError_t launch_linear_outputs_32(const LinearSweep& s, hipStream_t st) { return linear::outputs_of<32>(s, st); }
hipError_t launch_linear_gradients_32(const LinearSweep& dv, const LinearSweep& dk, const LinearSweep& dq, hipStream_t st) {
  return linear::gradients_of<32>(dv, dk, dq, st);
}
hipError_t launch_linear_decays_32(const LinearDecays& a, hipStream_t st) { return linear::decays_of<32>(a, st); }

}  // namespace falcon
