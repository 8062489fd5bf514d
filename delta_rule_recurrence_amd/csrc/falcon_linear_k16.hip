// Sweeps of linear attention over keys of 16.
#include "falcon_linear_kernel.h"

namespace falcon {

hipError_t launch_linear_sweep_16(const LinearSweep& s, hipStream_t st) { return linear::sweep_of<16>(s, st); }

}  // namespace falcon
