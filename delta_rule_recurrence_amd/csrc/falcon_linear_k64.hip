// Sweeps of linear attention over keys of 64.
#include "falcon_linear_kernel.h"

namespace falcon {

hipError_t launch_linear_sweep_64(const LinearSweep& s, hipStream_t st) { return linear::sweep_of<64>(s, st); }

}  // namespace falcon
