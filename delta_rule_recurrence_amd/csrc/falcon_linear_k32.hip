// Sweeps of linear attention over keys of 32.
#include "falcon_linear_kernel.h"

namespace falcon {

hipError_t launch_linear_sweep_32(const LinearSweep& s, hipStream_t st) { return linear::sweep_of<32>(s, st); }

}  // namespace falcon
