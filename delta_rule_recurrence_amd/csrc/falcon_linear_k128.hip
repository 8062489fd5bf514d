// Sweeps of linear attention over keys of 128.
#include "falcon_linear_kernel.h"

namespace falcon {

hipError_t launch_linear_sweep_128(const LinearSweep& s, hipStream_t st) { return linear::sweep_of<128>(s, st); }

}  // namespace falcon
