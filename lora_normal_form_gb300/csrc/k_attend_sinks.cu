// The one-token attention (k_attend.cuh) of windows whose first tokens stay visible.
#include "k_attend.cuh"

namespace scute {

cudaError_t launch_attend_sinks(const AttendArgs &a, int num_sms, cudaStream_t st) { return launch_attend_mode<SINKS>(a, num_sms, st); }

}  // namespace scute
