// The one-token attention (k_attend.cuh) of the tokens behind those that a group shares.
#include "k_attend.cuh"

namespace scute {

cudaError_t launch_attend_own(const AttendArgs &a, int num_sms, cudaStream_t st) { return launch_attend_mode<SHARED>(a, num_sms, st); }

}  // namespace scute
