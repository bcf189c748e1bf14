// The one-token attention (k_attend.cuh) of plain caches and windows.
#include "k_attend.cuh"

namespace scute {

size_t attend_part_floats(int num_sms) { return (size_t)num_sms * ATT_CTAS * 2 * PART_FLOATS; }
int attend_ctrs(int num_sms) { return num_sms * ATT_CTAS; }

cudaError_t launch_attend(const AttendArgs &a, int num_sms, cudaStream_t st) { return launch_attend_mode<PLAIN>(a, num_sms, st); }

}  // namespace scute
