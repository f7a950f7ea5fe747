// ngr_attend_f16.cu -- the paged attention's kernels for f16.
#include "ngr_attend.cuh"

namespace ngr {
int launch_attend_f16(const AttendArgs &a, cudaStream_t stream) { return run_attend<false, false>(a, stream); }
int launch_attend_join_f16(const AttendArgs &a, cudaStream_t stream) { return run_join<false>(a, stream); }
}  // namespace ngr
