// ngr_attend_bf16.cu -- the paged attention's kernels for bf16.
#include "ngr_attend.cuh"

namespace ngr {
int launch_attend_bf16(const AttendArgs &a, cudaStream_t stream) { return run_attend<true, false>(a, stream); }
int launch_attend_join_bf16(const AttendArgs &a, cudaStream_t stream) { return run_join<true>(a, stream); }
}  // namespace ngr
