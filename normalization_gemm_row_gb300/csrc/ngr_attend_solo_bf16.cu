// ngr_attend_solo_bf16.cu -- the paged attention's kernels for bf16 that take an
// item with one CTA.
#include "ngr_attend.cuh"

namespace ngr {
int launch_attend_solo_bf16(const AttendArgs &a, cudaStream_t stream) { return run_attend<true, true>(a, stream); }
}  // namespace ngr
