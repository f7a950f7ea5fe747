// ngr_attend_solo_f16.cu -- the paged attention's kernels for f16 that take an
// item with one CTA.
#include "ngr_attend.cuh"

namespace ngr {
int launch_attend_solo_f16(const AttendArgs &a, cudaStream_t stream) { return run_attend<false, true>(a, stream); }
}  // namespace ngr
