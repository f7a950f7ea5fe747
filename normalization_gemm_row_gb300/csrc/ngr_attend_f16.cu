// ngr_attend_f16.cu -- the paged attention's kernels for f16.
#define NGR_ATTEND_TYPE f16
#define NGR_ATTEND_BF16 false
#include "ngr_attend.cuh"
