// ngr_attend_bf16.cu -- the paged attention's kernels for bf16.
#define NGR_ATTEND_TYPE bf16
#define NGR_ATTEND_BF16 true
#include "ngr_attend.cuh"
