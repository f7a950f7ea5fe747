// ngr_entry.h -- what the entry points outside ngr_api.cu share with those in
// it.  Not installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace ngr {

// A value of the device error word beside kDevErrTimeout: a target outside
// the vocabulary (reported as NGR_ERR_ARG).
enum : int { kDevErrTarget = 2 };

// The current device's SM count: NGR_OK, NGR_ERR_ARCH or NGR_ERR_CUDA.
int device_sms(int *sms);

// NGR_TRACE: every call prints the kernel variant it chose to stderr.
bool trace_mode();

// The kernel timing (ngr_kernel_timing_start): the call's begin, a pair
// around each launch; then the call's end, which reports launch errors and,
// with NGR_DEBUG, the error word (`ws` may be null).
void call_begin();
void kernel_begin(cudaStream_t stream);
void kernel_end(cudaStream_t stream);
int call_end(int rc, void *ws, cudaStream_t stream);

// map_2d of a matrix whose rows are `pitch` elements apart.
bool map_2d_pitch(CUtensorMap *m, const void *ptr, bool bf16, int64_t rows, int64_t cols, uint32_t box_rows,
                  int64_t pitch);

}  // namespace ngr
