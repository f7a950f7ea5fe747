// ngr_join_backward_bf16_rms.cu -- the join's gradient in bf16, without a LayerNorm.
#include "ngr_join_backward.cuh"

namespace ngr {

int launch_join_backward_bf16_rms(int mode, const JoinArgs &a, int ctas, cudaStream_t stream)
{
    return run<true, false>(mode, a, ctas, stream);
}

}  // namespace ngr
