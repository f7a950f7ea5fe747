// ngr_join_backward_bf16_ln.cu -- the join's gradient in bf16, with a LayerNorm on either side.
#include "ngr_join_backward.cuh"

namespace ngr {

int launch_join_backward_bf16_ln(int mode, const JoinArgs &a, int ctas, cudaStream_t stream)
{
    return run<true, true>(mode, a, ctas, stream);
}

}  // namespace ngr
