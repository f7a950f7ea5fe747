// ngr_join_backward_f16_ln.cu -- the join's gradient in f16, with a LayerNorm on either side.
#include "ngr_join_backward.cuh"

namespace ngr {

int launch_join_backward_f16_ln(int mode, const JoinArgs &a, int ctas, cudaStream_t stream)
{
    return run<false, true>(mode, a, ctas, stream);
}

}  // namespace ngr
