// ngr_moe.h -- argument block of the mixture-of-experts layer for a few
// tokens (ngr_moe.cu).  Not installed.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace ngr {

constexpr int kMoeMaxTokens = 32;     // one bit of a word each
constexpr int kMoeMaxExperts = 1024;  // 32 logits a lane
constexpr int kMoeMaxTopK = 32;
constexpr int kMoeThreads = 256;
constexpr int kMoeSms = 152;          // sizing must not ask a device

struct MoeArgs {
    const void *x, *gamma, *beta;     // [M, K], [K]
    const void *Wr, *Wg, *Wu, *Wd;    // [E, K], [E, F, K], [E, F, K], [E, K, F]
    void *y;                          // [M, K]
    int *experts;                     // [M, top_k] or null: the caller's
    float *weights;
    int *ids;                         // [M, top_k]: the workspace's
    float *w;
    void *a;                          // [M, Kp] normalized rows, zeros up to Kp
    void *h;                          // [M top_k, Fp] weight x SiLU(gate) x up, zeros up to a multiple of 8
    int *err;
    int norm, M, K, F, E, top_k, renormalize;
    int Kp, Fp;                       // pitches, multiples of 64
    int cluster;                      // CTAs that share a token's router row
    int splits;                       // CTAs (a cluster) that share 16 rows of y
    float eps;
};

// vec_k, vec_f: rows of K (of F) elements start on 16-byte boundaries.
int launch_moe_router(bool bf16, bool vec_k, const MoeArgs &a, cudaStream_t stream);
int launch_moe_up(bool bf16, bool vec_k, const MoeArgs &a, cudaStream_t stream);
int launch_moe_down(bool bf16, bool vec_f, const MoeArgs &a, cudaStream_t stream);

}  // namespace ngr
