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
// Both product kernels run kMoeCtas CTAs, two for each of a GB300's SMs
// (sizing must not ask a device); their warps are the workers.
constexpr int kMoeCtas = 2 * 152;
constexpr int kMoeWorkers = kMoeCtas * (kMoeThreads / 32);
// Tokens of one matrix instruction: each has two of its 8 columns, its row
// rounded to the 16-bit type and what that rounding left out.
constexpr int kMoeGroup = 4;
// Steps of a worker at least: with 8, 5 tokens on 13 experts of 1000 x 2001
// take 43 us, with 4 41.
constexpr int kMoeMinShare = 4;
constexpr int kMoeCounters = 2 * kMoeWorkers;   // up, down: of a unit by its first worker

// Groups of tokens that share one reading of an expert's weights: 1 if the
// call has no more, 2 (nearly all experts' of a batch that spreads over many),
// or 4 where an expert has more than six on average, so that 8 would often
// not hold them.  4 against 2: 30 tokens, 6 of 20 experts of 6656 x 1088 185
// us (2: 225); 32 tokens, 4 of 16 of 4096 x 2048 167 (187); 23 tokens, 3 of 4
// of 8192 x 1344 111 (113); but 32 tokens, 2 of 8 of 4096 x 14336 528 (502).
inline int moe_groups(int64_t M, int64_t E, int64_t top_k)
{
    return M <= kMoeGroup ? 1 : M > 2 * kMoeGroup && M * top_k > 6 * E ? 4 : 2;
}
constexpr int kMoeMaxEntries = kMoeMaxExperts + kMoeMaxTokens * kMoeMaxTopK / (2 * kMoeGroup);

struct MoeArgs {
    const void *x, *gamma, *beta;     // [M, K], [K]
    const void *Wr, *Wg, *Wu, *Wd;    // [E, K], [E, F, K], [E, F, K], [E, K, F]
    void *y;                          // [M, K]
    int *experts;                     // [M, top_k] or null: the caller's
    float *weights;
    int *ids;                         // [M, top_k]: the workspace's
    float *w;
    void *a;                          // [M, 2, Kp] normalized rows in two parts, zeros up to a multiple of 8
    void *h;                          // [M top_k, 2, Fp] weight x SiLU(gate) x up in two parts, likewise
    // A worker's parts of the units that it shares, in FP32: two places of
    // part_bytes, the second for the unit that its run begins.  Up's are
    // [groups][32 lanes][gate, up], down's [tokens][16 rows]; up's are done
    // with when down's are made.
    float *parts;
    int part_bytes;
    int *counters;                    // [kMoeCounters], zeroed by the router
    int *err;
    int norm, M, K, F, E, top_k, renormalize;
    int Kp, Fp;                       // pitches, multiples of 64
    int groups;                       // see moe_groups
    int router;                       // CTAs of the cluster that takes a token's routing
    float eps;
};

// vec: rows of K (of F) elements start on 16-byte boundaries (router: x,
// gamma, beta and Wr).
int launch_moe_router(bool bf16, bool vec, const MoeArgs &a, cudaStream_t stream);
int launch_moe_up(bool bf16, bool vec, const MoeArgs &a, cudaStream_t stream);
int launch_moe_down(bool bf16, bool vec, const MoeArgs &a, cudaStream_t stream);

}  // namespace ngr
