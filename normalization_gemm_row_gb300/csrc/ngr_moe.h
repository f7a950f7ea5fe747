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
constexpr int kMoeMinShare = 4;       // steps of a worker at least
constexpr int kMoeCounters = 2 * kMoeWorkers;   // up, down: of a unit by its first worker

// Groups of tokens that share one reading of an expert's weights: 1 if the
// call has no more, 2 (nearly all experts' of a batch that spreads over many),
// or 4 where an expert has more than six on average, so that 8 would often
// not hold them.
inline int moe_groups(int64_t M, int64_t E, int64_t top_k) { return M <= kMoeGroup ? 1 : M > 2 * kMoeGroup && M * top_k > 6 * E ? 4 : 2; }
constexpr int kMoeMaxEntries = kMoeMaxExperts + kMoeMaxTokens * kMoeMaxTopK / (2 * kMoeGroup);
// Runs that share a unit at most: the last to finish adds their parts, at
// about 0.2 us each.
constexpr int kMoeMaxSharers = 24;

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
    // A worker's parts of the units that it shares, the second place for the
    // unit that begins with it: part_bytes each: up [groups][32 lanes][gate,
    // up], down [tokens][16 rows], FP32.  Up's are done with when
    // down's are made.
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
