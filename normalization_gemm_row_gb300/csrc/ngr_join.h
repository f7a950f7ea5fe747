// ngr_join.h -- argument blocks and launch geometry of the block join (norm
// after a block, gate, residual, norm before the next block) and of its
// gradient.  Not installed.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace ngr {

constexpr int kJoinThreads = 512;      // threads per CTA at most
constexpr int kJoinMaxCluster = 8;     // CTAs that share one row at most
constexpr int kJoinMaxVecs = 4;        // 8-element vectors per thread and row at most
constexpr int64_t kJoinMaxN = 65536;   // widest row
// Shared memory for the backward kernel's column sums, at most (of 227 KB).
constexpr int kJoinSumBytes = 200 * 1024;
// CTAs the backward kernel runs at most (its partial sums are one row per
// CTA, so their number is fixed here and not by the device: sizing needs no GPU).
constexpr int kJoinCtas = 152;

// How rows map to CTAs: `cluster` CTAs share a row, `cols` columns each (a
// multiple of 8); a CTA of tpr * slots threads works on `slots` rows at a
// time, tpr threads (a multiple of 32) of `vecs` vectors on each.
struct JoinShape {
    int cluster, cols, vecs, tpr, slots;
};

struct JoinArgs {
    const void *x, *residual, *gate;            // [M, N], [M, N] or null, [G, N] or null
    const void *gamma1, *beta1, *gamma2, *beta2;
    void *h, *y;                                // forward outputs (y null without norm2)
    const void *dy, *dh;                        // backward inputs (either may be null)
    void *dx, *dresidual, *dgate;               // backward outputs
    float4 *stats;                              // [M] (mu1, rstd1, mu2, rstd2)
    int *err;                                   // backward: the workspace's error word, cleared
    float *partials;                            // backward: per-CTA sums ([arrays but dgate][CTAs][N])
    int64_t M, rows_per_gate;
    int N, norm1, norm2;
    float eps1, eps2, residual_scale, block_scale;
    JoinShape shape;
    // Backward: the rows are cut into items of item_rows rows that lie in
    // one gate group each; group g has items [g * items_per_group, +items_per_group).
    int64_t items, item_rows;
    int items_per_group;
    // Row sums kept in shared memory and written to `partials`, -1 = not wanted:
    // the place of each among a CTA's `arrays` rows.
    // (dgate's, kept for one item at a time, is the last).
    int a_dgamma1, a_dbeta1, a_dgamma2, a_dbeta2, a_dgate, arrays;
    int dgate_direct;                           // one item per group: dgate is written by its CTA
    float *gate_partials;                       // [items][N] otherwise
};

// What ngr_join_backward's second kernel adds up.
struct JoinReduce {
    const float *src[5];        // rows of N floats
    int64_t row_stride[5];      // floats between the rows of one sum
    int rows[5];                // rows per sum
    void *dst[5];               // rows of N of the call's type, one per sum
    int64_t first[5];           // index of the first output row of source i among all
    int sources, N;
    int64_t total_outs;
};

JoinShape join_forward_shape(int64_t N);
JoinShape join_backward_shape(int64_t N, int arrays);
int launch_join_forward(bool bf16, bool vec, const JoinArgs &a, cudaStream_t stream);
int launch_join_backward(bool bf16, bool vec, const JoinArgs &a, int ctas, cudaStream_t stream);
int launch_join_reduce(bool bf16, const JoinReduce &r, cudaStream_t stream);

}  // namespace ngr
