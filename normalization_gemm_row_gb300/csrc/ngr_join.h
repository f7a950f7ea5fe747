// ngr_join.h -- argument blocks and launch geometry of the block join (norm
// after a block, gate, residual, norm before the next block) and of its
// gradient.  Not installed.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace ngr {

constexpr int kJoinThreads = 512;      // threads per CTA at most
constexpr int kJoinMaxCluster = 16;    // CTAs that share one row at most
constexpr int kJoinPortableCluster = 8;   // a larger cluster has to be asked for
constexpr int64_t kJoinMaxN = 65536;   // widest row
constexpr int64_t kJoinSmem = 224 * 1024;   // shared memory of an SM for its CTAs' rings and sums
constexpr int kJoinForwardCols = 16384;   // columns a CTA takes at most: 512 threads x 4 vectors
constexpr int kJoinBackwardCols = 8192;   // 512 threads x 2 vectors
// Both kernels are persistent, per_sm CTAs on each SM.  The backward's
// partial sums are rows per CTA, so the number of SMs is fixed here and not
// asked of the device: sizing needs no GPU.
constexpr int kJoinSms = 152;

// How a row's elements are reached, by the alignment of the call's pointers.
//   kJoinAligned  every row starts on a 16-byte boundary and has whole
//                 8-element vectors;
//   kJoinWindow   the [M, N] arrays have the same offset from a 16-byte
//                 boundary but N % 8 != 0 (or the offset is not 0): a row is
//                 covered by aligned vectors, those at its ends in part;
//   kJoinScalar   anything else, one 2-byte access per element.
enum { kJoinAligned = 0, kJoinWindow = 1, kJoinScalar = 2 };

// How rows map to CTAs: `cluster` CTAs share a row, `cols` columns each (a
// multiple of 8); a CTA of tpr * slots threads works on `slots` rows at a
// time, tpr threads (a multiple of 32) of `vecs` vectors on each.
struct JoinShape {
    int cluster, cols, vecs, tpr, slots, per_sm;
};

struct JoinArgs {
    const void *x, *residual, *gate;            // [M, N], [M, N] or null, [G, N] or null
    const void *gamma1, *beta1, *gamma2, *beta2;
    void *h, *y;                                // forward outputs (y null without norm2)
    const void *dy, *dh;                        // backward inputs (either may be null)
    void *dx, *dresidual, *dgate;               // backward outputs
    float4 *stats;                              // [M] (mu1, rstd1, mu2, rstd2)
    int *err;                                   // backward: the workspace's error word, cleared
    unsigned long long timeout_ns;              // backward: of a wait for the row's warps
    int64_t M, rows_per_gate;
    int N, norm1, norm2;
    float eps1, eps2, residual_scale, block_scale;
    int shift;                                  // kJoinWindow: the arrays' offset in elements
    JoinShape shape;
    // Backward: the rows are cut into items whose rows lie in one gate group
    // each; group g has items [g * items_per_group, +items_per_group).  Item i
    // of a group takes every period-th row of a run of item_rows rows: run
    // i / period, from its row i % period on.
    int64_t items, item_rows;
    int items_per_group, period;
    // Column sums, -1 = not wanted: their places among the `arrays` sums a
    // CTA keeps in shared memory.  Over an item: p = sum u1 D, q = sum D
    // (D the gradient of h), written to item_p, item_q [items][N].  Over a
    // CTA: dgamma2, dbeta2, written to cta_sums [2][CTAs][N].  With
    // fold_gate (small gate groups) p = sum gate u1 D and q = sum gate D run
    // over the CTA too (cta_sums [4]), and dgate is summed over its group
    // and written by the CTA itself.
    int a_p, a_q, a_dgamma2, a_dbeta2, a_dgate, arrays;
    int fold_gate;
    int depth;                                  // rows under way per CTA slot (1 to 3)
    float *item_p, *item_q, *cta_sums;
};

// The second kernel of the backward call: vectors of N from the rows of sums.
struct JoinReduce {
    const float *p, *q;          // [items][N] (or [CTAs][N] with fold_gate), null: not there
    const float *dgamma2_rows, *dbeta2_rows;   // [ctas][N]
    void *dgamma1, *dbeta1, *dgamma2, *dbeta2, *dgate;   // null: not wanted (or written already)
    const void *gate, *gamma1, *beta1;         // null: 1, 1, 0
    int64_t groups;
    int items_per_group, ctas, pq_rows, N;
    float block_scale;
    int fold_gate;
};

JoinShape join_forward_shape(int64_t N, int mode);
JoinShape join_backward_shape(int64_t N, int mode, int arrays);
int launch_join_forward(bool bf16, int mode, const JoinArgs &a, cudaStream_t stream);
int launch_join_backward(bool bf16, int mode, const JoinArgs &a, int ctas, cudaStream_t stream);
int launch_join_reduce(bool bf16, const JoinReduce &r, cudaStream_t stream);

}  // namespace ngr
