// ngr_ce.h -- argument blocks of the linear cross entropy's kernels.  Not
// installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace ngr {

// The four products of the operator.  z = x W^T by tiles, reduced to each
// row's (max, sum) in the epilogue or turned into dz; dx = dz W; dW = dz^T x.
enum { kCeLse = 0, kCeGrad = 1, kCeDx = 2, kCeDw = 3 };

constexpr int kCeTile = 256;      // rows, and columns at most, of a CTA pair's output tile

// What the kernels of a call learn of its tokens (device memory): `count`
// tokens have a target, and `weight` is the largest finite size of a gradient
// weight logit_scale dloss or logit_scale (dloss + dlse).  dz is held in 16
// bits as a multiple of weight / 2^13: it neither overflows nor loses small
// probabilities among fp16's subnormals, and where all tokens weigh the same
// (a mean) the target's -1 is exact.  `down` = weight / 2^13 undoes it in
// FP32.
struct CeInfo {
    int count;
    float weight, down;
};

// Per counted token: lse in powers of two, the weights of p and of the
// target's -1 in that unit, and the target.
struct CeRow {
    float lse2, weight_p, weight_t;
    int target;
};

struct alignas(128) CeGemmArgs {
    CUtensorMap map_a, map_b;
    CUtensorMap map_out;    // kCeDw: `out`, box {64 columns, 32 rows} (with `boxes`)
    const CeInfo *info;
    int *err;
    unsigned long long timeout_ns;
    int rows;               // kCeDw: vocabulary entries of the piece (output rows)
    int cols;               // output columns: vocabulary entries of the piece, or K
    int depth;              // contracted length (kCeDw: the counted tokens, from info)
    int splits;             // kCeDx: ranges of the contracted length, each with its own sums
    float scale2;           // kCeLse, kCeGrad: logit scale times log2(e)
    float scale;            // kCeLse: logit scale
    int v0;                 // first vocabulary entry of the piece
    const int *target;      // kCeLse: [count] targets of the counted tokens
    int width;              // columns of a tile: a multiple of 32, 256 at most (256 for dx, dW)
    float2 *part;           // kCeLse: [2 column tiles][part_pitch] (max, sum) in powers of two
    int64_t part_pitch;
    float *z_target;        // kCeLse: [count] the target's logit
    const CeRow *row;       // kCeGrad
    void *out;              // kCeGrad: dz [rows][pitch]; kCeDw: dW at v0; kCeDx: dx (finish)
    int64_t pitch;          // elements between rows of `out`
    int boxes;              // kCeDw: aligned rows, written as boxes (map_out)
    float *sums;            // kCeDx: FP32 [splits][sums_rows][sums_pitch]
    int64_t sums_rows, sums_pitch;
    int add;                // kCeDx: add to the sums of the pieces before
    int finish;             // kCeDx: this is the last piece and splits == 1: write dx itself
    const int *index;       // kCeDx (finish): a counted token's row of x
    int after_dx;           // kCeDw: the kernel before it is dx (and not dz, which it reads)
};

int launch_ce_gemm(int mode, bool bf16, const CeGemmArgs &a, int64_t units, cudaStream_t stream);

struct CeTokens {
    const void *x;          // [M, K] rows of K elements
    const int64_t *target;  // [M]
    const float *dloss;     // [M] or null (forward)
    const float *dlse;      // [M] or null
    const float *lse;       // [M] (backward)
    void *dx;               // [M, K] or null: rows of tokens that do not count are zeroed
    float logit_scale;
    int64_t M, K, V;
    int64_t K8, Kx;         // K up to multiples of 8 (what W's rows hold) and 64 (rows of xc)
    CeInfo *info;
    int *err;
    int *index;             // [M] counted tokens in order, the others behind them
    int *ctarget;           // [M] targets of the counted tokens
    CeRow *row;             // [M up to a tile] (backward)
    void *xc;               // [M up to 64][Kx] the counted tokens' rows, zeros behind
};

// W's rows at `pitch` elements (a multiple of 8).
int launch_ce_pad(const void *W, void *dst, int64_t rows, int64_t K, int64_t pitch, cudaStream_t stream);
// The tokens' index and the gathered rows: two kernels, or for few tokens the
// second alone.
bool launch_ce_index_apart(const CeTokens &t);
int launch_ce_index(const CeTokens &t, cudaStream_t stream);
int launch_ce_gather(const CeTokens &t, cudaStream_t stream);
int launch_ce_loss(const CeTokens &t, const float2 *part, int64_t part_pitch, int parts,
                   const float *z_target, float *loss, float *lse, cudaStream_t stream);
int launch_ce_dx(bool bf16, const CeTokens &t, const float *sums, int64_t sums_pitch, int splits,
                 cudaStream_t stream);

}  // namespace ngr
