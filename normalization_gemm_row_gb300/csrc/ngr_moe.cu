// ngr_moe.cu -- a mixture-of-experts layer with SwiGLU experts for at most 32
// tokens, in three launches.
//
//   a = norm(x),  z = a Wr^T,  p = softmax(z),  the top_k largest p of each
//   token (ties: the lowest expert), divided by their sum if asked;
//   h = p SiLU(a Wg^T) (a Wu^T) for a token and chosen expert,
//   y = sum over the chosen experts of h Wd^T.
//
// A chosen expert's three weights are read once, 6 F K bytes, for the few
// tokens that chose it: reading them bounds the layer.  The weights go
// straight from memory into the operands of 16 x 8 x 16 matrix instructions,
// their rows as the instruction's rows and the tokens as its columns: a lane
// reads 16 contiguous bytes of a row, and the contraction is taken in the
// order that this gives, for both operands alike.
//
// The steps of a product (64 columns of 16 weight rows) over all chosen
// experts stand in one row that is cut into equal runs, one a warp
// ("worker"), so that any number of experts and any sizes keep every warp
// busy to the end; only the device knows the choice.  A worker's loads run
// kDepth steps ahead, past the ends of units too.  A unit (16 rows' results)
// that several workers share is put together, in the workers' order, by the
// one that finishes last: the others leave their parts in memory and count.
//
// The instruction has 8 columns for 4 tokens: a token's row takes two, rounded
// to the 16-bit type and what that left out, so that rounding a and h costs
// no accuracy (a single rounding of each doubled y's error, 1.7e-3 to 3.4e-3
// in bf16), for no bytes of weights more.
#include "ngr.h"
#include "ngr_entry.h"
#include "ngr_internal.h"
#include "ngr_mma.cuh"
#include "ngr_moe.h"
#include "ngr_ptx.cuh"
#include "ngr_shift.cuh"

#include <cooperative_groups.h>

namespace ngr {

namespace cg = cooperative_groups;

namespace {

constexpr int kWarps = kMoeThreads / 32;

// ------------------------------------------------------------------ rows
__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// 8 elements from column k of a row of n (k a multiple of 8), zeros past its
// end.  VEC: the row starts on a 16-byte boundary and n is a multiple of 8.
template <bool VEC>
__device__ __forceinline__ uint4 row8(const uint16_t *row, int k, int n)
{
    if (k >= n) return zero4();
    if (VEC) return __ldg(reinterpret_cast<const uint4 *>(row + k));
    const int left = n - k;
    const uint4 d = load_shifted(row + k, 0, left < 8 ? left : 8);
    uint32_t w[4] = {d.x, d.y, d.z, d.w};
    // (what follows the row's end belongs to the next row)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] &= (2 * i < left ? 0xFFFFu : 0u) | (2 * i + 1 < left ? 0xFFFF0000u : 0u);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &d, float (&v)[8])
{
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 p = unpack16<BF16>(w[j]);
        v[2 * j] = p.x;
        v[2 * j + 1] = p.y;
    }
}

// Two values as their rounded parts and what the rounding left out.
template <bool BF16>
__device__ __forceinline__ uint2 two_parts(float x, float y)
{
    const uint32_t hi = pack16<BF16>(x, y);
    const float2 h = unpack16<BF16>(hi);
    // (an infinity has no second part)
    return make_uint2(hi, pack16<BF16>(fabsf(h.x) < INFINITY ? x - h.x : 0.0f, fabsf(h.y) < INFINITY ? y - h.y : 0.0f));
}

__device__ __forceinline__ float block_sum(float v, float *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w];
    return v;
}

// ---------------------------------------------------------------- router
// A cluster for a token.  Its CTAs share the experts, each with the token's
// normalized row in FP32, a piece at a time; the first CTA gathers the logits
// and chooses.
constexpr int kRouterPiece = 8192;
constexpr int kRouterPitch = kRouterPiece / 8 + 1;

// A float as an unsigned number of the same order, NaN as -inf.
__device__ __forceinline__ uint32_t order_of(float v)
{
    const uint32_t b = __float_as_uint(v == v ? v + 0.0f : -INFINITY);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kMoeThreads) moe_router_kernel(const __grid_constant__ MoeArgs a)
{
    // column k of a piece at [k % 8][k / 8]: a lane's 8 columns lie in 8 rows
    __shared__ float row[8 * kRouterPitch];
    __shared__ float logit[kMoeMaxExperts];
    __shared__ float mine[kMoeMaxExperts / 8];     // of experts i cluster + rank
    __shared__ float red[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int m = static_cast<int>(blockIdx.x) / a.cluster;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *x = static_cast<const uint16_t *>(a.x) + static_cast<int64_t>(m) * a.K;
    const uint16_t *gamma = static_cast<const uint16_t *>(a.gamma), *beta = static_cast<const uint16_t *>(a.beta);
    pdl_launch_dependents();
    cluster.barrier_arrive();      // (waited for before the first one's memory is written: it has to have started)
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
    for (int i = static_cast<int>(blockIdx.x) * kMoeThreads + threadIdx.x; i < kMoeWorkers;
         i += static_cast<int>(gridDim.x) * kMoeThreads)
        a.count_up[i] = a.count_down[i] = 0;

    float mean = 0.0f, scale = 1.0f;
    if (a.norm != kNormNone) {
        float v[8];
        if (a.norm == kNormLayer) {
            float s = 0.0f;
#pragma unroll 4
            for (int k = threadIdx.x * 8; k < a.K; k += kMoeThreads * 8) {
                unpack8<BF16>(row8<VEC>(x, k, a.K), v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s += v[j];
            }
            mean = block_sum(s, red) / a.K;
        }
        float s = 0.0f;
#pragma unroll 4
        for (int k = threadIdx.x * 8; k < a.K; k += kMoeThreads * 8) {
            unpack8<BF16>(row8<VEC>(x, k, a.K), v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float c = k + j < a.K ? v[j] - mean : 0.0f;
                s = fmaf(c, c, s);
            }
        }
        scale = 1.0f / sqrtf(block_sum(s, red) / a.K + a.eps);
    }
    for (int i = threadIdx.x; i < kMoeMaxExperts / 8; i += kMoeThreads) mine[i] = 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += kRouterPiece) {
        const int n = min(kRouterPiece, a.K - k0);
        __syncthreads();
        for (int c = threadIdx.x; c * 8 < n; c += kMoeThreads) {
            const int k = k0 + c * 8;
            float v[8];
            unpack8<BF16>(row8<VEC>(x, k, a.K), v);
            if (a.norm != kNormNone) {
                float g[8];
                unpack8<BF16>(row8<VEC>(gamma, k, a.K), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = k + j < a.K ? (v[j] - mean) * scale * g[j] : 0.0f;
                if (a.norm == kNormLayer) {
                    unpack8<BF16>(row8<VEC>(beta, k, a.K), g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += g[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) row[j * kRouterPitch + c] = v[j];
            if (rank == 0) {
                const uint2 p0 = two_parts<BF16>(v[0], v[1]), p1 = two_parts<BF16>(v[2], v[3]),
                            p2 = two_parts<BF16>(v[4], v[5]), p3 = two_parts<BF16>(v[6], v[7]);
                uint16_t *out = static_cast<uint16_t *>(a.a) + static_cast<int64_t>(2 * m) * a.Kp + k;
                *reinterpret_cast<uint4 *>(out) = make_uint4(p0.x, p1.x, p2.x, p3.x);
                *reinterpret_cast<uint4 *>(out + a.Kp) = make_uint4(p0.y, p1.y, p2.y, p3.y);
            }
        }
        __syncthreads();
        for (int i = warp; i * a.cluster + rank < a.E; i += kWarps) {
            const int e = i * a.cluster + rank;
            float z = 0.0f;
            const uint16_t *wr = static_cast<const uint16_t *>(a.Wr) + static_cast<int64_t>(e) * a.K;
#pragma unroll 8
            for (int c = lane; c * 8 < n; c += 32) {
                float w[8];
                unpack8<BF16>(row8<VEC>(wr, k0 + c * 8, a.K), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) z = fmaf(w[j], row[j * kRouterPitch + c], z);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            if (lane == 0) mine[i] += z;
        }
    }
    cluster.barrier_wait();
    float *logits = cluster.map_shared_rank(logit, 0);
    __syncthreads();
    for (int i = threadIdx.x; i * a.cluster + rank < a.E; i += kMoeThreads) logits[i * a.cluster + rank] = mine[i];
    cluster.sync();
    if (rank != 0 || warp != 0) return;

    // One warp chooses; lane l has the experts l, l + 32, ...
    float top = -INFINITY;
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, logit[e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float all = 0.0f;
    for (int e = lane; e < a.E; e += 32) all += expf(logit[e] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    uint32_t taken = 0;            // of this lane's experts
    float p = 0.0f, sum = 0.0f;    // lane s: choice s
    int id = 0;
    for (int s = 0; s < a.top_k; ++s) {
        // the largest logit that is left, of equal ones the lowest expert's;
        // NaN counts as -inf, so that there is always a choice
        uint32_t best = 0;         // (below any logit's order)
        int at = kMoeMaxExperts;
        for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
            const uint32_t v = order_of(logit[e]);
            if (!((taken >> i) & 1u) && v > best) {
                best = v;
                at = e;
            }
        }
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        at = __reduce_min_sync(0xffffffffu, best == most ? at : kMoeMaxExperts);
        if ((at & 31) == lane) taken |= 1u << (at >> 5);
        const float q = expf(logit[at] - top) / all;
        sum += q;
        if (lane == s) {
            p = q;
            id = at;
        }
    }
    if (lane < a.top_k) {
        if (a.renormalize) p /= sum;
        const int i = m * a.top_k + lane;
        a.ids[i] = id;
        a.w[i] = p;
        if (a.experts) a.experts[i] = id;
        if (a.weights) a.weights[i] = p;
    }
}

// -------------------------------------------------------------- products
// The experts that somebody chose, in order, for every CTA in its shared
// memory.  The rows of h stand by expert and then by token.
struct Chosen {
    uint16_t expert[kMoeMaxExperts], base[kMoeMaxExperts + 2];
    uint8_t token[kMoeMaxTokens * kMoeMaxTopK];        // of a row of h
    int count;
};
// `tokens`: room for kMoeMaxExperts words.
__device__ __forceinline__ void find_chosen(const MoeArgs &a, Chosen &c, uint32_t *tokens)
{
    const int lane = threadIdx.x & 31, all = a.M * a.top_k;
    for (int e = threadIdx.x; e < a.E; e += kMoeThreads) tokens[e] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < all; i += kMoeThreads) atomicOr(&tokens[a.ids[i]], 1u << (i / a.top_k));
    __syncthreads();
    if (threadIdx.x < 32) {
        int n = 0, rows = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const uint32_t t = e0 + lane < a.E ? tokens[e0 + lane] : 0u;
            const uint32_t some = __ballot_sync(0xffffffffu, t != 0u);
            if (some == 0u) continue;
            const int mine = __popc(t);
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (t != 0u) {
                const int at = n + __popc(some & ((1u << lane) - 1u));
                int r = rows + incl - mine;
                c.expert[at] = static_cast<uint16_t>(e0 + lane);
                c.base[at] = static_cast<uint16_t>(r);
                for (uint32_t left = t; left; left &= left - 1u) c.token[r++] = static_cast<uint8_t>(__ffs(left) - 1);
            }
            n += __popc(some);
            rows += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            c.count = n;
            c.base[n] = static_cast<uint16_t>(all);
        }
    }
    __syncthreads();
}

// A stage of a worker's ring: a step's 16 weight rows of 128 bytes, or of the
// nine 16-byte words that they lie in where rows are off the boundary, and
// the first group's 8 token rows of 128 bytes.
template <bool VEC>
struct Stage {
    static constexpr int kPitch = VEC ? 128 : 144;
    static constexpr int kTokens = 16 * kPitch;
    static constexpr int kBytes = kTokens + 8 * 128;
};

// Where a segment (the steps over one expert's 16 rows) has its operands.
// Rows 0 to 7 start at r0, rows 8 to 15 at r1, `pitch` elements apart, n0 and
// n1 of each are there; the tokens' rows are those of `tokens` rows from
// `base` on, of h, or of a through the list.
struct Segment {
    const uint16_t *r0, *r1;
    int n0, n1;
    int base, tokens, expert;
};

// The row (of a or h) of a token's part: column `col` of group j.
template <bool DOWN>
__device__ __forceinline__ const uint16_t *token_row(const MoeArgs &a, const Chosen &c, const Segment &s, int j, int col)
{
    const int r = j * kMoeGroup + (col >> 1);
    if (r >= s.tokens) return nullptr;
    if (DOWN) return static_cast<const uint16_t *>(a.h) + (static_cast<int64_t>(s.base + r) * 2 + (col & 1)) * a.Fp;
    return static_cast<const uint16_t *>(a.a) + (static_cast<int64_t>(c.token[s.base + r]) * 2 + (col & 1)) * a.Kp;
}

template <bool DOWN>
__device__ __forceinline__ Segment segment(const MoeArgs &a, const Chosen &c, int64_t index)
{
    Segment s;
    if (DOWN) {      // by 16 rows of Wd, then by expert
        const int tile = static_cast<int>(index / c.count), i = static_cast<int>(index - static_cast<int64_t>(tile) * c.count);
        s.expert = i;
        s.r0 = static_cast<const uint16_t *>(a.Wd) + (static_cast<int64_t>(c.expert[i]) * a.K + tile * 16) * a.F;
        s.r1 = s.r0 + static_cast<int64_t>(8) * a.F;
        s.n0 = a.K - tile * 16;
        s.n1 = s.n0 - 8;
    } else {         // by expert, then by 8 rows of Wg and of Wu
        const int tiles = (a.F + 7) / 8;
        const int i = static_cast<int>(index / tiles), tile = static_cast<int>(index - static_cast<int64_t>(i) * tiles);
        const int64_t at = (static_cast<int64_t>(c.expert[i]) * a.F + tile * 8) * a.K;
        s.expert = i;
        s.r0 = static_cast<const uint16_t *>(a.Wg) + at;
        s.r1 = static_cast<const uint16_t *>(a.Wu) + at;
        s.n0 = s.n1 = a.F - tile * 8;
    }
    s.base = c.base[s.expert];
    s.tokens = c.base[s.expert + 1] - s.base;
    return s;
}

// The copies of one step, columns [k, k + 64) of n.
template <bool DOWN, bool VEC>
__device__ __forceinline__ void fetch(const MoeArgs &a, const Chosen &c, const Segment &s, int k, uint32_t stage, int lane)
{
    const int n = DOWN ? a.F : a.K;
    if (VEC) {
        const int col = lane & 7, at = k + col * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 4 + (lane >> 3), q = r & 7;
            const uint16_t *row = r < 8 ? s.r0 : s.r1;
            const bool there = at < n && q < (r < 8 ? s.n0 : s.n1);
            cp_async16(stage + r * 128 + ((col ^ q) << 4), there ? row + static_cast<int64_t>(q) * n + at : row, there);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const int w = i * 32 + lane, r = w / 9, col = w - r * 9, q = r & 7;
            if (r >= 16) continue;
            // the aligned word `col` after the one that column k lies in:
            // there if it holds any of the columns up to n
            const uint16_t *p = (r < 8 ? s.r0 : s.r1) + static_cast<int64_t>(q) * n + k;
            const int d = static_cast<int>((reinterpret_cast<uintptr_t>(p) >> 1) & 7u);
            const bool there = k + col * 8 - d < n && (col < 8 || d > 0) && q < (r < 8 ? s.n0 : s.n1);
            cp_async16(stage + r * 144 + col * 16, there ? static_cast<const void *>(p - d + col * 8) : a.h, there);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = i * 4 + (lane >> 3), at = k + (lane & 7) * 8;
        const uint16_t *row = token_row<DOWN>(a, c, s, 0, col);
        const bool there = row && at < n;
        cp_async16(stage + Stage<VEC>::kTokens + col * 128 + (((lane & 7) ^ col) << 4),
                   there ? static_cast<const void *>(row + at) : a.h, there);
    }
}

// A 32-bit operand word of a row off the 16-byte boundary: columns e, e + 1 of
// the stage's row whose first word starts `d` elements before column 0.
__device__ __forceinline__ uint32_t pair_at(uint32_t row, int d, int e)
{
    const int at = d + e;
    uint32_t lo;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(lo) : "r"(row + (at >> 1) * 4) : "memory");
    if (!(at & 1)) return lo;
    uint32_t hi;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(hi) : "r"(row + (at >> 1) * 4 + 4) : "memory");
    return __funnelshift_r(lo, hi, 16);
}

// The products of one step.
template <bool BF16, bool DOWN, bool VEC, int NT>
__device__ __forceinline__ void take(float (&acc)[NT][4], const MoeArgs &a, const Chosen &c, const Segment &s, int k,
                                     uint32_t stage, int lane)
{
    const int g = lane >> 2, t = lane & 3, n = DOWN ? a.F : a.K;
    uint32_t w[4][4];      // the weights' operands of four contractions of 16
    if (VEC) {
        const int r = ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) ldmatrix4(w[i], stage + r * 128 + (((2 * i + half) ^ (r & 7)) << 4));
    } else {
        const uint16_t *p0 = s.r0 + static_cast<int64_t>(g) * n + k, *p1 = s.r1 + static_cast<int64_t>(g) * n + k;
        const int d0 = static_cast<int>((reinterpret_cast<uintptr_t>(p0) >> 1) & 7u);
        const int d1 = static_cast<int>((reinterpret_cast<uintptr_t>(p1) >> 1) & 7u);
        const uint32_t row0 = stage + g * 144, row1 = stage + (g + 8) * 144;
        const int left = n - k;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int e = i * 16 + h * 8 + 2 * t;
                // (what follows the row's end belongs to the next row)
                const uint32_t keep = (e < left ? 0xFFFFu : 0u) | (e + 1 < left ? 0xFFFF0000u : 0u);
                w[i][2 * h] = pair_at(row0, d0, e) & keep;
                w[i][2 * h + 1] = pair_at(row1, d1, e) & keep;
            }
    }
    {
        const int col = lane & 7, quarter = lane >> 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t b[4];
            ldmatrix4(b, stage + Stage<VEC>::kTokens + col * 128 + (((4 * i + quarter) ^ col) << 4));
            mma_16816<BF16>(acc[0], w[2 * i][0], w[2 * i][1], w[2 * i][2], w[2 * i][3], b[0], b[1]);
            mma_16816<BF16>(acc[0], w[2 * i + 1][0], w[2 * i + 1][1], w[2 * i + 1][2], w[2 * i + 1][3], b[2], b[3]);
        }
    }
    // Experts with more tokens: their rows straight from memory, which holds
    // them near (they are read for every 16 rows of the weights).
#pragma unroll
    for (int j = 1; j < NT; ++j) {
        if (j * kMoeGroup >= s.tokens) break;
        const uint16_t *row = token_row<DOWN>(a, c, s, j, g);
        uint32_t b[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = k + i * 16 + h * 8;
                b[i][h] = row && at < n ? __ldg(reinterpret_cast<const uint32_t *>(row + at + 2 * t)) : 0u;
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_16816<BF16>(acc[j], w[i][0], w[i][1], w[i][2], w[i][3], b[i][0], b[i][1]);
    }
}

// Which workers share the steps [begin, end).
struct Sharers {
    int first, last;
};
__device__ __forceinline__ Sharers sharers(int64_t begin, int64_t end, int64_t share)
{
    return Sharers{static_cast<int>(begin / share), static_cast<int>((end - 1) / share)};
}
// Count a part in, after its memory: true for the last.
__device__ __forceinline__ bool counted_last(int *count, const Sharers &w, int lane)
{
    __threadfence();
    __syncwarp();
    int before = 0;
    if (lane == 0) before = atomicAdd(count + w.first, 1);
    const bool last = __shfl_sync(0xffffffffu, before, 0) == w.last - w.first;
    if (last) __threadfence();
    return last;
}

constexpr int depth_of(int NT) { return NT == 8 ? 3 : 4; }
template <bool DOWN, bool VEC, int NT>
constexpr int smem_of()
{
    return kWarps * (depth_of(NT) * Stage<VEC>::kBytes + (DOWN ? NT * kMoeGroup * 17 * 4 : 0));
}

template <bool BF16, bool DOWN, bool VEC, int NT>
__global__ void __launch_bounds__(kMoeThreads, 2) moe_kernel(const __grid_constant__ MoeArgs a)
{
    constexpr int S = depth_of(NT);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Chosen c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    if (!DOWN) pdl_launch_dependents();
    pdl_wait();
    find_chosen(a, c, reinterpret_cast<uint32_t *>(smem));

    const int n = DOWN ? a.F : a.K;
    const int length = (n + 63) / 64;      // steps of a segment
    const int64_t segments = static_cast<int64_t>(c.count) * (DOWN ? (a.K + 15) / 16 : (a.F + 7) / 8);
    const int64_t total = segments * length;
    int64_t share = (total + kMoeWorkers - 1) / kMoeWorkers;
    if (share < kMoeMinShare) share = kMoeMinShare;
    const int worker = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    const int64_t first = worker * share;
    if (first >= total) return;
    const int count = static_cast<int>(min(share, total - first));

    const uint32_t ring = smem_u32(smem) + warp * (S * Stage<VEC>::kBytes);
    // DOWN: the tokens' sums of the 16 rows under way, [token][17]
    float *sums = reinterpret_cast<float *>(smem + kWarps * S * Stage<VEC>::kBytes) + warp * (NT * kMoeGroup * 17);
    int64_t index = first / length, ahead = index;
    int step = static_cast<int>(first - index * length), ahead_step = step;
    Segment s = segment<DOWN>(a, c, index), f = s;
    auto issue = [&](int stage) {
        fetch<DOWN, VEC>(a, c, f, ahead_step * 64, ring + stage * Stage<VEC>::kBytes, lane);
        if (++ahead_step == length) {
            ahead_step = 0;
            if (++ahead < segments) f = segment<DOWN>(a, c, ahead);
        }
    };
#pragma unroll
    for (int i = 0; i < S; ++i) {
        if (i < count) issue(i);
        cp_async_commit();
    }
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = 0.0f;
    if (DOWN) {
        for (int i = lane; i < NT * kMoeGroup * 17; i += 32) sums[i] = 0.0f;
        __syncwarp();
    }
    // steps of the unit (a segment, or DOWN the segments of 16 rows)
    const int64_t unit = DOWN ? static_cast<int64_t>(c.count) * length : length;
    int stage = 0;
    for (int i = 0; i < count; ++i) {
        cp_async_wait<S - 1>();
        __syncwarp();
        take<BF16, DOWN, VEC, NT>(acc, a, c, s, step * 64, ring + stage * Stage<VEC>::kBytes, lane);
        __syncwarp();
        if (i + S < count) issue(stage);
        cp_async_commit();
        stage = stage + 1 == S ? 0 : stage + 1;
        const bool ends = ++step == length, done = i + 1 == count;
        if (!ends && !done) continue;

        // the segment's end, or the run's
        const int64_t at = first + i + 1;                  // steps so far in the whole row
        const int64_t begin = (at - 1) / unit * unit, end = begin + unit;
        const bool whole = begin >= first && end <= at, close = at == end || done;
        const Sharers w = sharers(begin, end, share);
        const int64_t slot = static_cast<int64_t>(worker) * 2 + (worker == w.first ? 1 : 0);
        if (!DOWN) {
            const int f0 = static_cast<int>(index - index / ((a.F + 7) / 8) * ((a.F + 7) / 8)) * 8;
            float2 v[NT];      // gate and up of row g for token t of each group
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                v[j] = make_float2(acc[j][0] + acc[j][1], acc[j][2] + acc[j][3]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[j][r] = 0.0f;
            }
            bool finish = whole;
            if (!whole) {
                float2 *part = reinterpret_cast<float2 *>(a.part_up) + slot * (NT * 32) + lane;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j * kMoeGroup < s.tokens) part[j * 32] = v[j];
                finish = counted_last(a.count_up, w, lane);
                if (finish) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) v[j] = make_float2(0.0f, 0.0f);
                    for (int p = w.first; p <= w.last; ++p) {
                        const float2 *from = reinterpret_cast<const float2 *>(a.part_up) +
                                             (static_cast<int64_t>(p) * 2 + (p == w.first ? 1 : 0)) * (NT * 32) + lane;
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            if (j * kMoeGroup < s.tokens) {
                                const float2 x = __ldcg(from + j * 32);
                                v[j].x += x.x;
                                v[j].y += x.y;
                            }
                    }
                }
            }
            if (finish) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int r = j * kMoeGroup + t;
                    if (r >= s.tokens) continue;
                    const int token = c.token[s.base + r];
                    float p = 0.0f;
                    for (int q = 0; q < a.top_k; ++q)
                        if (a.ids[token * a.top_k + q] == c.expert[s.expert]) p = a.w[token * a.top_k + q];
                    // The token's weight goes into h, so that the last
                    // product is a plain sum over the experts.
                    const float h = g < s.n0 ? p * (v[j].x / (1.0f + expf(-v[j].x)) * v[j].y) : 0.0f;
                    const uint2 parts = two_parts<BF16>(h, 0.0f);
                    uint16_t *out = static_cast<uint16_t *>(a.h) + static_cast<int64_t>(s.base + r) * 2 * a.Fp + f0 + g;
                    out[0] = static_cast<uint16_t>(parts.x);
                    out[a.Fp] = static_cast<uint16_t>(parts.y);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int r = j * kMoeGroup + t;
                if (r < s.tokens) {
                    float *to = sums + c.token[s.base + r] * 17;
                    to[g] += acc[j][0] + acc[j][1];
                    to[g + 8] += acc[j][2] + acc[j][3];
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[j][q] = 0.0f;
            }
            __syncwarp();
            if (close) {
                const int row0 = static_cast<int>(begin / unit) * 16, values = a.M * 16;
                bool finish = whole;
                if (!whole) {
                    float *part = a.part_down + slot * (NT * kMoeGroup * 16);
                    for (int v = lane; v < values; v += 32) part[v] = sums[(v >> 4) * 17 + (v & 15)];
                    finish = counted_last(a.count_down, w, lane);
                    if (finish) {
                        for (int v = lane; v < values; v += 32) {
                            float x = 0.0f;
#pragma unroll 4
                            for (int p = w.first; p <= w.last; ++p)
                                x += __ldcg(a.part_down + (static_cast<int64_t>(p) * 2 + (p == w.first ? 1 : 0)) * (NT * kMoeGroup * 16) + v);
                            sums[(v >> 4) * 17 + (v & 15)] = x;
                        }
                    }
                }
                if (finish)
                    for (int v = lane; v < values; v += 32)
                        if (row0 + (v & 15) < a.K)
                            static_cast<uint16_t *>(a.y)[static_cast<int64_t>(v >> 4) * a.K + row0 + (v & 15)] =
                                static_cast<uint16_t>(pack16<BF16>(sums[(v >> 4) * 17 + (v & 15)], 0.0f));
                __syncwarp();
                for (int v = lane; v < NT * kMoeGroup * 17; v += 32) sums[v] = 0.0f;
                __syncwarp();
            }
        }
        if (ends) {
            step = 0;
            if (++index < segments) s = segment<DOWN>(a, c, index);
        }
    }
    cp_async_wait<0>();
}

template <typename F>
cudaError_t launch(F *kern, unsigned grid, int cluster, size_t smem, bool after, const MoeArgs &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 0) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (after) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(n);
    if (smem > 0) {
        // (an attribute of the current device's copy of the function)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool BF16, bool DOWN, bool VEC>
cudaError_t product(const MoeArgs &a, cudaStream_t stream)
{
    switch (moe_groups(a.M)) {
    case 1: return launch(moe_kernel<BF16, DOWN, VEC, 1>, kMoeCtas, 0, smem_of<DOWN, VEC, 1>(), true, a, stream);
    case 2: return launch(moe_kernel<BF16, DOWN, VEC, 2>, kMoeCtas, 0, smem_of<DOWN, VEC, 2>(), true, a, stream);
    case 4: return launch(moe_kernel<BF16, DOWN, VEC, 4>, kMoeCtas, 0, smem_of<DOWN, VEC, 4>(), true, a, stream);
    default: return launch(moe_kernel<BF16, DOWN, VEC, 8>, kMoeCtas, 0, smem_of<DOWN, VEC, 8>(), true, a, stream);
    }
}

int status(const char *what, cudaError_t e) { return e == cudaSuccess ? 0 : record_cuda_error(what, e, cudaGetErrorString(e)); }

}  // namespace

int launch_moe_router(bool bf16, bool vec, const MoeArgs &a, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(a.M * a.cluster);
    const auto kern = bf16 ? (vec ? moe_router_kernel<true, true> : moe_router_kernel<true, false>)
                           : (vec ? moe_router_kernel<false, true> : moe_router_kernel<false, false>);
    return status("expert router launch", launch(kern, grid, a.cluster, 0, false, a, stream));
}

int launch_moe_up(bool bf16, bool vec, const MoeArgs &a, cudaStream_t stream)
{
    return status("expert gate and up launch", bf16 ? (vec ? product<true, false, true>(a, stream) : product<true, false, false>(a, stream))
                                                    : (vec ? product<false, false, true>(a, stream) : product<false, false, false>(a, stream)));
}

int launch_moe_down(bool bf16, bool vec, const MoeArgs &a, cudaStream_t stream)
{
    return status("expert down launch", bf16 ? (vec ? product<true, true, true>(a, stream) : product<true, true, false>(a, stream))
                                             : (vec ? product<false, true, true>(a, stream) : product<false, true, false>(a, stream)));
}

}  // namespace ngr
