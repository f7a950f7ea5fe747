// ngr_join_forward.cu -- the join of a block to its residual stream (see
// ngr_join_kernel.cuh): TPR threads on a row, the row held in registers.
//
// The statistics are two-pass (mean, then centred squares), so a row far from
// zero mean or with a few very large channels loses nothing.  Four vectors a
// thread and four CTAs of 256 threads an SM (64 registers) keep enough loads
// in flight: at 8192 x 8192, RMSNorm on both sides, three or five CTAs, two
// or eight vectors, persistent CTAs that fetch the next row early, or a ring
// of rows in shared memory all ran 2-60 % slower.
#include <algorithm>

#include "ngr_join_kernel.cuh"

namespace ngr {

namespace {

// Threads of a CTA: 256 (four CTAs an SM), 512 for the widest rows.
__host__ __device__ constexpr int forward_threads(int tpr) { return tpr > 256 ? tpr : 256; }
// CTAs an SM: three of the window mode take 398 us against 239 at 8192 x 8191,
// LN/LN.
__host__ __device__ constexpr int forward_ctas(int mode, int tpr)
{
    return (mode == kJoinScalar ? 512 : 1024) / forward_threads(tpr);
}
// A warp a row while five vectors a lane cover it (its sums need no barrier),
// then three or four vectors a thread.
constexpr Width kWidths[] = {{32, 1}, {32, 2}, {32, 3}, {32, 4}, {32, 5}, {64, 3}, {64, 4},
                             {128, 3}, {128, 4}, {256, 3}, {256, 4}, {512, 3}, {512, 4}};
constexpr unsigned kWave = 4 * kJoinSms;   // CTAs that run at once

// ONE: a CTA to a row (no cluster).
template <bool BF16, int MODE, int TPR, int VECS, bool ONE>
__global__ void __launch_bounds__(forward_threads(TPR), forward_ctas(MODE, TPR))
    join_forward_kernel(const __grid_constant__ JoinArgs a)
{
    constexpr int kSlots = forward_threads(TPR) / TPR;
    __shared__ RowSumSmem sums;
    int half = 0;
    const int cluster = ONE ? 1 : a.shape.cluster;
    const uint32_t rank = cluster > 1 ? cluster_ctarank() : 0u;
    const int slot = threadIdx.x / TPR;
    const int c0 = static_cast<int>(rank) * a.shape.cols;
    constexpr int kFull = ONE ? full_vectors(kWidths, TPR, VECS, MODE) : -1;
    const Place<MODE, TPR, kFull> p(c0, min(a.N, c0 + a.shape.cols), threadIdx.x % TPR);
    const int64_t row = static_cast<int64_t>(blockIdx.x / cluster) * kSlots + slot;
    const bool active = kSlots == 1 || row < a.M;
    const int64_t off = active ? row * a.N : 0;
    const int s = row_shift<MODE>(a, row);
    const float inv_n = 1.0f / static_cast<float>(a.N);

    uint4 xp[VECS], rp[VECS];
#pragma unroll
    for (int v = 0; v < VECS; ++v) xp[v] = rp[v] = make_uint4(0u, 0u, 0u, 0u);
    if (active) {
#pragma unroll
        for (int v = 0; v < VECS; ++v) xp[v] = load8(elements(a.x, off), p, v, s);
        if (a.residual) {
#pragma unroll
            for (int v = 0; v < VECS; ++v) rp[v] = load8(elements(a.residual, off), p, v, s);
        }
    }
    const uint16_t *gate = nullptr;
    if (a.gate) gate = elements(a.gate, a.rows_per_gate >= a.M || !active ? 0 : row / a.rows_per_gate * a.N);
    // In a call of one wave the vectors are in no cache: they are on their way
    // while x is reduced.  (With more rows the CTAs before have brought them,
    // and asking again for each row tripled the time at narrow widths.)
    if (gridDim.x <= kWave) {
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const int c = p.col(v, 0, 0);
            if (c < p.c1) {
                if (gate) prefetch_l1(gate + c);
                if (a.gamma1) prefetch_l1(elements(a.gamma1, c));
                if (a.gamma2) prefetch_l1(elements(a.gamma2, c));
            }
        }
    }
    // Every CTA of the cluster runs before its shared memory is written.
    if (cluster > 1) cluster_sync_all();

    float mu1 = 0.0f, rs1 = 1.0f;
    if (a.norm1 == kNormLayer) {
        float2 t = both(0.0f);
#pragma unroll
        for (int v = 0; v < VECS; ++v) sum8(t, unpack8<BF16>(xp[v]));   // zero past the row
        float k[1] = {t.x + t.y};
        row_sum<1, TPR>(k, sums, half, cluster, rank);
        mu1 = k[0] * inv_n;
    }
    if (a.norm1 != kNormNone) {
        float2 t = both(0.0f);
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            Vec8 d = unpack8<BF16>(xp[v]);
            if (a.norm1 == kNormLayer) d = masked(d + -mu1, p, v, s);
            dot8(t, d, d);
        }
        float k[1] = {t.x + t.y};
        row_sum<1, TPR>(k, sums, half, cluster, rank);
        rs1 = rsqrtf(k[0] * inv_n + a.eps1);
    }

    Vec8 h[VECS];
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
        Vec8 n = unpack8<BF16>(xp[v]);
        if (a.norm1 == kNormLayer) n = n + -mu1;
        if (a.norm1 != kNormNone) n = n * rs1 * param8<BF16>(elements(a.gamma1), p, v, s);
        if (a.norm1 == kNormLayer) n = n + param8<BF16>(elements(a.beta1), p, v, s);
        if (gate) n = n * param8<BF16>(gate, p, v, s);
        h[v] = fma8(unpack8<BF16>(rp[v]), a.residual_scale, n * a.block_scale);
        if (active) store8(elements(a.h, off), p, v, s, pack8<BF16>(h[v]));
    }

    float mu2 = 0.0f, rs2 = 1.0f;
    if (a.norm2 == kNormLayer) {
        float2 t = both(0.0f);
#pragma unroll
        for (int v = 0; v < VECS; ++v) sum8(t, masked(h[v], p, v, s));
        float k[1] = {t.x + t.y};
        row_sum<1, TPR>(k, sums, half, cluster, rank);
        mu2 = k[0] * inv_n;
    }
    if (a.norm2 != kNormNone) {
        float2 t = both(0.0f);
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            if (a.norm2 == kNormLayer) h[v] = h[v] + -mu2;
            const Vec8 d = masked(h[v], p, v, s);
            dot8(t, d, d);
        }
        float k[1] = {t.x + t.y};
        row_sum<1, TPR>(k, sums, half, cluster, rank);
        rs2 = rsqrtf(k[0] * inv_n + a.eps2);
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            Vec8 y = h[v] * rs2 * param8<BF16>(elements(a.gamma2), p, v, s);
            if (a.norm2 == kNormLayer) y = y + param8<BF16>(elements(a.beta2), p, v, s);
            if (active) store8(elements(a.y, off), p, v, s, pack8<BF16>(y));
        }
    }
    if (a.stats && active && threadIdx.x % TPR == 0 && rank == 0) a.stats[row] = make_float4(mu1, rs1, mu2, rs2);
}

template <bool BF16, int MODE>
int run(const JoinArgs &a, cudaStream_t stream)
{
    const int64_t ctas = (a.M + a.shape.slots - 1) / a.shape.slots;
#define NGR_WIDTH(T, V, ONE)                                                    \
    if (a.shape.tpr == T && a.shape.vecs == V && (a.shape.cluster == 1) == ONE) \
        return launch_join(join_forward_kernel<BF16, MODE, T, V, ONE>, ctas, a.shape, 0, a, stream, "join launch");
    // (a CTA of a cluster has more than 8192 columns)
    NGR_WIDTH(256, 4, true)
    NGR_WIDTH(512, 4, true)
    NGR_WIDTH(512, 4, false)
    if constexpr (MODE != kJoinScalar) {
        NGR_WIDTH(32, 1, true)
        NGR_WIDTH(32, 2, true)
        NGR_WIDTH(32, 3, true)
        NGR_WIDTH(32, 4, true)
        NGR_WIDTH(32, 5, true)
        NGR_WIDTH(64, 3, true)
        NGR_WIDTH(64, 4, true)
        NGR_WIDTH(128, 3, true)
        NGR_WIDTH(128, 4, true)
        NGR_WIDTH(256, 3, true)
        NGR_WIDTH(512, 3, true)
        NGR_WIDTH(512, 3, false)
    }
#undef NGR_WIDTH
    return -9;
}

}  // namespace

JoinShape join_forward_shape(int64_t N, int mode)
{
    JoinShape s;
    s.cluster = 1;
    auto cols = [&] { return up8((N + s.cluster - 1) / s.cluster); };
    while (cols() + (mode == kJoinWindow ? 8 : 0) > kJoinForwardCols) s.cluster *= 2;
    s.cols = static_cast<int>(cols());
    // (a cluster works on one row at a time; the scalar mode, for pointers
    // that no other takes, has two widths only)
    for (const Width &w : kWidths) {
        s.tpr = w.tpr;
        s.vecs = w.vecs;
        if (w.tpr * w.vecs < join_vectors(s, mode) || (s.cluster > 1 && w.tpr < 256)) continue;
        if (mode != kJoinScalar || (w.tpr >= 256 && w.vecs == 4)) break;
    }
    s.slots = forward_threads(s.tpr) / s.tpr;
    s.per_sm = 0;
    return s;
}

int launch_join_forward(bool bf16, int mode, const JoinArgs &a, cudaStream_t stream)
{
    if (mode == kJoinAligned) return bf16 ? run<true, kJoinAligned>(a, stream) : run<false, kJoinAligned>(a, stream);
    if (mode == kJoinWindow) return bf16 ? run<true, kJoinWindow>(a, stream) : run<false, kJoinWindow>(a, stream);
    return bf16 ? run<true, kJoinScalar>(a, stream) : run<false, kJoinScalar>(a, stream);
}

}  // namespace ngr
