// ngr_join_backward.cuh -- the gradient of the block join (see
// ngr_join_kernel.cuh).  One translation unit for each element type and for
// joins with and without a LayerNorm, so that they compile in parallel.
//
// A CTA (or cluster) takes items of rows, `slots` rows at a time, and keeps
// column sums of its rows in shared memory, each thread adding to its own
// columns, so nothing is atomic and the order is fixed.  Since a gate row
// holds for a whole item, dgamma1, dbeta1 and dgate all follow from
// p = sum u1 D and q = sum D of the items:
//   dgamma1 = sum_items s gate p,  dbeta1 = sum_items s gate q,
//   dgate = s (gamma1 sum p + beta1 sum q) over the group's items.
//
// With the forward's statistics at hand one row reduction is enough: D =
// dA - c0 - c1 u2 with dA = dh + rstd2 gamma2 dy is linear in the two means
// c0, c1 of the second pullback, so the sums the first pullback needs of D
// are formed from sums that do not need them.  (Recomputing the statistics
// would take three to five dependent reductions a row.)  Between the
// reduction and the stores u1, u2 and dA stay in registers.
//
// Persistent; every thread keeps its elements of the next rows coming
// through a ring of its own in shared memory (asynchronous 16-byte copies),
// so that the loads fly under the reduction and the stores.
#pragma once

#include <algorithm>

#include "ngr_join_kernel.cuh"

namespace ngr {

namespace {

__host__ __device__ constexpr int backward_slots(int tpr) { return tpr < 256 ? 256 / tpr : 1; }
// CTAs an SM: its registers hold 768 threads with one vector, 512 with two.
__host__ __device__ constexpr int backward_ctas(int tpr, int vecs)
{
    return (vecs == 1 ? 768 : 512) / (tpr * backward_slots(tpr));
}

// Floats of a row of sums (see `at`).
__host__ __device__ constexpr int join_sum_cols(int cols, int mode) { return mode == kJoinWindow ? cols + 16 : cols; }

// Two vectors a thread, but one at 96 and 160 threads, where the SM holds half
// as many threads again (two vectors measured beside them: 16000 x 1152 LN/LN
// with 16 gate rows 69.8 us against 73.2 and 32000 x 768 RMS/RMS 62.8 against
// 63.8; the other norms the other way round, 56.4 against 52.7 and 89.0
// against 81.5).
constexpr Width kWidths[] = {{32, 1}, {32, 2}, {96, 1}, {64, 2}, {160, 1}, {96, 2},
                             {128, 2}, {192, 2}, {256, 2}, {384, 2}, {512, 2}};

__device__ __forceinline__ void copy_async16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// CENTER: a LayerNorm on either side (8 sums a row, beta1); without one 3.
// ONE: a CTA to a row (no cluster).
template <bool BF16, int MODE, int TPR, int VECS, bool CENTER, bool ONE>
__global__ void __launch_bounds__(TPR * backward_slots(TPR), backward_ctas(TPR, VECS))
    join_backward_kernel(const __grid_constant__ JoinArgs a)
{
    constexpr int kSlots = backward_slots(TPR);
    constexpr int kThreads = TPR * kSlots;
    constexpr int kStage = (4 * VECS + 1) * kThreads;   // 16-byte slots of one stage of the ring
    extern __shared__ uint4 ring[];   // [depth][vecs of x, residual, dy, dh; statistics][threads]
    float *const acc = reinterpret_cast<float *>(ring + a.depth * kStage);   // [arrays][slots][cols]
    __shared__ RowSumSmem sums;
    int half = 0;
    // With a LayerNorm, what does not need the row's sums is done between a
    // warp's arrival at their barrier and its wait: 32768 x 2048 198 -> 176 us,
    // 8192 x 5000 146 -> 133.  (With one vector a thread 16000 x 1152 took 72
    // against 69 us, and RMSNorm alone 5 % longer: fewer instructions to put
    // there, and the next rows asked for later.  In the window mode a column's
    // thread changes with the shift, and the barrier orders its sums.)
    constexpr bool kArrive = CENTER && ONE && TPR > 32 && VECS > 1 && MODE == kJoinAligned;
    __shared__ uint64_t given;
    uint32_t given_phase = 0;
    bool waits = true;
    const int cluster = ONE ? 1 : a.shape.cluster;
    const uint32_t rank = cluster > 1 ? cluster_ctarank() : 0u;
    const int64_t cta = blockIdx.x / cluster;
    const int64_t n_ctas = gridDim.x / cluster;
    const int slot = threadIdx.x / TPR;
    const int c0 = static_cast<int>(rank) * a.shape.cols;
    constexpr int kFull = ONE ? full_vectors(kWidths, TPR, VECS, MODE) : -1;
    const Place<MODE, TPR, kFull> p(c0, min(a.N, c0 + a.shape.cols), threadIdx.x % TPR);
    const int ncols = p.c1 - p.c0;
    const float inv_n = 1.0f / static_cast<float>(a.N);
    const bool norm1 = a.norm1 != kNormNone, norm2 = a.norm2 != kNormNone;
    const bool ln1 = CENTER && a.norm1 == kNormLayer, ln2 = CENTER && a.norm2 == kNormLayer;

    if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
    const int cols = a.shape.cols, sum_cols = join_sum_cols(cols, MODE), arr = kSlots * sum_cols;
    for (int i = threadIdx.x; i < a.arrays * arr; i += kThreads) acc[i] = 0.0f;
    // an array that the call does not have is zeros
    uint4 *const mine = ring + threadIdx.x;
    for (int i = 0; i < a.depth * (4 * VECS + 1); ++i) mine[i * kThreads] = make_uint4(0u, 0u, 0u, 0u);
    if (kArrive && threadIdx.x == 0) {
        mbar_init(&given, kThreads / 32);
        fence_mbarrier_init();
    }
    __syncthreads();
    if (cluster > 1) cluster_sync_all();   // every CTA runs before its shared memory is written

    // Where column c (from c0) of a sum lies, so that a warp's accesses fall
    // into different banks: aligned vectors as two planes of 16-byte halves,
    // shifted ones as eight planes of elements, which have room for a vector's
    // columns before c0 and behind the last (8192 x 5003: 182 -> 173 us against
    // a test for every element).
    const int plane = sum_cols >> 3;
    auto at = [&](int c) {
        if constexpr (MODE == kJoinAligned) return ((c >> 2) & 1) * (cols >> 1) + (c >> 3) * 4 + (c & 3);
        if constexpr (MODE == kJoinWindow) return (c & 7) * plane + (c >> 3) + 1;
        return c;
    };
    // sum `b` (of this slot) of vector v += d
    auto add8 = [&](float *b, int v, int s, const Vec8 &d) {
        if constexpr (MODE == kJoinAligned) {
            if (!p.whole(v, s)) return;
            float4 *lo = reinterpret_cast<float4 *>(b) + (threadIdx.x % TPR) + v * TPR;
            float4 *hi = reinterpret_cast<float4 *>(b + (cols >> 1)) + (threadIdx.x % TPR) + v * TPR;
            float4 x = *lo, y = *hi;
            const float2 x0 = __fadd2_rn(make_float2(x.x, x.y), d.p[0]), x1 = __fadd2_rn(make_float2(x.z, x.w), d.p[1]);
            const float2 y0 = __fadd2_rn(make_float2(y.x, y.y), d.p[2]), y1 = __fadd2_rn(make_float2(y.z, y.w), d.p[3]);
            *lo = make_float4(x0.x, x0.y, x1.x, x1.y);
            *hi = make_float4(y0.x, y0.y, y1.x, y1.y);
        } else if constexpr (MODE == kJoinWindow) {
            if (!p.some(v, s)) return;
            b += threadIdx.x % TPR + v * TPR;
#pragma unroll
            for (int j = 0; j < 8; ++j) {   // at(col - c0)
                const int e = j + 8 - s;
                b[e * plane + (e >= 8 ? 1 - 8 * plane : 0)] += (j & 1) ? d.p[j >> 1].y : d.p[j >> 1].x;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (p.valid(v, j, s))
                    b[at(p.col(v, j, s) - p.c0)] += (j & 1) ? d.p[j >> 1].y : d.p[j >> 1].x;
        }
    };
    auto sum_of = [&](int k) { return acc + (k < 0 ? 0 : k) * arr + slot * sum_cols; };
    float *const sum_p = sum_of(a.a_p), *const sum_q = sum_of(a.a_q);
    float *const sum_g2 = sum_of(a.a_dgamma2), *const sum_b2 = sum_of(a.a_dbeta2);
    // The CTA's sum k over its slots, by columns, to `put`; then zero.
    auto flush = [&](int k, auto put) {
        float *b = acc + k * arr;
        for (int c = threadIdx.x; c < ncols; c += kThreads) {
            float t = 0.0f;
            for (int q = 0; q < kSlots; ++q) {
                t += b[q * sum_cols + at(c)];
                b[q * sum_cols + at(c)] = 0.0f;
            }
            put(p.c0 + c, t);
        }
    };

    const int period = MODE == kJoinWindow ? a.period : 1;
    // The CTA's way through the rows of its items: one cursor for the rows it
    // works on, one for those it fetches.
    struct Cursor {
        int64_t item, base, r1, group;
    };
    auto open = [&](Cursor &c) {
        if (c.item >= a.items) return;
        c.group = c.item / a.items_per_group;
        const int64_t g0 = c.group * a.rows_per_gate;
        const int64_t g1 = g0 + a.rows_per_gate < a.M ? g0 + a.rows_per_gate : a.M;
        const int64_t i = c.item - c.group * a.items_per_group, run = MODE == kJoinWindow ? i / a.period : i;
        c.base = g0 + run * a.item_rows;
        c.r1 = c.base + a.item_rows < g1 ? c.base + a.item_rows : g1;
        if (MODE == kJoinWindow) c.base += i - run * a.period;
    };
    // the next rows of this item, or the first of the CTA's next item
    auto advance = [&](Cursor &c) {
        c.base += kSlots * period;
        if (c.base >= c.r1) {
            c.item += n_ctas;
            open(c);
        }
    };
    // The cursor's row into stage `st` of the ring.
    auto fetch = [&](const Cursor &c, uint4 *st) {
        const int64_t row = c.base + slot * period;
        if (c.item < a.items && row < c.r1) {
            const int s = row_shift<MODE>(a, row);
            const int64_t off = row * a.N;
            const void *src[4] = {a.x, a.residual, a.dy, a.dh};
            copy_async16(st + 4 * VECS * kThreads, a.stats + row);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (src[k] == nullptr) continue;
                const uint16_t *b = elements(src[k], off);
#pragma unroll
                for (int v = 0; v < VECS; ++v) {
                    uint4 *d = st + (k * VECS + v) * kThreads;
                    if constexpr (MODE == kJoinScalar) *d = load_elements(b, p, v, s);
                    else if (p.some(v, s)) copy_async16(d, b + p.col(v, 0, s));
                }
            }
        } else {
            // (what the slots held before may be anything; rstd 0 makes all terms
            // of a row that is not there 0)
#pragma unroll
            for (int i = 0; i < 4 * VECS + 1; ++i) st[i * kThreads] = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    Cursor now{cta, 0, 0, 0}, ahead{cta, 0, 0, 0};
    open(now);
    open(ahead);
    // w = s gate gamma1, wb = s gate beta1, g2 = gamma2 at this thread's
    // columns.  They hold for an item; in the window mode the columns move
    // with the row, so there as long as the rows have one shift.
    Vec8 w[VECS], wb[CENTER ? VECS : 1], g2[VECS];
    auto params = [&](int s) {
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const Vec8 gs = (a.gate ? param8<BF16>(elements(a.gate, now.group * a.N), p, v, s)
                                    : masked(filled(1.0f), p, v, s)) * a.block_scale;
            w[v] = norm1 ? gs * param8<BF16>(elements(a.gamma1), p, v, s) : gs;
            if constexpr (CENTER) wb[v] = ln1 ? gs * param8<BF16>(elements(a.beta1), p, v, s) : filled(0.0f);
            g2[v] = norm2 ? param8<BF16>(elements(a.gamma2), p, v, s) : filled(0.0f);
        }
    };
    for (int i = 0; i < a.depth; ++i) {
        fetch(ahead, mine + i * kStage);
        advance(ahead);
    }
    if (MODE != kJoinWindow && now.item < a.items) params(0);
    int shift = -1;   // kJoinWindow: the parameters' (-1: of another item)
    int stage = 0;
    while (now.item < a.items) {
        const int64_t row = now.base + slot * period;
        const bool active = row < now.r1;
        const int64_t off = row * a.N;
        const int s = row_shift<MODE>(a, row);
        // the oldest of the rows under way has arrived (each thread reads what
        // it copied itself)
        if (a.depth == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (a.depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 2;" ::: "memory");
        uint4 *const in = mine + stage * kStage;
        const float4 st = *reinterpret_cast<const float4 *>(in + 4 * VECS * kThreads);
        const float rs2 = norm2 ? st.w : 0.0f;
        if (MODE == kJoinWindow && s != shift) {
            params(s);
            shift = s;
        }

        Vec8 u1[VECS], u2[VECS], D[VECS];
        float2 t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = both(0.0f);
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            u1[v] = unpack8<BF16>(own_elements(in[v * kThreads], p, v, s));
            if constexpr (CENTER) u1[v] = u1[v] + -st.x;
            u1[v] = u1[v] * st.y;
            const Vec8 wu = w[v] * u1[v];
            Vec8 h = fma8(unpack8<BF16>(own_elements(in[(VECS + v) * kThreads], p, v, s)), a.residual_scale, wu);
            if constexpr (CENTER) h = h + wb[v] + -st.z;
            u2[v] = h * rs2;
            const Vec8 dy = unpack8<BF16>(own_elements(in[(2 * VECS + v) * kThreads], p, v, s));
            const Vec8 q = g2[v] * dy;
            D[v] = fma8(q, rs2, unpack8<BF16>(own_elements(in[(3 * VECS + v) * kThreads], p, v, s)));
            dot8(t[0], q, u2[v]);
            dot8(t[1], wu, D[v]);
            dot8(t[2], wu, u2[v]);
            if constexpr (CENTER) {
                sum8(t[3], q);
                dot8(t[4], w[v], D[v]);
                sum8(t[5], w[v]);
                dot8(t[6], w[v], u2[v]);
                sum8(t[7], wu);
            }
            if constexpr (!kArrive) {
                if (CENTER && a.a_dbeta2 >= 0) add8(sum_b2, v, s, dy);
                if (a.a_dgamma2 >= 0) add8(sum_g2, v, s, dy * u2[v]);
            }
        }
        if constexpr (!kArrive) {
            fetch(ahead, in);
            advance(ahead);
            stage = stage + 1 == a.depth ? 0 : stage + 1;
        }

        float k[CENTER ? 8 : 4];
#pragma unroll
        for (int i = 0; i < (CENTER ? 8 : 4); ++i) k[i] = t[i].x + t[i].y;
        if constexpr (kArrive) {
            row_sum<8, TPR>(k, sums, half, cluster, rank, [&] {
                __syncwarp();
                if ((threadIdx.x & 31) == 0) mbar_arrive(&given);
                if (a.a_dgamma2 >= 0) {
#pragma unroll
                    for (int v = 0; v < VECS; ++v) {
                        const Vec8 dy = unpack8<BF16>(own_elements(in[(2 * VECS + v) * kThreads], p, v, s));
                        if (a.a_dbeta2 >= 0) add8(sum_b2, v, s, dy);
                        add8(sum_g2, v, s, dy * u2[v]);
                    }
                }
                fetch(ahead, in);
                advance(ahead);
                stage = stage + 1 == a.depth ? 0 : stage + 1;
                // A wait that runs out is reported, and those to come try once.
                // (Here and not by the shared bounded wait: its call in this
                // loop, registers saved around it, took 32768 x 2048 from 177 to
                // 191 us.)
                uint64_t since = 0;
                for (uint32_t it = 1; !mbar_try_wait(&given, given_phase) && waits; ++it) {
                    if ((it & 63u) != 0) continue;
                    if (since == 0) since = global_timer_ns();
                    if (global_timer_ns() - since > a.timeout_ns) {
                        atomicExch(a.err, kDevErrTimeout);
                        waits = false;
                    }
                }
                given_phase ^= 1u;
            });
        } else {
            row_sum<CENTER ? 8 : 4, TPR>(k, sums, half, cluster, rank);
        }
        const float c1 = rs2 * k[0] * inv_n;
        float c_0 = 0.0f, t0 = 0.0f, t1 = norm1 ? k[1] - c1 * k[2] : 0.0f;
        if constexpr (CENTER) {
            if (ln2) c_0 = rs2 * k[3] * inv_n;
            if (ln1) t0 = (k[4] - c_0 * k[5] - c1 * k[6]) * inv_n;
            if (norm1) t1 -= c_0 * k[7];
        }
        t1 *= inv_n;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            D[v] = fma8(u2[v], -c1, D[v]);
            if constexpr (CENTER) D[v] = D[v] + -c_0;
            if (active) {
                Vec8 o = fma8(u1[v], -t1, w[v] * D[v]);
                if constexpr (CENTER) o = o + -t0;
                store8(elements(a.dx, off), p, v, s, pack8<BF16>(o * st.y));
                if (a.dresidual) store8(elements(a.dresidual, off), p, v, s, pack8<BF16>(D[v] * a.residual_scale));
            }
            if (a.fold_gate) {
                // (few rows to a gate row: gate applied here, dgate by groups)
                if (!active) continue;
                Vec8 n = norm1 ? u1[v] * param8<BF16>(elements(a.gamma1), p, v, s) : u1[v];
                if (ln1) n = n + param8<BF16>(elements(a.beta1), p, v, s);
                add8(sum_of(a.a_dgate), v, s, n * D[v] * a.block_scale);
                D[v] = D[v] * param8<BF16>(elements(a.gate, now.group * a.N), p, v, s) * a.block_scale;
            }
            if (a.a_p >= 0) add8(sum_p, v, s, u1[v] * D[v]);
            if (CENTER && a.a_q >= 0) add8(sum_q, v, s, D[v]);
        }
        const int64_t item = now.item, group = now.group;
        advance(now);
        if (now.item != item) {
            __syncthreads();
            if (a.fold_gate) {
                flush(a.a_dgate, [&](int c, float f) {
                    if (a.dgate) elements(a.dgate, group * a.N)[c] = round16<BF16>(f);
                });
            } else {
                if (a.a_p >= 0) flush(a.a_p, [&](int c, float f) { a.item_p[item * a.N + c] = f; });
                if (a.a_q >= 0) flush(a.a_q, [&](int c, float f) { a.item_q[item * a.N + c] = f; });
            }
            if (MODE != kJoinWindow && now.item < a.items) params(0);
            shift = -1;
            __syncthreads();
        }
    }
    __syncthreads();
    const int64_t row = cta * a.N;
    if (a.a_dgamma2 >= 0) flush(a.a_dgamma2, [&](int c, float f) { a.cta_sums[row + c] = f; });
    if (a.a_dbeta2 >= 0) flush(a.a_dbeta2, [&](int c, float f) { a.cta_sums[n_ctas * a.N + row + c] = f; });
    if (a.fold_gate) {
        if (a.a_p >= 0) flush(a.a_p, [&](int c, float f) { a.item_p[row + c] = f; });
        if (a.a_q >= 0) flush(a.a_q, [&](int c, float f) { a.item_q[row + c] = f; });
    }
}

inline int64_t ring_row(const JoinShape &s) { return (4ll * s.vecs + 1) * s.tpr * s.slots * 16; }
inline int64_t sum_bytes(const JoinShape &s, int arrays, int mode)
{
    return static_cast<int64_t>(arrays) * s.slots * join_sum_cols(s.cols, mode) * 4;
}

template <bool BF16, int MODE, bool CENTER>
int run_mode(JoinArgs a, int ctas, cudaStream_t stream)
{
    // as deep a ring as the SM's shared memory has room for beside the sums
    const int64_t row = ring_row(a.shape), sums = sum_bytes(a.shape, a.arrays, MODE);
    a.depth = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(3, (kJoinSmem / a.shape.per_sm - 2048 - sums) / row)));
    const size_t smem = static_cast<size_t>(sums + a.depth * row);
#define NGR_WIDTH(T, V, ONE)                                                                                    \
    if (a.shape.tpr == T && a.shape.vecs == V && (a.shape.cluster == 1) == ONE)                                 \
        return launch_join(join_backward_kernel<BF16, MODE, T, V, CENTER, ONE>, ctas, a.shape, smem, a, stream, \
                           "join gradient launch");
    NGR_WIDTH(512, 2, true)
    NGR_WIDTH(64, 2, true)
    NGR_WIDTH(512, 2, false)
    if constexpr (MODE != kJoinScalar) {
        NGR_WIDTH(32, 1, true)
        NGR_WIDTH(32, 2, true)
        NGR_WIDTH(96, 1, true)
        NGR_WIDTH(160, 1, true)
        NGR_WIDTH(96, 2, true)
        NGR_WIDTH(128, 2, true)
        NGR_WIDTH(192, 2, true)
        NGR_WIDTH(256, 2, true)
        NGR_WIDTH(384, 2, true)
        NGR_WIDTH(384, 2, false)
        // (five sums alone cut a row into CTAs of fewer than 4097 columns)
        if constexpr (CENTER) NGR_WIDTH(256, 2, false)
    }
#undef NGR_WIDTH
    return -9;
}

template <bool BF16, bool CENTER>
int run(int mode, const JoinArgs &a, int ctas, cudaStream_t stream)
{
    if (mode == kJoinAligned) return run_mode<BF16, kJoinAligned, CENTER>(a, ctas, stream);
    if (mode == kJoinWindow) return run_mode<BF16, kJoinWindow, CENTER>(a, ctas, stream);
    return run_mode<BF16, kJoinScalar, CENTER>(a, ctas, stream);
}

}  // namespace

}  // namespace ngr
