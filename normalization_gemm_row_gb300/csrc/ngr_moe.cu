// ngr_moe.cu -- a mixture-of-experts layer with SwiGLU experts for at most 32
// tokens, in three launches.
//
//   a = norm(x),  z = a Wr^T,  p = softmax(z),  the top_k largest p of each
//   token (ties: the lowest expert), divided by their sum if asked;
//   h = p SiLU(a Wg^T) (a Wu^T) for a token and chosen expert,
//   y = sum over the chosen experts of h Wd^T.
//
// A chosen expert's three weights, 6 F K bytes, serve the few tokens that
// chose it: reading them bounds the layer.  Each warp has a ring of stages in
// shared memory that its own asynchronous copies fill with weights and token
// rows, and takes them with 16 x 8 x 16 matrix instructions, the weight's rows
// as the instruction's rows and the tokens as its columns; it waits for
// nothing but its own copies.  (Weights loaded straight into the operands: 802
// us where the rings take 362, below.)
//
// The steps of a product (64 columns of 16 weight rows) over all chosen
// experts stand in one row that is cut into equal runs, one a warp
// ("worker"), so that any number of experts and any sizes keep every warp
// busy to the end; only the device knows the choice.  A worker's copies run
// some steps ahead, past the ends of units too.  A unit (16 rows' results)
// that several workers share is put together, in the workers' order, by the
// one that finishes last: the others leave their parts in memory and count.
//
// The instruction has 8 columns for 4 tokens: a token's row takes two, rounded
// to the 16-bit type and what that left out, so that rounding a and h costs
// no accuracy (a single rounding of each doubled y's error, 1.7e-3 to 3.4e-3
// in bf16), for no bytes of weights more.
//
// bf16, 32 tokens, 6 of 64 experts of 4096 x 1536: 362 us, gate and up 249 us
// (6.4 TB/s), down 125; one token, 2 of 8 experts of 4096 x 14336: 125 us.
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

// Two values as their rounded parts and what the rounding left out.  fp16's
// narrow range is moved for it: the value is taken times 2^-8, so that up to
// 2^24 fits, and the second part times 2^11 more, as it is that much smaller.
// Both together are off by at most 2^-22 of the value, or 2^-28.  (Without the
// scales what passed 65504 was infinite, and a value below 2^-14 had no second
// part: it was up to 2^-25 off.)
template <bool BF16>
constexpr float kValueScale = BF16 ? 1.0f : 1.0f / 256.0f;
template <bool BF16>
constexpr float kLowScale = BF16 ? 1.0f : 2048.0f;
template <bool BF16>
__device__ __forceinline__ uint2 two_parts(float x, float y)
{
    x *= kValueScale<BF16>;
    y *= kValueScale<BF16>;
    const uint32_t hi = pack16<BF16>(x, y);
    const float2 h = unpack16<BF16>(hi);
    // (an infinity has no second part)
    return make_uint2(hi, pack16<BF16>(fabsf(h.x) < INFINITY ? (x - h.x) * kLowScale<BF16> : 0.0f,
                                       fabsf(h.y) < INFINITY ? (y - h.y) * kLowScale<BF16> : 0.0f));
}
// A sum of products with values in two parts, from those with each of them.
template <bool BF16>
__device__ __forceinline__ float both_parts(float hi, float lo)
{
    if (BF16) return hi + lo;
    return fmaf(lo, 1.0f / kLowScale<BF16>, hi) * (1.0f / kValueScale<BF16>);
}

// ---------------------------------------------------------------- router
// A cluster of a.router CTAs (8, or 16 for many experts) for a token.  Its
// CTAs share the experts, each with the token's normalized row in FP32, a
// piece at a time; the first CTA gathers the logits and chooses.  Bound by the
// latency of what it does one after the other: row, statistics, logits,
// choice (10 us at 32 tokens of 4096, 32 experts, memory's caches flushed).
constexpr int kRouterPiece = 8192;
constexpr int kRouterPitch = kRouterPiece / 8 + 1;
constexpr int kRouterThreads = 512, kRouterWarps = kRouterThreads / 32;
constexpr int kRouterAtOnce = 2;      // experts of a warp

__device__ __forceinline__ float block_sum(float v, float *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kRouterWarps; ++w) v += red[w];
    return v;
}

// A float as an unsigned number of the same order, NaN as -inf.
__device__ __forceinline__ uint32_t order_of(float v)
{
    const uint32_t b = __float_as_uint(v == v ? v + 0.0f : -INFINITY);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kRouterThreads) moe_router_kernel(const __grid_constant__ MoeArgs a)
{
    // column k of a piece at [k % 8][k / 8]: a lane's 8 columns lie in 8 rows
    __shared__ float row[8 * kRouterPitch];
    __shared__ float logit[kMoeMaxExperts];
    __shared__ float mine[kMoeMaxExperts / 8][kRouterWarps];     // parts of the CTA's experts' logits
    __shared__ float red[kRouterWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int m = static_cast<int>(blockIdx.x) / a.router;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *x = static_cast<const uint16_t *>(a.x) + static_cast<int64_t>(m) * a.K;
    const uint16_t *gamma = static_cast<const uint16_t *>(a.gamma), *beta = static_cast<const uint16_t *>(a.beta);
    pdl_launch_dependents();
    cluster.barrier_arrive();      // (waited for before the first one's memory is written: it has to have started)
    // The CTA's experts rank, rank + a.router, ...: a warp takes two at once,
    // or a part of their rows where there are fewer pairs than warps.
    const int experts = rank < a.E ? (a.E - rank + a.router - 1) / a.router : 0;
    const int pairs = (experts + kRouterAtOnce - 1) / kRouterAtOnce;      // one a warp, or a part of its rows
    const int split = pairs >= 16 ? 1 : pairs >= 8 ? 2 : pairs >= 4 ? 4 : pairs >= 2 ? 8 : 16;
    const int slots = kRouterWarps / split, mine_of = warp / split, part = warp % split;
    uint4 held[kRouterPiece / 8 / kRouterThreads];      // the row, if it is no longer than a piece
    uint4 held_gamma[kRouterPiece / 8 / kRouterThreads];
    const bool short_row = a.K <= kRouterPiece;
    if (short_row && a.norm != kNormNone) {
#pragma unroll
        for (int i = 0; i < kRouterPiece / 8 / kRouterThreads; ++i)
            held_gamma[i] = row8<VEC>(gamma, (i * kRouterThreads + static_cast<int>(threadIdx.x)) * 8, a.K);
    }
    if (short_row) {
#pragma unroll
        for (int i = 0; i < kRouterPiece / 8 / kRouterThreads; ++i)
            held[i] = row8<VEC>(x, (i * kRouterThreads + static_cast<int>(threadIdx.x)) * 8, a.K);
    }
    // What is read last is on its way to L2 meanwhile.
    for (int i = mine_of; i < experts; i += slots) {
        const char *wr = static_cast<const char *>(a.Wr) + (static_cast<int64_t>(i) * a.router + rank) * a.K * 2;
        for (int at = (part * 32 + lane) * 128; at < a.K * 2; at += split * 32 * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(wr + at));
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
    for (int i = static_cast<int>(blockIdx.x) * kRouterThreads + threadIdx.x; i < kMoeCounters;
         i += static_cast<int>(gridDim.x) * kRouterThreads)
        a.counters[i] = 0;
    // f(values, column) over the row, 8 columns a thread at a time
    auto over_row = [&](auto f) {
        float v[8];
        if (short_row) {
#pragma unroll
            for (int i = 0; i < kRouterPiece / 8 / kRouterThreads; ++i) {
                const int k = (i * kRouterThreads + static_cast<int>(threadIdx.x)) * 8;
                if (k >= a.K) break;
                unpack8<BF16>(held[i], v);
                f(v, k);
            }
        } else {
#pragma unroll 4
            for (int k = threadIdx.x * 8; k < a.K; k += kRouterThreads * 8) {
                unpack8<BF16>(row8<VEC>(x, k, a.K), v);
                f(v, k);
            }
        }
    };
    float mean = 0.0f, scale = 1.0f;
    if (a.norm != kNormNone) {
        if (a.norm == kNormLayer) {
            float s = 0.0f;
            over_row([&](const float (&v)[8], int) {
#pragma unroll
                for (int j = 0; j < 8; ++j) s += v[j];
            });
            mean = block_sum(s, red) / a.K;
        }
        float s = 0.0f;
        over_row([&](const float (&v)[8], int k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float c = k + j < a.K ? v[j] - mean : 0.0f;
                s = fmaf(c, c, s);
            }
        });
        scale = 1.0f / sqrtf(block_sum(s, red) / a.K + a.eps);
    }
    for (int i = threadIdx.x; i < kMoeMaxExperts / 8 * kRouterWarps; i += kRouterThreads) mine[i / kRouterWarps][i % kRouterWarps] = 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += kRouterPiece) {
        const int n = min(kRouterPiece, a.K - k0);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRouterPiece / 8 / kRouterThreads; ++i) {
            const int c = i * kRouterThreads + static_cast<int>(threadIdx.x), k = k0 + c * 8;
            if (c * 8 >= n) break;
            float v[8];
            unpack8<BF16>(short_row ? held[i] : row8<VEC>(x, k, a.K), v);
            if (a.norm != kNormNone) {
                float g[8];
                unpack8<BF16>(short_row ? held_gamma[i] : row8<VEC>(gamma, k, a.K), g);
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
        // several experts of a warp at once: their rows' loads together, the
        // token's columns read once
        for (int i0 = mine_of; i0 < experts; i0 += kRouterAtOnce * slots) {
            float z[kRouterAtOnce] = {};
            const uint16_t *wr = static_cast<const uint16_t *>(a.Wr) + (static_cast<int64_t>(i0) * a.router + rank) * a.K;
            const int64_t next = static_cast<int64_t>(slots) * a.router * a.K;
            const bool both = i0 + slots < experts;
#pragma unroll 8
            for (int c = part * 32 + lane; c * 8 < n; c += split * 32) {
                uint4 d[kRouterAtOnce];
                d[0] = row8<VEC>(wr, k0 + c * 8, a.K);
                d[1] = both ? row8<VEC>(wr + next, k0 + c * 8, a.K) : zero4();
                float r[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = row[j * kRouterPitch + c];
#pragma unroll
                for (int u = 0; u < kRouterAtOnce; ++u) {
                    float w[8];
                    unpack8<BF16>(d[u], w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[u] = fmaf(w[j], r[j], z[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < kRouterAtOnce; ++u) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) z[u] += __shfl_xor_sync(0xffffffffu, z[u], o);
                if (lane == 0 && (u == 0 || both)) mine[i0 + u * slots][part] += z[u];
            }
        }
    }
    cluster.barrier_wait();
    float *logits = cluster.map_shared_rank(logit, 0);
    __syncthreads();
    for (int i = threadIdx.x; i < experts; i += kRouterThreads) {
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < kRouterWarps; ++w) z += mine[i][w];
        logits[i * a.router + rank] = z;
    }
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
    // The largest logit that is left, of equal ones the lowest expert's; NaN
    // counts as -inf, so that there is always a choice.  (Any logit's order is
    // above 0.)
    int id = 0;                    // lane s: choice s
    auto choose = [&](auto best_of, auto take) {
        for (int s = 0; s < a.top_k; ++s) {
            uint32_t best = 0;
            int at = kMoeMaxExperts;
            best_of(best, at);
            const uint32_t most = __reduce_max_sync(0xffffffffu, best);
            at = __reduce_min_sync(0xffffffffu, best == most ? at : kMoeMaxExperts);
            if ((at & 31) == lane) take(at >> 5);
            if (lane == s) id = at;
        }
    };
    constexpr int kHeld = 8;
    if (a.E <= 32 * kHeld) {
        uint32_t order[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) order[i] = lane + 32 * i < a.E ? order_of(logit[lane + 32 * i]) : 0u;
        choose(
            [&](uint32_t &best, int &at) {
#pragma unroll
                for (int i = 0; i < kHeld; ++i)
                    if (order[i] > best) {
                        best = order[i];
                        at = lane + 32 * i;
                    }
            },
            [&](int t) {
#pragma unroll
                for (int i = 0; i < kHeld; ++i)
                    if (i == t) order[i] = 0u;
            });
    } else {
        uint32_t taken = 0;        // of this lane's experts
        choose(
            [&](uint32_t &best, int &at) {
                for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
                    const uint32_t v = order_of(logit[e]);
                    if (!((taken >> i) & 1u) && v > best) {
                        best = v;
                        at = e;
                    }
                }
            },
            [&](int t) { taken |= 1u << t; });
    }
    float p = lane < a.top_k ? expf(logit[id] - top) / all : 0.0f, sum = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
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
// memory; one that more than ENTRY tokens chose stands there once for each
// ENTRY of them, and its weights' second reader finds them in L2 (it
// runs at the same time).  So every step costs the same, whatever the choice:
// with all of an expert's tokens in one entry the runs with the busiest
// experts kept the others waiting (down at 32 tokens, 32 experts of 4096 x
// 1536: a third of the warps' time; 433 us in all for the 32 tokens and 64
// experts above, against 362).  The rows of h stand by expert and then by
// token.
struct Chosen {
    uint16_t expert[kMoeMaxEntries], base[kMoeMaxEntries];
    uint8_t tokens[kMoeMaxEntries];
    uint8_t token[kMoeMaxTokens * kMoeMaxTopK];        // of a row of h
    int count;
};
struct ChosenScratch {
    uint32_t tokens[kMoeMaxExperts];                   // bits
    uint16_t base[kMoeMaxExperts];                     // by expert
};
// `p`, if not null, takes the weight of each row of h.
template <int THREADS, int ENTRY>
__device__ __forceinline__ void find_chosen(const MoeArgs &a, Chosen &c, ChosenScratch &x, float *p)
{
    const int lane = threadIdx.x & 31, all = a.M * a.top_k;
    // a thread's choices, most calls' only ones held
    const int i0 = threadIdx.x;
    int id0 = 0;
    float w0 = 0.0f;
    if (i0 < all) {
        id0 = __ldcg(a.ids + i0);
        if (p) w0 = __ldcg(a.w + i0);
    }
    for (int e = threadIdx.x; e < a.E; e += THREADS) x.tokens[e] = 0u;
    __syncthreads();
    for (int i = i0; i < all; i += THREADS) atomicOr(&x.tokens[i == i0 ? id0 : __ldcg(a.ids + i)], 1u << (i / a.top_k));
    __syncthreads();
    if (threadIdx.x < 32) {
        int n = 0, rows = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const uint32_t t = e0 + lane < a.E ? x.tokens[e0 + lane] : 0u;
            if (__ballot_sync(0xffffffffu, t != 0u) == 0u) continue;
            const int mine = __popc(t), entries = (mine + ENTRY - 1) / ENTRY;
            int incl = mine | entries << 16;      // both sums at once
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (t != 0u) {
                int at = n + (incl >> 16) - entries, r = rows + (incl & 0xFFFF) - mine, left = mine;
                x.base[e0 + lane] = static_cast<uint16_t>(r);
                for (int i = 0; i < entries; ++i, ++at, left -= ENTRY) {
                    c.expert[at] = static_cast<uint16_t>(e0 + lane);
                    c.base[at] = static_cast<uint16_t>(r + i * ENTRY);
                    c.tokens[at] = static_cast<uint8_t>(min(left, ENTRY));
                }
                for (uint32_t bits = t; bits; bits &= bits - 1u) c.token[r++] = static_cast<uint8_t>(__ffs(bits) - 1);
            }
            const int sums = __shfl_sync(0xffffffffu, incl, 31);
            n += sums >> 16;
            rows += sums & 0xFFFF;
        }
        if (lane == 0) c.count = n;
    }
    __syncthreads();
    if (p) {
        for (int i = i0; i < all; i += THREADS) {
            const int e = i == i0 ? id0 : __ldcg(a.ids + i), m = i / a.top_k;
            p[x.base[e] + __popc(x.tokens[e] & ((1u << m) - 1u))] = i == i0 ? w0 : __ldcg(a.w + i);
        }
    }
    __syncthreads();
}

// How one kernel is laid out, with room for NT groups of tokens in an entry.
constexpr int moe_warps(bool down, int nt) { return nt == 4 ? 5 : nt == 2 && down ? 7 : 8; }
template <bool DOWN, bool VEC, int NT>
struct Layout {
    static constexpr int kStages = NT == 1 ? 4 : 3;
    // A stage: a step's 16 weight rows of 128 bytes, or of the nine 16-byte
    // words that they lie in where rows are off the boundary, and 8 token
    // rows of 128 bytes a group.
    static constexpr int kGroups = NT, kEntry = NT * kMoeGroup;
    static constexpr int kPitch = VEC ? 128 : 144, kCopies = VEC ? 4 : 5;
    static constexpr int kTokens = 16 * kPitch, kStage = kTokens + NT * 1024;
    // DOWN: the tokens' sums of the 16 rows under way, [token][17]
    static constexpr int kMost = NT == 1 ? kMoeGroup : kMoeMaxTokens;
    static constexpr int kSums = DOWN ? kMost * 17 * 4 : 0;
    static constexpr int kWarp = kStages * kStage + kSums;
    // Two CTAs have to fit into an SM's shared memory.
    static constexpr int kWarps = moe_warps(DOWN, NT), kThreads = 32 * kWarps, kWorkers = kMoeCtas * kWarps;
    static constexpr int kWeights = DOWN ? 0 : kMost * kMoeMaxTopK * 4;
    static constexpr int kBytes = kWarps * kWarp + kWeights;
    static_assert(kWarps * kWarp >= static_cast<int>(sizeof(ChosenScratch)), "the rings hold it first");
    static_assert(2 * (kBytes + static_cast<int>(sizeof(Chosen)) + 1024) <= 228 * 1024, "two CTAs an SM");
    static_assert(kWorkers <= kMoeWorkers, "places of the parts");
};

// A segment: the steps over one expert's 16 rows.  DOWN: by 16 rows of Wd,
// then by expert; else by expert, then by 8 rows of Wg and of Wu.
struct Segment {
    int tile, i;
    int base, tokens;      // its rows of h
};
template <bool DOWN>
__device__ __forceinline__ void tokens_of(const Chosen &c, Segment &s)
{
    s.base = c.base[s.i];
    s.tokens = c.tokens[s.i];
}
// The next one: false behind the last.
template <bool DOWN>
__device__ __forceinline__ bool next(const Chosen &c, Segment &s, int tiles)
{
    if (DOWN) {
        if (++s.i == c.count) {
            s.i = 0;
            if (++s.tile == tiles) return false;
        }
    } else if (++s.tile == tiles) {
        s.tile = 0;
        if (++s.i == c.count) return false;
    }
    tokens_of<DOWN>(c, s);
    return true;
}

// The row (of a or h) of a token's part: column `col` of group j; null if
// there is none.
template <bool DOWN>
__device__ __forceinline__ const uint16_t *token_row(const MoeArgs &a, const Chosen &c, const Segment &s, int j, int col)
{
    const int r = j * kMoeGroup + (col >> 1);
    if (r >= s.tokens) return nullptr;
    if (DOWN) return static_cast<const uint16_t *>(a.h) + (static_cast<int64_t>(s.base + r) * 2 + (col & 1)) * a.Fp;
    return static_cast<const uint16_t *>(a.a) + (static_cast<int64_t>(c.token[s.base + r]) * 2 + (col & 1)) * a.Kp;
}

// A weight's 16 rows of the segment: the q-th of the first or second 8.
template <bool DOWN>
__device__ __forceinline__ const uint16_t *weight_row(const MoeArgs &a, const Chosen &c, const Segment &s, int half, int q)
{
    const int64_t e = c.expert[s.i];
    if (DOWN) return static_cast<const uint16_t *>(a.Wd) + (e * a.K + s.tile * 16 + half * 8 + q) * a.F;
    return static_cast<const uint16_t *>(half ? a.Wu : a.Wg) + (e * a.F + s.tile * 8 + q) * a.K;
}
template <bool DOWN>
__device__ __forceinline__ bool weight_there(const MoeArgs &a, const Segment &s, int half, int q)
{
    return DOWN ? s.tile * 16 + half * 8 + q < a.K : s.tile * 8 + q < a.F;
}

// A lane's copies of a segment's steps: 16 bytes from `from`, 128 further a
// step, for the first `steps` of them (then zeros).
template <typename L>
struct Copies {
    const uint16_t *from[L::kCopies], *token[2 * L::kGroups];
    int steps[L::kCopies], token_steps[2 * L::kGroups];

    template <bool VEC>
    __device__ __forceinline__ void weights(int step, uint32_t stage, int lane)
    {
#pragma unroll
        for (int i = 0; i < L::kCopies; ++i) {
            if (VEC) {
                const int r = i * 4 + (lane >> 3);
                cp_async16_ahead(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4), from[i], step < steps[i]);
            } else if (i * 32 + lane < 144) {
                cp_async16_ahead(stage + (i * 32 + lane) * 16, from[i], step < steps[i]);
            }
        }
        skip_weights();
    }
    __device__ __forceinline__ void tokens(int step, uint32_t stage, int lane)
    {
#pragma unroll
        for (int i = 0; i < 2 * L::kGroups; ++i) {
            const int col = (i & 1) * 4 + (lane >> 3);
            cp_async16(stage + L::kTokens + (i >> 1) * 1024 + col * 128 + (((lane & 7) ^ col) << 4), token[i],
                       step < token_steps[i]);
            token[i] += 64;
        }
    }
    __device__ __forceinline__ void skip_weights()
    {
#pragma unroll
        for (int i = 0; i < L::kCopies; ++i) from[i] += 64;
    }
    // On to the next 8 rows of the same experts' weights, of n elements, behind
    // a segment's `length` steps: the rows' distances from the boundary stay.
    __device__ __forceinline__ void next_rows(int n, int length)
    {
#pragma unroll
        for (int i = 0; i < L::kCopies; ++i) from[i] += 8 * static_cast<int64_t>(n) - length * 64;
#pragma unroll
        for (int i = 0; i < 2 * L::kGroups; ++i) token[i] -= length * 64;
    }
    __device__ __forceinline__ void skip(int steps)
    {
#pragma unroll
        for (int i = 0; i < L::kCopies; ++i) from[i] += steps * 64;
#pragma unroll
        for (int i = 0; i < 2 * L::kGroups; ++i) token[i] += steps * 64;
    }
};
template <bool DOWN, bool VEC, typename L>
__device__ __forceinline__ void plan_copies(const MoeArgs &a, const Chosen &c, const Segment &s, Copies<L> &p, int lane)
{
    const int n = DOWN ? a.F : a.K;
#pragma unroll
    for (int i = 0; i < L::kCopies; ++i) {
        if (VEC) {
            const int r = i * 4 + (lane >> 3), col = (lane & 7) * 8;
            const bool there = weight_there<DOWN>(a, s, r >> 3, r & 7);
            p.from[i] = weight_row<DOWN>(a, c, s, there ? r >> 3 : 0, there ? r & 7 : 0) + col;
            p.steps[i] = there ? (n - col + 63) >> 6 : 0;
        } else {
            // word `col` after the aligned one that the row's start lies in:
            // there as long as it holds any column below n
            const int w = i * 32 + lane, r = w / 9, col = w - r * 9;
            const bool there = r < 16 && weight_there<DOWN>(a, s, r >> 3, r & 7);
            const uint16_t *row = weight_row<DOWN>(a, c, s, there ? r >> 3 : 0, there ? r & 7 : 0);
            const int d = static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) & 7u);
            p.from[i] = row - d + col * 8;
            p.steps[i] = there && (col < 8 || d > 0) ? (n - col * 8 + d + 63) >> 6 : 0;
        }
    }
#pragma unroll
    for (int i = 0; i < 2 * L::kGroups; ++i) {
        const uint16_t *row = token_row<DOWN>(a, c, s, i >> 1, (i & 1) * 4 + (lane >> 3));
        const int col = (lane & 7) * 8;
        p.token[i] = (row ? row : static_cast<const uint16_t *>(a.h)) + col;
        p.token_steps[i] = row ? (n - col + 63) >> 6 : 0;
    }
}
// The 32-bit operand word at `at` of a row off the 16-byte boundary: from there
// if its columns start with a word, else (shift 16) from the middle of it to
// that of the next.  (Both are read: neighbouring rows' distances differ, and
// a branch would part the warp.)
__device__ __forceinline__ uint32_t pair_at(uint32_t at, uint32_t shift)
{
    uint32_t lo, hi;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(lo) : "r"(at) : "memory");
    asm volatile("ld.shared.u32 %0, [%1 + 4];" : "=r"(hi) : "r"(at) : "memory");
    return __funnelshift_r(lo, hi, shift);
}

// The products of one step, `left` columns from the row's end.  d0, d1: how
// far rows g and g + 8 start from the boundary.
template <bool BF16, bool DOWN, bool VEC, int NT>
__device__ __forceinline__ void take(float (&acc)[NT][4], int tokens, int left, int d0, int d1, uint32_t stage, int lane)
{
    using L = Layout<DOWN, VEC, NT>;
    const int g = lane >> 2, t = lane & 3;
    uint32_t w[4][4];      // the weights' operands of four contractions of 16
    if (VEC) {
        const int r = ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) ldmatrix4(w[i], stage + r * 128 + (((2 * i + half) ^ (r & 7)) << 4));
    } else {
        const uint32_t at0 = stage + g * 144 + (d0 >> 1) * 4 + t * 4, at1 = stage + (g + 8) * 144 + (d1 >> 1) * 4 + t * 4;
        const uint32_t shift0 = (d0 & 1) * 16, shift1 = (d1 & 1) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[i][2 * h] = pair_at(at0 + i * 32 + h * 16, shift0);
                w[i][2 * h + 1] = pair_at(at1 + i * 32 + h * 16, shift1);
            }
        if (left < 64) {      // what follows the row's end belongs to the next row
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = i * 16 + h * 8 + 2 * t;
                    const uint32_t keep = (e < left ? 0xFFFFu : 0u) | (e + 1 < left ? 0xFFFF0000u : 0u);
                    w[i][2 * h] &= keep;
                    w[i][2 * h + 1] &= keep;
                }
        }
    }
#pragma unroll
    for (int j = 0; j < L::kGroups; ++j) {
        if (j > 0 && j * kMoeGroup >= tokens) break;
        const int col = lane & 7, quarter = lane >> 3;
        const uint32_t row = stage + L::kTokens + j * 1024 + col * 128;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t b[4];
            ldmatrix4(b, row + (((4 * i + quarter) ^ col) << 4));
            mma_16816<BF16>(acc[j], w[2 * i][0], w[2 * i][1], w[2 * i][2], w[2 * i][3], b[0], b[1]);
            mma_16816<BF16>(acc[j], w[2 * i + 1][0], w[2 * i + 1][1], w[2 * i + 1][2], w[2 * i + 1][3], b[2], b[3]);
        }
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

// The parts of 16 rows' sums for all tokens, added in the workers' order into
// sums [token][17].  A part is M x 4 pieces of 16 bytes: few tokens' are read
// several at a time, each by some of the lanes; of many a lane reads several
// pieces at a time.
template <int PIECES>
__device__ __forceinline__ void gather_pieces(const MoeArgs &a, const Sharers &w, float *sums, int lane, int each)
{
    const float4 *parts = reinterpret_cast<const float4 *>(a.parts);
    const int pitch = a.part_bytes / 16, group = lane / each, groups = 32 / each, v = lane % each;
    float4 x[PIECES] = {};
#pragma unroll 4
    for (int p = w.first + group; p <= w.last; p += groups) {
        const float4 *from = parts + (static_cast<int64_t>(p) * 2 + (p == w.first ? 1 : 0)) * pitch + v;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            if (v + i * 32 < a.M * 4) {
                const float4 y = __ldcg(from + i * 32);
                x[i].x += y.x;
                x[i].y += y.y;
                x[i].z += y.z;
                x[i].w += y.w;
            }
        }
    }
    for (int o = 16; o >= each; o >>= 1) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            x[i].x += __shfl_xor_sync(0xffffffffu, x[i].x, o);
            x[i].y += __shfl_xor_sync(0xffffffffu, x[i].y, o);
            x[i].z += __shfl_xor_sync(0xffffffffu, x[i].z, o);
            x[i].w += __shfl_xor_sync(0xffffffffu, x[i].w, o);
        }
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int at = v + i * 32;
        if (group == 0 && at < a.M * 4) {
            float *to = sums + (at >> 2) * 17 + (at & 3) * 4;
            to[0] = x[i].x;
            to[1] = x[i].y;
            to[2] = x[i].z;
            to[3] = x[i].w;
        }
    }
    __syncwarp();
}
__device__ __forceinline__ void gather_parts(const MoeArgs &a, const Sharers &w, float *sums, int lane)
{
    if (a.M <= 8) gather_pieces<1>(a, w, sums, lane, a.M == 1 ? 4 : a.M == 2 ? 8 : a.M <= 4 ? 16 : 32);
    else gather_pieces<4>(a, w, sums, lane, 32);
}

template <bool BF16, bool DOWN, bool VEC, int NT>
__global__ void __launch_bounds__(32 * moe_warps(DOWN, NT), 2) moe_kernel(const __grid_constant__ MoeArgs a)
{
    using L = Layout<DOWN, VEC, NT>;
    constexpr int S = L::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Chosen c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    float *weights = DOWN ? nullptr : reinterpret_cast<float *>(smem + L::kWarps * L::kWarp);
    // Up waits for the router and lets down start only then, so that down may
    // read the choice before it waits for up.
    if (!DOWN) {
        pdl_wait();
        pdl_launch_dependents();
    }
    find_chosen<L::kThreads, L::kEntry>(a, c, *reinterpret_cast<ChosenScratch *>(smem), weights);

    const int n = DOWN ? a.F : a.K;
    const int length = (n + 63) / 64, tiles = DOWN ? (a.K + 15) / 16 : (a.F + 7) / 8;
    const int64_t total = static_cast<int64_t>(c.count) * tiles * length;
    // (steps of a unit: a segment, or DOWN the segments of 16 rows)
    const int64_t unit = DOWN ? static_cast<int64_t>(c.count) * length : length;
    // Steps of a worker: at least as many as a unit then has workers, whose
    // last one adds their parts at about a step's time each (down's parts of
    // fewer than 8 tokens: several at once, in that measure).  19 tokens, 4 of
    // 8 experts of 192 x 4544 (12 units of down): 43 us, of half or twice as
    // many workers 50 and 46, without this limit 98; 29 tokens, 5 of 122 of 156
    // x 3958 (10 units): 148 us, 165 and 158, at 24 workers 194; one token, 2 of
    // 8 of 256 x 16384: 29 us, as with 8 tokens' measure 31.
    const float cost = DOWN && a.M < 8 ? static_cast<float>(a.M) * 0.125f : 1.0f;
    const int64_t share = max(max(static_cast<int64_t>(kMoeMinShare), static_cast<int64_t>(sqrtf(cost * static_cast<float>(unit)))),
                              (total + L::kWorkers - 1) / L::kWorkers);
    const int worker = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    const int64_t first = worker * share;
    if (first >= total) return;
    const int count = static_cast<int>(min(share, total - first));

    const uint32_t ring = smem_u32(smem) + warp * L::kWarp;
    float *sums = reinterpret_cast<float *>(smem + warp * L::kWarp + S * L::kStage);
    int *counts = a.counters + (DOWN ? kMoeWorkers : 0);
    Segment s;
    const int64_t index = first / length;
    int step = static_cast<int>(first - index * length), ahead = step;
    s.i = static_cast<int>(DOWN ? index % c.count : index / tiles);
    s.tile = static_cast<int>(DOWN ? index / c.count : index % tiles);
    tokens_of<DOWN>(c, s);
    Segment f = s;
    Copies<L> copies;
    plan_copies<DOWN, VEC, L>(a, c, f, copies, lane);
    copies.skip(step);
    auto advance = [&] {
        if (++ahead == length) {
            ahead = 0;
            const int i = f.i;
            if (next<DOWN>(c, f, tiles)) {
                if (!DOWN && f.i == i && f.tile + 1 < tiles) copies.next_rows(n, length);
                else plan_copies<DOWN, VEC, L>(a, c, f, copies, lane);
            }
        }
    };
    if (DOWN) {
        // The first stages' weights are on their way while up ends: the
        // choice is known since up began.
        const Segment f0 = f;
        const Copies<L> copies0 = copies;
        const int ahead0 = ahead;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            if (i < count) {
                copies.template weights<VEC>(ahead, ring + i * L::kStage, lane);
                advance();
            }
        }
        pdl_wait();
        f = f0;
        copies = copies0;
        ahead = ahead0;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
        if (i < count) {
            if (DOWN) copies.skip_weights();
            else copies.template weights<VEC>(ahead, ring + i * L::kStage, lane);
            copies.tokens(ahead, ring + i * L::kStage, lane);
            advance();
        }
        cp_async_commit();
    }
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = 0.0f;
    if (DOWN) {
        for (int i = lane; i < L::kMost * 17; i += 32) sums[i] = 0.0f;
        __syncwarp();
    }
    int64_t begin = DOWN ? s.tile * unit : index * length;
    int d0 = 0, d1 = 0, stage = 0;
    bool fresh = true;
    for (int i = 0; i < count; ++i) {
        if (!VEC && fresh) {
            d0 = static_cast<int>((reinterpret_cast<uintptr_t>(weight_row<DOWN>(a, c, s, 0, g)) >> 1) & 7u);
            d1 = static_cast<int>((reinterpret_cast<uintptr_t>(weight_row<DOWN>(a, c, s, 1, g)) >> 1) & 7u);
            fresh = false;
        }
        cp_async_wait<S - 1>();
        __syncwarp();
        take<BF16, DOWN, VEC, NT>(acc, s.tokens, n - step * 64, d0, d1, ring + stage * L::kStage, lane);
        __syncwarp();
        if (i + S < count) {
            copies.template weights<VEC>(ahead, ring + stage * L::kStage, lane);
            copies.tokens(ahead, ring + stage * L::kStage, lane);
            advance();
        }
        cp_async_commit();
        stage = stage + 1 == S ? 0 : stage + 1;
        const bool ends = ++step == length, done = i + 1 == count;
        if (!ends && !done) continue;

        // the segment's end, or the run's
        const int64_t end = begin + unit, at = first + i + 1;
        const bool close = at == end || done, whole = begin >= first && end <= at;
        Sharers w = {0, 0};
        int64_t slot = 0;
        if (close && !whole) {
            w = sharers(begin, end, share);
            slot = static_cast<int64_t>(worker) * 2 + (worker == w.first ? 1 : 0);
        }
        if (!DOWN) {
            float2 v[NT];      // gate and up of row g for token t of each group
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                v[j] = make_float2(both_parts<BF16>(acc[j][0], acc[j][1]), both_parts<BF16>(acc[j][2], acc[j][3]));
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[j][r] = 0.0f;
            }
            bool finish = whole;
            if (!whole) {
                float2 *part = reinterpret_cast<float2 *>(a.parts) + slot * (a.part_bytes / 8) + lane;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j * kMoeGroup < s.tokens) part[j * 32] = v[j];
                finish = counted_last(counts, w, lane);
                if (finish) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) v[j] = make_float2(0.0f, 0.0f);
#pragma unroll 4
                    for (int p = w.first; p <= w.last; ++p) {
                        const float2 *from = reinterpret_cast<const float2 *>(a.parts) +
                                             (static_cast<int64_t>(p) * 2 + (p == w.first ? 1 : 0)) * (a.part_bytes / 8) + lane;
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
                    // The token's weight goes into h, so that the last
                    // product is a plain sum over the experts.
                    const float h = weight_there<DOWN>(a, s, 0, g)
                                        ? weights[s.base + r] * (v[j].x / (1.0f + expf(-v[j].x)) * v[j].y)
                                        : 0.0f;
                    const uint2 parts = two_parts<BF16>(h, 0.0f);
                    uint16_t *out = static_cast<uint16_t *>(a.h) + static_cast<int64_t>(s.base + r) * 2 * a.Fp + s.tile * 8 + g;
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
                    to[g] += both_parts<BF16>(acc[j][0], acc[j][1]);
                    to[g + 8] += both_parts<BF16>(acc[j][2], acc[j][3]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[j][q] = 0.0f;
            }
            __syncwarp();
            if (close) {
                const int row0 = s.tile * 16, values = a.M * 16;
                bool finish = whole;
                if (!whole) {
                    // (16-byte pieces: M tokens x 4 of them)
                    float4 *part = reinterpret_cast<float4 *>(a.parts) + slot * (a.part_bytes / 16);
                    for (int v = lane; v < a.M * 4; v += 32) {
                        const float *from = sums + (v >> 2) * 17 + (v & 3) * 4;
                        part[v] = make_float4(from[0], from[1], from[2], from[3]);
                    }
                    finish = counted_last(counts, w, lane);
                    if (finish) gather_parts(a, w, sums, lane);
                }
                if (finish)
                    for (int v = lane; v < values; v += 32)
                        if (row0 + (v & 15) < a.K)
                            static_cast<uint16_t *>(a.y)[static_cast<int64_t>(v >> 4) * a.K + row0 + (v & 15)] =
                                static_cast<uint16_t>(pack16<BF16>(sums[(v >> 4) * 17 + (v & 15)], 0.0f));
                __syncwarp();
                for (int v = lane; v < L::kMost * 17; v += 32) sums[v] = 0.0f;
                __syncwarp();
            }
        }
        if (ends) {
            step = 0;
            fresh = true;
            if (at == end) begin = end;
            next<DOWN>(c, s, tiles);
        }
    }
    cp_async_wait<0>();
}

template <typename F>
cudaError_t launch(F *kern, unsigned grid, unsigned threads, int cluster, size_t smem, bool after, const MoeArgs &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
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
    if (cluster > 8) {      // a size that has to be asked for
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    if (smem > 0) {
        // (an attribute of the current device's copy of the function)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool BF16, bool DOWN, bool VEC, int NT>
cudaError_t product(const MoeArgs &a, cudaStream_t stream)
{
    using L = Layout<DOWN, VEC, NT>;
    return launch(moe_kernel<BF16, DOWN, VEC, NT>, kMoeCtas, L::kThreads, 0, L::kBytes, true, a, stream);
}

template <bool BF16, bool DOWN, bool VEC>
cudaError_t product(const MoeArgs &a, cudaStream_t stream)
{
    switch (a.groups) {
    case 1: return product<BF16, DOWN, VEC, 1>(a, stream);
    case 2: return product<BF16, DOWN, VEC, 2>(a, stream);
    default: return product<BF16, DOWN, VEC, 4>(a, stream);
    }
}

int status(const char *what, cudaError_t e) { return e == cudaSuccess ? 0 : record_cuda_error(what, e, cudaGetErrorString(e)); }

}  // namespace

int launch_moe_router(bool bf16, bool vec, const MoeArgs &a, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(a.M * a.router);
    const auto kern = bf16 ? (vec ? moe_router_kernel<true, true> : moe_router_kernel<true, false>)
                           : (vec ? moe_router_kernel<false, true> : moe_router_kernel<false, false>);
    return status("expert router launch", launch(kern, grid, kRouterThreads, a.router, 0, false, a, stream));
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
