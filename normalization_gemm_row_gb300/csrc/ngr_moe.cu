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
// order that this gives, for both operands alike.  Nothing is staged, so a
// warp's loads of a whole tile are under way together.
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

template <bool BF16>
__device__ __forceinline__ float load16(const void *p, int64_t i)
{
    const uint16_t v = static_cast<const uint16_t *>(p)[i];
    if (BF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    return __half2float(__ushort_as_half(v));
}

// 8 elements from column k of a row of n (k a multiple of 8), zeros past its
// end.  VEC: the row starts on a 16-byte boundary and n is a multiple of 8.
// Read once: not kept in L1.
template <bool VEC>
__device__ __forceinline__ uint4 row8(const uint16_t *row, int k, int n)
{
    uint4 d = make_uint4(0u, 0u, 0u, 0u);
    if (k >= n) return d;
    if (VEC) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(d.x), "=r"(d.y), "=r"(d.z), "=r"(d.w)
                     : "l"(row + k));
        return d;
    }
    const int left = n - k;
    d = load_shifted(row + k, 0, left < 8 ? left : 8);
    if (left < 8) {
        uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] &= (2 * j < left ? 0xFFFFu : 0u) | (2 * j + 1 < left ? 0xFFFF0000u : 0u);
        d = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return d;
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

// The router: a cluster for a token.  Its CTAs share the experts, each with
// the token's normalized row in FP32, a piece at a time; the first CTA
// gathers the logits and chooses.
constexpr int kRouterPiece = 4096;
constexpr int kRouterPitch = kRouterPiece / 8 + 1;
constexpr int kRouterEach = kMoeMaxExperts / 8 / kWarps;    // experts a warp, with 8 CTAs

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kMoeThreads) moe_router_kernel(const __grid_constant__ MoeArgs a)
{
    // column k of a piece at [k % 8][k / 8]: a lane's 8 columns lie in 8 rows
    __shared__ float row[8 * kRouterPitch];
    __shared__ float logit[kMoeMaxExperts];
    __shared__ float red[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int m = static_cast<int>(blockIdx.x) / a.cluster;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *x = static_cast<const uint16_t *>(a.x) + static_cast<int64_t>(m) * a.K;
    pdl_launch_dependents();
    cluster.barrier_arrive();      // (waited for before the first one's memory is written: it has to have started)
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;

    float mean = 0.0f, scale = 1.0f;
    if (a.norm != kNormNone) {
        if (a.norm == kNormLayer) {
            float s = 0.0f;
            for (int k = threadIdx.x; k < a.K; k += kMoeThreads) s += load16<BF16>(x, k);
            mean = block_sum(s, red) / a.K;
        }
        float s = 0.0f;
        for (int k = threadIdx.x; k < a.K; k += kMoeThreads) {
            const float v = load16<BF16>(x, k) - mean;
            s += v * v;
        }
        scale = 1.0f / sqrtf(block_sum(s, red) / a.K + a.eps);
    }
    float z[kRouterEach];      // logits of experts (i warps + warp) cluster + rank
#pragma unroll
    for (int i = 0; i < kRouterEach; ++i) z[i] = 0.0f;
    for (int k0 = 0; k0 < a.Kp; k0 += kRouterPiece) {
        const int n = min(kRouterPiece, a.K - k0);
        __syncthreads();
        for (int k = threadIdx.x; k < kRouterPiece; k += kMoeThreads) {
            float v = 0.0f;
            if (k < n) {
                v = load16<BF16>(x, k0 + k);
                if (a.norm != kNormNone) {
                    v = (v - mean) * scale * load16<BF16>(a.gamma, k0 + k);
                    if (a.norm == kNormLayer) v += load16<BF16>(a.beta, k0 + k);
                }
            }
            row[(k & 7) * kRouterPitch + (k >> 3)] = v;
            // The experts' products take the row in the inputs' type, as the
            // library's other products do; the router takes it unrounded.
            if (rank == 0 && k0 + k < a.Kp)
                static_cast<uint16_t *>(a.a)[static_cast<int64_t>(m) * a.Kp + k0 + k] =
                    static_cast<uint16_t>(pack16<BF16>(v, 0.0f));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRouterEach; ++i) {
            const int e = (i * kWarps + warp) * a.cluster + rank;
            if (e >= a.E) continue;
            const uint16_t *wr = static_cast<const uint16_t *>(a.Wr) + static_cast<int64_t>(e) * a.K + k0;
#pragma unroll 4
            for (int k = lane * 8; k < n; k += 256) {
                const uint4 d = row8<VEC>(wr, k, n);
                const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = unpack16<BF16>(w[j]);
                    z[i] = fmaf(v.x, row[2 * j * kRouterPitch + (k >> 3)], z[i]);
                    z[i] = fmaf(v.y, row[(2 * j + 1) * kRouterPitch + (k >> 3)], z[i]);
                }
            }
        }
    }
    cluster.barrier_wait();
    float *logits = cluster.map_shared_rank(logit, 0);
#pragma unroll
    for (int i = 0; i < kRouterEach; ++i) {
        const int e = (i * kWarps + warp) * a.cluster + rank;
        if (e >= a.E) continue;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z[i] += __shfl_xor_sync(0xffffffffu, z[i], o);
        if (lane == 0) logits[e] = z[i];
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
    uint32_t taken = 0;            // of this lane's experts
    float p = 0.0f, sum = 0.0f;    // lane s: choice s
    int id = 0;
    for (int s = 0; s < a.top_k; ++s) {
        // the largest logit that is left, of equal ones the lowest expert's;
        // NaN counts as -inf, so that there is always a choice
        float best = -INFINITY;
        int at = kMoeMaxExperts;
        for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
            const float v = logit[e];
            if ((taken >> i) & 1u) continue;
            if (at == kMoeMaxExperts || v > best) {
                best = v == v ? v : -INFINITY;
                at = e;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float v = __shfl_xor_sync(0xffffffffu, best, o);
            const int other = __shfl_xor_sync(0xffffffffu, at, o);
            // (a lane without any expert left has at = kMoeMaxExperts)
            if (other < kMoeMaxExperts && (at == kMoeMaxExperts || v > best || (v == best && other < at))) {
                best = v;
                at = other;
            }
        }
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

// The experts that somebody chose, in order, for every CTA in its shared
// memory: the tokens of each as bits, and the first of its rows of h, which
// stand by expert and then by token.
struct Chosen {
    uint32_t tokens[kMoeMaxExperts];
    uint16_t expert[kMoeMaxExperts];
    uint16_t base[kMoeMaxExperts];
    int count;
};
__device__ __forceinline__ void find_chosen(const MoeArgs &a, Chosen &c)
{
    const int lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < a.E; e += kMoeThreads) c.tokens[e] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < a.M * a.top_k; i += kMoeThreads) atomicOr(&c.tokens[a.ids[i]], 1u << (i / a.top_k));
    __syncthreads();
    if (threadIdx.x < 32) {
        int n = 0, rows = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const uint32_t t = e < a.E ? c.tokens[e] : 0u;
            const uint32_t some = __ballot_sync(0xffffffffu, t != 0u);
            const int mine = __popc(t);
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const int at = n + __popc(some & ((1u << lane) - 1u));
            __syncwarp();
            // (places up to e only: nothing that is still to be read)
            if (t != 0u) {
                c.expert[at] = static_cast<uint16_t>(e);
                c.base[at] = static_cast<uint16_t>(rows + incl - mine);
                c.tokens[at] = t;
            }
            __syncwarp();
            n += __popc(some);
            rows += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) c.count = n;
    }
    __syncthreads();
}

// The row of h of a token and expert.
__device__ __forceinline__ int h_row(const Chosen &c, int i, int token)
{
    return c.base[i] + __popc(c.tokens[i] & ((1u << token) - 1u));
}

// One step of a contraction: 64 columns of the 16 rows r0 (rows 0 to 7) and
// r1 (8 to 15) of a weight against the tokens' rows b (NT x 8 columns of the
// instruction; null: no such token).
template <bool BF16, bool VEC, int NT>
__device__ __forceinline__ void step64(float (&acc)[NT][4], const uint16_t *r0, const uint16_t *r1, int k, int n,
                                       const uint16_t *const (&b)[NT], uint32_t live)
{
    const uint4 p0 = r0 ? row8<VEC>(r0, k, n) : make_uint4(0u, 0u, 0u, 0u);
    const uint4 q0 = r1 ? row8<VEC>(r1, k, n) : make_uint4(0u, 0u, 0u, 0u);
    const uint4 p1 = r0 ? row8<VEC>(r0, k + 32, n) : make_uint4(0u, 0u, 0u, 0u);
    const uint4 q1 = r1 ? row8<VEC>(r1, k + 32, n) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (NT > 1 && !((live >> j) & 1u)) continue;     // (the same for the whole warp)
        uint4 c0 = make_uint4(0u, 0u, 0u, 0u), c1 = c0;
        if (b[j]) {
            if (k < n) c0 = __ldg(reinterpret_cast<const uint4 *>(b[j] + k));
            if (k + 32 < n) c1 = __ldg(reinterpret_cast<const uint4 *>(b[j] + k + 32));
        }
        mma_16816<BF16>(acc[j], p0.x, q0.x, p0.y, q0.y, c0.x, c0.y);
        mma_16816<BF16>(acc[j], p0.z, q0.z, p0.w, q0.w, c0.z, c0.w);
        mma_16816<BF16>(acc[j], p1.x, q1.x, p1.y, q1.y, c1.x, c1.y);
        mma_16816<BF16>(acc[j], p1.z, q1.z, p1.w, q1.w, c1.z, c1.w);
    }
}

// Which of the NT groups of 8 tokens an expert has.
template <int NT>
__device__ __forceinline__ uint32_t live_groups(uint32_t tokens)
{
    uint32_t live = 0;
#pragma unroll
    for (int j = 0; j < NT; ++j) live |= ((tokens >> (8 * j)) & 255u) ? 1u << j : 0u;
    return live;
}

// Gate and up: a unit is 8 columns of h of one expert, the gate's weight rows
// as the instruction's rows 0 to 7 and the up's as 8 to 15, so that both
// products of an element end in one lane.  The warps share the contraction.
template <bool BF16, bool VEC, int NT>
__global__ void __launch_bounds__(kMoeThreads, 2) moe_up_kernel(const __grid_constant__ MoeArgs a)
{
    __shared__ Chosen c;
    __shared__ float red[2][kWarps][NT * 4][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait();
    find_chosen(a, c);
    const int tiles = (a.F + 7) / 8;
    const int64_t units = static_cast<int64_t>(c.count) * tiles;
    const int u1 = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    int buf = 0;
    for (int u = static_cast<int>(units * blockIdx.x / gridDim.x); u < u1; ++u, buf ^= 1) {
        const int i = u / tiles, f0 = (u - i * tiles) * 8, e = c.expert[i];
        const uint32_t tokens = c.tokens[i], live = live_groups<NT>(tokens);
        const int64_t wrow = (static_cast<int64_t>(e) * a.F + f0 + g) * a.K;
        const bool in = f0 + g < a.F;
        const uint16_t *wg = in ? static_cast<const uint16_t *>(a.Wg) + wrow : nullptr;
        const uint16_t *wu = in ? static_cast<const uint16_t *>(a.Wu) + wrow : nullptr;
        const uint16_t *b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
            b[j] = (tokens >> (8 * j + g)) & 1u ? static_cast<const uint16_t *>(a.a) + static_cast<int64_t>(8 * j + g) * a.Kp
                                                 : nullptr;
        float acc[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[j][r] = 0.0f;
#pragma unroll 4
        for (int k = warp * 64 + t * 8; k < a.Kp; k += kWarps * 64)
            step64<BF16, VEC, NT>(acc, wg, wu, k, a.K, b, live);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[buf][warp][j * 4 + r][lane] = acc[j][r];
        __syncthreads();
        if (warp < 2 * NT) {
            const int j = warp >> 1, col = warp & 1, token = 8 * j + 2 * t + col;
            if ((tokens >> token) & 1u) {
                float gate = 0.0f, up = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    gate += red[buf][w][j * 4 + col][lane];
                    up += red[buf][w][j * 4 + 2 + col][lane];
                }
                float p = 0.0f;
                for (int s = 0; s < a.top_k; ++s)
                    if (a.ids[token * a.top_k + s] == e) p = a.w[token * a.top_k + s];
                // The token's weight goes into h before it is rounded, so that
                // the last product is a plain sum over the experts.
                const float v = in ? p * (gate / (1.0f + expf(-gate)) * up) : 0.0f;
                static_cast<uint16_t *>(a.h)[static_cast<int64_t>(h_row(c, i, token)) * a.Fp + f0 + g] =
                    static_cast<uint16_t>(pack16<BF16>(v, 0.0f));
            }
        }
    }
}

// Down: a cluster makes 16 columns of y for all tokens; the chosen experts'
// rows of Wd, 64 columns a step, are shared by the cluster's warps.
template <bool BF16, bool VEC, int NT>
__global__ void __launch_bounds__(kMoeThreads, 2) moe_down_kernel(const __grid_constant__ MoeArgs a)
{
    __shared__ Chosen c;
    __shared__ float red[kWarps][NT * 4][32];
    __shared__ float part[NT * 4 * 32];
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int rank = static_cast<int>(cluster.block_rank());
    const int k0 = static_cast<int>(blockIdx.x) / a.splits * 16;
    pdl_wait();
    find_chosen(a, c);
    const int steps = (a.F + 63) / 64, all = c.count * steps;
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = 0.0f;
#pragma unroll 2
    for (int s = rank * kWarps + warp; s < all; s += a.splits * kWarps) {
        const int i = s / steps, f = (s - i * steps) * 64 + t * 8;
        const uint32_t tokens = c.tokens[i], live = live_groups<NT>(tokens);
        const uint16_t *wd = static_cast<const uint16_t *>(a.Wd) + (static_cast<int64_t>(c.expert[i]) * a.K + k0 + g) * a.F;
        const uint16_t *r0 = k0 + g < a.K ? wd : nullptr;
        const uint16_t *r1 = k0 + 8 + g < a.K ? wd + static_cast<int64_t>(8) * a.F : nullptr;
        const uint16_t *b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
            b[j] = (tokens >> (8 * j + g)) & 1u
                       ? static_cast<const uint16_t *>(a.h) + static_cast<int64_t>(h_row(c, i, 8 * j + g)) * a.Fp
                       : nullptr;
        step64<BF16, VEC, NT>(acc, r0, r1, f, a.F, b, live);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[warp][j * 4 + r][lane] = acc[j][r];
    __syncthreads();
    for (int v = threadIdx.x; v < NT * 128; v += kMoeThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += red[w][v >> 5][v & 31];
        part[v] = sum;
    }
    if (a.splits > 1) cluster.sync();
    else __syncthreads();
    if (rank == 0) {
        for (int v = threadIdx.x; v < NT * 128; v += kMoeThreads) {
            float sum = part[v];
            for (int r = 1; r < a.splits; ++r) sum += cluster.map_shared_rank(part, r)[v];
            const int l = v & 31, q = v >> 5, token = (q >> 2) * 8 + 2 * (l & 3) + (q & 1);
            const int k = k0 + (l >> 2) + ((q >> 1) & 1) * 8;
            if (token < a.M && k < a.K)
                static_cast<uint16_t *>(a.y)[static_cast<int64_t>(token) * a.K + k] =
                    static_cast<uint16_t>(pack16<BF16>(sum, 0.0f));
        }
    }
    if (a.splits > 1) cluster.sync();      // (the others' sums are read until here)
}

template <typename F>
cudaError_t launch(F *kern, unsigned grid, int cluster, bool after, const MoeArgs &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kMoeThreads);
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
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool BF16, bool VEC>
cudaError_t up(const MoeArgs &a, cudaStream_t stream)
{
    const unsigned grid = 2 * kMoeSms;
    if (a.M <= 8) return launch(moe_up_kernel<BF16, VEC, 1>, grid, 0, true, a, stream);
    if (a.M <= 16) return launch(moe_up_kernel<BF16, VEC, 2>, grid, 0, true, a, stream);
    return launch(moe_up_kernel<BF16, VEC, 4>, grid, 0, true, a, stream);
}

template <bool BF16, bool VEC>
cudaError_t down(const MoeArgs &a, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>((a.K + 15) / 16 * a.splits);
    if (a.M <= 8) return launch(moe_down_kernel<BF16, VEC, 1>, grid, a.splits, true, a, stream);
    if (a.M <= 16) return launch(moe_down_kernel<BF16, VEC, 2>, grid, a.splits, true, a, stream);
    return launch(moe_down_kernel<BF16, VEC, 4>, grid, a.splits, true, a, stream);
}

int status(const char *what, cudaError_t e) { return e == cudaSuccess ? 0 : record_cuda_error(what, e, cudaGetErrorString(e)); }

}  // namespace

int launch_moe_router(bool bf16, bool vec_k, const MoeArgs &a, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(a.M * a.cluster);
    const auto kern = bf16 ? (vec_k ? moe_router_kernel<true, true> : moe_router_kernel<true, false>)
                           : (vec_k ? moe_router_kernel<false, true> : moe_router_kernel<false, false>);
    return status("expert router launch", launch(kern, grid, a.cluster, false, a, stream));
}

int launch_moe_up(bool bf16, bool vec_k, const MoeArgs &a, cudaStream_t stream)
{
    return status("expert gate and up launch", bf16 ? (vec_k ? up<true, true>(a, stream) : up<true, false>(a, stream))
                                                    : (vec_k ? up<false, true>(a, stream) : up<false, false>(a, stream)));
}

int launch_moe_down(bool bf16, bool vec_f, const MoeArgs &a, cudaStream_t stream)
{
    return status("expert down launch", bf16 ? (vec_f ? down<true, true>(a, stream) : down<true, false>(a, stream))
                                             : (vec_f ? down<false, true>(a, stream) : down<false, false>(a, stream)));
}

}  // namespace ngr
