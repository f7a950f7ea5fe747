// ngr_ce.cu -- the linear cross entropy around its products: which tokens
// count, their rows gathered, the last step of the loss, the last sums of dx.
//
// Tokens whose target is negative take no part: the counted tokens' rows are
// copied together, so that the products run over those alone, nothing a
// masked row holds (infinities, NaN) reaches a sum, and the rows start on
// 128-byte lines whatever K is.  The copy moves 4 K bytes a token against the
// 2 K V operations of one product.
#include "ngr_ce.h"
#include "ngr_internal.h"
#include "ngr_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace ngr {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kDzUnit = 8192.0f;   // dz's largest weight
constexpr int kIndexThreads = 1024, kIndexEach = 8;
constexpr int kGatherThreads = 128;
constexpr int kLossThreads = 1024;

// One CTA: a prefix sum over the tokens gives each counted token its place
// (their order kept) and the others theirs from the end; the largest weight
// is the unit of dz.
__global__ void __launch_bounds__(kIndexThreads) ce_index_kernel(const __grid_constant__ CeTokens t)
{
    __shared__ int warp_sum[kIndexThreads / 32];
    __shared__ float warp_max[kIndexThreads / 32];
    __shared__ int bad;
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    int64_t base = 0;   // counted tokens before this round
    float top = 0.0f;
    for (int64_t r0 = 0; r0 < t.M; r0 += kIndexThreads * kIndexEach) {
        const int64_t i0 = r0 + static_cast<int64_t>(threadIdx.x) * kIndexEach;
        int64_t target[kIndexEach];
        int mine = 0;
#pragma unroll
        for (int j = 0; j < kIndexEach; ++j) {
            target[j] = i0 + j < t.M ? t.target[i0 + j] : -1;
            if (target[j] >= t.V) {
                bad = 1;
                target[j] = -1;
            }
            mine += target[j] >= 0;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int before = 0, total = 0;
        for (int w = 0; w < kIndexThreads / 32; ++w) {
            if (w < warp) before += warp_sum[w];
            total += warp_sum[w];
        }
        int64_t at = base + before + incl - mine;
#pragma unroll
        for (int j = 0; j < kIndexEach; ++j) {
            const int64_t i = i0 + j;
            if (i >= t.M) continue;
            if (target[j] >= 0) {
                t.index[at] = static_cast<int>(i);
                t.ctarget[at] = static_cast<int>(target[j]);
                ++at;
                if (t.lse) {
                    const float g = t.dloss ? t.dloss[i] : 0.0f, l = t.dlse ? t.dlse[i] : 0.0f;
                    top = fmaxf(top, fmaxf(fabsf(g), fabsf(g + l)));
                }
            } else {
                t.index[t.M - 1 - (i - at)] = static_cast<int>(i);
            }
        }
        base += total;
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) warp_max[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 0; w < kIndexThreads / 32; ++w) top = fmaxf(top, warp_max[w]);
        top *= fabsf(t.logit_scale);
        // (no weight, or one that is not finite: unscaled)
        if (!(top >= 1.0e-30f && top <= 1.0e38f)) top = kDzUnit;
        CeInfo info;
        info.count = static_cast<int>(base);
        info.weight = top;
        info.down = top / kDzUnit;
        *t.info = info;
        *t.err = bad ? kDevErrTarget : 0;
    }
}

// One CTA per row of the gathered matrix at a time: a counted token's row
// (padded with zeros to Kx), zero rows up to the next 64 (the contracted
// length of dW), and in the backward call each row's softmax constants and
// zeros for the dx rows of the tokens that do not count.
template <bool VEC>
__global__ void __launch_bounds__(kGatherThreads) ce_gather_kernel(const __grid_constant__ CeTokens t)
{
    pdl_launch_dependents();
    pdl_wait();
    const int count = t.info->count;
    const int64_t filled = (static_cast<int64_t>(max(count, 1)) + 63) / 64 * 64;
    const int64_t last = filled > t.M ? filled : t.M;
    const int vecs = static_cast<int>(t.Kx / 8), whole = static_cast<int>(t.K / 8);
    for (int64_t r = blockIdx.x; r < last; r += gridDim.x) {
        const int64_t token = r < t.M ? t.index[r] : 0;
        if (r < filled) {
            uint4 *dst = static_cast<uint4 *>(t.xc) + r * vecs;
            const uint16_t *src = static_cast<const uint16_t *>(t.x) + token * t.K;
#pragma unroll 4
            for (int v = threadIdx.x; v < vecs; v += kGatherThreads) {
                uint4 d = make_uint4(0u, 0u, 0u, 0u);
                if (r < count) {
                    if constexpr (VEC) {
                        if (v < whole) d = reinterpret_cast<const uint4 *>(src)[v];
                    } else {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int64_t c = 8 * static_cast<int64_t>(v) + 2 * j;
                            const uint32_t lo = c < t.K ? src[c] : 0u;
                            const uint32_t hi = c + 1 < t.K ? src[c + 1] : 0u;
                            w[j] = lo | (hi << 16);
                        }
                        d = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                dst[v] = d;
            }
        }
        if (t.row && r < count && threadIdx.x == 0) {
            const float top = t.info->weight;
            const float g = t.dloss ? t.dloss[token] : 0.0f, l = t.dlse ? t.dlse[token] : 0.0f;
            t.row[r] = CeRow{t.lse[token] * kLog2e, (g + l) * t.logit_scale / top * kDzUnit,
                             g * t.logit_scale / top * kDzUnit, t.ctarget[r]};
        }
        if (t.dx && r >= count && r < t.M) {
            uint16_t *dst = static_cast<uint16_t *>(t.dx) + token * t.K;
            if constexpr (VEC) {
                for (int v = threadIdx.x; v < whole; v += kGatherThreads)
                    reinterpret_cast<uint4 *>(dst)[v] = make_uint4(0u, 0u, 0u, 0u);
            } else {
                for (int64_t c = threadIdx.x; c < t.K; c += kGatherThreads) dst[c] = 0;
            }
        }
    }
}

// (max, sum) pairs in powers of two, merged in a fixed order.
__device__ __forceinline__ void merge(float &m, float &s, float om, float os)
{
    const float top = fmaxf(m, om);
    const float base = top == -INFINITY ? 0.0f : top;
    s = s * exp2f(m - base) + os * exp2f(om - base);
    m = top;
}

// A row's pairs over the column tiles -> its lse and loss.  `rows` rows per
// CTA (1 or 32), the CTA's other threads along the pairs.
__global__ void __launch_bounds__(kLossThreads) ce_loss_kernel(
    const __grid_constant__ CeTokens t, const float2 *__restrict__ part, int64_t part_pitch, int parts,
    const float *__restrict__ z_target, float *loss, float *lse, int rows)
{
    __shared__ float2 pair[kLossThreads];
    const int lanes = kLossThreads / rows;
    const int x = threadIdx.x % rows, y = threadIdx.x / rows;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * rows + x;
    pdl_wait();
    const int count = t.info->count;
    float m = -INFINITY, s = 0.0f;
    if (r < count) {
#pragma unroll 4
        for (int p = y; p < parts; p += lanes) {
            const float2 v = part[p * part_pitch + r];
            merge(m, s, v.x, v.y);
        }
    }
    pair[threadIdx.x] = make_float2(m, s);
    __syncthreads();
    for (int h = lanes / 2; h > 0; h >>= 1) {
        if (y < h) {
            const float2 o = pair[threadIdx.x + h * rows];
            merge(m, s, o.x, o.y);
            pair[threadIdx.x] = make_float2(m, s);
        }
        __syncthreads();
    }
    if (y == 0 && r < t.M) {
        const int token = t.index[r];
        const float l = r < count ? m * kLn2 + logf(s) : 0.0f;
        lse[token] = l;
        loss[token] = r < count ? l - z_target[r] : 0.0f;
    }
}

// dx rows from the sums of the ranges of the vocabulary, in range order.
template <bool BF16>
__global__ void __launch_bounds__(256) ce_dx_kernel(const __grid_constant__ CeTokens t,
                                                    const float *__restrict__ sums, int64_t sums_rows, int splits)
{
    pdl_wait();
    const int count = t.info->count;
    const float down = t.info->down;
    const int64_t total = static_cast<int64_t>(count) * t.K;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / t.K;
        float v = 0.0f;
        for (int k = 0; k < splits; ++k) v += sums[k * sums_rows * t.K + i];
        v *= down;
        uint16_t *d = static_cast<uint16_t *>(t.dx) + t.index[r] * t.K + (i - r * t.K);
        if constexpr (BF16) *d = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        else *d = __half_as_ushort(__float2half_rn(v));
    }
}

// A launch as a programmatic dependent of the kernel before it: it may start
// while that one ends, and waits for it before it reads (pdl_wait).  A call's
// first kernel is not launched so.
template <typename... P, typename... A>
int launch_after(const char *what, void (*kern)(P...), unsigned grid, unsigned threads, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e == cudaSuccess ? 0 : record_cuda_error(what, e, cudaGetErrorString(e));
}

unsigned blocks(int64_t n, int64_t most) { return static_cast<unsigned>(n < 1 ? 1 : n < most ? n : most); }

}  // namespace

int launch_ce_index(const CeTokens &t, cudaStream_t stream)
{
    ce_index_kernel<<<1, kIndexThreads, 0, stream>>>(t);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : record_cuda_error("cross entropy token index launch", e, cudaGetErrorString(e));
}

int launch_ce_gather(const CeTokens &t, cudaStream_t stream)
{
    const bool vec = t.K % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.dx)) & 15u) == 0;
    const int64_t rows = (t.M + 63) / 64 * 64;
    const unsigned grid = blocks(rows, 152 * 16);
    return launch_after("cross entropy gather launch", vec ? ce_gather_kernel<true> : ce_gather_kernel<false>, grid,
                        kGatherThreads, stream, t);
}

int launch_ce_loss(const CeTokens &t, const float2 *part, int64_t part_pitch, int parts,
                   const float *z_target, float *loss, float *lse, cudaStream_t stream)
{
    // A CTA per row while the rows are few, else 32 rows side by side so
    // that a warp reads whole lines of the pairs.
    const int rows = t.M < 512 ? 1 : 32;
    return launch_after("cross entropy loss launch", ce_loss_kernel, static_cast<unsigned>((t.M + rows - 1) / rows),
                        kLossThreads, stream, t, part, part_pitch, parts, z_target, loss, lse, rows);
}

int launch_ce_dx(bool bf16, const CeTokens &t, const float *sums, int64_t sums_rows, int splits,
                 cudaStream_t stream)
{
    const unsigned grid = blocks((t.M * t.K + 255) / 256, 152 * 8);
    return launch_after("cross entropy dx sums launch", bf16 ? ce_dx_kernel<true> : ce_dx_kernel<false>, grid, 256u,
                        stream, t, sums, sums_rows, splits);
}

}  // namespace ngr
