// ngr_ce.cu -- the linear cross entropy around its products: which tokens
// count, their rows gathered, the last step of the loss, the last sums of dx.
//
// Tokens whose target is negative take no part: the counted tokens' rows are
// copied together, so that the products run over those alone, nothing a
// masked row holds (infinities, NaN) reaches a sum, and the rows start on
// 128-byte lines whatever K is.  The copy moves 4 K bytes a token against the
// 2 K V operations of one product.
#include "ngr_ce.h"
#include "ngr_entry.h"
#include "ngr_internal.h"
#include "ngr_ptx.cuh"
#include "ngr_shift.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace ngr {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kDzUnit = 8192.0f;   // dz's largest weight
constexpr int kIndexThreads = 1024, kIndexEach = 8;
constexpr int kGatherThreads = 128;
constexpr int kFewTokens = kGatherThreads * kIndexEach;   // index and gather in one kernel up to this

// W's rows of K elements (K % 8 != 0) as rows on 128-byte lines, zeros up to
// the next multiple of 8: one 16-byte piece a thread, from the aligned words
// it lies in.
__global__ void __launch_bounds__(256) ce_pad_kernel(const uint16_t *__restrict__ src, uint4 *__restrict__ dst,
                                                     int64_t rows, int K, int pitch_vecs)
{
    const int vecs = (K + 7) / 8;
    const int64_t total = rows * vecs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / vecs;
        const int v = static_cast<int>(i - r * vecs), left = K - 8 * v;
        uint4 d = load_shifted(src + r * K + 8 * v, 0, left < 8 ? left : 8);
        if (left < 8) {   // what follows belongs to the next row
            uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] &= (2 * j < left ? 0xFFFFu : 0u) | (2 * j + 1 < left ? 0xFFFF0000u : 0u);
            d = make_uint4(w[0], w[1], w[2], w[3]);
        }
        dst[r * pitch_vecs + v] = d;
    }
}

// A prefix sum over the tokens [r0, r0 + THREADS x kIndexEach) gives each
// counted token its place (their order kept) and the others theirs from the
// end: put(place, token, target or -1).  `base` counts the tokens of the
// rounds before and is carried on; `top` takes the largest finite weight of
// this thread's tokens; *bad is set by a target outside the vocabulary.
template <int THREADS, typename Put>
__device__ __forceinline__ void place_tokens(const CeTokens &t, int64_t r0, int64_t &base, float &top, int *bad,
                                             int *warp_sum, Put put)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t i0 = r0 + static_cast<int64_t>(threadIdx.x) * kIndexEach;
    int64_t target[kIndexEach];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kIndexEach; ++j) {
        target[j] = i0 + j < t.M ? t.target[i0 + j] : -1;
        if (target[j] >= t.V) {
            *bad = 1;
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
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    int64_t at = base + before + incl - mine;
#pragma unroll
    for (int j = 0; j < kIndexEach; ++j) {
        const int64_t i = i0 + j;
        if (i >= t.M) continue;
        if (target[j] >= 0) {
            put(at, static_cast<int>(i), static_cast<int>(target[j]));
            ++at;
            if (t.lse) {
                const float g = t.dloss ? t.dloss[i] : 0.0f, l = t.dlse ? t.dlse[i] : 0.0f;
                const float w = fmaxf(fabsf(g), fabsf(g + l));
                // (an infinite weight is no unit for the others')
                if (w < INFINITY) top = fmaxf(top, w);
            }
        } else {
            put(t.M - 1 - (i - at), static_cast<int>(i), -1);
        }
    }
    base += total;
    __syncthreads();
}

// The largest weight over the CTA's threads (all get it) as the unit of dz.
template <int THREADS>
__device__ __forceinline__ CeInfo tokens_info(const CeTokens &t, int64_t count, float top, float *warp_max)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, warp_max[w]);
    top *= fabsf(t.logit_scale);
    // (no weight, or one at the ends of FP32's range: unscaled)
    if (!(top >= 1.0e-30f && top <= 1.0e38f)) top = kDzUnit;
    CeInfo info;
    info.count = static_cast<int>(count);
    info.weight = top;
    info.down = top / kDzUnit;
    return info;
}

__global__ void __launch_bounds__(kIndexThreads) ce_index_kernel(const __grid_constant__ CeTokens t)
{
    __shared__ int warp_sum[kIndexThreads / 32];
    __shared__ float warp_max[kIndexThreads / 32];
    __shared__ int bad;
    pdl_launch_dependents();
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    int64_t base = 0;
    float top = 0.0f;
    for (int64_t r0 = 0; r0 < t.M; r0 += kIndexThreads * kIndexEach)
        place_tokens<kIndexThreads>(t, r0, base, top, &bad, warp_sum, [&](int64_t at, int token, int target) {
            t.index[at] = token;
            if (target >= 0) t.ctarget[at] = target;
        });
    const CeInfo info = tokens_info<kIndexThreads>(t, base, top, warp_max);
    if (threadIdx.x == 0) {
        *t.info = info;
        *t.err = bad ? kDevErrTarget : 0;
    }
}

// Row r of the gathered matrix: a counted token's row (padded with zeros to
// Kx), a zero row up to the next 64 (the contracted length of dW), and in the
// backward call the row's softmax constants and zeros for the dx row of a
// token that does not count.
template <bool VEC>
__device__ __forceinline__ void gather_row(const CeTokens &t, const CeInfo &info, int64_t r, int64_t token, int target)
{
    const int count = info.count;
    const int vecs = static_cast<int>(t.Kx / 8), whole = static_cast<int>(t.K / 8);
    if (r < (static_cast<int64_t>(max(count, 1)) + 63) / 64 * 64) {
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
        const float g = t.dloss ? t.dloss[token] : 0.0f, l = t.dlse ? t.dlse[token] : 0.0f;
        t.row[r] = CeRow{t.lse[token] * kLog2e, (g + l) * t.logit_scale / info.weight * kDzUnit,
                         g * t.logit_scale / info.weight * kDzUnit, target};
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

template <bool VEC>
__global__ void __launch_bounds__(kGatherThreads) ce_gather_kernel(const __grid_constant__ CeTokens t)
{
    pdl_launch_dependents();
    pdl_wait();
    const CeInfo info = *t.info;
    const int64_t rows = (t.M + 63) / 64 * 64;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        gather_row<VEC>(t, info, r, r < t.M ? t.index[r] : 0, r < info.count ? t.ctarget[r] : -1);
}

// Index and gather in one kernel for few tokens: every CTA places them all
// for itself in shared memory, which costs less than a launch.
template <bool VEC>
__global__ void __launch_bounds__(kGatherThreads) ce_index_gather_kernel(const __grid_constant__ CeTokens t)
{
    __shared__ int index[kFewTokens], ctarget[kFewTokens];
    __shared__ int warp_sum[kGatherThreads / 32];
    __shared__ float warp_max[kGatherThreads / 32];
    __shared__ int bad;
    pdl_launch_dependents();
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    int64_t base = 0;
    float top = 0.0f;
    place_tokens<kGatherThreads>(t, 0, base, top, &bad, warp_sum, [&](int64_t at, int token, int target) {
        index[at] = token;
        ctarget[at] = target;
    });
    const CeInfo info = tokens_info<kGatherThreads>(t, base, top, warp_max);
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < t.M; i += kGatherThreads) {
            t.index[i] = index[i];
            t.ctarget[i] = ctarget[i];
        }
        if (threadIdx.x == 0) {
            *t.info = info;
            *t.err = bad ? kDevErrTarget : 0;
        }
    }
    const int64_t rows = (t.M + 63) / 64 * 64;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        gather_row<VEC>(t, info, r, r < t.M ? index[r] : 0, r < t.M ? ctarget[r] : -1);
}

// (max, sum) pairs in powers of two, merged in a fixed order.
__device__ __forceinline__ void merge(float &m, float &s, float om, float os)
{
    const float top = fmaxf(m, om);
    const float base = fabsf(top) == INFINITY ? 0.0f : top;   // (inf - inf is no number)
    s = s * exp2f(m - base) + os * exp2f(om - base);
    m = top;
}

// A row's pairs over the column tiles -> its lse and loss.  ROWS 32: 32 rows
// side by side, so that a warp reads whole lines of the pairs, and 32 threads
// along the pairs of each; ROWS 1, while the rows are few: a CTA per row.
template <int ROWS>
__global__ void __launch_bounds__(ROWS == 1 ? 256 : 1024) ce_loss_kernel(
    const __grid_constant__ CeTokens t, const float2 *__restrict__ part, int64_t part_pitch, int parts,
    const float *__restrict__ z_target, float *loss, float *lse)
{
    constexpr int kLanes = ROWS == 1 ? 256 : 32;   // threads along a row's pairs
    __shared__ float2 pair[ROWS == 1 ? 8 : 32][33];
    const int x = threadIdx.x % ROWS, y = threadIdx.x / ROWS;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * ROWS + x;
    pdl_wait();
    const int count = t.info->count;
    float m = -INFINITY, s = 0.0f;
    if (r < count) {
#pragma unroll 4
        for (int p = y; p < parts; p += kLanes) {
            const float2 v = part[p * part_pitch + r];
            merge(m, s, v.x, v.y);
        }
    }
    // ROWS 32: turn the tile round, so that a warp holds one row's 32 lanes.
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if constexpr (ROWS == 32) {
        pair[y][x] = make_float2(m, s);
        __syncthreads();
        const float2 v = pair[lane][warp];
        m = v.x;
        s = v.y;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o);
        merge(m, s, om, os);
    }
    if constexpr (ROWS == 1) {
        if (lane == 0) pair[warp][0] = make_float2(m, s);
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int w = 1; w < 8; ++w) merge(m, s, pair[w][0].x, pair[w][0].y);
        }
    }
    const int64_t row = ROWS == 1 ? r : static_cast<int64_t>(blockIdx.x) * ROWS + warp;
    if (lane == 0 && (ROWS == 32 || warp == 0) && row < t.M) {
        const int token = t.index[row];
        const float l = row < count ? m * kLn2 + logf(s) : 0.0f;
        lse[token] = l;
        loss[token] = row < count ? l - z_target[row] : 0.0f;
    }
}

// dx rows from the sums of the ranges of the vocabulary, in range order.
template <bool BF16>
__global__ void __launch_bounds__(256) ce_dx_kernel(const __grid_constant__ CeTokens t,
                                                    const float *__restrict__ sums, int64_t sums_pitch, int splits)
{
    pdl_wait();
    const int count = t.info->count;
    const float down = t.info->down;
    const int64_t total = static_cast<int64_t>(count) * t.K;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = i / t.K;
        float v = 0.0f;
        const int64_t c = i - r * t.K;
        for (int k = 0; k < splits; ++k) v += sums[(k * t.M + r) * sums_pitch + c];
        v *= down;
        uint16_t *d = static_cast<uint16_t *>(t.dx) + t.index[r] * t.K + c;
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

int launch_ce_pad(const void *W, void *dst, int64_t rows, int64_t K, int64_t pitch, cudaStream_t stream)
{
    ce_pad_kernel<<<blocks((rows * ((K + 7) / 8) + 255) / 256, 152 * 8), 256, 0, stream>>>(
        static_cast<const uint16_t *>(W), static_cast<uint4 *>(dst), rows, static_cast<int>(K),
        static_cast<int>(pitch / 8));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : record_cuda_error("cross entropy weight copy launch", e, cudaGetErrorString(e));
}

bool launch_ce_index_apart(const CeTokens &t) { return t.M > kFewTokens; }

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
    const unsigned grid = blocks((t.M + 63) / 64 * 64, 152 * 16);
    if (!launch_ce_index_apart(t)) {
        if (vec) ce_index_gather_kernel<true><<<grid, kGatherThreads, 0, stream>>>(t);
        else ce_index_gather_kernel<false><<<grid, kGatherThreads, 0, stream>>>(t);
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? 0 : record_cuda_error("cross entropy gather launch", e, cudaGetErrorString(e));
    }
    return launch_after("cross entropy gather launch", vec ? ce_gather_kernel<true> : ce_gather_kernel<false>, grid,
                        kGatherThreads, stream, t);
}

int launch_ce_loss(const CeTokens &t, const float2 *part, int64_t part_pitch, int parts,
                   const float *z_target, float *loss, float *lse, cudaStream_t stream)
{
    if (t.M < 1024)
        return launch_after("cross entropy loss launch", ce_loss_kernel<1>, static_cast<unsigned>(t.M), 256u, stream,
                            t, part, part_pitch, parts, z_target, loss, lse);
    return launch_after("cross entropy loss launch", ce_loss_kernel<32>, static_cast<unsigned>((t.M + 31) / 32), 1024u,
                        stream, t, part, part_pitch, parts, z_target, loss, lse);
}

int launch_ce_dx(bool bf16, const CeTokens &t, const float *sums, int64_t sums_pitch, int splits,
                 cudaStream_t stream)
{
    const unsigned grid = blocks((t.M * t.K + 255) / 256, 152 * 8);
    return launch_after("cross entropy dx sums launch", bf16 ? ce_dx_kernel<true> : ce_dx_kernel<false>, grid, 256u,
                        stream, t, sums, sums_pitch, splits);
}

}  // namespace ngr
