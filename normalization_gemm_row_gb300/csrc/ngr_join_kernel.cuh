// ngr_join_kernel.cuh -- the join of a transformer block to its residual
// stream, in one pass over the rows, and its gradient: what the forward and
// the backward kernel share.
//
//   u1 = core1(x)            n = gamma1 u1 + beta1      (norm after the block)
//   h  = a residual + s gate n                          (gate, residual scale)
//   u2 = core2(h)            y = gamma2 u2 + beta2      (norm before the next)
//
// core: LayerNorm (v - mean) / sqrt(var + eps), RMSNorm v / sqrt(ms + eps),
// or none (n = x; no y).  All arithmetic is FP32; h and y are rounded once,
// and y is the norm of the unrounded h.
//
// Gradient, with D the whole gradient of h and pull(d) = rstd (d - u mean(d u)
// [- mean(d) for LayerNorm]) the pullback of a core:
//   D = dh + pull2(gamma2 dy)       dresidual = a D
//   dgate = s sum_group n D         dn = s gate D
//   dgamma1 = sum u1 dn, dbeta1 = sum dn, dx = pull1(gamma1 dn)
//   dgamma2 = sum u2 dy, dbeta2 = sum dy
//
// Both kernels are bound by HBM: the forward reads x and residual and writes
// h and y (8 bytes an element), the backward reads x, residual, dy and dh
// and writes dx and dresidual (12 bytes an element); everything else is a
// vector of the row's width or four floats a row.  What comes next is the
// issue of instructions, most of them integer: so the number of threads on a
// row and of vectors a thread are compile-time constants, which makes every
// offset from a row's start an immediate (with both at run time the forward
// issued 34 instructions an element, 16 of them integer and 7 of arithmetic).
#pragma once

#include "ngr_internal.h"
#include "ngr_join.h"
#include "ngr_ptx.cuh"
#include "ngr_shift.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace ngr {

// ------------------------------------------------------------ 16-bit vectors
// 8 elements as four FP32 pairs: the arithmetic runs on pairs (one
// instruction for two elements), which halves the instructions that come
// near the time of the loads in the backward kernel.
struct Vec8 {
    float2 p[4];
};

template <bool BF16>
__device__ __forceinline__ Vec8 unpack8(const uint4 &q)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    Vec8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16)
            f.p[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        else
            f.p[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    }
    return f;
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const Vec8 &f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f.p[i].x, f.p[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        } else {
            const __half2 v = __floats2half2_rn(f.p[i].x, f.p[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16>
__device__ __forceinline__ uint16_t round16(float v)
{
    if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else return __half_as_ushort(__float2half_rn(v));
}

template <bool BF16>
__device__ __forceinline__ float widen16(uint16_t v)
{
    if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else return __half2float(__ushort_as_half(v));
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ Vec8 filled(float v)
{
    Vec8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = both(v);
    return f;
}
__device__ __forceinline__ Vec8 operator*(const Vec8 &a, const Vec8 &b)
{
    Vec8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = __fmul2_rn(a.p[i], b.p[i]);
    return f;
}
__device__ __forceinline__ Vec8 operator*(const Vec8 &a, float b)
{
    Vec8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = __fmul2_rn(a.p[i], both(b));
    return f;
}
__device__ __forceinline__ Vec8 operator+(const Vec8 &a, const Vec8 &b)
{
    Vec8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = __fadd2_rn(a.p[i], b.p[i]);
    return f;
}
__device__ __forceinline__ Vec8 operator+(const Vec8 &a, float b)
{
    Vec8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = __fadd2_rn(a.p[i], both(b));
    return f;
}
// a b + c
__device__ __forceinline__ Vec8 fma8(const Vec8 &a, float b, const Vec8 &c)
{
    Vec8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = __ffma2_rn(a.p[i], both(b), c.p[i]);
    return f;
}
// s += a (as pairs), s += a b
__device__ __forceinline__ void sum8(float2 &s, const Vec8 &a)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __fadd2_rn(s, a.p[i]);
}
__device__ __forceinline__ void dot8(float2 &s, const Vec8 &a, const Vec8 &b)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __ffma2_rn(a.p[i], b.p[i], s);
}

// A thread's place in its row: which columns its vector v holds, and how
// they are read and written (kJoin* modes).  Vector v of thread t is the
// (v TPR + t)-th of the CTA's columns [c0, c1); in the window mode the
// vectors are shifted back by `s` elements, the row's distance from the
// 16-byte boundary before it; those that reach over an end are read whole
// (the aligned 16 bytes hold an element of the row, so they are the
// caller's), what is not the row's is put to zero, and they are written by
// elements.  In the scalar mode element j of vector v is column
// c0 + (v 8 + j) TPR + t, so that neighbouring threads touch neighbouring
// elements.  Where a CTA has whole rows, vectors from 1 on do not reach over
// a row's start, nor the first FULL vectors over its end (see full_vectors),
// and the tests for that fall away (8192 x 14337, LN/LN: 374 -> 273 us, the
// gradient at 32768 x 2048 174 -> 142 us).  FULL -1: nothing is known.
template <int MODE, int TPR, int FULL>
struct Place {
    int c0, c1, first;   // first: the column of element 0 of vector 0 (unshifted)
    __device__ __forceinline__ Place(int c0_, int c1_, int t)
        : c0(c0_), c1(c1_), first(MODE == kJoinScalar ? c0_ + t : c0_ + t * 8) {}
    __device__ __forceinline__ int col(int v, int j, int s) const
    {
        if constexpr (MODE == kJoinScalar) return first + (v * 8 + j) * TPR;
        if constexpr (MODE == kJoinAligned) return first + v * TPR * 8 + j;
        return first + v * TPR * 8 + j - s;
    }
    __device__ __forceinline__ bool valid(int v, int j, int s) const
    {
        if constexpr (MODE == kJoinAligned) return whole(v, s);
        if (inner(v)) return true;
        const int c = col(v, j, s);
        return (c >= c0 || (FULL >= 0 && v > 0)) && (c < c1 || v < FULL);
    }
    // any of them
    __device__ __forceinline__ bool some(int v, int s) const
    {
        const int c = col(v, 0, s);
        return (c < c1 || v < FULL) && (MODE == kJoinAligned || c + 8 > c0 || (FULL >= 0 && v > 0));
    }
    // all 8 columns of the vector (one 16-byte access)
    __device__ __forceinline__ bool whole(int v, int s) const
    {
        if constexpr (MODE == kJoinScalar) return false;
        if (inner(v)) return true;
        const int c = col(v, 0, s);
        if constexpr (MODE == kJoinAligned) return c < c1;
        return (c >= c0 || (FULL >= 0 && v > 0)) && (c + 8 <= c1 || v < FULL);
    }
    // known to be whole
    __device__ __forceinline__ static constexpr bool inner(int v) { return v < FULL && (MODE == kJoinAligned || v > 0); }
};

// The vector's elements one by one (zero where the thread has no column).
template <typename P>
__device__ __forceinline__ uint4 load_elements(const uint16_t *row, const P &p, int v, int s)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = p.valid(v, 2 * i, s) ? row[p.col(v, 2 * i, s)] : 0u;
        const uint32_t hi = p.valid(v, 2 * i + 1, s) ? row[p.col(v, 2 * i + 1, s)] : 0u;
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A vector's elements with zeros where the thread has no column.
template <int MODE, int TPR, int FULL>
__device__ __forceinline__ uint4 own_elements(const uint4 &d, const Place<MODE, TPR, FULL> &p, int v, int s)
{
    if (MODE != kJoinWindow || p.whole(v, s)) return d;
    uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] &= (p.valid(v, 2 * i, s) ? 0xFFFFu : 0u) | (p.valid(v, 2 * i + 1, s) ? 0xFFFF0000u : 0u);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// `row` is the address of the row's column 0.
template <int MODE, int TPR, int FULL>
__device__ __forceinline__ uint4 load8(const uint16_t *row, const Place<MODE, TPR, FULL> &p, int v, int s)
{
    if constexpr (MODE == kJoinScalar) return load_elements(row, p, v, s);
    if (!p.some(v, s)) return make_uint4(0u, 0u, 0u, 0u);
    return own_elements(*reinterpret_cast<const uint4 *>(row + p.col(v, 0, s)), p, v, s);
}

template <int MODE, int TPR, int FULL>
__device__ __forceinline__ void store8(uint16_t *row, const Place<MODE, TPR, FULL> &p, int v, int s, const uint4 &d)
{
    if (p.whole(v, s)) {
        *reinterpret_cast<uint4 *>(row + p.col(v, 0, s)) = d;
        return;
    }
    if constexpr (MODE != kJoinAligned) {
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (p.valid(v, j, s))
                row[p.col(v, j, s)] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
}

// The same columns of a vector of the row's width (gamma, beta, a gate row):
// read-only for the whole call, zero where the thread has no column.
template <bool BF16, int MODE, int TPR, int FULL>
__device__ __forceinline__ Vec8 param8(const uint16_t *b, const Place<MODE, TPR, FULL> &p, int v, int s)
{
    if constexpr (MODE == kJoinAligned) {
        return unpack8<BF16>(p.whole(v, s) ? __ldg(reinterpret_cast<const uint4 *>(b + p.col(v, 0, s)))
                                           : make_uint4(0u, 0u, 0u, 0u));
    } else {
        if constexpr (MODE == kJoinWindow) {
            if (!p.some(v, s)) return filled(0.0f);
            const int c = p.col(v, 0, s);
            return unpack8<BF16>(own_elements(load_shifted(b + c, p.inner(v) ? 0 : max(p.c0 - c, 0), p.inner(v) ? 8 : min(p.c1 - c, 8)), p, v, s));
        }
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = p.valid(v, j, s) ? widen16<BF16>(__ldg(b + p.col(v, j, s))) : 0.0f;
        Vec8 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.p[i] = make_float2(f[2 * i], f[2 * i + 1]);
        return r;
    }
}

// v with zeros where the thread has no column.
template <int MODE, int TPR, int FULL>
__device__ __forceinline__ Vec8 masked(const Vec8 &a, const Place<MODE, TPR, FULL> &p, int v, int s)
{
    if (MODE != kJoinScalar && p.whole(v, s)) return a;
    Vec8 f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f.p[i] = make_float2(p.valid(v, 2 * i, s) ? a.p[i].x : 0.0f, p.valid(v, 2 * i + 1, s) ? a.p[i].y : 0.0f);
    return f;
}

__device__ __forceinline__ const uint16_t *elements(const void *p, int64_t off = 0)
{
    return static_cast<const uint16_t *>(p) + off;
}
__device__ __forceinline__ uint16_t *elements(void *p, int64_t off = 0) { return static_cast<uint16_t *>(p) + off; }

template <int MODE>
__device__ __forceinline__ int row_shift(const JoinArgs &a, int64_t row)
{
    return MODE == kJoinWindow ? static_cast<int>((a.shift + row * a.N) & 7) : 0;
}

// ------------------------------------------------------------------ row sums
struct RowSumSmem {
    float4 warp[2][kJoinThreads / 32][2];
    float peer[2][kJoinMaxCluster][8];
};

// Adds K values (1, 4 or 8) over the TPR threads of a row, in an order that
// depends on the shape alone; every thread of the row gets the sums.  Lanes
// halve the values they carry while they exchange them, so K values cost
// about K + 5 - log2 K shuffles and not 5 K; then the row's warps and the
// cluster's CTAs add up through shared memory.  The two halves of the
// buffers take turns, so one barrier a call is enough.  All threads of the
// CTA (of the cluster) call it together.  `barrier` stands between the warps'
// writes and reads.
template <int K, int TPR, typename Barrier>
__device__ __forceinline__ void row_sum(float (&v)[K], RowSumSmem &s, int &half, int cluster, uint32_t rank,
                                        Barrier barrier)
{
    static_assert(K == 1 || K == 4 || K == 8, "values");
    constexpr int kWarps = TPR / 32;
    const int lane = threadIdx.x & 31;
    constexpr int kLast = K == 1 ? 16 : K == 4 ? 4 : 2;   // distance of the first plain exchange
#pragma unroll
    for (int n = K / 2, o = 16; n >= 1; n >>= 1, o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
#pragma unroll
    for (int o = kLast; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    // lanes [k 32 / K, +32 / K) now hold value k of the warp
    if (kWarps == 1 && cluster == 1) {
        const float mine = v[0];
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, mine, k * (32 / K));
        // (shared memory that other lanes wrote before is seen after, as with
        // the barrier of wider rows)
        __syncwarp();
        return;
    }
    half ^= 1;
    const int warp = threadIdx.x >> 5;
    if (lane % (32 / K) == 0) reinterpret_cast<float *>(s.warp[half][warp])[lane / (32 / K)] = v[0];
    barrier();
    const int first = warp / kWarps * kWarps;   // the row's warps
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if constexpr (K == 1) {
            v[0] += s.warp[half][first + w][0].x;
        } else {
#pragma unroll
            for (int k = 0; k < K; k += 4) {
                const float4 q = s.warp[half][first + w][k / 4];
                v[k] += q.x;
                v[k + 1] += q.y;
                v[k + 2] += q.z;
                v[k + 3] += q.w;
            }
        }
    }
    if (cluster > 1) {
        if (threadIdx.x < cluster) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const uint32_t dst = mapa_shared(smem_u32(&s.peer[half][rank][k]), threadIdx.x);
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(v[k]) : "memory");
            }
        }
        cluster_sync_all();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = 0.0f;
        for (int r = 0; r < cluster; ++r)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += s.peer[half][r][k];
    }
}

template <int K, int TPR>
__device__ __forceinline__ void row_sum(float (&v)[K], RowSumSmem &s, int &half, int cluster, uint32_t rank)
{
    row_sum<K, TPR>(v, s, half, cluster, rank, [] { __syncthreads(); });
}

// ----------------------------------------------------------------- launching
// Threads on a row and vectors a thread; a kernel's widths are listed by the
// vectors they hold, and a row takes the first that holds its own.
struct Width {
    int tpr, vecs;
};
// How many vectors of every thread surely end inside the row: it has more
// vectors than the width before holds, the last of them in part (in the
// window mode they are counted as for the worst shift, one too many).
template <int N>
constexpr int full_vectors(const Width (&widths)[N], int tpr, int vecs, int mode)
{
    if (mode == kJoinScalar) return -1;
    for (int i = 0, before = 0; i < N; before = widths[i].tpr * widths[i].vecs, ++i)
        if (widths[i].tpr == tpr && widths[i].vecs == vecs)
            return (mode == kJoinWindow && before > 0 ? before - 1 : before) / tpr;
    return -1;
}
// Vectors that cover the CTA's columns (one more where rows are shifted).
inline int64_t join_vectors(const JoinShape &s, int mode) { return s.cols / 8 + (mode == kJoinWindow ? 1 : 0); }
inline int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

template <typename K>
int launch_join(K kern, int64_t ctas, const JoinShape &sh, size_t smem, const JoinArgs &a, cudaStream_t stream,
                const char *what)
{
    if (smem > 40 * 1024) {   // (static shared memory counts towards the 48 KB that need no asking)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess)
            return record_cuda_error("cudaFuncSetAttribute(max dynamic smem)", e, cudaGetErrorString(e));
    }
    if (sh.cluster > kJoinPortableCluster) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess)
            return record_cuda_error("cudaFuncSetAttribute(cluster size)", e, cudaGetErrorString(e));
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas * sh.cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(sh.tpr * sh.slots));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(sh.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = sh.cluster > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    return e == cudaSuccess ? 0 : record_cuda_error(what, e, cudaGetErrorString(e));
}

}  // namespace ngr
