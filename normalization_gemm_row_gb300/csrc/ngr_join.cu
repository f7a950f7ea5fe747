// ngr_join.cu -- the join of a transformer block to its residual stream, in
// one pass over the rows, and its gradient:
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
// vector of the row's width or four floats a row.
#include "ngr_internal.h"
#include "ngr_join.h"
#include "ngr_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace ngr {

namespace {

// ------------------------------------------------------------ 16-bit vectors
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &p, float (&f)[8])
{
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        } else {
            const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's place in its row.  VEC: vector v covers columns
// [c0 + (v tpr + t) 8, +8) with 16-byte accesses (every row starts on a
// 16-byte boundary and has whole vectors).  Otherwise element j of vector v
// is column c0 + (v 8 + j) tpr + t, each a 2-byte access, so that any width
// and any 2-byte aligned address works and neighbouring threads still touch
// neighbouring elements.
template <bool VEC>
struct Place {
    int c0, c1, tpr, t;   // the CTA's columns [c0, c1)
    __device__ __forceinline__ int col(int v, int j) const
    {
        return VEC ? c0 + (v * tpr + t) * 8 + j : c0 + (v * 8 + j) * tpr + t;
    }
    __device__ __forceinline__ bool valid(int v, int j) const
    {
        return col(v, VEC ? 0 : j) < c1;
    }
};

template <bool VEC>
__device__ __forceinline__ uint4 load8(const void *base, int64_t row_off, const Place<VEC> &p, int v,
                                       bool active)
{
    const uint16_t *b = static_cast<const uint16_t *>(base) + row_off;
    if constexpr (VEC) {
        if (active && p.valid(v, 0)) return *reinterpret_cast<const uint4 *>(b + p.col(v, 0));
        return make_uint4(0u, 0u, 0u, 0u);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = active && p.valid(v, 2 * i) ? b[p.col(v, 2 * i)] : 0u;
            const uint32_t hi = active && p.valid(v, 2 * i + 1) ? b[p.col(v, 2 * i + 1)] : 0u;
            w[i] = lo | (hi << 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(void *base, int64_t row_off, const Place<VEC> &p, int v,
                                       bool active, const uint4 &d)
{
    uint16_t *b = static_cast<uint16_t *>(base) + row_off;
    if constexpr (VEC) {
        if (active && p.valid(v, 0)) *reinterpret_cast<uint4 *>(b + p.col(v, 0)) = d;
    } else {
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (active && p.valid(v, j))
                b[p.col(v, j)] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
}

// ------------------------------------------------------------------ row sums
constexpr int kMaxSums = 8;

struct RowSumSmem {
    float warp[2][kJoinThreads / 32][kMaxSums];
    float peer[2][kJoinMaxCluster][kMaxSums];
};

// Adds K values over the threads of a row (shuffles, then shared memory,
// then the shared memory of the cluster's CTAs), in an order that depends on
// the shape alone; every thread of the row gets the sums.  The two halves of
// the buffers take turns, so one barrier a call is enough.  All threads of
// the CTA (of the cluster) call it together.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], RowSumSmem &s, int &half, const JoinShape &sh,
                                        int slot, uint32_t rank)
{
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    const int warps = sh.tpr >> 5;
    if (warps == 1 && sh.cluster == 1) return;
    half ^= 1;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) s.warp[half][warp][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.0f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += s.warp[half][slot * warps + w][k];
    if (sh.cluster > 1) {
        if (threadIdx.x < sh.cluster) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const uint32_t dst = mapa_shared(smem_u32(&s.peer[half][rank][k]), threadIdx.x);
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(v[k]) : "memory");
            }
        }
        cluster_sync_all();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = 0.0f;
        for (int r = 0; r < sh.cluster; ++r)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += s.peer[half][r][k];
    }
}

__device__ __forceinline__ int64_t gate_row(const JoinArgs &a, int64_t row)
{
    return a.rows_per_gate >= a.M ? 0 : row / a.rows_per_gate;
}

// ------------------------------------------------------------------- forward
// One group of threads per row, the row held in registers (vecs x 8 elements
// a thread).  The statistics are two-pass (mean, then centred squares), so a
// row far from zero mean or with a few very large channels loses nothing.
template <bool BF16, bool VEC, int VECS>
__global__ void __launch_bounds__(kJoinThreads) join_forward_kernel(const __grid_constant__ JoinArgs a)
{
    __shared__ RowSumSmem sums;
    int half = 0;
    const JoinShape &sh = a.shape;
    const uint32_t rank = sh.cluster > 1 ? cluster_ctarank() : 0u;
    const int slot = threadIdx.x / sh.tpr;
    Place<VEC> p;
    p.tpr = sh.tpr;
    p.t = threadIdx.x - slot * sh.tpr;
    p.c0 = static_cast<int>(rank) * sh.cols;
    p.c1 = min(a.N, p.c0 + sh.cols);
    // Every CTA of the cluster runs before its shared memory is written.
    if (sh.cluster > 1) cluster_sync_all();
    const int64_t row = static_cast<int64_t>(blockIdx.x / sh.cluster) * sh.slots + slot;
    const bool active = row < a.M;
    const int64_t off = row * a.N;
    const float inv_n = 1.0f / static_cast<float>(a.N);

    uint4 xp[VECS], rp[VECS];
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
        xp[v] = load8<VEC>(a.x, off, p, v, active);
        rp[v] = a.residual ? load8<VEC>(a.residual, off, p, v, active) : make_uint4(0u, 0u, 0u, 0u);
    }

    float mu1 = 0.0f, rs1 = 1.0f;
    if (a.norm1 == kNormLayer) {
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            float x[8];
            unpack8<BF16>(xp[v], x);   // invalid elements are zero
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += x[j];
        }
        row_sum(s, sums, half, sh, slot, rank);
        mu1 = s[0] * inv_n;
    }
    if (a.norm1 != kNormNone) {
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            float x[8];
            unpack8<BF16>(xp[v], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = p.valid(v, j) ? x[j] - mu1 : 0.0f;
                s[0] += d * d;
            }
        }
        row_sum(s, sums, half, sh, slot, rank);
        rs1 = rsqrtf(s[0] * inv_n + a.eps1);
    }

    float h[VECS][8];
    const int64_t goff = a.gate && active ? gate_row(a, row) * a.N : 0;
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
        float x[8], t[8];
        unpack8<BF16>(xp[v], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (x[j] - mu1) * rs1;
        if (a.norm1 != kNormNone) {
            unpack8<BF16>(load8<VEC>(a.gamma1, 0, p, v, true), t);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= t[j];
            if (a.norm1 == kNormLayer) {
                unpack8<BF16>(load8<VEC>(a.beta1, 0, p, v, true), t);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] += t[j];
            }
        }
        if (a.gate) {
            unpack8<BF16>(load8<VEC>(a.gate, goff, p, v, active), t);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= t[j];
        }
        unpack8<BF16>(rp[v], t);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[v][j] = a.residual_scale * t[j] + a.block_scale * x[j];
        store8<VEC>(a.h, off, p, v, active, pack8<BF16>(h[v]));
    }

    float mu2 = 0.0f, rs2 = 1.0f;
    if (a.norm2 == kNormLayer) {
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < VECS; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += p.valid(v, j) ? h[v][j] : 0.0f;
        row_sum(s, sums, half, sh, slot, rank);
        mu2 = s[0] * inv_n;
    }
    if (a.norm2 != kNormNone) {
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < VECS; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = p.valid(v, j) ? h[v][j] - mu2 : 0.0f;
                s[0] += d * d;
            }
        row_sum(s, sums, half, sh, slot, rank);
        rs2 = rsqrtf(s[0] * inv_n + a.eps2);
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            float t[8], y[8];
            unpack8<BF16>(load8<VEC>(a.gamma2, 0, p, v, true), t);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (h[v][j] - mu2) * rs2 * t[j];
            if (a.norm2 == kNormLayer) {
                unpack8<BF16>(load8<VEC>(a.beta2, 0, p, v, true), t);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] += t[j];
            }
            store8<VEC>(a.y, off, p, v, active, pack8<BF16>(y));
        }
    }
    if (a.stats && active && p.t == 0 && rank == 0) a.stats[row] = make_float4(mu1, rs1, mu2, rs2);
}

// ------------------------------------------------------------------ backward
// A CTA (or cluster) takes items of rows, `slots` rows at a time, and keeps
// the column sums of its rows (dgamma1, dbeta1, dgamma2, dbeta2, and dgate
// within an item) in shared memory, each thread adding to its own columns,
// so nothing is atomic and the order is fixed.
//
// With the forward's statistics at hand one row reduction is enough: the
// pullback through the second norm is linear in the two means of that norm,
// so the sums the first norm's pullback needs of D are formed from six sums
// that do not need those means.  (Recomputing the statistics would take
// three to five dependent reductions a row.)
template <bool BF16, bool VEC, int VECS>
__global__ void __launch_bounds__(kJoinThreads, 1) join_backward_kernel(const __grid_constant__ JoinArgs a)
{
    extern __shared__ float acc[];   // [arrays][slots][cols]
    __shared__ RowSumSmem sums;
    int half = 0;
    const JoinShape &sh = a.shape;
    const uint32_t rank = sh.cluster > 1 ? cluster_ctarank() : 0u;
    const int64_t group_cta = blockIdx.x / sh.cluster;
    const int64_t n_ctas = gridDim.x / sh.cluster;
    const int slot = threadIdx.x / sh.tpr;
    Place<VEC> p;
    p.tpr = sh.tpr;
    p.t = threadIdx.x - slot * sh.tpr;
    p.c0 = static_cast<int>(rank) * sh.cols;
    p.c1 = min(a.N, p.c0 + sh.cols);
    const int ncols = p.c1 - p.c0;
    const float inv_n = 1.0f / static_cast<float>(a.N);
    const bool norm1 = a.norm1 != kNormNone, norm2 = a.norm2 != kNormNone;
    const bool ln1 = a.norm1 == kNormLayer, ln2 = a.norm2 == kNormLayer;

    if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0;
    const int arr = sh.slots * sh.cols;
    for (int i = threadIdx.x; i < a.arrays * arr; i += blockDim.x) acc[i] = 0.0f;
    __syncthreads();
    if (sh.cluster > 1) cluster_sync_all();   // every CTA runs before its shared memory is written
    // This thread's sums of vector v: 8 floats of array k.  In the order of
    // the thread's elements, so a warp's accesses are whole 16-byte rows (VEC)
    // or consecutive floats.
    auto add8 = [&](int k, int v, const float (&d)[8]) {
        if (k < 0) return;
        float *b = acc + static_cast<size_t>(k) * arr + slot * sh.cols;
        if constexpr (VEC) {
            if (p.valid(v, 0)) {
                float4 *q = reinterpret_cast<float4 *>(b + p.col(v, 0) - p.c0);
                float4 lo = q[0], hi = q[1];
                lo.x += d[0]; lo.y += d[1]; lo.z += d[2]; lo.w += d[3];
                hi.x += d[4]; hi.y += d[5]; hi.z += d[6]; hi.w += d[7];
                q[0] = lo;
                q[1] = hi;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (p.valid(v, j)) b[p.col(v, j) - p.c0] += d[j];
        }
    };

    for (int64_t item = group_cta; item < a.items; item += n_ctas) {
        const int64_t group = item / a.items_per_group;
        const int64_t g0 = group * a.rows_per_gate;
        const int64_t g1 = g0 + a.rows_per_gate < a.M ? g0 + a.rows_per_gate : a.M;
        const int64_t r0 = g0 + (item - group * a.items_per_group) * a.item_rows;
        const int64_t r1 = r0 + a.item_rows < g1 ? r0 + a.item_rows : g1;
        const int64_t goff = group * a.N;
        for (int64_t base = r0; base < r1; base += sh.slots) {
            const int64_t row = base + slot;
            const bool active = row < r1;
            const int64_t off = row * a.N;
            uint4 xp[VECS], rp[VECS], yp[VECS], hp[VECS];
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                xp[v] = load8<VEC>(a.x, off, p, v, active);
                rp[v] = a.residual ? load8<VEC>(a.residual, off, p, v, active) : zero;
                yp[v] = a.dy ? load8<VEC>(a.dy, off, p, v, active) : zero;
                hp[v] = a.dh ? load8<VEC>(a.dh, off, p, v, active) : zero;
            }
            const float4 st = active ? a.stats[row] : make_float4(0.f, 0.f, 0.f, 0.f);

            // Everything of vector v that both phases need.
            auto terms = [&](int v, float (&u1)[8], float (&n)[8], float (&u2)[8], float (&w)[8],
                             float (&gs)[8], float (&dA)[8], float (&dyh)[8]) {
                float t[8], b[8];
                unpack8<BF16>(xp[v], u1);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    u1[j] = norm1 ? (u1[j] - st.x) * st.y : u1[j];
                    gs[j] = a.block_scale;
                }
                if (a.gate) {
                    unpack8<BF16>(load8<VEC>(a.gate, goff, p, v, true), t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) gs[j] *= t[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    n[j] = u1[j];
                    w[j] = gs[j];
                }
                if (norm1) {
                    unpack8<BF16>(load8<VEC>(a.gamma1, 0, p, v, true), t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        n[j] *= t[j];
                        w[j] *= t[j];
                    }
                    if (ln1) {
                        unpack8<BF16>(load8<VEC>(a.beta1, 0, p, v, true), t);
#pragma unroll
                        for (int j = 0; j < 8; ++j) n[j] += t[j];
                    }
                }
                unpack8<BF16>(rp[v], t);
                unpack8<BF16>(hp[v], dA);
                unpack8<BF16>(yp[v], dyh);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float h = a.residual_scale * t[j] + gs[j] * n[j];
                    u2[j] = norm2 ? (h - st.z) * st.w : 0.0f;
                }
                if (norm2) {
                    unpack8<BF16>(load8<VEC>(a.gamma2, 0, p, v, true), b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        b[j] *= dyh[j];          // gamma2 dy
                        dA[j] += st.w * b[j];    // dh + rstd2 gamma2 dy
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) b[j] = 0.0f;
                }
                // columns past the row take no part
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!p.valid(v, j)) u1[j] = u2[j] = w[j] = dA[j] = b[j] = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) dyh[j] = b[j];
            };

            float s[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = 0.0f;
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                float u1[8], n[8], u2[8], w[8], gs[8], dA[8], dyh[8];
                terms(v, u1, n, u2, w, gs, dA, dyh);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float wu = w[j] * u1[j];
                    s[0] += dyh[j];
                    s[1] += dyh[j] * u2[j];
                    s[2] += w[j] * dA[j];
                    s[3] += w[j];
                    s[4] += w[j] * u2[j];
                    s[5] += wu * dA[j];
                    s[6] += wu;
                    s[7] += wu * u2[j];
                }
            }
            row_sum(s, sums, half, sh, slot, rank);
            // D = dA - c0 - c1 u2
            const float c0 = ln2 ? st.w * s[0] * inv_n : 0.0f;
            const float c1 = norm2 ? st.w * s[1] * inv_n : 0.0f;
            const float t0 = ln1 ? (s[2] - c0 * s[3] - c1 * s[4]) * inv_n : 0.0f;
            const float t1 = norm1 ? (s[5] - c0 * s[6] - c1 * s[7]) * inv_n : 0.0f;
            const float rs1 = norm1 ? st.y : 1.0f;
#pragma unroll
            for (int v = 0; v < VECS; ++v) {
                float u1[8], n[8], u2[8], w[8], gs[8], D[8], dyh[8], o[8];
                terms(v, u1, n, u2, w, gs, D, dyh);
#pragma unroll
                for (int j = 0; j < 8; ++j) D[j] -= c0 + c1 * u2[j];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = rs1 * (w[j] * D[j] - t0 - t1 * u1[j]);
                store8<VEC>(a.dx, off, p, v, active, pack8<BF16>(o));
                if (a.dresidual) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = a.residual_scale * D[j];
                    store8<VEC>(a.dresidual, off, p, v, active, pack8<BF16>(o));
                }
                if (!active) continue;
                if (a.a_dgate >= 0) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = a.block_scale * n[j] * D[j];
                    add8(a.a_dgate, v, o);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) D[j] *= gs[j];   // dn
                add8(a.a_dbeta1, v, D);
                if (a.a_dgamma1 >= 0) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = D[j] * u1[j];
                    add8(a.a_dgamma1, v, o);
                }
                unpack8<BF16>(yp[v], dyh);
                add8(a.a_dbeta2, v, dyh);
                if (a.a_dgamma2 >= 0) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = dyh[j] * u2[j];
                    add8(a.a_dgamma2, v, o);
                }
            }
        }
        if (a.a_dgate >= 0) {
            __syncthreads();
            float *b = acc + static_cast<size_t>(a.a_dgate) * arr;
            for (int c = threadIdx.x; c < ncols; c += blockDim.x) {
                float t = 0.0f;
                for (int k = 0; k < sh.slots; ++k) {
                    t += b[k * sh.cols + c];
                    b[k * sh.cols + c] = 0.0f;
                }
                if (a.dgate_direct) {
                    uint16_t *q = static_cast<uint16_t *>(a.dgate) + goff + p.c0 + c;
                    if constexpr (BF16) *q = __bfloat16_as_ushort(__float2bfloat16_rn(t));
                    else *q = __half_as_ushort(__float2half_rn(t));
                } else {
                    a.gate_partials[item * a.N + p.c0 + c] = t;
                }
            }
            __syncthreads();
        }
    }
    __syncthreads();
    // The CTA's sums: row (array, CTA) of `partials`, the item's gate sums aside.
    for (int k = 0; k < a.arrays; ++k) {
        if (k == a.a_dgate) continue;
        float *dst = a.partials + (static_cast<int64_t>(k) * n_ctas + group_cta) * a.N + p.c0;
        const float *b = acc + static_cast<size_t>(k) * arr;
        for (int c = threadIdx.x; c < ncols; c += blockDim.x) {
            float t = 0.0f;
            for (int q = 0; q < sh.slots; ++q) t += b[q * sh.cols + c];
            dst[c] = t;
        }
    }
}

// ---------------------------------------------------------------- last sums
constexpr int kReduceCols = 32, kReduceLanes = 16;

// Output row o of width N = the sum of its source's rows, added in a fixed order.
template <bool BF16>
__global__ void __launch_bounds__(kReduceCols *kReduceLanes) join_reduce_kernel(const __grid_constant__ JoinReduce r)
{
    __shared__ float part[kReduceLanes][kReduceCols];
    const int tx = threadIdx.x % kReduceCols, ty = threadIdx.x / kReduceCols;
    const int col = blockIdx.x * kReduceCols + tx;
    for (int64_t o = blockIdx.y; o < r.total_outs; o += gridDim.y) {
        int i = 0;
        while (i + 1 < r.sources && o >= r.first[i + 1]) ++i;
        const int64_t k = o - r.first[i];
        const float *src = r.src[i] + k * r.rows[i] * r.row_stride[i];
        float t = 0.0f;
        if (col < r.N)
            for (int q = ty; q < r.rows[i]; q += kReduceLanes) t += src[q * r.row_stride[i] + col];
        part[ty][tx] = t;
        __syncthreads();
        if (ty == 0 && col < r.N) {
            t = 0.0f;
#pragma unroll
            for (int q = 0; q < kReduceLanes; ++q) t += part[q][tx];
            uint16_t *d = static_cast<uint16_t *>(r.dst[i]) + k * r.N + col;
            if constexpr (BF16) *d = __bfloat16_as_ushort(__float2bfloat16_rn(t));
            else *d = __half_as_ushort(__float2half_rn(t));
        }
        __syncthreads();
    }
}

int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

// Threads and vectors for `cols` columns: at most `want` threads of a row if
// four vectors each are enough for that.
void row_threads(int64_t cols, int want, int *vecs, int *tpr)
{
    int v = 1;
    while (v < kJoinMaxVecs && (cols + 8 * v - 1) / (8 * v) > want) v *= 2;
    const int64_t t = (cols + 8 * v - 1) / (8 * v);
    *vecs = v;
    *tpr = static_cast<int>((t + 31) / 32 * 32);
}

template <typename K>
int launch_cluster(K kern, unsigned rows, const JoinShape &sh, size_t smem, const JoinArgs &a,
                   cudaStream_t stream, const char *what)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * static_cast<unsigned>(sh.cluster));
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

template <bool BF16, bool VEC, int VECS>
int run_forward(const JoinArgs &a, cudaStream_t stream)
{
    const int64_t rows = (a.M + a.shape.slots - 1) / a.shape.slots;
    return launch_cluster(join_forward_kernel<BF16, VEC, VECS>, static_cast<unsigned>(rows), a.shape, 0, a,
                          stream, "cudaLaunchKernelEx (join)");
}

template <bool BF16, bool VEC, int VECS>
int run_backward(const JoinArgs &a, int ctas, cudaStream_t stream)
{
    auto kern = join_backward_kernel<BF16, VEC, VECS>;
    const size_t smem = static_cast<size_t>(a.arrays) * a.shape.slots * a.shape.cols * sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kJoinSumBytes);
    if (e != cudaSuccess)
        return record_cuda_error("cudaFuncSetAttribute(max dynamic smem)", e, cudaGetErrorString(e));
    return launch_cluster(kern, static_cast<unsigned>(ctas), a.shape, smem, a, stream,
                          "cudaLaunchKernelEx (join gradient)");
}

}  // namespace

JoinShape join_forward_shape(int64_t N)
{
    JoinShape s;
    s.cluster = 1;
    while (up8((N + s.cluster - 1) / s.cluster) > kJoinThreads * kJoinMaxVecs * 8) s.cluster *= 2;
    s.cols = static_cast<int>(up8((N + s.cluster - 1) / s.cluster));
    row_threads(s.cols, 256, &s.vecs, &s.tpr);
    s.slots = s.cluster > 1 || s.tpr > 128 ? 1 : 256 / s.tpr;
    return s;
}

JoinShape join_backward_shape(int64_t N, int arrays)
{
    JoinShape s;
    s.cluster = 1;
    auto cols = [&] { return up8((N + s.cluster - 1) / s.cluster); };
    while (cols() > kJoinThreads * kJoinMaxVecs * 8 || arrays * cols() * 4 > kJoinSumBytes) s.cluster *= 2;
    s.cols = static_cast<int>(cols());
    row_threads(s.cols, kJoinThreads, &s.vecs, &s.tpr);
    s.slots = s.cluster > 1 ? 1 : kJoinThreads / s.tpr;
    while (s.slots > 1 && static_cast<int64_t>(arrays) * s.slots * s.cols * 4 > kJoinSumBytes) --s.slots;
    return s;
}

#define NGR_JOIN_CASES(CALL)                                                \
    switch (a.shape.vecs) {                                                 \
    case 1: return bf16 ? (vec ? CALL(true, true, 1) : CALL(true, false, 1)) \
                        : (vec ? CALL(false, true, 1) : CALL(false, false, 1)); \
    case 2: return bf16 ? (vec ? CALL(true, true, 2) : CALL(true, false, 2)) \
                        : (vec ? CALL(false, true, 2) : CALL(false, false, 2)); \
    case 4: return bf16 ? (vec ? CALL(true, true, 4) : CALL(true, false, 4)) \
                        : (vec ? CALL(false, true, 4) : CALL(false, false, 4)); \
    }                                                                       \
    return -9;

int launch_join_forward(bool bf16, bool vec, const JoinArgs &a, cudaStream_t stream)
{
#define NGR_FWD(B, V, K) run_forward<B, V, K>(a, stream)
    NGR_JOIN_CASES(NGR_FWD)
#undef NGR_FWD
}

int launch_join_backward(bool bf16, bool vec, const JoinArgs &a, int ctas, cudaStream_t stream)
{
#define NGR_BWD(B, V, K) run_backward<B, V, K>(a, ctas, stream)
    NGR_JOIN_CASES(NGR_BWD)
#undef NGR_BWD
}

int launch_join_reduce(bool bf16, const JoinReduce &r, cudaStream_t stream)
{
    if (r.sources == 0) return 0;
    const dim3 grid(static_cast<unsigned>((r.N + kReduceCols - 1) / kReduceCols),
                    static_cast<unsigned>(r.total_outs < 1024 ? r.total_outs : 1024));
    if (bf16) join_reduce_kernel<true><<<grid, kReduceCols * kReduceLanes, 0, stream>>>(r);
    else join_reduce_kernel<false><<<grid, kReduceCols * kReduceLanes, 0, stream>>>(r);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : record_cuda_error("join sums launch", e, cudaGetErrorString(e));
}

}  // namespace ngr
