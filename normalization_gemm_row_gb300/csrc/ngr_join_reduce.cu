// ngr_join_reduce.cu -- the second kernel of the join's gradient: the vectors
// of the row's width from the sums that the CTAs left, and the choice of the
// first kernel's shape.
#include "ngr_join_backward.cuh"

namespace ngr {

namespace {

// ---------------------------------------------------------------- last sums
constexpr int kReduceCols = 32, kReduceLanes = 16;

// Output row o (0-3 dgamma1, dbeta1, dgamma2, dbeta2, then the gate's rows)
// at 32 x VEC columns: the rows of sums are added in a fixed order, 16 lanes
// of threads taking every 16th row, eight loads under way in each (16000 x
// 1152: the gradient 74.6 -> 68.6 us).  The launch overlaps the gradient
// kernel's tail; 32 lanes were 2 % slower at 8192 columns.
template <bool BF16, int VEC>
__global__ void __launch_bounds__(kReduceCols *kReduceLanes) join_reduce_kernel(const __grid_constant__ JoinReduce r)
{
    __shared__ float part[kReduceLanes][2][kReduceCols * VEC];
    const int tx = threadIdx.x % kReduceCols, ty = threadIdx.x / kReduceCols;
    const int col = (blockIdx.x * kReduceCols + tx) * VEC;
    const bool in = col < r.N;
    pdl_wait();
    const uint16_t *gate = static_cast<const uint16_t *>(r.gate);
    auto load = [&](const float *rows, int64_t i, float (&f)[VEC]) {
        const float *p = rows + i * r.N + col;
        if constexpr (VEC == 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p);
            f[0] = q.x;
            f[1] = q.y;
            f[2] = q.z;
            f[3] = q.w;
        } else {
            f[0] = *p;
        }
    };
    for (int64_t o = blockIdx.y; o < 4 + (r.dgate ? r.groups : 0); o += gridDim.y) {
        void *dst = o == 0 ? r.dgamma1 : o == 1 ? r.dbeta1 : o == 2 ? r.dgamma2 : o == 3 ? r.dbeta2 : r.dgate;
        if (!dst) continue;
        float t[VEC] = {}, u[VEC] = {}, f[VEC];
        if (in && o < 2) {
            const float *src = o == 0 ? r.p : r.q;
#pragma unroll 8
            for (int i = ty; i < r.pq_rows; i += kReduceLanes) {
                load(src, i, f);
                const uint16_t *g = gate + static_cast<int64_t>(i / r.items_per_group) * r.N + col;
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    t[j] += r.fold_gate ? f[j] : gate ? r.block_scale * widen16<BF16>(g[j]) * f[j] : r.block_scale * f[j];
            }
        } else if (in && o < 4) {
            const float *src = o == 2 ? r.dgamma2_rows : r.dbeta2_rows;
#pragma unroll 8
            for (int i = ty; i < r.ctas; i += kReduceLanes) {
                load(src, i, f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) t[j] += f[j];
            }
        } else if (in) {
            const int64_t i0 = (o - 4) * r.items_per_group;
#pragma unroll 8
            for (int i = ty; i < r.items_per_group; i += kReduceLanes) {
                load(r.p, i0 + i, f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) t[j] += f[j];
                if (r.q) {
                    load(r.q, i0 + i, f);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) u[j] += f[j];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            part[ty][0][j * kReduceCols + tx] = t[j];
            part[ty][1][j * kReduceCols + tx] = u[j];
        }
        __syncthreads();
        // (column j of thread tx: VEC of the CTA's warps add one j each)
        const int c = col + ty;
        if (ty < VEC && in) {
            float sum = 0.0f, sum_q = 0.0f;
#pragma unroll
            for (int q = 0; q < kReduceLanes; ++q) {
                sum += part[q][0][ty * kReduceCols + tx];
                sum_q += part[q][1][ty * kReduceCols + tx];
            }
            if (o >= 4) {
                const uint16_t *g1 = static_cast<const uint16_t *>(r.gamma1), *b1 = static_cast<const uint16_t *>(r.beta1);
                sum *= g1 ? widen16<BF16>(g1[c]) : 1.0f;
                if (b1) sum += sum_q * widen16<BF16>(b1[c]);
                sum *= r.block_scale;
            }
            static_cast<uint16_t *>(dst)[(o >= 4 ? (o - 4) * r.N : 0) + c] = round16<BF16>(sum);
        }
        __syncthreads();
    }
}

template <int VEC>
cudaError_t reduce(bool bf16, const JoinReduce &r, int64_t outs, cudaStream_t stream)
{
    constexpr int kCols = kReduceCols * VEC;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((r.N + kCols - 1) / kCols), static_cast<unsigned>(outs < 1024 ? outs : 1024));
    cfg.blockDim = dim3(kReduceCols * kReduceLanes);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bf16 ? join_reduce_kernel<true, VEC> : join_reduce_kernel<false, VEC>, r);
}

}  // namespace

// The row's columns over as few CTAs as hold them and their sums.  Clusters of
// 8 hold every row up to 65536 columns but for two kinds that are wider than
// 60000: shifted rows, which need a vector more than 8 CTAs have, and rows
// with five sums, which need more shared memory; those take 16 CTAs.
JoinShape join_backward_shape(int64_t N, int mode, int arrays)
{
    JoinShape s;
    s.cluster = 1;
    auto cols = [&] { return up8((N + s.cluster - 1) / s.cluster); };
    while (cols() + (mode == kJoinWindow ? 8 : 0) > kJoinBackwardCols) s.cluster *= 2;
    for (;; s.cluster *= 2) {
        s.cols = static_cast<int>(cols());
        const int64_t n = join_vectors(s, mode);
        // (a cluster works on one row at a time; the scalar mode, for pointers
        // that no other takes, has two widths only)
        s.tpr = 512;
        s.vecs = 2;
        for (const Width &w : kWidths) {
            if (w.tpr * w.vecs < n || (s.cluster > 1 && w.tpr < 256)) continue;
            if (mode == kJoinScalar && !(w.tpr == 64 && w.vecs == 2)) continue;
            s.tpr = w.tpr;
            s.vecs = w.vecs;
            break;
        }
        s.slots = backward_slots(s.tpr);
        // As many CTAs as the SM has registers for, and shared memory for
        // their sums and a row each.
        const int64_t bytes = sum_bytes(s, arrays, mode) + ring_row(s) + 2048;
        s.per_sm = static_cast<int>(std::min<int64_t>(backward_ctas(s.tpr, s.vecs), kJoinSmem / bytes));
        if (s.per_sm >= 1) return s;
    }
}

int launch_join_backward_bf16_ln(int mode, const JoinArgs &a, int ctas, cudaStream_t stream);
int launch_join_backward_bf16_rms(int mode, const JoinArgs &a, int ctas, cudaStream_t stream);
int launch_join_backward_f16_ln(int mode, const JoinArgs &a, int ctas, cudaStream_t stream);
int launch_join_backward_f16_rms(int mode, const JoinArgs &a, int ctas, cudaStream_t stream);

int launch_join_backward(bool bf16, int mode, const JoinArgs &a, int ctas, cudaStream_t stream)
{
    if (a.norm1 == kNormLayer || a.norm2 == kNormLayer)
        return bf16 ? launch_join_backward_bf16_ln(mode, a, ctas, stream) : launch_join_backward_f16_ln(mode, a, ctas, stream);
    return bf16 ? launch_join_backward_bf16_rms(mode, a, ctas, stream) : launch_join_backward_f16_rms(mode, a, ctas, stream);
}

int launch_join_reduce(bool bf16, const JoinReduce &r, cudaStream_t stream)
{
    if (!r.dgamma1 && !r.dbeta1 && !r.dgamma2 && !r.dbeta2 && !r.dgate) return 0;
    const int64_t outs = 4 + (r.dgate ? r.groups : 0);
    // Four columns a thread in rows so wide that four outputs have a CTA for
    // every SM: the gradient at 8192 x 8192 154.3 -> 151.4 us, but at 32768 x
    // 2048 141.6 -> 142.9 and at 16000 x 1152 56.5 -> 62.7.
    const bool wide = r.N % 4 == 0 && r.N / (4 * kReduceCols) * 4 >= kJoinSms;
    const cudaError_t e = wide ? reduce<4>(bf16, r, outs, stream) : reduce<1>(bf16, r, outs, stream);
    return e == cudaSuccess ? 0 : record_cuda_error("join sums launch", e, cudaGetErrorString(e));
}

}  // namespace ngr
