// ngr_join_api.cu -- entry points of the block join (ngr_join.cu): argument
// checks, workspace layout, how the backward pass cuts the rows.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "ngr.h"
#include "ngr_internal.h"
#include "ngr_join.h"

namespace ngr {

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool norm_kind(int n) { return n >= kNormNone && n <= kNormRms; }

struct JoinPlan {
    JoinShape shape;
    int a_dgamma1 = -1, a_dbeta1 = -1, a_dgamma2 = -1, a_dbeta2 = -1, a_dgate = -1, arrays = 0;
    int64_t groups = 1, group_rows = 0, items = 0, item_rows = 0;
    int items_per_group = 1, ctas = 0;
    size_t off_partials = 256, off_gate = 0, total = 256;
};

// The rows are cut so that every CTA gets the same number of rows as nearly
// as the gate's groups allow: of the numbers of items per group, the one
// with the least rows on the busiest CTA, an item counted as one row more
// for writing its gate sums (N floats against a row's twelve bytes a column).
JoinPlan join_plan(int64_t M, int64_t N, int64_t rows_per_gate, int norm1, int norm2)
{
    JoinPlan p;
    if (norm1 != kNormNone) p.a_dgamma1 = p.arrays++;
    if (norm1 == kNormLayer) p.a_dbeta1 = p.arrays++;
    if (norm2 != kNormNone) p.a_dgamma2 = p.arrays++;
    if (norm2 == kNormLayer) p.a_dbeta2 = p.arrays++;
    const bool gate = rows_per_gate > 0;
    if (gate) p.a_dgate = p.arrays++;
    p.shape = join_backward_shape(N, p.arrays);
    p.group_rows = gate ? std::min(rows_per_gate, M) : M;
    if (M == 0) return p;
    p.groups = (M + p.group_rows - 1) / p.group_rows;
    const int64_t P = kJoinCtas / p.shape.cluster;
    const int64_t steps = (p.group_rows + p.shape.slots - 1) / p.shape.slots;
    const int64_t most = std::min(steps, std::max<int64_t>(1, 4 * P / p.groups));
    int64_t best = 0, best_cost = 0;
    for (int64_t c = 1; c <= most; ++c) {
        const int64_t rows = (steps + c - 1) / c + (gate ? 1 : 0);
        const int64_t cost = (p.groups * c + P - 1) / P * rows;
        if (best == 0 || cost < best_cost) {
            best = c;
            best_cost = cost;
        }
    }
    p.items_per_group = static_cast<int>(best);
    p.item_rows = (steps + best - 1) / best * p.shape.slots;
    p.items = p.groups * best;
    p.ctas = static_cast<int>(std::min(P, p.items));
    const size_t row = static_cast<size_t>(N) * sizeof(float);
    p.off_gate = p.off_partials + static_cast<size_t>(p.arrays - (gate ? 1 : 0)) * p.ctas * row;
    p.total = p.off_gate + (gate && best > 1 ? static_cast<size_t>(p.items) * row : 0);
    return p;
}

int join_sizes(int64_t M, int64_t N, int dtype)
{
    if (dtype != NGR_F16 && dtype != NGR_BF16) return NGR_ERR_DTYPE;
    if (M < 0 || N <= 0 || M >= (int64_t(1) << 31) || N > kJoinMaxN) return NGR_ERR_SHAPE;
    return NGR_OK;
}

// Whether the 16-byte kernels can run: NGR_ERR_ALIGN if not even 2-byte ones can.
int join_alignment(std::initializer_list<const void *> ptrs, int64_t N, bool *vec)
{
    *vec = N % 8 == 0;
    for (const void *p : ptrs) {
        if (!aligned(p, 2)) return NGR_ERR_ALIGN;
        *vec = *vec && aligned(p, 16);
    }
    return NGR_OK;
}

int join_norms(int norm1, int norm2, const void *gamma1, const void *beta1, const void *gamma2,
               const void *beta2, float eps1, float eps2, float residual_scale, float block_scale)
{
    if (!norm_kind(norm1) || !norm_kind(norm2)) return NGR_ERR_ARG;
    if ((norm1 != kNormNone && !(eps1 >= 0.0f)) || (norm2 != kNormNone && !(eps2 >= 0.0f))) return NGR_ERR_ARG;
    if (!std::isfinite(residual_scale) || !std::isfinite(block_scale)) return NGR_ERR_ARG;
    if ((norm1 != kNormNone && !gamma1) || (norm1 == kNormLayer && !beta1) ||
        (norm2 != kNormNone && !gamma2) || (norm2 == kNormLayer && !beta2))
        return NGR_ERR_NULL;
    return NGR_OK;
}

JoinArgs join_args(const void *x, const void *residual, const void *gate, int64_t rows_per_gate,
                   int norm1, const void *gamma1, const void *beta1, float eps1, int norm2,
                   const void *gamma2, const void *beta2, float eps2, float residual_scale,
                   float block_scale, int64_t M, int64_t N)
{
    JoinArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.residual = residual;
    a.gate = gate;
    a.rows_per_gate = gate ? std::min(rows_per_gate, M) : M;
    a.norm1 = norm1;
    a.gamma1 = norm1 != kNormNone ? gamma1 : nullptr;
    a.beta1 = norm1 == kNormLayer ? beta1 : nullptr;
    a.eps1 = eps1;
    a.norm2 = norm2;
    a.gamma2 = norm2 != kNormNone ? gamma2 : nullptr;
    a.beta2 = norm2 == kNormLayer ? beta2 : nullptr;
    a.eps2 = eps2;
    a.residual_scale = residual_scale;
    a.block_scale = block_scale;
    a.M = M;
    a.N = static_cast<int>(N);
    return a;
}

int zero_vector(void *p, int64_t n, cudaStream_t stream)
{
    if (!p) return NGR_OK;
    const cudaError_t e = cudaMemsetAsync(p, 0, static_cast<size_t>(n) * 2, stream);
    return e == cudaSuccess ? NGR_OK : record_cuda_error("cudaMemsetAsync (gradient)", e, cudaGetErrorString(e));
}

}  // namespace

}  // namespace ngr

using namespace ngr;

extern "C" {

int ngr_fused_norm_gate_residual_norm(int norm1, int norm2, const void *x, const void *residual,
                                      const void *gate, int64_t rows_per_gate, const void *gamma1,
                                      const void *beta1, const void *gamma2, const void *beta2,
                                      float eps1, float eps2, float residual_scale, float block_scale,
                                      int64_t M, int64_t N, int dtype, void *h, void *y, float *stats,
                                      ngr_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int rc = join_norms(norm1, norm2, gamma1, beta1, gamma2, beta2, eps1, eps2, residual_scale, block_scale);
    if (rc != NGR_OK) return rc;
    rc = join_sizes(M, N, dtype);
    if (rc != NGR_OK) return rc;
    if (gate && rows_per_gate <= 0) return NGR_ERR_ARG;
    if (M == 0) return NGR_OK;
    if (!x || !h || (norm2 != kNormNone && !y)) return NGR_ERR_NULL;
    if (!aligned(stats, 16)) return NGR_ERR_ALIGN;
    JoinArgs a = join_args(x, residual, gate, rows_per_gate, norm1, gamma1, beta1, eps1, norm2, gamma2,
                           beta2, eps2, residual_scale, block_scale, M, N);
    a.h = h;
    a.y = norm2 != kNormNone ? y : nullptr;
    a.stats = reinterpret_cast<float4 *>(stats);
    bool vec = false;
    rc = join_alignment({x, residual, gate, a.gamma1, a.beta1, a.gamma2, a.beta2, h, a.y}, N, &vec);
    if (rc != NGR_OK) return rc;
    int sms = 0;
    rc = device_sms(&sms);
    if (rc != NGR_OK) return rc;
    a.shape = join_forward_shape(N);
    call_begin();
    kernel_begin(stream);
    rc = launch_join_forward(dtype == NGR_BF16, vec, a, stream);
    kernel_end(stream);
    return call_end(rc, nullptr, stream);
}

size_t ngr_norm_gate_residual_norm_workspace_bytes(int norm1, int norm2, int64_t rows_per_gate, int64_t M,
                                                   int64_t N)
{
    if (!norm_kind(norm1) || !norm_kind(norm2) || join_sizes(M, N, NGR_F16) != NGR_OK) return 0;
    return join_plan(M, N, rows_per_gate, norm1, norm2).total;
}

int ngr_fused_norm_gate_residual_norm_backward(
    int norm1, int norm2, const void *dy, const void *dh, const void *x, const void *residual,
    const void *gate, int64_t rows_per_gate, const void *gamma1, const void *beta1, const void *gamma2,
    const float *stats, float residual_scale, float block_scale, int64_t M, int64_t N, int dtype, void *dx, void *dresidual, void *dgate, void *dgamma1, void *dbeta1, void *dgamma2,
    void *dbeta2, void *workspace, size_t workspace_bytes, ngr_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    // (beta2 has no part in the gradient: gamma2 stands in for it in the checks)
    int rc = join_norms(norm1, norm2, gamma1, beta1, gamma2, gamma2, 0.0f, 0.0f, residual_scale, block_scale);
    if (rc != NGR_OK) return rc;
    rc = join_sizes(M, N, dtype);
    if (rc != NGR_OK) return rc;
    if (gate && rows_per_gate <= 0) return NGR_ERR_ARG;
    // outputs that the call does not have are not written
    if (!gate) dgate = nullptr;
    if (norm1 == kNormNone) dgamma1 = nullptr;
    if (norm1 != kNormLayer) dbeta1 = nullptr;
    if (norm2 == kNormNone) dgamma2 = nullptr;
    if (norm2 != kNormLayer) dbeta2 = nullptr;
    if (M > 0 && (!x || !stats || !dx || (!dy && !dh) || (norm2 == kNormNone && !dh) ||
                  (!residual && dresidual)))
        return NGR_ERR_NULL;
    if (norm2 == kNormNone) dy = nullptr;
    if (!aligned(stats, 16)) return NGR_ERR_ALIGN;
    bool vec = false;
    JoinArgs a = join_args(x, residual, gate, rows_per_gate, norm1, gamma1, beta1, 0.0f, norm2, gamma2,
                           nullptr, 0.0f, residual_scale, block_scale, M, N);
    rc = join_alignment({dy, dh, x, residual, gate, a.gamma1, a.beta1, a.gamma2, dx, dresidual,
                         dgate, dgamma1, dbeta1, dgamma2, dbeta2}, N, &vec);
    if (rc != NGR_OK) return rc;
    const JoinPlan p = join_plan(M, N, gate ? rows_per_gate : 0, norm1, norm2);
    if (!workspace || workspace_bytes < p.total) return NGR_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return NGR_ERR_ALIGN;
    int sms = 0;
    rc = device_sms(&sms);
    if (rc != NGR_OK) return rc;
    char *ws = static_cast<char *>(workspace);
    if (M == 0) {   // empty sums
        rc = zero_vector(ws, 2, stream);
        for (void *v : {dgamma1, dbeta1, dgamma2, dbeta2})
            if (rc == NGR_OK) rc = zero_vector(v, N, stream);
        return rc;
    }
    a.dy = dy;
    a.dh = dh;
    a.dx = dx;
    a.dresidual = dresidual;
    a.dgate = dgate;
    a.stats = const_cast<float4 *>(reinterpret_cast<const float4 *>(stats));
    a.err = reinterpret_cast<int *>(ws);
    a.partials = reinterpret_cast<float *>(ws + p.off_partials);
    a.gate_partials = reinterpret_cast<float *>(ws + p.off_gate);
    a.shape = p.shape;
    a.items = p.items;
    a.item_rows = p.item_rows;
    a.items_per_group = p.items_per_group;
    a.a_dgamma1 = p.a_dgamma1;
    a.a_dbeta1 = p.a_dbeta1;
    a.a_dgamma2 = p.a_dgamma2;
    a.a_dbeta2 = p.a_dbeta2;
    a.a_dgate = dgate ? p.a_dgate : -1;
    a.arrays = p.arrays - (gate && !dgate ? 1 : 0);
    a.dgate_direct = p.items_per_group == 1;

    JoinReduce r;
    std::memset(&r, 0, sizeof(r));
    r.N = static_cast<int>(N);
    auto source = [&](const float *src, int rows, void *dst, int64_t outs) {
        if (!dst) return;
        r.src[r.sources] = src;
        r.row_stride[r.sources] = N;
        r.rows[r.sources] = rows;
        r.dst[r.sources] = dst;
        r.first[r.sources] = r.total_outs;
        r.total_outs += outs;
        ++r.sources;
    };
    auto sum_of = [&](int k) { return a.partials + static_cast<int64_t>(k) * p.ctas * N; };
    source(sum_of(p.a_dgamma1), p.ctas, dgamma1, 1);
    source(sum_of(p.a_dbeta1), p.ctas, dbeta1, 1);
    source(sum_of(p.a_dgamma2), p.ctas, dgamma2, 1);
    source(sum_of(p.a_dbeta2), p.ctas, dbeta2, 1);
    if (!a.dgate_direct) source(a.gate_partials, p.items_per_group, dgate, p.groups);

    const bool bf16 = dtype == NGR_BF16;
    call_begin();
    kernel_begin(stream);
    rc = launch_join_backward(bf16, vec, a, p.ctas, stream);
    kernel_end(stream);
    if (rc == NGR_OK && r.sources > 0) {
        kernel_begin(stream);
        rc = launch_join_reduce(bf16, r, stream);
        kernel_end(stream);
    }
    return call_end(rc, nullptr, stream);
}

}  // extern "C"
