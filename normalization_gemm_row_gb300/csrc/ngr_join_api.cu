// ngr_join_api.cu -- entry points of the block join (ngr_join_forward.cu,
// ngr_join_backward.cuh, ngr_join_reduce.cu): argument checks, workspace
// layout, how the backward pass cuts the rows.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "ngr.h"
#include "ngr_entry.h"
#include "ngr_internal.h"
#include "ngr_join.h"

namespace ngr {

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool norm_kind(int n) { return n >= kNormNone && n <= kNormRms; }

// Where the parts of the backward call's workspace lie, and how it cuts the
// rows (see JoinArgs).
struct JoinPlan {
    JoinShape shape;
    int a_p = -1, a_q = -1, a_dgamma2 = -1, a_dbeta2 = -1, a_dgate = -1, arrays = 0;
    int64_t groups = 1, group_rows = 0, items = 0, item_rows = 0, pq_rows = 0;
    int items_per_group = 1, period = 1, ctas = 0;
    bool fold_gate = false;
    size_t off_p = 256, off_q = 0, off_cta = 0, total = 256;
};

// A gate row of fewer tokens than this is applied row by row: writing the
// sums p and q of an item costs 8 bytes a column, as much as two thirds of
// a row's loads and stores, and the rows of sums would be as many as the
// tokens.
constexpr int64_t kFoldRows = 16;

// The rows are cut so that every CTA gets the same number of rows as nearly
// as the gate's groups allow: of the numbers of items per group that fill the
// CTAs one to four times over, the one with the least rows on the busiest
// CTA, an item counted as one row more for writing its sums.
//
// In the window mode the rows' shifts repeat after 8 / gcd(N, 8) rows, and the
// parameters, which lie under the row's columns, are loaded again when the
// shift changes: an item there has rows of one shift, if that leaves it
// kPeriodRows rows (8192 x 5003, RMS/RMS: 217 -> 182 us).
constexpr int64_t kPeriodRows = 4;

JoinPlan join_plan(int mode, int64_t M, int64_t N, int64_t rows_per_gate, int norm1, int norm2)
{
    JoinPlan p;
    const bool gate = rows_per_gate > 0;
    p.group_rows = gate ? std::min(rows_per_gate, M) : M;
    p.fold_gate = gate && p.group_rows < kFoldRows && p.group_rows < M;
    if (norm1 != kNormNone || (gate && !p.fold_gate)) p.a_p = p.arrays++;
    if (norm1 == kNormLayer) p.a_q = p.arrays++;
    if (norm2 != kNormNone) p.a_dgamma2 = p.arrays++;
    if (norm2 == kNormLayer) p.a_dbeta2 = p.arrays++;
    if (p.fold_gate) p.a_dgate = p.arrays++;
    p.shape = join_backward_shape(N, mode, p.arrays);
    if (M == 0) return p;
    p.groups = (M + p.group_rows - 1) / p.group_rows;
    const int64_t P = std::max<int64_t>(1, kJoinSms * p.shape.per_sm / p.shape.cluster);
    auto cut = [&](int64_t period) {
        const int64_t step = p.shape.slots * period, steps = (p.group_rows + step - 1) / step;
        int64_t best = 1;
        auto cost = [&](int64_t c) { return (p.groups * c * period + P - 1) / P * ((steps + c - 1) / c + 1); };
        for (int64_t waves = 1; waves <= 4 && !p.fold_gate; ++waves) {
            const int64_t c = std::min(steps, std::max<int64_t>(1, waves * P / (p.groups * period)));
            if (cost(c) < cost(best)) best = c;
        }
        p.period = static_cast<int>(period);
        p.items_per_group = static_cast<int>(best * period);
        p.item_rows = (steps + best - 1) / best * step;
        p.items = p.groups * p.items_per_group;
        return (steps + best - 1) / best;
    };
    const int64_t period = mode != kJoinWindow || p.fold_gate || N % 8 == 0 ? 1 : N % 2 ? 8 : N % 4 ? 4 : 2;
    if (cut(period) < kPeriodRows && period > 1) cut(1);
    p.ctas = static_cast<int>(std::min(P, p.items));
    p.pq_rows = p.fold_gate ? p.ctas : p.items;
    const size_t row = static_cast<size_t>(N) * sizeof(float);
    p.off_q = p.off_p + (p.a_p >= 0 ? static_cast<size_t>(p.pq_rows) * row : 0);
    p.off_cta = p.off_q + (p.a_q >= 0 ? static_cast<size_t>(p.pq_rows) * row : 0);
    p.total = p.off_cta + static_cast<size_t>((p.a_dgamma2 >= 0) + (p.a_dbeta2 >= 0)) * p.ctas * row;
    return p;
}

int join_sizes(int64_t M, int64_t N, int dtype)
{
    if (dtype != NGR_F16 && dtype != NGR_BF16) return NGR_ERR_DTYPE;
    if (M < 0 || N <= 0 || M >= (int64_t(1) << 31) || N > kJoinMaxN) return NGR_ERR_SHAPE;
    return NGR_OK;
}

// How the rows can be reached (kJoin* mode, and `shift` for the window
// mode): NGR_ERR_ALIGN if an address is not even that of a 16-bit element.
int join_alignment(std::initializer_list<const void *> rows, std::initializer_list<const void *> vectors,
                   int64_t N, int *mode, int *shift)
{
    bool same = true, vec = N % 8 == 0;
    *shift = -1;
    for (const void *p : rows) {
        if (!aligned(p, 2)) return NGR_ERR_ALIGN;
        if (!p) continue;
        const int at = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / 2);
        if (*shift < 0) *shift = at;
        same = same && at == *shift;
    }
    for (const void *p : vectors) {
        if (!aligned(p, 2)) return NGR_ERR_ALIGN;
        vec = vec && aligned(p, 16);
    }
    if (*shift < 0) *shift = 0;
    *mode = !same ? kJoinScalar : vec && *shift == 0 ? kJoinAligned : kJoinWindow;
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

void trace(const char *what, int mode, const JoinArgs &a, int64_t ctas)
{
    if (!trace_mode()) return;
    std::fprintf(stderr, "ngr: %s M=%lld N=%d norms=%d,%d %s cluster=%d cols=%d threads=%d x %d vecs=%d grid=%lld\n", what,
                 static_cast<long long>(a.M), a.N, a.norm1, a.norm2,
                 mode == kJoinAligned ? "aligned" : mode == kJoinWindow ? "shifted" : "by elements", a.shape.cluster,
                 a.shape.cols, a.shape.slots, a.shape.tpr, a.shape.vecs, static_cast<long long>(ctas * a.shape.cluster));
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
    int mode = 0;
    rc = join_alignment({x, residual, h, a.y}, {gate, a.gamma1, a.beta1, a.gamma2, a.beta2}, N, &mode, &a.shift);
    if (rc != NGR_OK) return rc;
    if (a.y == h) return NGR_ERR_ARG;
    int sms = 0;
    rc = device_sms(&sms);
    if (rc != NGR_OK) return rc;
    a.shape = join_forward_shape(N, mode);
    trace("block join", mode, a, (M + a.shape.slots - 1) / a.shape.slots);
    call_begin();
    kernel_begin(stream);
    rc = launch_join_forward(dtype == NGR_BF16, mode, a, stream);
    kernel_end(stream);
    return call_end(rc, nullptr, stream);
}

size_t ngr_norm_gate_residual_norm_workspace_bytes(int norm1, int norm2, int64_t rows_per_gate, int64_t M,
                                                   int64_t N)
{
    if (!norm_kind(norm1) || !norm_kind(norm2) || join_sizes(M, N, NGR_F16) != NGR_OK) return 0;
    // (the alignment of the pointers is not known here: the most of the modes)
    size_t most = 0;
    for (int mode : {kJoinAligned, kJoinWindow, kJoinScalar})
        most = std::max(most, join_plan(mode, M, N, rows_per_gate, norm1, norm2).total);
    return most;
}

int ngr_fused_norm_gate_residual_norm_backward(
    int norm1, int norm2, const void *dy, const void *dh, const void *x, const void *residual,
    const void *gate, int64_t rows_per_gate, const void *gamma1, const void *beta1, const void *gamma2,
    const float *stats, float residual_scale, float block_scale, int64_t M, int64_t N, int dtype, void *dx,
    void *dresidual, void *dgate, void *dgamma1, void *dbeta1, void *dgamma2, void *dbeta2, void *workspace,
    size_t workspace_bytes, ngr_stream_t stream_)
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
    JoinArgs a = join_args(x, residual, gate, rows_per_gate, norm1, gamma1, beta1, 0.0f, norm2, gamma2,
                           nullptr, 0.0f, residual_scale, block_scale, M, N);
    int mode = 0;
    rc = join_alignment({dy, dh, x, residual, dx, dresidual},
                        {gate, a.gamma1, a.beta1, a.gamma2, dgate, dgamma1, dbeta1, dgamma2, dbeta2}, N, &mode,
                        &a.shift);
    if (rc != NGR_OK) return rc;
    const JoinPlan p = join_plan(mode, M, N, gate ? rows_per_gate : 0, norm1, norm2);
    if (!workspace || workspace_bytes < p.total) return NGR_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return NGR_ERR_ALIGN;
    if (M > 0 && dresidual == dx) return NGR_ERR_ARG;
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
    a.timeout_ns = wait_timeout_ns();
    a.shape = p.shape;
    a.items = p.items;
    a.item_rows = p.item_rows;
    a.items_per_group = p.items_per_group;
    a.period = p.period;
    a.a_p = p.a_p;
    a.a_q = p.a_q;
    a.a_dgamma2 = p.a_dgamma2;
    a.a_dbeta2 = p.a_dbeta2;
    a.a_dgate = p.a_dgate;
    a.arrays = p.arrays;
    a.fold_gate = p.fold_gate;
    a.item_p = reinterpret_cast<float *>(ws + p.off_p);
    a.item_q = reinterpret_cast<float *>(ws + p.off_q);
    a.cta_sums = reinterpret_cast<float *>(ws + p.off_cta);

    JoinReduce r;
    std::memset(&r, 0, sizeof(r));
    r.p = p.a_p >= 0 ? a.item_p : nullptr;
    r.q = p.a_q >= 0 ? a.item_q : nullptr;
    r.dgamma2_rows = a.cta_sums;
    r.dbeta2_rows = a.cta_sums + static_cast<int64_t>(p.ctas) * N;
    r.dgamma1 = dgamma1;
    r.dbeta1 = dbeta1;
    r.dgamma2 = dgamma2;
    r.dbeta2 = dbeta2;
    r.dgate = p.fold_gate ? nullptr : dgate;
    r.gate = gate;
    r.gamma1 = a.gamma1;
    r.beta1 = a.beta1;
    r.groups = p.groups;
    r.items_per_group = p.items_per_group;
    r.ctas = p.ctas;
    r.pq_rows = static_cast<int>(p.pq_rows);
    r.N = static_cast<int>(N);
    r.block_scale = block_scale;
    r.fold_gate = p.fold_gate;

    const bool bf16 = dtype == NGR_BF16;
    trace("block join gradient", mode, a, p.ctas);
    call_begin();
    kernel_begin(stream);
    rc = launch_join_backward(bf16, mode, a, p.ctas, stream);
    kernel_end(stream);
    if (rc == NGR_OK && (dgamma1 || dbeta1 || dgamma2 || dbeta2 || r.dgate)) {
        kernel_begin(stream);
        rc = launch_join_reduce(bf16, r, stream);
        kernel_end(stream);
    }
    return call_end(rc, workspace, stream);
}

}  // extern "C"
