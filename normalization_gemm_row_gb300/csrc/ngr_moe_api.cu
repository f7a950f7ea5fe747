// ngr_moe_api.cu -- entry point of the mixture-of-experts layer for a few
// tokens (ngr_moe.cu): argument checks, workspace layout, launch sizes.
#include <algorithm>
#include <cstdio>
#include <cstring>

#include "ngr.h"
#include "ngr_entry.h"
#include "ngr_internal.h"
#include "ngr_moe.h"

namespace ngr {

namespace {

static_assert(NGR_MOE_MAX_M == kMoeMaxTokens && NGR_MOE_MAX_EXPERTS == kMoeMaxExperts && NGR_MOE_MAX_TOP_K == kMoeMaxTopK,
              "ngr.h and the kernels agree");

// More experts than this take clusters of 16 CTAs in the router, if the tokens
// are few enough for each CTA to have an SM: 8 tokens, 512 experts 118 us with
// 16, 122.7 with 8; 128 experts 97 and 98.5; one token, 256 experts of 7168 x
// 2048 142 and 146; but 32 tokens, 512 experts 331 and 323.5; 12 tokens, 128
// experts 131 and 129.
constexpr int64_t kMoeManyExperts = 64, kMoeFewTokens = 9;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Whether two arrays share no byte (a null one does not).
bool apart(const void *p, size_t p_bytes, const void *q, size_t q_bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return !p || !q || a + p_bytes <= b || b + q_bytes <= a;
}
int64_t up_to(int64_t v, int64_t n) { return (v + n - 1) / n * n; }

int moe_sizes(int64_t M, int64_t K, int64_t F, int64_t E, int64_t top_k)
{
    if (M < 0 || M > NGR_MOE_MAX_M || K <= 0 || K > NGR_MOE_MAX_WIDTH || F <= 0 || F > NGR_MOE_MAX_WIDTH || E <= 0 || E > NGR_MOE_MAX_EXPERTS ||
        top_k <= 0 || top_k > E || top_k > NGR_MOE_MAX_TOP_K)
        return NGR_ERR_SHAPE;
    return NGR_OK;
}

struct MoePlan {
    size_t ids, w, a, h, parts, counters, total;
    int64_t Kp, Fp, part_bytes;
    int groups;
};

MoePlan moe_plan(int64_t M, int64_t K, int64_t F, int64_t E, int64_t top_k)
{
    MoePlan p;
    p.Kp = up_to(K, 64);
    p.Fp = up_to(F, 64);
    size_t off = 256;
    auto take = [&](int64_t bytes) {
        const size_t at = off;
        off += (static_cast<size_t>(bytes) + 255) & ~static_cast<size_t>(255);
        return at;
    };
    p.ids = take(M * top_k * 4);
    p.w = take(M * top_k * 4);
    p.a = take(M * 2 * p.Kp * 2);
    p.h = take(M * top_k * 2 * p.Fp * 2);
    p.groups = moe_groups(M, E, top_k);
    p.part_bytes = std::max<int64_t>(p.groups * 256, M * 64);
    p.parts = take(static_cast<int64_t>(kMoeWorkers) * 2 * p.part_bytes);
    p.counters = take(kMoeCounters * 4);
    p.total = off;
    return p;
}

}  // namespace

}  // namespace ngr

using namespace ngr;

extern "C" {

size_t ngr_moe_swiglu_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t E, int64_t top_k)
{
    if (moe_sizes(M, K, F, E, top_k) != NGR_OK) return 0;
    return moe_plan(M, K, F, E, top_k).total;
}

int ngr_fused_moe_swiglu(int norm, const void *x, const void *gamma, const void *beta, const void *Wr, const void *Wg,
                         const void *Wu, const void *Wd, float eps, int64_t top_k, int renormalize, int64_t M, int64_t K,
                         int64_t F, int64_t E, int dtype, void *y, int32_t *experts, float *weights, void *workspace,
                         size_t workspace_bytes, ngr_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (dtype != NGR_F16 && dtype != NGR_BF16) return NGR_ERR_DTYPE;
    if (norm != NGR_NORM_NONE && norm != NGR_NORM_LAYER && norm != NGR_NORM_RMS) return NGR_ERR_ARG;
    int rc = moe_sizes(M, K, F, E, top_k);
    if (rc != NGR_OK) return rc;
    if (norm != NGR_NORM_NONE && !(eps >= 0.0f)) return NGR_ERR_ARG;
    if (M == 0) return NGR_OK;
    if (!x || !Wr || !Wg || !Wu || !Wd || !y || (norm != NGR_NORM_NONE && !gamma) || (norm == NGR_NORM_LAYER && !beta))
        return NGR_ERR_NULL;
    for (const void *p : {x, gamma, beta, Wr, Wg, Wu, Wd, static_cast<const void *>(y)})
        if (!aligned(p, 2)) return NGR_ERR_ALIGN;
    if (!aligned(experts, 4) || !aligned(weights, 4)) return NGR_ERR_ALIGN;
    // x is read to its end before y is written, but while the choice is; what
    // is returned is apart from one another.
    const size_t rows = static_cast<size_t>(M * K) * 2, choices = static_cast<size_t>(M * top_k) * 4;
    if (!apart(experts, choices, x, rows) || !apart(weights, choices, x, rows) || !apart(experts, choices, y, rows) ||
        !apart(weights, choices, y, rows) || !apart(experts, choices, weights, choices))
        return NGR_ERR_ARG;
    const MoePlan p = moe_plan(M, K, F, E, top_k);
    if (!workspace || workspace_bytes < p.total) return NGR_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return NGR_ERR_ALIGN;
    int sms = 0;
    rc = device_sms(&sms);
    if (rc != NGR_OK) return rc;
    char *ws = static_cast<char *>(workspace);
    MoeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.gamma = norm != NGR_NORM_NONE ? gamma : nullptr;
    a.beta = norm == NGR_NORM_LAYER ? beta : nullptr;
    a.Wr = Wr;
    a.Wg = Wg;
    a.Wu = Wu;
    a.Wd = Wd;
    a.y = y;
    a.experts = experts;
    a.weights = weights;
    a.ids = reinterpret_cast<int *>(ws + p.ids);
    a.w = reinterpret_cast<float *>(ws + p.w);
    a.a = ws + p.a;
    a.h = ws + p.h;
    a.parts = reinterpret_cast<float *>(ws + p.parts);
    a.part_bytes = static_cast<int>(p.part_bytes);
    a.groups = p.groups;
    a.counters = reinterpret_cast<int *>(ws + p.counters);
    a.err = reinterpret_cast<int *>(ws);
    a.norm = norm;
    a.M = static_cast<int>(M);
    a.K = static_cast<int>(K);
    a.F = static_cast<int>(F);
    a.E = static_cast<int>(E);
    a.top_k = static_cast<int>(top_k);
    a.renormalize = renormalize != 0;
    a.Kp = static_cast<int>(p.Kp);
    a.Fp = static_cast<int>(p.Fp);
    a.eps = eps;
    a.router = E > kMoeManyExperts && M <= kMoeFewTokens ? 16 : 8;
    const bool bf16 = dtype == NGR_BF16;
    const bool vec_r = K % 8 == 0 && aligned(Wr, 16) && aligned(x, 16) && aligned(a.gamma, 16) && aligned(a.beta, 16);
    const bool vec_k = K % 8 == 0 && aligned(Wg, 16) && aligned(Wu, 16);
    const bool vec_f = F % 8 == 0 && aligned(Wd, 16);
    if (trace_mode())
        std::fprintf(stderr, "ngr: experts M=%d K=%d F=%d E=%d top_k=%d norm=%d groups=%d%s%s\n",
                     a.M, a.K, a.F, a.E, a.top_k, norm, a.groups, vec_k ? "" : ", gate and up shifted",
                     vec_f ? "" : ", down shifted");
    call_begin();
    kernel_begin(stream);
    rc = launch_moe_router(bf16, vec_r, a, stream);
    kernel_end(stream);
    if (rc == NGR_OK) {
        kernel_begin(stream);
        rc = launch_moe_up(bf16, vec_k, a, stream);
        kernel_end(stream);
    }
    if (rc == NGR_OK) {
        kernel_begin(stream);
        rc = launch_moe_down(bf16, vec_f, a, stream);
        kernel_end(stream);
    }
    return call_end(rc, workspace, stream);
}

}  // extern "C"
