// ngr_ce_api.cu -- entry points of the linear cross entropy (ngr_ce.cu,
// ngr_ce_gemm.cu): argument checks, workspace layout, the pieces of the
// vocabulary.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "ngr.h"
#include "ngr_ce.h"
#include "ngr_entry.h"
#include "ngr_internal.h"

namespace ngr {

namespace {

constexpr int64_t kMaxDim31 = int64_t(1) << 31;
// dz of one piece of the vocabulary takes at most this much memory (unless a
// piece of kMinPiece entries needs more): large enough that a piece's
// products fill the GPU for hundreds of microseconds.
constexpr int64_t kPieceBytes = int64_t(256) << 20;
constexpr int64_t kMinPiece = 4096;
// CTA pairs a GB300 runs at once; sizing must not ask a device.
constexpr int64_t kPairs = 76;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t up_to(int64_t v, int64_t n) { return (v + n - 1) / n * n; }

// Columns of the tiles of z (rows x cols): the width, a multiple of 32, at
// which the CTA pairs are busiest, a tile counted as kTileCost columns more.
constexpr int64_t kTileCost = 32;
int tile_width(int64_t rows, int64_t cols)
{
    const int64_t m = (std::max<int64_t>(rows, 1) + kCeTile - 1) / kCeTile;
    int best = kCeTile;
    int64_t least = 0;
    for (int w = kCeTile; w >= 128; w -= 32) {
        const int64_t cost = (m * ((cols + w - 1) / w) + kPairs - 1) / kPairs * (w + kTileCost);
        if (least == 0 || cost < least) {
            least = cost;
            best = w;
        }
    }
    return best;
}

// Few output tiles of dx: the vocabulary is cut into ranges whose sums are
// added afterwards.  The number of ranges that leaves the busiest pair the
// least k blocks, a tile counted as kSplitCost k blocks more (its epilogue
// and first loads), and the sums' way to memory and back (8 bytes an element
// of dx and range) as one k block for 2 MB; at least 8 k blocks a range.
constexpr int64_t kSplitCost = 12;
int64_t dx_splits(int64_t tiles, int64_t k_blocks, int64_t elements)
{
    if (tiles >= 8 * kPairs) return 1;
    int64_t best = 1, least = 0;
    for (int64_t s = 1; s <= 32 && (s == 1 || k_blocks / s >= 8); ++s) {
        const int64_t cost = (tiles * s + kPairs - 1) / kPairs * ((k_blocks + s - 1) / s + kSplitCost) +
                             (s > 1 ? s * elements / 250000 : 0);
        if (least == 0 || cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

struct CePlan {
    int64_t K8, Kx, w_pitch, piece, pieces, splits, parts;
    bool finish;
    size_t info, index, ctarget, xc, wp, row, part, z_target, dz, sums, total;
};

CePlan ce_plan(bool backward, int64_t M, int64_t K, int64_t V)
{
    CePlan p;
    std::memset(&p, 0, sizeof(p));
    p.K8 = up_to(K, 8);
    p.Kx = up_to(K, kBK);
    size_t off = 256;   // error word
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~static_cast<size_t>(255);
        return at;
    };
    p.info = take(sizeof(CeInfo));
    p.index = take(static_cast<size_t>(M) * 4);
    p.ctarget = take(static_cast<size_t>(M) * 4);
    p.xc = take(static_cast<size_t>(up_to(std::max<int64_t>(M, 1), 64)) * p.Kx * 2);
    p.w_pitch = K % 8 == 0 ? K : p.Kx;
    if (K % 8 != 0) p.wp = take(static_cast<size_t>(V) * p.w_pitch * 2);
    if (!backward) {
        const int64_t w = tile_width(M, V);
        p.parts = (V + w - 1) / w * 2;
        p.part = take(static_cast<size_t>(p.parts) * M * sizeof(float2));
        p.z_target = take(static_cast<size_t>(M) * 4);
    } else {
        const int64_t rows = up_to(std::max<int64_t>(M, 1), kCeTile);
        int64_t most = std::max(kMinPiece, kPieceBytes / (2 * rows) / kCeTile * kCeTile);
        p.pieces = (V + most - 1) / most;
        p.piece = up_to((V + p.pieces - 1) / p.pieces, kCeTile);
        p.pieces = (V + p.piece - 1) / p.piece;
        p.row = take(static_cast<size_t>(rows) * sizeof(CeRow));
        p.dz = take(static_cast<size_t>(rows) * p.piece * 2);
        p.splits = dx_splits(rows / kCeTile * ((K + kCeTile - 1) / kCeTile), p.piece / kBK, M * K);
        // dx itself is written by the last piece's product where its rows take
        // 16-byte pieces and nothing is left to add.
        p.finish = p.splits == 1 && K % 8 == 0;
        if (!p.finish || p.pieces > 1)
            p.sums = take(static_cast<size_t>(p.splits) * M * p.Kx * sizeof(float));
    }
    p.total = off;
    return p;
}

int ce_sizes(int64_t M, int64_t K, int64_t V, int dtype)
{
    if (dtype != NGR_F16 && dtype != NGR_BF16) return NGR_ERR_DTYPE;
    if (M < 0 || K <= 0 || V <= 0 || M >= kMaxDim31 || K >= kMaxDim31 || V >= kMaxDim31) return NGR_ERR_SHAPE;
    return NGR_OK;
}

struct CeCall {
    CeTokens t;
    CePlan p;
    char *ws;
    const void *W;   // rows of K8 elements, w_pitch apart
    bool bf16;
    cudaStream_t stream;
};

// What forward and backward have in common: checks of the workspace, the
// tokens' arguments, W with rows of a 16-byte pitch (a call's first launch).
int ce_begin(CeCall *c, bool backward, const void *x, const void *W, const int64_t *target, float logit_scale,
             int64_t M, int64_t K, int64_t V, int dtype, void *workspace, size_t workspace_bytes)
{
    if (!std::isfinite(logit_scale)) return NGR_ERR_ARG;
    if (!aligned(x, 2) || !aligned(W, K % 8 == 0 ? 16 : 2) || !aligned(target, 8)) return NGR_ERR_ALIGN;
    c->p = ce_plan(backward, M, K, V);
    if (!workspace || workspace_bytes < c->p.total) return NGR_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return NGR_ERR_ALIGN;
    int sms = 0;
    const int rc = device_sms(&sms);
    if (rc != NGR_OK) return rc;
    char *ws = static_cast<char *>(workspace);
    c->ws = ws;
    c->bf16 = dtype == NGR_BF16;
    c->W = K % 8 == 0 ? W : ws + c->p.wp;
    CeTokens &t = c->t;
    t.x = x;
    t.target = target;
    t.logit_scale = logit_scale;
    t.M = M;
    t.K = K;
    t.V = V;
    t.K8 = c->p.K8;
    t.Kx = c->p.Kx;
    t.info = reinterpret_cast<CeInfo *>(ws + c->p.info);
    t.err = reinterpret_cast<int *>(ws);
    t.index = reinterpret_cast<int *>(ws + c->p.index);
    t.ctarget = reinterpret_cast<int *>(ws + c->p.ctarget);
    t.xc = ws + c->p.xc;
    call_begin();
    if (K % 8 == 0) return NGR_OK;
    kernel_begin(c->stream);
    const int pad = launch_ce_pad(W, ws + c->p.wp, V, K, c->p.w_pitch, c->stream);
    kernel_end(c->stream);
    return pad == NGR_OK ? NGR_OK : call_end(pad, nullptr, c->stream);
}

CeGemmArgs ce_args(const CeCall &c)
{
    CeGemmArgs a;
    std::memset(&a, 0, sizeof(a));
    a.info = c.t.info;
    a.err = c.t.err;
    a.timeout_ns = wait_timeout_ns();
    a.scale = c.t.logit_scale;
    a.scale2 = c.t.logit_scale * 1.4426950408889634f;
    a.splits = 1;
    a.width = kCeTile;
    return a;
}

int64_t tiles_of(int64_t rows, int64_t cols, int64_t width = kCeTile)
{
    return (std::max<int64_t>(rows, 1) + kCeTile - 1) / kCeTile * ((cols + width - 1) / width);
}

#define NGR_TIMED(CALL)          \
    do {                         \
        kernel_begin(stream);    \
        rc = (CALL);             \
        kernel_end(stream);      \
        if (rc != NGR_OK) return call_end(rc, nullptr, stream); \
    } while (0)

int ce_forward(const void *x, const void *W, const int64_t *target, float logit_scale, int64_t M, int64_t K,
               int64_t V, int dtype, float *loss, float *lse, void *workspace, size_t workspace_bytes,
               cudaStream_t stream)
{
    int rc = ce_sizes(M, K, V, dtype);
    if (rc != NGR_OK) return rc;
    if (M == 0) return NGR_OK;
    if (!x || !W || !target || !loss || !lse) return NGR_ERR_NULL;
    if (!aligned(loss, 4) || !aligned(lse, 4)) return NGR_ERR_ALIGN;
    CeCall c;
    std::memset(&c, 0, sizeof(c));
    c.stream = stream;
    rc = ce_begin(&c, false, x, W, target, logit_scale, M, K, V, dtype, workspace, workspace_bytes);
    if (rc != NGR_OK) return rc;
    CeGemmArgs a = ce_args(c);
    a.width = tile_width(M, V);
    if (!map_2d(&a.map_a, c.t.xc, c.bf16, up_to(M, 64), c.t.Kx, kBM) ||
        !map_2d_pitch(&a.map_b, c.W, c.bf16, V, c.t.K8, static_cast<uint32_t>(a.width / 2), c.p.w_pitch))
        return NGR_ERR_CUDA;
    a.cols = static_cast<int>(V);
    a.depth = static_cast<int>(c.t.K8);
    a.target = c.t.ctarget;
    a.part = reinterpret_cast<float2 *>(c.ws + c.p.part);
    a.part_pitch = M;
    a.z_target = reinterpret_cast<float *>(c.ws + c.p.z_target);
    if (launch_ce_index_apart(c.t)) NGR_TIMED(launch_ce_index(c.t, stream));
    NGR_TIMED(launch_ce_gather(c.t, stream));
    NGR_TIMED(launch_ce_gemm(kCeLse, c.bf16, a, tiles_of(M, V, a.width), stream));
    NGR_TIMED(launch_ce_loss(c.t, a.part, M, static_cast<int>(c.p.parts), a.z_target, loss, lse, stream));
    return call_end(rc, workspace, stream);
}

int ce_backward(const float *dloss, const float *dlse, const float *lse, const void *x, const void *W,
                const int64_t *target, float logit_scale, int64_t M, int64_t K, int64_t V, int dtype, void *dx,
                void *dW, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    int rc = ce_sizes(M, K, V, dtype);
    if (rc != NGR_OK) return rc;
    if (!dx && !dW) return NGR_ERR_NULL;
    if (M > 0 && (!x || !W || !target || !lse || (!dloss && !dlse))) return NGR_ERR_NULL;
    if (!aligned(dx, 2) || !aligned(dW, 2) || !aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dlse, 4))
        return NGR_ERR_ALIGN;
    CeCall c;
    std::memset(&c, 0, sizeof(c));
    c.stream = stream;
    if (M == 0) {   // an empty sum
        if (!dW) return NGR_OK;
        int sms = 0;
        rc = device_sms(&sms);
        if (rc != NGR_OK) return rc;
        const cudaError_t e = cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * K * 2, stream);
        return e == cudaSuccess ? NGR_OK : record_cuda_error("cudaMemsetAsync (dW)", e, cudaGetErrorString(e));
    }
    c.t.dloss = dloss;
    c.t.dlse = dlse;
    c.t.lse = lse;
    c.t.dx = dx;
    rc = ce_begin(&c, true, x, W, target, logit_scale, M, K, V, dtype, workspace, workspace_bytes);
    if (rc != NGR_OK) return rc;
    c.t.row = reinterpret_cast<CeRow *>(c.ws + c.p.row);
    if (launch_ce_index_apart(c.t)) NGR_TIMED(launch_ce_index(c.t, stream));
    NGR_TIMED(launch_ce_gather(c.t, stream));
    const int64_t rows = up_to(M, kCeTile);
    char *dz = c.ws + c.p.dz;
    float *sums = reinterpret_cast<float *>(c.ws + c.p.sums);
    for (int64_t i = 0; i < c.p.pieces; ++i) {
        const int64_t v0 = i * c.p.piece, n = std::min(c.p.piece, V - v0);
        const char *Wi = static_cast<const char *>(c.W) + v0 * c.p.w_pitch * 2;
        CeGemmArgs a = ce_args(c);
        a.width = tile_width(M, n);
        if (!map_2d(&a.map_a, c.t.xc, c.bf16, up_to(M, 64), c.t.Kx, kBM) ||
            !map_2d_pitch(&a.map_b, Wi, c.bf16, n, c.t.K8, static_cast<uint32_t>(a.width / 2), c.p.w_pitch))
            return NGR_ERR_CUDA;
        a.cols = static_cast<int>(n);
        a.depth = static_cast<int>(c.t.K8);
        a.v0 = static_cast<int>(v0);
        a.row = c.t.row;
        a.out = dz;
        a.pitch = c.p.piece;
        NGR_TIMED(launch_ce_gemm(kCeGrad, c.bf16, a, tiles_of(M, n, a.width), stream));
        if (dx) {
            a = ce_args(c);
            if (!map_2d_pitch(&a.map_a, dz, c.bf16, rows, n, kBM, c.p.piece) ||
                !map_2d_pitch(&a.map_b, Wi, c.bf16, n, c.t.K8, kBK, c.p.w_pitch))
                return NGR_ERR_CUDA;
            a.cols = static_cast<int>(K);
            a.depth = static_cast<int>(n);
            a.splits = static_cast<int>(c.p.splits);
            a.sums = sums;
            a.sums_rows = M;
            a.sums_pitch = c.p.Kx;
            a.add = i > 0;
            a.finish = i == c.p.pieces - 1 && c.p.finish;
            a.out = dx;
            a.pitch = K;
            a.index = c.t.index;
            NGR_TIMED(launch_ce_gemm(kCeDx, c.bf16, a, tiles_of(M, K) * c.p.splits, stream));
        }
        if (dW) {
            a = ce_args(c);
            if (!map_2d_pitch(&a.map_a, dz, c.bf16, rows, n, kBK, c.p.piece) ||
                !map_2d(&a.map_b, c.t.xc, c.bf16, up_to(M, 64), c.t.Kx, kBK))
                return NGR_ERR_CUDA;
            a.rows = static_cast<int>(n);
            a.cols = static_cast<int>(K);
            a.out = static_cast<char *>(dW) + v0 * K * 2;
            a.pitch = K;
            a.after_dx = dx != nullptr;
            a.boxes = K % 8 == 0 && aligned(dW, 16);
            if (a.boxes && !map_2d(&a.map_out, a.out, c.bf16, n, K, 32)) return NGR_ERR_CUDA;
            NGR_TIMED(launch_ce_gemm(kCeDw, c.bf16, a, tiles_of(n, K), stream));
        }
    }
    if (dx && !c.p.finish)
        NGR_TIMED(launch_ce_dx(c.bf16, c.t, sums, c.p.Kx, static_cast<int>(c.p.splits), stream));
    return call_end(rc, workspace, stream);
}

}  // namespace

}  // namespace ngr

using namespace ngr;

extern "C" {

size_t ngr_linear_cross_entropy_workspace_bytes(int backward, int64_t M, int64_t K, int64_t V)
{
    if (ce_sizes(M, K, V, NGR_F16) != NGR_OK) return 0;
    return ce_plan(backward != 0, M, K, V).total;
}

int ngr_fused_linear_cross_entropy(const void *x, const void *W, const int64_t *target, float logit_scale,
                                   int64_t M, int64_t K, int64_t V, int dtype, float *loss, float *lse,
                                   void *workspace, size_t workspace_bytes, ngr_stream_t stream)
{
    return ce_forward(x, W, target, logit_scale, M, K, V, dtype, loss, lse, workspace, workspace_bytes,
                      reinterpret_cast<cudaStream_t>(stream));
}

int ngr_fused_linear_cross_entropy_backward(const float *dloss, const float *dlse, const float *lse,
                                            const void *x, const void *W, const int64_t *target,
                                            float logit_scale, int64_t M, int64_t K, int64_t V, int dtype,
                                            void *dx, void *dW, void *workspace, size_t workspace_bytes,
                                            ngr_stream_t stream)
{
    return ce_backward(dloss, dlse, lse, x, W, target, logit_scale, M, K, V, dtype, dx, dW, workspace,
                       workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
