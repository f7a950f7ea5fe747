// ngr_kv_api.cu -- entry points of the paged key-value cache (ngr_append.cu,
// ngr_attend.cuh): argument checks, workspace layout, how many workers.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <numeric>
#include <utility>

#include "ngr.h"
#include "ngr_entry.h"
#include "ngr_internal.h"
#include "ngr_kv.h"

namespace ngr {

namespace {

constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;
// Units of a call that are several to a thread: as many as the SMs have room
// for threads, twice over.  Four heads a thread against one: 8192 tokens of 80
// heads of 128 64 and 84 us, 2048 tokens of 48 heads 10.5 and 16.6; calls
// below this would leave SMs without a block.
constexpr int64_t kAppendMany = int64_t(2) * 152 * 2048;
// Fewer tiles than this are not worth a worker of their own: one row of 4096
// tokens, 8 key heads: 14.5 us, with 1 15.2, with 4 14.6.
constexpr int64_t kMinShare = 2;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The step of a dimension that may have one entry (any step means the same).
int64_t step(int64_t stride, int64_t entries) { return entries > 1 ? stride : 0; }

int kv_view(const ngr_kv_cache *c, int64_t G, KvView *v)
{
    if (!c || !c->k || !c->v || !c->table) return NGR_ERR_NULL;
    if (c->pages <= 0 || c->pages > kMax31 || c->page_size <= 0 || c->page_size > kMax31 || c->table_rows <= 0 ||
        c->table_rows > kMax31 || c->table_pages <= 0 || c->table_pages > kMax31)
        return NGR_ERR_SHAPE;
    if (!aligned(c->table, 4) || !aligned(c->k, 2) || !aligned(c->v, 2)) return NGR_ERR_ALIGN;
    v->k = c->k;
    v->v = c->v;
    v->k_page = step(c->k_page_stride, c->pages);
    v->k_token = step(c->k_token_stride, c->page_size);
    v->k_head = step(c->k_head_stride, G);
    v->v_page = step(c->v_page_stride, c->pages);
    v->v_token = step(c->v_token_stride, c->page_size);
    v->v_head = step(c->v_head_stride, G);
    // (rows of the table may be parts of wider ones)
    if ((c->table_rows > 1 && c->table_stride < c->table_pages) ||
        (v->k_page | v->k_token | v->k_head | v->v_page | v->v_token | v->v_head) < 0)
        return NGR_ERR_ARG;
    v->table = c->table;
    v->table_stride = c->table_stride;
    v->capacity = c->table_pages * c->page_size;
    v->pages = static_cast<int>(c->pages);
    v->page_size = static_cast<int>(c->page_size);
    v->rows = static_cast<int>(c->table_rows);
    // ceil(2^(31 + s) / page_size) with 2^s the next power of two: exact below 2^31
    v->page_mul = v->page_sh = 0;
    if (c->page_size > 1) {
        int s = 1;
        while ((int64_t(1) << s) < c->page_size) ++s;
        v->page_mul = static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + c->page_size - 1) / c->page_size);
        v->page_sh = static_cast<uint32_t>(s - 1);
    }
    return NGR_OK;
}

// All of a view's 16-byte units, counted from its start, have numbers of 32
// bits, and its last head starts below the largest, which stands for none
// (strides are multiples of 8 elements).
bool within_32(int64_t page, int64_t token, int64_t head, const KvView &v, int64_t G, int64_t D)
{
    const double last = static_cast<double>(page / 8) * (v.pages - 1) + static_cast<double>(token / 8) * (v.page_size - 1) +
                        static_cast<double>(head / 8) * static_cast<double>(G - 1);
    return last < 4294967295.0 && last + static_cast<double>(D / 8) <= 4294967296.0;
}

// Elements that every address of these strides is a multiple of: 8, 4, 2 or 1.
int granule(std::initializer_list<const void *> bases, std::initializer_list<int64_t> steps)
{
    int64_t bits = 8;
    for (const void *p : bases) bits |= static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) >> 1);
    for (int64_t s : steps) bits |= s;
    return static_cast<int>(bits & -bits);
}

// What a tensor occupies: pieces of `bytes`, `count` of them at steps of
// `step` in each dimension (bytes, not negative), the smaller steps first.
struct Places {
    static constexpr int kDims = 3;
    uintptr_t at;
    int64_t bytes, count[kDims], step[kDims];
    int dims = 0;

    // dimensions as {entries, step in elements of `size` bytes}
    Places(const void *p, int64_t piece, int64_t size, std::initializer_list<std::pair<int64_t, int64_t>> of)
        : at(reinterpret_cast<uintptr_t>(p)), bytes(piece * size)
    {
        for (const auto &d : of) {
            if (d.first <= 1 || d.second == 0) continue;
            int i = dims++;
            for (; i > 0 && step[i - 1] > d.second * size; --i) {
                step[i] = step[i - 1];
                count[i] = count[i - 1];
            }
            step[i] = d.second * size;
            count[i] = d.first;
        }
    }
    // from the first byte to behind the last, of the first n dimensions
    int64_t extent(int n) const
    {
        int64_t e = bytes;
        for (int i = 0; i < n; ++i) e += (count[i] - 1) * step[i];
        return e;
    }
    // Every piece lies behind those of smaller steps: none shares a byte with another.
    bool nested() const
    {
        for (int i = 0; i < dims; ++i)
            if (step[i] < extent(i)) return false;
        return true;
    }
};
// Whether two tensors share no byte: one lies behind the other, or what the
// smaller steps span lies apart within a distance that all others are
// multiples of (parts of one array's rows or pages, say).
bool apart(const Places &a, const Places &b)
{
    if (a.at + a.extent(a.dims) <= b.at || b.at + b.extent(b.dims) <= a.at) return true;
    for (int i = a.dims; i >= 0; --i)
        for (int j = b.dims; j >= 0; --j) {
            int64_t period = 0;
            for (int d = i; d < a.dims; ++d) period = std::gcd(period, a.step[d]);
            for (int d = j; d < b.dims; ++d) period = std::gcd(period, b.step[d]);
            if (period == 0) continue;
            const int64_t off = static_cast<int64_t>((b.at % period + period - a.at % period) % period);
            if (off >= a.extent(i) && off + b.extent(j) <= period) return true;
        }
    return false;
}

// Contexts whose items take a CTA each: tiles of each of its warps at most, 6
// or a sixth of the items.  Few items leave SMs idle, but there is no second
// launch and nothing to join.  64 query heads on 8 of 128, alone against
// split, memory's caches flushed: one row of 1000 tokens 16.5 us (split 17.5),
// of 2040 21.7 (17.5); 12 rows of 4000 49 (56), 16 of 2040 36 (46), 16 of
// 4000 61 (71); 16 of 400 to 4000 44 (46); 16 of 100 11 (17).  The longest row
// sets the time, and only the table's room is known here, not the lengths: one
// row of 2000 among 15 of 100 25 us (split 19), of 4000 37.5 (23), of 1500
// among 7 of 50 21 (19).  With longer tables that would cost more than even
// batches gain (one of 8000 tokens 54 us, split 24): they stay split.
constexpr int64_t kSoloTiles = 6, kSoloItems = 6;

struct AttendPlan {
    bool solo;
    int64_t at_once;      // key heads of a launch
    int64_t workers, groups, slots, part_rows, blocks, items;
    size_t flags, jobs, ml, o, total;
};

// The workers that the longest sequences the table has room for keep busy,
// up to every warp of the device.
AttendPlan attend_plan(int64_t B, int64_t H, int64_t G, int64_t D, int64_t capacity, int64_t window)
{
    AttendPlan p;
    std::memset(&p, 0, sizeof(p));
    const int64_t group = H / G;
    const int dim = attend_dim(D), warps = attend_warps(dim, attend_heads(group));
    const int64_t longest = window > 0 ? std::min(window, capacity) : capacity;
    p.blocks = (group + kAttendRows - 1) / kAttendRows;
    // (so many heads that not each can have a worker take several launches)
    p.at_once = std::min(G, std::max<int64_t>(1, kAttendSms * warps / p.blocks));
    p.items = B * p.at_once * p.blocks;
    p.part_rows = std::min<int64_t>(group, kAttendRows);
    const int64_t tiles = (longest + kAttendTile - 1) / kAttendTile;
    p.total = 256;
    // (a block more looks for bad pages)
    p.solo = p.items < kAttendSms && tiles <= std::max(kSoloTiles, p.items / kSoloItems) * warps;
    // Longer tables' batches have a split's workspace all the same, so that one
    // for a batch is enough for smaller batches, which are split.
    if (p.solo && tiles <= kSoloTiles * warps) return p;
    // (a place more for each item: kItemPlaces)
    const double all = static_cast<double>(p.items) * static_cast<double>(tiles + 1);
    const int64_t ctas = all >= static_cast<double>(kAttendSms * kMinShare)
                             ? kAttendSms
                             : std::max<int64_t>(1, (p.items * (tiles + 1) + kMinShare - 1) / kMinShare);
    p.workers = ctas * warps;
    p.groups = p.workers / (p.at_once * p.blocks);
    p.slots = std::min(p.items, p.workers);
    size_t off = 256;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~static_cast<size_t>(255);
        return at;
    };
    p.flags = take(static_cast<size_t>(p.workers) * sizeof(int));
    p.jobs = take(static_cast<size_t>(p.slots) * sizeof(AttendJob));
    p.ml = take(static_cast<size_t>(p.workers) * 2 * p.part_rows * sizeof(float2));
    p.o = take(static_cast<size_t>(p.workers) * 2 * p.part_rows * dim * sizeof(float));
    p.total = off;
    return p;
}

int heads(int64_t H, int64_t G, int64_t D, bool queries)
{
    if (G <= 0 || D <= 0 || D > kAttendMaxDim || G > kMax31) return NGR_ERR_SHAPE;
    if (queries && (H <= 0 || H > kMax31 || H % G != 0)) return NGR_ERR_SHAPE;
    return NGR_OK;
}

int attend_sizes(int64_t B, int64_t H, int64_t G, int64_t D)
{
    const int rc = heads(H, G, D, true);
    if (rc != NGR_OK) return rc;
    if (D % 8 != 0 || B < 0 || B > kMax31 || (B > 0 && H > kMax31 / B)) return NGR_ERR_SHAPE;
    if (H / G > kAttendMaxGroup) return NGR_ERR_SHAPE;
    return NGR_OK;
}

}  // namespace

}  // namespace ngr

using namespace ngr;

extern "C" {

int ngr_fused_rope_append_kv(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                             int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                             int64_t v_head_stride, const ngr_kv_cache *cache, const int32_t *positions,
                             const int32_t *rows, const float *inv_freq, int64_t rot, int interleaved, int64_t T,
                             int64_t H, int64_t G, int64_t D, int dtype, void *q_out, int64_t q_out_token_stride,
                             int64_t q_out_head_stride, void *workspace, size_t workspace_bytes, ngr_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (dtype != NGR_F16 && dtype != NGR_BF16) return NGR_ERR_DTYPE;
    int rc = heads(H, G, D, false);
    if (rc != NGR_OK) return rc;
    if (T < 0 || T > kMax31 || (q && (H <= 0 || H > kMax31))) return NGR_ERR_SHAPE;
    if (rot < 0 || rot > D || rot % 2 != 0) return NGR_ERR_ARG;
    if (workspace && workspace_bytes < NGR_ROPE_APPEND_KV_WORKSPACE) return NGR_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return NGR_ERR_ALIGN;
    if (T == 0) return NGR_OK;
    if (!k || !v || !positions || (rot > 0 && !inv_freq) || (q && !q_out)) return NGR_ERR_NULL;
    AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    rc = kv_view(cache, G, &a.kv);
    if (rc != NGR_OK) return rc;
    if (!rows && cache->table_rows < T) return NGR_ERR_SHAPE;
    if (!aligned(positions, 4) || !aligned(rows, 4) || !aligned(inv_freq, 4)) return NGR_ERR_ALIGN;
    if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(q_out, 2)) return NGR_ERR_ALIGN;
    if (!q) {
        H = 0;
        q_out = nullptr;
    }
    q_token_stride = step(q_token_stride, q ? T : 0);
    q_head_stride = step(q_head_stride, H);
    q_out_token_stride = step(q_out_token_stride, q ? T : 0);
    q_out_head_stride = step(q_out_head_stride, H);
    k_token_stride = step(k_token_stride, T);
    k_head_stride = step(k_head_stride, G);
    v_token_stride = step(v_token_stride, T);
    v_head_stride = step(v_head_stride, G);
    if (q_token_stride < 0 || q_head_stride < 0 || k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 ||
        v_head_stride < 0 || q_out_token_stride < 0 || q_out_head_stride < 0)
        return NGR_ERR_ARG;
    // what is written has a place of its own for every element
    const KvView &kv = a.kv;
    const Places k_cache(kv.k, D, 2, {{G, kv.k_head}, {kv.page_size, kv.k_token}, {kv.pages, kv.k_page}}),
        v_cache(kv.v, D, 2, {{G, kv.v_head}, {kv.page_size, kv.v_token}, {kv.pages, kv.v_page}});
    if ((q && T > 1 && q_out_token_stride == 0) || (H > 1 && q_out_head_stride == 0) || (G > 1 && (kv.k_head == 0 || kv.v_head == 0)) ||
        (kv.page_size > 1 && (kv.k_token == 0 || kv.v_token == 0)) || (kv.pages > 1 && (kv.k_page == 0 || kv.v_page == 0)))
        return NGR_ERR_ARG;
    if (!k_cache.nested() || !v_cache.nested() || !apart(k_cache, v_cache)) return NGR_ERR_ARG;
    if (q) {
        const Places out(q_out, D, 2, {{H, q_out_head_stride}, {T, q_out_token_stride}});
        if (!out.nested()) return NGR_ERR_ARG;
        if (q == q_out) {      // the same elements in the same places
            if (q_token_stride != q_out_token_stride || q_head_stride != q_out_head_stride) return NGR_ERR_ARG;
        } else if (!apart(out, Places(q, D, 2, {{H, q_head_stride}, {T, q_token_stride}})) ||
                   !apart(out, Places(k, D, 2, {{G, k_head_stride}, {T, k_token_stride}})) ||
                   !apart(out, Places(v, D, 2, {{G, v_head_stride}, {T, v_token_stride}}))) {
            return NGR_ERR_ARG;
        }
    }
    int vec = granule({q, k, v, q_out, a.kv.k, a.kv.v},
                      {D, q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                       q_out_token_stride, q_out_head_stride, a.kv.k_page, a.kv.k_token, a.kv.k_head, a.kv.v_page,
                       a.kv.v_token, a.kv.v_head});
    vec = std::min(vec, granule({}, {interleaved ? rot : rot / 2, interleaved ? 0 : rot}));
    int sms = 0;
    rc = device_sms(&sms);
    if (rc != NGR_OK) return rc;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.qo_token = q_out_token_stride;
    a.qo_head = q_out_head_stride;
    a.positions = positions;
    a.rows = rows;
    a.inv_freq = inv_freq;
    a.err = static_cast<int *>(workspace);
    a.T = static_cast<int>(T);
    a.H = static_cast<int>(H);
    a.G = static_cast<int>(G);
    a.D = static_cast<int>(D);
    a.rot = static_cast<int>(rot);
    // Few tokens spread over as many blocks as they fill; of many a thread
    // takes several heads, whose loads are under way together and whose
    // angles are the same.
    const int64_t all = H + 2 * G;
    a.units = append_units(vec, interleaved != 0, D, rot);
    if (all > kMax31 / 256) return NGR_ERR_SHAPE;
    a.each = all * a.units * T >= kAppendMany ? kAppendEach : 1;
    const int64_t at_once = (kAppendThreads / a.units) * a.each, blocks = (all + at_once - 1) / at_once;
    if (blocks > (kMax31 - 1) / T) return NGR_ERR_SHAPE;
    a.blocks_per_token = static_cast<int>(blocks);
    a.threads = static_cast<int>((all + blocks * a.each - 1) / (blocks * a.each)) * a.units;
    if (trace_mode())
        std::fprintf(stderr, "ngr: rotated append T=%d H=%d G=%d D=%d rot=%d%s page=%d elements at once=%d blocks a token=%d\n",
                     a.T, a.H, a.G, a.D, a.rot, interleaved ? " interleaved" : "", a.kv.page_size, vec, a.blocks_per_token);
    call_begin();
    kernel_begin(stream);
    rc = launch_append(dtype == NGR_BF16, vec, interleaved != 0, a, stream);
    kernel_end(stream);
    return call_end(rc, workspace, stream);
}

size_t ngr_paged_attention_workspace_bytes(int64_t B, int64_t H, int64_t G, int64_t D, int64_t capacity,
                                           int64_t window)
{
    if (attend_sizes(B, H, G, D) != NGR_OK || capacity <= 0 || window < 0) return 0;
    return attend_plan(B, H, G, D, std::min(capacity, kMax31), window).total;
}

int ngr_fused_paged_attention(const void *q, int64_t q_row_stride, int64_t q_head_stride, const ngr_kv_cache *cache,
                              const int32_t *lengths, float scale, int64_t window, int64_t B, int64_t H, int64_t G,
                              int64_t D, int dtype, void *out, float *lse, void *workspace, size_t workspace_bytes,
                              ngr_stream_t stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (dtype != NGR_F16 && dtype != NGR_BF16) return NGR_ERR_DTYPE;
    int rc = attend_sizes(B, H, G, D);
    if (rc != NGR_OK) return rc;
    const float scale2 = scale * 1.4426950408889634f;      // of exponents of 2
    if (!std::isfinite(scale2) || window < 0) return NGR_ERR_ARG;
    if (B == 0) return NGR_OK;
    if (!q || !lengths || !out) return NGR_ERR_NULL;
    AttendArgs a;
    std::memset(&a, 0, sizeof(a));
    rc = kv_view(cache, G, &a.kv);
    if (rc != NGR_OK) return rc;
    if (cache->table_rows < B) return NGR_ERR_SHAPE;
    q_row_stride = step(q_row_stride, B);
    q_head_stride = step(q_head_stride, H);
    if (q_row_stride < 0 || q_head_stride < 0) return NGR_ERR_ARG;
    if (!aligned(lengths, 4) || !aligned(lse, 4) || !aligned(out, 16) ||
        granule({q, a.kv.k, a.kv.v}, {q_row_stride, q_head_stride, a.kv.k_page, a.kv.k_token, a.kv.k_head, a.kv.v_page,
                                      a.kv.v_token, a.kv.v_head}) != 8)
        return NGR_ERR_ALIGN;
    // Each query is read by its own item's warps, which then write its place
    // in out: in q's memory only where both lie alike.
    const Places q_at(q, D, 2, {{H, q_head_stride}, {B, q_row_stride}}), out_at(out, B * H * D, 2, {}), lse_at(lse, B * H, 4, {});
    const bool in_place = q == out && (H == 1 || q_head_stride == D) && (B == 1 || q_row_stride == H * D);
    if (!in_place && !apart(q_at, out_at)) return NGR_ERR_ARG;
    if (lse && (!apart(q_at, lse_at) || !apart(out_at, lse_at))) return NGR_ERR_ARG;
    if (!within_32(a.kv.k_page, a.kv.k_token, a.kv.k_head, a.kv, G, D) ||
        !within_32(a.kv.v_page, a.kv.v_token, a.kv.v_head, a.kv, G, D))
        return NGR_ERR_SHAPE;
    a.k_page = static_cast<uint32_t>(a.kv.k_page / 8);
    a.k_token = static_cast<uint32_t>(a.kv.k_token / 8);
    a.k_head = static_cast<uint32_t>(a.kv.k_head / 8);
    a.v_page = static_cast<uint32_t>(a.kv.v_page / 8);
    a.v_token = static_cast<uint32_t>(a.kv.v_token / 8);
    a.v_head = static_cast<uint32_t>(a.kv.v_head / 8);
    a.alike = a.k_page == a.v_page && a.k_token == a.v_token && a.k_head == a.v_head;
    const AttendPlan p = attend_plan(B, H, G, D, std::min(a.kv.capacity, kMax31), window);
    if (!workspace || workspace_bytes < p.total) return NGR_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return NGR_ERR_ALIGN;
    int sms = 0;
    rc = device_sms(&sms);
    if (rc != NGR_OK) return rc;
    char *ws = static_cast<char *>(workspace);
    a.q = q;
    a.q_row = q_row_stride;
    a.q_head = q_head_stride;
    a.lengths = lengths;
    a.out = out;
    a.lse = lse;
    a.scale2 = scale2;
    a.window = static_cast<int>(std::min(window, kMax31));
    a.B = static_cast<int>(B);
    a.H = static_cast<int>(H);
    a.D = static_cast<int>(D);
    a.group = static_cast<int>(H / G);
    a.blocks = static_cast<int>(p.blocks);
    a.workers = static_cast<int>(p.workers);
    a.groups = static_cast<int>(p.groups);
    a.min_share = static_cast<int>(kMinShare);
    a.part_rows = static_cast<int>(p.part_rows);
    a.flags = reinterpret_cast<int *>(ws + p.flags);
    a.jobs = reinterpret_cast<AttendJob *>(ws + p.jobs);
    a.part_ml = reinterpret_cast<float2 *>(ws + p.ml);
    a.part_o = reinterpret_cast<float *>(ws + p.o);
    a.err = reinterpret_cast<int *>(ws);
    if (trace_mode())
        std::fprintf(stderr, "ngr: paged attention B=%d H=%d G=%d D=%d page=%d window=%d dim=%d %s=%d jobs=%d\n", a.B, a.H,
                     static_cast<int>(G), a.D, a.kv.page_size, a.window, attend_dim(D), p.solo ? "items" : "workers",
                     p.solo ? static_cast<int>(p.items) : a.workers, static_cast<int>(p.slots));
    const bool bf16 = dtype == NGR_BF16;
    call_begin();
    for (int64_t g = 0; g < G && rc == NGR_OK; g += p.at_once) {
        a.G = static_cast<int>(std::min(p.at_once, G - g));
        a.q = static_cast<const uint16_t *>(q) + g * a.group * q_head_stride;
        a.kv.k = static_cast<uint16_t *>(const_cast<void *>(cache->k)) + g * a.kv.k_head;
        a.kv.v = static_cast<uint16_t *>(const_cast<void *>(cache->v)) + g * a.kv.v_head;
        a.out = static_cast<uint16_t *>(out) + g * a.group * D;
        a.lse = lse ? lse + g * a.group : nullptr;
        a.slots = static_cast<int>(std::min(B * a.G * p.blocks, p.workers));
        a.slot_by_item = B * a.G * p.blocks <= p.workers;
        a.err_keep = g > 0;
        kernel_begin(stream);
        rc = p.solo ? (bf16 ? launch_attend_solo_bf16(a, stream) : launch_attend_solo_f16(a, stream))
                    : (bf16 ? launch_attend_bf16(a, stream) : launch_attend_f16(a, stream));
        kernel_end(stream);
        if (rc == NGR_OK && !p.solo) {
            kernel_begin(stream);
            rc = bf16 ? launch_attend_join_bf16(a, stream) : launch_attend_join_f16(a, stream);
            kernel_end(stream);
        }
    }
    return call_end(rc, workspace, stream);
}

}  // extern "C"
