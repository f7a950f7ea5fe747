// ngr_attend.cuh -- attention of one new token for each sequence over a paged
// key-value cache.
//
//   s_j = scale q . k_j,  lse = log sum_j exp s_j,  out = sum_j exp(s_j - lse) v_j
//
// A key or value read serves the H / G query heads of its head: 2 H / G
// operations a byte, so reading the cache bounds it.  The cache is streamed
// once, by warps: each has a ring of stages in shared memory that
// asynchronous copies of 16 tokens' keys and values fill, and takes them with
// 16 x 8 x 16 matrix instructions, tokens (then dimensions) as the rows and 8
// query heads as the columns, with a running maximum and sum.  (With heads as
// rows, 8 heads would leave half of every instruction and of its registers
// unused.)  The warps have nothing to wait for but their own copies: no
// barrier.
//
// The sequences' tiles of 16 tokens stand in one row, with a place more before
// each sequence for what its beginning costs, and the row is cut into equal
// runs.  A group of warps ("workers") takes a run, a warp for each key head
// (and block of 16 query heads where there are more).  A batch of any lengths
// is balanced so, and nothing but the device has to know the lengths; and what
// is read at a time lies together: the heads of a token share lines of L2 (64
// rows of 8000 tokens, 8 key heads of 80: 215 us; with the items' tiles in one
// row, head after head, 329, as much as with 128 dimensions).  An item (a
// sequence and key head) that lies in one run is finished there; the others'
// parts (FP32 sums, maximum, sum of exponentials) are joined by a second kernel
// in the tokens' order, so a call repeated gives the same bits.
//
// Few items of short contexts take a CTA each ("solo"): its warps share the
// item's tiles and join their parts in shared memory, without a second launch.
//
// Scores, maxima, exponentials and sums are FP32.  A softmax weight goes into
// its product with v in two parts of the inputs' type, and a tile's products
// are added to the sums by rounding additions, not by the instruction's own
// long chain.
//
// bf16, 64 query heads on 8 of 128: 64 rows of 2048 to 8192 tokens 213 us (6.3
// TB/s), one of 131072 tokens 95 us (5.6 TB/s, of which 7 are the join), one
// of 1000 tokens 14 us.
#pragma once

#include "ngr.h"
#include "ngr_entry.h"
#include "ngr_internal.h"
#include "ngr_kv.h"
#include "ngr_mma.cuh"
#include "ngr_ptx.cuh"

#include <type_traits>

namespace ngr {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
// What the softmax weights are multiplied by for their product with v, and the
// sums divided by in the end.  A weight is at most 1, of the run's largest: in
// fp16 those below 2^-14 would be subnormal and those below 2^-25 gone, while
// the sum of the exponentials counts them (27000 tokens at e^-17.3 of one of
// weight 1: 1.6e-3 in their place of 8.3e-4).  Times 2^15 all are normal from
// 2^-29 on.
template <bool BF16>
constexpr float kWeightScale = BF16 ? 1.0f : 32768.0f;

// A warp's ring: stages of 16 tokens' keys or values in turn, 192 KB over the
// CTA's warps.
template <int DP, int NB>
struct Ring {
    static constexpr int kWarps = attend_warps(DP, NB), kThreads = 32 * kWarps;
    static constexpr int kStage = kAttendTile * DP * 2, kFit = 192 * 1024 / kWarps / kStage;
    static constexpr int kStages = kFit < 6 ? kFit : 6, kBytes = kStages * kStage;
    static_assert(kStages >= 3, "a tile's values and the next one's keys go while its keys are used");
    // tiles that are under way at once
    static constexpr int kTiles = 4;
};

// What a row of the batch has: its first token and how many.
struct Span {
    int start, n, tiles;
    bool used;
};
__device__ __forceinline__ Span span_of(const AttendArgs &a, int b, bool *bad)
{
    int len = a.lengths[b];
    Span s;
    s.used = len >= 0;
    if (len > a.kv.capacity) {
        *bad = true;
        len = static_cast<int>(a.kv.capacity);
    }
    s.start = a.window > 0 && len > a.window ? len - a.window : 0;
    s.n = len > 0 ? len - s.start : 0;
    // (a row without tokens is visited too: it has an output; a row may have
    // 2^31 - 1 tokens, so nothing is added to n: the last tile's last token is
    // number 2^31 - 1)
    s.tiles = s.n > 0 ? s.n / kAttendTile + (s.n % kAttendTile != 0) : 1;
    return s;
}

// Places of the row before each sequence's tiles: taking up an item (queries,
// output) costs about as much as a tile (37 rows of 12 heads, some of them
// with a tile alone: the worker of those ended at 50 us, the others at 35).
constexpr int kItemPlaces = 1;

// A tile of the row, for one of the items.
struct Place {
    int b, item, tile;     // sequence, item among the sequence's, tile of the item
    Span s;
};
// On to the next one; returns how many places further it is.
__device__ __forceinline__ int advance(const AttendArgs &a, Place &p, bool *bad)
{
    if (++p.tile < p.s.tiles) return 1;
    p.tile = 0;
    if (++p.b < a.B) p.s = span_of(a, p.b, bad);
    return 1 + kItemPlaces;
}

// The entry of the table for a token of a tile, one in lane % 16, and its slot
// in the page; kNone past the sequence's end, which no entry is (negative ones
// are no pages, and -1 then).
constexpr int kNone = -2147483647 - 1;
__device__ __forceinline__ int page_entry(const AttendArgs &a, const Place &p, int lane, int *slot)
{
    const int j = p.tile * kAttendTile + (lane & 15);
    if (j >= p.s.n) return kNone;
    const int token = p.s.start + j;
    const int page = a.kv.page_mul ? __umulhi(token, a.kv.page_mul) >> a.kv.page_sh : token;
    *slot = token - page * a.kv.page_size;
    return max(a.kv.table[p.b * a.kv.table_stride + page], -1);
}

// Piece c of row r of a stage lies at c ^ turn(r), so that eight rows' pieces
// of one column lie in all banks: the rows are P pieces apart, and 8 of them
// fill the 8 places of 16 bytes modulo 128.
template <int DP>
__device__ __forceinline__ constexpr int turn(int r)
{
    static_assert(DP / 8 % 8 == 0 || DP / 8 % 8 == 2 || DP / 8 % 8 == 4, "");
    return DP / 8 % 8 == 0 ? r & 7 : DP / 8 % 8 == 4 ? (r >> 1) & 3 : (r >> 2) & 1;
}

// A lane's 16-byte pieces of a tile's rows, D / 8 a row: piece lane + 32 i.
// FULL: D = DP.
template <int DP, bool FULL>
struct Pieces {
    static constexpr int kEach = DP / 8, kMost = kAttendTile * kEach / 32;
    // a lane's pieces lie in one column, kRows rows apart
    static constexpr bool kColumn = FULL && 32 % kEach == 0;
    static constexpr int kRows = kColumn ? 32 / kEach : 1, kHeld = kColumn ? 1 : kMost;
    int count;                              // of all the tile's
    int at[kHeld], row[kHeld], col[kHeld];  // in the stage; the token; the piece of its row
    __device__ __forceinline__ Pieces(int D, int lane)
    {
        const int each = FULL ? kEach : D / 8;
        count = kAttendTile * each;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int p = min(i * 32 + lane, count - 1), r = p / each, c = p - r * each;
            at[i] = r * (DP * 2) + ((c ^ turn<DP>(r)) << 4);
            row[i] = r;
            col[i] = c;
        }
    }
    __device__ __forceinline__ int at_of(int i) const
    {
        // (the first row is below kRows, whose multiples' bits are apart from it)
        return kColumn ? (at[0] ^ (turn<DP>(i * kRows) << 4)) + i * kRows * DP * 2 : at[kColumn ? 0 : i];
    }
    __device__ __forceinline__ int row_of(int i) const { return kColumn ? row[0] + i * kRows : row[kColumn ? 0 : i]; }
    __device__ __forceinline__ int col_of(int i) const { return col[kColumn ? 0 : i]; }
};
constexpr uint32_t kNowhere = 0xffffffffu;
// The rows at these offsets (one in lane % 16, in 16-byte units) to a stage;
// zeros for those nowhere, if not `all` are somewhere.
template <int DP, bool FULL>
__device__ __forceinline__ void fetch(const void *cache, const Pieces<DP, FULL> &p, uint32_t offset, bool all, uint32_t stage,
                                      int lane)
{
    using P = Pieces<DP, FULL>;
    const uint4 *from = static_cast<const uint4 *>(cache) + (P::kColumn ? p.col_of(0) : 0);
    if (all) {
#pragma unroll
        for (int i = 0; i < P::kMost; ++i) {
            if (!FULL && i * 32 >= p.count) break;
            const uint32_t at = __shfl_sync(0xffffffffu, offset, p.row_of(i)) + (P::kColumn ? 0 : p.col_of(i));
            if (FULL || i * 32 + lane < p.count) cp_async16(stage + p.at_of(i), from + at);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < P::kMost; ++i) {
        if (!FULL && i * 32 >= p.count) break;
        const uint32_t at = __shfl_sync(0xffffffffu, offset, p.row_of(i));
        const bool there = at != kNowhere;
        if (FULL || i * 32 + lane < p.count)
            cp_async16(stage + p.at_of(i), from + (there ? at + (P::kColumn ? 0 : p.col_of(i)) : 0u), there);
    }
}

// One row of an item's output from at most 32 parts, by a warp: ml(i) is part
// i's (maximum, sum), o(i, at) its sums of dimensions at to at + 3.
template <bool BF16, int DP, typename Ml, typename O>
__device__ __forceinline__ void join_row(const AttendArgs &a, int parts, int64_t head, Ml ml, O o)
{
    constexpr int kEach = (DP / 4 + 31) / 32;
    const int lane = threadIdx.x & 31;
    const float2 mine = lane < parts ? ml(lane) : make_float2(-INFINITY, 0.0f);
    float top = mine.x;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float w = exp2_fast(mine.x - (top == -INFINITY ? 0.0f : top));
    float total = w * mine.y;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
    float4 acc[kEach] = {};
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int at = (e * 32 + lane) * 4;
            if (at >= DP) break;
            const float4 v = o(i, at);
            acc[e].x = fmaf(wi, v.x, acc[e].x);
            acc[e].y = fmaf(wi, v.y, acc[e].y);
            acc[e].z = fmaf(wi, v.z, acc[e].z);
            acc[e].w = fmaf(wi, v.w, acc[e].w);
        }
    }
    const float by = total == 0.0f ? 0.0f : 1.0f / total;
    uint16_t *out = static_cast<uint16_t *>(a.out) + head * a.D;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
        if ((e * 32 + lane) * 4 < a.D)
            *reinterpret_cast<uint2 *>(out + (e * 32 + lane) * 4) =
                make_uint2(pack16<BF16>(acc[e].x * by, acc[e].y * by), pack16<BF16>(acc[e].z * by, acc[e].w * by));
    if (a.lse && lane == 0) a.lse[head] = total == 0.0f ? -INFINITY : top * kLn2 + logf(total);
}

// The error word by one block: lengths beyond the table, and pages that are
// not there, of all rows.  8 lanes take a row, 8 entries each at once, so that
// the block is done before those that attend (150 rows of 2000 tokens one
// after the other, a block wide: 108 us).
__device__ __forceinline__ void check_pages(const AttendArgs &a)
{
    constexpr int kLanes = 8, kHeld = 8;
    bool bad = false;
    for (int b = static_cast<int>(threadIdx.x) / kLanes; b < a.B; b += static_cast<int>(blockDim.x) / kLanes) {
        const Span s = span_of(a, b, &bad);
        if (s.n == 0) continue;
        const int last = (s.start + s.n - 1) / a.kv.page_size;
        for (int64_t i = s.start / a.kv.page_size + static_cast<int>(threadIdx.x) % kLanes; i <= last; i += kLanes * kHeld) {
            int page[kHeld];
#pragma unroll
            for (int h = 0; h < kHeld; ++h) page[h] = i + h * kLanes <= last ? a.kv.table[b * a.kv.table_stride + i + h * kLanes] : 0;
#pragma unroll
            for (int h = 0; h < kHeld; ++h) bad = bad || page[h] < 0 || page[h] >= a.kv.pages;
        }
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.err = any ? kDevErrPage : 0;
}

// NB: blocks of 8 query heads that a warp takes at once, 1 or 2.
template <bool BF16, int DP, int NB, bool FULL, bool SOLO>
__global__ void __launch_bounds__(32 * attend_warps(DP, NB), 1) attend_kernel(const __grid_constant__ AttendArgs a)
{
    using R = Ring<DP, NB>;
    constexpr int kWarps = R::kWarps, kThreads = R::kThreads, S = R::kStages;
    constexpr int kSteps = DP / 16;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ long long before[SOLO ? 1 : kThreads + 1];
    __shared__ long long warp_total[SOLO ? 1 : kWarps];
    __shared__ uint32_t seen[kWarps][R::kTiles];
    __shared__ float2 solo_ml[SOLO ? kWarps : 1][kAttendRows];
    static_assert(kAttendRows / 2 * NB * DP * 4 <= R::kBytes, "a part in a warp's ring");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int items = a.G * a.blocks;
    pdl_launch_dependents();
    // (columns from D on are zeros, which no copy touches)
    if (!FULL)
        for (int i = threadIdx.x; i < kWarps * R::kBytes / 16; i += kThreads)
            reinterpret_cast<uint4 *>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);

    bool bad = false;
    Place c;
    long long share = 1, place = 0, end = 0;      // the worker's run: from tile c's place up to `end`
    int worker = warp, group = 0;
    if constexpr (SOLO) {
        if (static_cast<int>(blockIdx.x) == a.B * items) {      // a block that only looks for bad pages
            check_pages(a);
            return;
        }
        c.b = static_cast<int>(blockIdx.x) / items;
        c.item = static_cast<int>(blockIdx.x) - c.b * items;
        c.s = span_of(a, c.b, &bad);
        share = (c.s.tiles + kWarps - 1) / kWarps;
        c.tile = worker * static_cast<int>(share);
        place = c.tile;
        end = min(place + share, static_cast<long long>(c.s.tiles));
        if (!FULL) __syncthreads();
    } else {
        // Tiles before each run of `each` sequences.
        const int each = (a.B + kThreads - 1) / kThreads;
        long long mine = 0;
        for (int i = 0; i < each; ++i) {
            const int b = static_cast<int>(threadIdx.x) * each + i;
            if (b < a.B) mine += span_of(a, b, &bad).tiles + kItemPlaces;
        }
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_total[warp] = incl;
        __syncthreads();
        long long base = 0;
        for (int w = 0; w < warp; ++w) base += warp_total[w];
        before[threadIdx.x + 1] = base + incl;
        if (threadIdx.x == 0) before[0] = 0;
        __syncthreads();
        bad = false;      // (counted by whoever works on the sequence)
        const long long total = before[kThreads];
        share = (total + a.groups - 1) / a.groups;
        if (share < a.min_share) share = a.min_share;
        // Few workers spread over the SMs, a group's by fours (64 rows of 2048
        // to 8192 tokens 212.5 us, each on an SM of its own 217; eights as fours).
        constexpr int kTogether = 4;
        worker = ((warp / kTogether) * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x)) * kTogether + warp % kTogether;
        c.item = worker % items;
        group = worker / items;
        if (group < a.groups) {
            place = group * share;
            end = min(place + share, total);
        }
        if (place < end) {
            int lo = 0, hi = kThreads;       // before[lo] <= place < before[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (before[mid] <= place) lo = mid;
                else hi = mid;
            }
            long long at = before[lo];
            int b = lo * each;
            Span s = span_of(a, b, &bad);
            while (at + s.tiles + kItemPlaces <= place) {
                at += s.tiles + kItemPlaces;
                s = span_of(a, ++b, &bad);
            }
            c.b = b;
            c.s = s;
            at += kItemPlaces;      // of the first tile
            c.tile = static_cast<int>(max(0LL, place - at));
            place = at + c.tile;
        }
    }
    AttendJob job = {-1, -1, 0, 0};
    const Place at_start = c;      // solo: the CTA's item

    if (place < end) {
        Place f = c;
        long long f_place = place;
        const Pieces<DP, FULL> pieces(a.D, lane);
        const uint32_t base = smem_u32(ring) + warp * R::kBytes;
        // Keys and values go by turns; the values' offsets are kept from the
        // keys'.  What the cursor f does not reach is an empty group.
        uint32_t k_at = kNowhere, v_at = kNowhere;
        bool all = false;                  // the tile has all its tokens
        bool real = false;                 // the last keys issued were a tile's
        int issued = 0;                    // tiles
        auto locate = [&](const Place &f, int entry, int slot) {
            k_at = v_at = kNowhere;
            if (entry != kNone) {
                if (entry >= 0 && entry < a.kv.pages) {
                    const uint32_t head = a.blocks == 1 ? f.item : f.item / a.blocks;
                    k_at = entry * a.k_page + slot * a.k_token + head * a.k_head;
                    v_at = a.alike ? k_at : entry * a.v_page + slot * a.v_token + head * a.v_head;
                } else {
                    bad = true;
                }
            }
        };
        auto issue_keys = [&](const Place &f, long long f_at, int entry, int slot, int stage) {
            real = f_at < end;
            if (real) {
                locate(f, entry, slot);
                const uint32_t there = __ballot_sync(0xffffffffu, k_at != kNowhere);
                all = there == 0xffffffffu;
                if (lane == 0) seen[warp][issued % R::kTiles] = there;
                fetch<DP, FULL>(a.kv.k, pieces, k_at, all, base + stage * R::kStage, lane);
                ++issued;
            }
            cp_async_commit();
        };
        auto issue_values = [&](int stage) {      // of the tile whose keys went last
            if (real) fetch<DP, FULL>(a.kv.v, pieces, v_at, all, base + stage * R::kStage, lane);
            cp_async_commit();
        };
        auto entry_ahead = [&](int *slot) { return f_place < end ? page_entry(a, f, lane, slot) : kNone; };
        {
            // The first tiles' table entries are asked for together.
            constexpr int kFirst = (S + 1) / 2;
            Place at[kFirst];
            long long place_of[kFirst];
            int entry[kFirst], slot[kFirst] = {};
#pragma unroll
            for (int j = 0; j < kFirst; ++j) {
                at[j] = f;
                place_of[j] = f_place;
                entry[j] = entry_ahead(&slot[j]);
                if (f_place < end) f_place += advance(a, f, &bad);
            }
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (i % 2 == 0) issue_keys(at[i / 2], place_of[i / 2], entry[i / 2], slot[i / 2], i);
                else issue_values(i);
            }
        }

        // of dimension block j, head block n: dimensions 16 j + g (o[0], o[1])
        // and 16 j + g + 8, heads 8 n + 2t and the next; maximum and this
        // lane's share of the sum of each of those heads
        float o[kSteps][NB][4], top[NB][2], sum[NB][2];
        uint32_t q[kSteps][NB][2];
        bool fresh = true;         // a new item
        bool whole = !SOLO && c.tile == 0;  // this worker has the item's beginning
        int stage = 0;
        for (int i = 0; place < end; ++i) {
            int slot = 0;
            const int entry = entry_ahead(&slot);
            if (fresh) {
                const int kv_head = c.item / a.blocks, block = c.item - kv_head * a.blocks;
                const int rows = min(kAttendRows, a.group - block * kAttendRows);
                const uint16_t *from = static_cast<const uint16_t *>(a.q) + c.b * a.q_row +
                                       (kv_head * a.group + block * kAttendRows) * a.q_head;
#pragma unroll
                for (int n = 0; n < NB; ++n) {
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = 8 * n + g, d = k * 16 + h * 8 + 2 * t;
                            q[k][n][h] = r < rows && d < a.D ? *reinterpret_cast<const uint32_t *>(from + r * a.q_head + d) : 0u;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[k][n][e] = 0.0f;
                    }
                    top[n][0] = top[n][1] = -INFINITY;
                    sum[n][0] = sum[n][1] = 0.0f;
                }
                fresh = false;
            }
            cp_async_wait<S - 1>();
            __syncwarp();
            const uint32_t there = seen[warp][i % R::kTiles] & 0xffffu;

            // scores of tokens g (z[0], z[1]) and g + 8 with heads 2t, 2t + 1
            float z[NB][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[n][e] = 0.0f;
            {
                const int r = lane & 15, half = lane >> 4;
                const uint32_t row = base + stage * R::kStage + r * (DP * 2);
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    uint32_t w[4];
                    ldmatrix4(w, row + (((2 * k + half) ^ turn<DP>(r)) << 4));
#pragma unroll
                    for (int n = 0; n < NB; ++n) mma_16816<BF16>(z[n], w[0], w[1], w[2], w[3], q[k][n][0], q[k][n][1]);
                }
            }
            __syncwarp();
            auto next_keys = [&] {
                issue_keys(f, f_place, entry, slot, stage);
                if (real) {
                    f_place += advance(a, f, &bad);
                    // a new item's queries on their way, for when its first tile is taken
                    if (f.tile == 0 && f_place < end && lane < kAttendRows) {
                        const int kv_head = f.item / a.blocks, block = f.item - kv_head * a.blocks;
                        const int r = kv_head * a.group + block * kAttendRows + lane;
                        if (lane < min(kAttendRows, a.group - block * kAttendRows))
#pragma unroll
                            for (int d = 0; d < DP * 2; d += 128)      // (of the head alone: what follows the last may be nobody's)
                                if (FULL || d < a.D * 2)
                                    asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const uint8_t *>(a.q) + (f.b * a.q_row + r * a.q_head) * 2 + d));
                    }
                }
            };
            if (S % 2 == 0) next_keys();
            else issue_values(stage);
            stage = stage + 1 == S ? 0 : stage + 1;
            // in units of log 2, those that are not there out
            bool more = false;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[n][e] *= a.scale2;
            if (there != 0xffffu) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((there >> (g + (e >> 1) * 8)) & 1u)) z[n][e] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) more = more || z[n][e] > top[n][e & 1];
            // Only where a head's maximum grows is it exchanged.
            if (__any_sync(0xffffffffu, more)) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float high = fmaxf(z[n][h], z[n][2 + h]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, x));
                        const float to = fmaxf(top[n][h], high);
                        const float by = to == top[n][h] ? 1.0f : exp2_fast(top[n][h] - to);
                        top[n][h] = to;
                        sum[n][h] *= by;
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            o[k][n][h] *= by;
                            o[k][n][2 + h] *= by;
                        }
                    }
            }
            // The weights go to the second product in two parts of the inputs'
            // type: the weight cut off, and what that left out.  (In one part,
            // tokens of equal scores have weights that are all off alike, by
            // up to half a step, which the sum of the unrounded ones does not
            // have: as much again as the output's own rounding.)  The second
            // part's last bit is set where the first is not 0, so that both are
            // above 0 and an infinite value gives its infinity, not one minus
            // another or times 0.  Together they are off by at most 3 x 2^-15
            // of the weight (fp16 3 x 2^-21, or 3 x 2^-40 of the largest where
            // its steps end); a weight of 0 is 0.
            uint32_t p[2][NB][2];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // (nothing seen so far: 2^(-inf - 0) = 0)
                    const float off = top[n][e & 1] == -INFINITY ? 0.0f : top[n][e & 1];
                    z[n][e] = exp2_fast(z[n][e] - off);
                    sum[n][e & 1] += z[n][e];
                    z[n][e] *= kWeightScale<BF16>;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t high = cut16<BF16>(z[n][2 * h], z[n][2 * h + 1]);
                    const float2 v = unpack16<BF16>(high);
                    p[0][n][h] = transpose8(high);
                    p[1][n][h] = transpose8(pack16<BF16>(z[n][2 * h] - v.x, z[n][2 * h + 1] - v.y) | __vminu2(high, 0x10001u));
                }
            }
            cp_async_wait<S - 1>();
            __syncwarp();
            {
                const int r = lane & 7, tokens = (lane >> 4) << 3, half = (lane >> 3) & 1;
                const uint32_t row = base + stage * R::kStage + (tokens + r) * (DP * 2);
                // A tile's sums are a chain of their own, for the sake of long
                // ones (mma_16816_from_zero).  Four dimension blocks at once,
                // so that few products wait for one before them: 64 rows of
                // 2048 to 8192 tokens 213 us (with the weights in one part and
                // one long chain 211), 16 rows of 8000, 16 heads to a key head
                // of 192, 99 (two blocks at once 103, one 121), of 256 151 (one
                // part, one chain 133).
                constexpr int kAtOnce = 4;
#pragma unroll
                for (int k0 = 0; k0 < kSteps; k0 += kAtOnce) {
                    uint32_t w[kAtOnce][4];
#pragma unroll
                    for (int k = 0; k < kAtOnce && k0 + k < kSteps; ++k)
                        ldmatrix4_t(w[k], row + (((2 * (k0 + k) + half) ^ turn<DP>(r)) << 4));
                    float d[kAtOnce][NB][4];
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k = 0; k < kAtOnce && k0 + k < kSteps; ++k)
#pragma unroll
                            for (int n = 0; n < NB; ++n) {
                                if (part == 0) mma_16816_from_zero<BF16>(d[k][n], w[k][0], w[k][1], w[k][2], w[k][3], p[0][n][0], p[0][n][1]);
                                else mma_16816<BF16>(d[k][n], w[k][0], w[k][1], w[k][2], w[k][3], p[1][n][0], p[1][n][1]);
                            }
#pragma unroll
                    for (int k = 0; k < kAtOnce && k0 + k < kSteps; ++k)
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[k0 + k][n][e] += d[k][n][e];
                }
            }
            __syncwarp();
            if (S % 2 == 0) issue_values(stage);
            else next_keys();
            stage = stage + 1 == S ? 0 : stage + 1;

            const bool ends = c.tile + 1 == c.s.tiles;
            if (ends || place + 1 >= end) {
                const int kv_head = c.item / a.blocks, block = c.item - kv_head * a.blocks;
                const int rows = min(kAttendRows, a.group - block * kAttendRows);
                const int head = kv_head * a.group + block * kAttendRows;
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) sum[n][h] += __shfl_xor_sync(0xffffffffu, sum[n][h], x);
                if (!BF16) {
#pragma unroll
                    for (int k = 0; k < kSteps; ++k)
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[k][n][e] *= 1.0f / kWeightScale<BF16>;
                }
                if (!SOLO && ends && whole) {
                    if (c.s.used) {
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int r = 8 * n + 2 * t + h;
                                if (r >= rows) continue;
                                const float total = sum[n][h], by = total == 0.0f ? 0.0f : 1.0f / total;
                                const int64_t at = static_cast<int64_t>(c.b) * a.H + head + r;
                                uint16_t *out = static_cast<uint16_t *>(a.out) + at * a.D;
#pragma unroll
                                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (k * 16 + e * 8 < a.D)
                                            out[k * 16 + e * 8 + g] =
                                                static_cast<uint16_t>(pack16<BF16>(o[k][n][2 * e + h] * by, 0.0f));
                                if (a.lse && g == 0) a.lse[at] = total == 0.0f ? -INFINITY : top[n][h] * kLn2 + logf(total);
                            }
                    }
                    if (a.slot_by_item && lane == 0)
                        a.jobs[static_cast<int64_t>(c.b) * items + c.item] = AttendJob{-1, -1, 0, 0};
                } else {
                    const int64_t part = ((static_cast<int64_t>(c.item) * a.groups + group) * 2 + (whole ? 1 : 0)) * a.part_rows;
                    if (SOLO) {      // (the ring is empty: its copies are done)
                        cp_async_wait<0>();
                        __syncwarp();
                    }
                    float2 *part_ml = SOLO ? solo_ml[SOLO ? warp : 0] : a.part_ml + part;
                    float *part_o = SOLO ? reinterpret_cast<float *>(ring + warp * R::kBytes) : a.part_o + part * DP;
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = 8 * n + 2 * t + h;
                            if (r >= rows) continue;
                            if (g == 0) part_ml[r] = make_float2(top[n][h], sum[n][h]);
                            float *po = part_o + r * DP + g;
#pragma unroll
                            for (int k = 0; k < kSteps; ++k) {
                                po[k * 16] = o[k][n][h];
                                po[k * 16 + 8] = o[k][n][2 + h];
                            }
                        }
                    if (whole) {      // the others' parts follow
                        const long long last = place + (c.s.tiles - 1 - c.tile);
                        job = AttendJob{group, static_cast<int>(last / share), c.b, c.item};
                        if (a.slot_by_item && lane == 0) a.jobs[static_cast<int64_t>(c.b) * items + c.item] = job;
                    }
                }
                fresh = whole = true;
            }
            place += advance(a, c, &bad);
        }
        cp_async_wait<0>();
    }
    if constexpr (SOLO) {
        __syncthreads();
        const int kv_head = at_start.item / a.blocks, block = at_start.item - kv_head * a.blocks;
        const int rows = min(kAttendRows, a.group - block * kAttendRows);
        const int parts = (at_start.s.tiles + static_cast<int>(share) - 1) / static_cast<int>(share);
        if (!at_start.s.used) return;
        for (int row = warp; row < rows; row += kWarps)
            join_row<BF16, DP>(
                a, parts, static_cast<int64_t>(at_start.b) * a.H + kv_head * a.group + block * kAttendRows + row,
                [&](int i) { return solo_ml[i][row]; },
                [&](int i, int at) { return *reinterpret_cast<const float4 *>(ring + i * R::kBytes + (row * DP + at) * 4); });
        return;
    }
    if (!a.slot_by_item && lane == 0) a.jobs[worker] = job;
    const bool any = __any_sync(0xffffffffu, bad);
    if (lane == 0) a.flags[worker] = any;
}

// The parts of an item that several workers share.  Up to 32 parts (a batch)
// a warp takes a row by itself, its parts' weights in its lanes; more (few
// long sequences) are taken by all warps of a block together, a row of blocks
// for each row; HELD of its parts a warp has under way at once.  8 where items
// have many parts on average (131072 tokens of 8 key heads: 98.9 -> 97.4 us
// with 8 instead of 4), else 4, whose registers let more blocks run (64 rows of
// 8192 tokens: the join 12 us instead of 17).
constexpr int kJoinWarps = 16;

template <int N>
__device__ __forceinline__ void add_scaled(float4 (&to)[N], const float4 (&v)[N], float w)
{
#pragma unroll
    for (int e = 0; e < N; ++e) {
        to[e].x = fmaf(w, v[e].x, to[e].x);
        to[e].y = fmaf(w, v[e].y, to[e].y);
        to[e].z = fmaf(w, v[e].z, to[e].z);
        to[e].w = fmaf(w, v[e].w, to[e].w);
    }
}

template <bool BF16, int DP, int HELD>
__global__ void __launch_bounds__(32 * kJoinWarps) attend_join_kernel(const __grid_constant__ AttendArgs a)
{
    extern __shared__ float weight[];     // [groups][weight, weight x sum]
    __shared__ __align__(16) float sums[kJoinWarps][DP];
    __shared__ float red[kJoinWarps];
    constexpr int kEach = (DP / 4 + 31) / 32;      // 16-byte pieces of a part's row that a lane has
    auto has = [&](int e) { return (e * 32 + (static_cast<int>(threadIdx.x) & 31)) * 4 < DP; };
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        int bad = 0;
        for (int w = threadIdx.x; w < a.workers; w += 32 * kJoinWarps) bad |= a.flags[w];
        const int any = __syncthreads_or(bad);
        if (threadIdx.x == 0 && (any || !a.err_keep)) *a.err = any ? kDevErrPage : 0;
    }
    const AttendJob job = a.jobs[blockIdx.x];
    if (job.first < 0) return;
    const int kv_head = job.item / a.blocks, block = job.item - kv_head * a.blocks;
    const int rows = min(kAttendRows, a.group - block * kAttendRows), parts = job.last - job.first + 1;
    const int64_t head0 = static_cast<int64_t>(job.row) * a.H + kv_head * a.group + block * kAttendRows;
    auto part = [&](int i, int row) {
        return ((static_cast<int64_t>(job.item) * a.groups + job.first + i) * 2 + (i == 0 ? 1 : 0)) * a.part_rows + row;
    };
    auto load = [&](float4 (&v)[kEach], int i, int row) {
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            v[e] = has(e) ? __ldcg(reinterpret_cast<const float4 *>(a.part_o + part(i, row) * DP) + e * 32 + lane)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };

    if (parts <= 32) {
        if (blockIdx.y > 0) return;
        for (int row = warp; row < rows; row += kJoinWarps)
            join_row<BF16, DP>(
                a, parts, head0 + row, [&](int i) { return a.part_ml[part(i, row)]; },
                [&](int i, int at) { return __ldcg(reinterpret_cast<const float4 *>(a.part_o + part(i, row) * DP + at)); });
        return;
    }
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        // A warp's first sums are on their way before their weights are known.
        float4 held[HELD][kEach];
#pragma unroll
        for (int h = 0; h < HELD; ++h)
            if (warp + h * kJoinWarps < parts) load(held[h], warp + h * kJoinWarps, row);
        float top = -INFINITY;
        for (int i = threadIdx.x; i < parts; i += 32 * kJoinWarps) top = fmaxf(top, a.part_ml[part(i, row)].x);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        if (lane == 0) red[warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, red[w]);
        const float off = top == -INFINITY ? 0.0f : top;
        for (int i = threadIdx.x; i < parts; i += 32 * kJoinWarps) {
            const float2 ml = a.part_ml[part(i, row)];
            const float w = exp2_fast(ml.x - off);
            weight[2 * i] = w;
            weight[2 * i + 1] = w * ml.y;
        }
        __syncthreads();
        // (every warp sums the denominators the same way)
        float total = 0.0f;
        for (int i = lane; i < parts; i += 32) total += weight[2 * i + 1];
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
        {
            float4 acc[kEach] = {};
#pragma unroll
            for (int h = 0; h < HELD; ++h)
                if (warp + h * kJoinWarps < parts) add_scaled(acc, held[h], weight[2 * (warp + h * kJoinWarps)]);
#pragma unroll 4
            for (int i = warp + HELD * kJoinWarps; i < parts; i += kJoinWarps) {
                float4 v[kEach];
                load(v, i, row);
                add_scaled(acc, v, weight[2 * i]);
            }
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                if (has(e)) *reinterpret_cast<float4 *>(&sums[warp][(e * 32 + lane) * 4]) = acc[e];
        }
        __syncthreads();
        const float by = total == 0.0f ? 0.0f : 1.0f / total;
        if (threadIdx.x < DP / 2 && static_cast<int>(threadIdx.x) * 2 < a.D) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                x += sums[w][2 * threadIdx.x];
                y += sums[w][2 * threadIdx.x + 1];
            }
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + (head0 + row) * a.D + 2 * threadIdx.x) =
                pack16<BF16>(x * by, y * by);
        }
        if (a.lse && threadIdx.x == 0) a.lse[head0 + row] = total == 0.0f ? -INFINITY : top * kLn2 + logf(total);
    }
}

template <bool BF16, int DP, int NB, bool FULL, bool SOLO>
cudaError_t attend(const AttendArgs &a, cudaStream_t stream)
{
    using R = Ring<DP, NB>;
    constexpr int kSmem = R::kWarps * R::kBytes;
    // (an attribute of the device's copy of the function: set at every call,
    // as the current device may be another)
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<BF16, DP, NB, FULL, SOLO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attend_kernel<BF16, DP, NB, FULL, SOLO><<<SOLO ? a.B * a.G * a.blocks + 1 : a.workers / R::kWarps, R::kThreads, kSmem, stream>>>(a);
    return cudaGetLastError();
}
template <bool BF16, int DP, bool PADDED, bool SOLO>
cudaError_t attend(const AttendArgs &a, cudaStream_t stream)
{
    if constexpr (PADDED) {
        if (a.D < DP)
            return attend_heads(a.group) == 1 ? attend<BF16, DP, 1, false, SOLO>(a, stream) : attend<BF16, DP, 2, false, SOLO>(a, stream);
    }
    return attend_heads(a.group) == 1 ? attend<BF16, DP, 1, true, SOLO>(a, stream) : attend<BF16, DP, 2, true, SOLO>(a, stream);
}

template <bool BF16, int DP>
cudaError_t join(const AttendArgs &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    // (blocks for single rows where there are few jobs, which are the long ones)
    const int apart = 1024 / a.slots;
    cfg.gridDim = dim3(static_cast<unsigned>(a.slots),
                       static_cast<unsigned>(apart < 1 ? 1 : apart < a.part_rows ? apart : a.part_rows));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.groups) * 2 * sizeof(float);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.slots * 32 <= a.workers ? attend_join_kernel<BF16, DP, 8> : attend_join_kernel<BF16, DP, 4>, a);
}

// Calls f with the padded dimension, and whether smaller ones share it.
template <typename F>
cudaError_t by_dim(int64_t D, F f)
{
    switch (attend_dim(D)) {
    case 64: return f(std::integral_constant<int, 64>(), std::true_type());
    case 80: return f(std::integral_constant<int, 80>(), std::false_type());
    case 96: return f(std::integral_constant<int, 96>(), std::false_type());
    case 128: return f(std::integral_constant<int, 128>(), std::true_type());
    case 192: return f(std::integral_constant<int, 192>(), std::false_type());
    default: return f(std::integral_constant<int, 256>(), std::true_type());
    }
}

template <bool BF16, bool SOLO>
int run_attend(const AttendArgs &a, cudaStream_t stream)
{
    const cudaError_t e = by_dim(a.D, [&](auto dim, auto padded) { return attend<BF16, dim(), padded(), SOLO>(a, stream); });
    return e == cudaSuccess ? 0 : record_cuda_error("paged attention launch", e, cudaGetErrorString(e));
}
template <bool BF16>
int run_join(const AttendArgs &a, cudaStream_t stream)
{
    const cudaError_t e = by_dim(a.D, [&](auto dim, auto) { return join<BF16, dim()>(a, stream); });
    return e == cudaSuccess ? 0 : record_cuda_error("paged attention join launch", e, cudaGetErrorString(e));
}

}  // namespace

}  // namespace ngr
