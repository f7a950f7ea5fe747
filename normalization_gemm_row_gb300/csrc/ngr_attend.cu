// ngr_attend.cu -- attention of one new token for each sequence over a paged
// key-value cache.
//
//   s_j = scale q . k_j,  lse = log sum_j exp s_j,  out = sum_j exp(s_j - lse) v_j
//
// A key or value read serves the H / G query heads of its head: 2 H / G
// operations a byte, so reading the cache bounds it.  The cache is streamed
// once, by warps: each has a ring of stages in shared memory that
// asynchronous copies of 16 tokens' keys and values fill, and takes them with
// 16 x 8 x 16 matrix instructions, the query heads (at most 16) as rows,
// with a running maximum and sum.  The warps have nothing to wait for but
// their own copies: no barrier.
//
// All items' tiles of 16 tokens (an item: a sequence and key head, and a block
// of 16 query heads where there are more) stand in one row, which is cut into
// equal runs, one a warp ("worker").  A batch of any lengths is balanced so,
// and nothing but the device has to know the lengths.  An item that lies in
// one run is finished there; the others' parts (FP32 sums, maximum, sum of
// exponentials) are joined by a second kernel in the tokens' order, so a call
// repeated gives the same bits.
#include "ngr.h"
#include "ngr_entry.h"
#include "ngr_internal.h"
#include "ngr_kv.h"
#include "ngr_mma.cuh"
#include "ngr_ptx.cuh"

namespace ngr {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Stages of a warp's ring: 24 KB at 64 and 128 dimensions, 48 KB at 256.
constexpr int stages_of(int DP) { return DP == 64 ? 6 : 3; }
constexpr int stage_bytes(int DP) { return 2 * kAttendTile * DP * 2; }
constexpr int warp_bytes(int DP) { return stages_of(DP) * stage_bytes(DP); }

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
    // (a row without tokens is visited too: it has an output)
    s.tiles = s.n > 0 ? (s.n + kAttendTile - 1) / kAttendTile : 1;
    return s;
}

// A place in the row of tiles.
struct Place {
    int b, item, tile;     // sequence, item among the sequence's, tile of the item
    Span s;
};
__device__ __forceinline__ void advance(const AttendArgs &a, Place &p, bool *bad)
{
    if (++p.tile < p.s.tiles) return;
    p.tile = 0;
    if (++p.item < a.G * a.blocks) return;
    p.item = 0;
    if (++p.b < a.B) p.s = span_of(a, p.b, bad);
}

// Where the tokens of a tile lie in the caches, a token in lane % 16: element
// offsets, or -1 where there is nothing to read.
struct Tokens {
    int64_t k, v;
};
__device__ __forceinline__ int page_entry(const AttendArgs &a, const Place &p, int lane, int *slot)
{
    const int j = p.tile * kAttendTile + (lane & 15);
    if (j >= p.s.n) return -2;
    const int token = p.s.start + j, page = token / a.kv.page_size;
    *slot = token - page * a.kv.page_size;
    return a.kv.table[p.b * a.kv.table_stride + page];
}
__device__ __forceinline__ Tokens tokens_at(const AttendArgs &a, const Place &p, int entry, int slot)
{
    Tokens t = {-1, -1};
    if (entry == -2) return t;
    const int g = p.item / a.blocks;
    t.k = entry * a.kv.k_page + slot * a.kv.k_token + g * a.kv.k_head;
    t.v = entry * a.kv.v_page + slot * a.kv.v_token + g * a.kv.v_head;
    return t;
}

template <int DP>
__device__ __forceinline__ void fetch(const AttendArgs &a, const Tokens &t, uint32_t stage, int lane)
{
    constexpr int kPieces = DP / 8, kRows = 32 / kPieces;
    const int col = lane % kPieces, r0 = lane / kPieces;
    const bool in = col * 8 < a.D;
    const uint16_t *k = static_cast<const uint16_t *>(a.kv.k), *v = static_cast<const uint16_t *>(a.kv.v);
#pragma unroll
    for (int i = 0; i < kAttendTile / kRows; ++i) {
        const int r = i * kRows + r0;
        const int64_t ko = __shfl_sync(0xffffffffu, t.k, r), vo = __shfl_sync(0xffffffffu, t.v, r);
        const bool there = in && ko >= 0;
        const uint32_t at = stage + r * (DP * 2) + ((col ^ (r & 7)) << 4);
        cp_async16(at, there ? k + ko + col * 8 : k, there);
        cp_async16(at + kAttendTile * DP * 2, there ? v + vo + col * 8 : v, there);
    }
}

template <bool BF16, int DP>
__global__ void __launch_bounds__(32 * (DP == 256 ? 4 : 8), 1) attend_kernel(const __grid_constant__ AttendArgs a)
{
    constexpr int kWarps = DP == 256 ? 4 : 8, kThreads = 32 * kWarps, S = stages_of(DP);
    constexpr int kSteps = DP / 16, kCols = DP / 8;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ long long before[kThreads + 1];
    __shared__ long long warp_total[kWarps];
    __shared__ uint32_t seen[kWarps][S];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int items = a.G * a.blocks;
    pdl_launch_dependents();

    // Tiles before each run of `each` sequences.
    const int each = (a.B + kThreads - 1) / kThreads;
    bool bad = false;
    {
        long long mine = 0;
        for (int i = 0; i < each; ++i) {
            const int b = static_cast<int>(threadIdx.x) * each + i;
            if (b < a.B) mine += static_cast<long long>(span_of(a, b, &bad).tiles) * items;
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
    }
    bad = false;      // (counted by whoever works on the sequence)
    const long long total = before[kThreads];
    long long share = (total + a.workers - 1) / a.workers;
    if (share < a.min_share) share = a.min_share;
    // Neighbouring runs on different SMs: a few runs have an SM each.
    const int worker = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    const long long first = worker * share;
    long long left = total - first;
    const int count = static_cast<int>(left <= 0 ? 0 : left < share ? left : share);
    AttendJob job = {-1, -1, 0, 0};

    if (count > 0) {
        Place c;
        {
            int lo = 0, hi = kThreads;       // before[lo] <= first < before[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (before[mid] <= first) lo = mid;
                else hi = mid;
            }
            long long at = before[lo];
            int b = lo * each;
            Span s = span_of(a, b, &bad);
            while (at + static_cast<long long>(s.tiles) * items <= first) {
                at += static_cast<long long>(s.tiles) * items;
                s = span_of(a, ++b, &bad);
            }
            c.b = b;
            c.s = s;
            c.item = static_cast<int>((first - at) / s.tiles);
            c.tile = static_cast<int>((first - at) - static_cast<long long>(c.item) * s.tiles);
        }
        Place f = c;
        const uint32_t base = smem_u32(ring) + warp * warp_bytes(DP);
        auto issue = [&](int entry, int slot, int stage) {
            if (entry != -2 && (entry < 0 || entry >= a.kv.pages)) {
                bad = true;
                entry = -2;
            }
            const Tokens at = tokens_at(a, f, entry, slot);
            const uint32_t there = __ballot_sync(0xffffffffu, at.k >= 0);
            if (lane == 0) seen[warp][stage] = there;
            fetch<DP>(a, at, base + stage * stage_bytes(DP), lane);
            advance(a, f, &bad);
        };
#pragma unroll
        for (int i = 0; i < S; ++i) {
            if (i < count) {
                int slot = 0;
                const int entry = page_entry(a, f, lane, &slot);
                issue(entry, slot, i);
            }
            cp_async_commit();
        }

        float o[kCols][4], top[2], sum[2];
        uint32_t qa[kSteps][4];
        bool fresh = true;         // a new item
        bool whole = c.tile == 0;  // this worker has the item's beginning
        int stage = 0;
        for (int i = 0; i < count; ++i) {
            int slot = 0, entry = -2;
            if (i + S < count) entry = page_entry(a, f, lane, &slot);
            const int kv_head = c.item / a.blocks, block = c.item - kv_head * a.blocks;
            const int rows = min(kAttendRows, a.group - block * kAttendRows);
            const int head = kv_head * a.group + block * kAttendRows;
            if (fresh) {
                const uint16_t *q = static_cast<const uint16_t *>(a.q) + c.b * a.q_row + head * a.q_head;
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int r = g + (h & 1) * 8, d = k * 16 + (h >> 1) * 8 + 2 * t;
                        qa[k][h] = r < rows && d < a.D ? *reinterpret_cast<const uint32_t *>(q + r * a.q_head + d) : 0u;
                    }
#pragma unroll
                for (int j = 0; j < kCols; ++j)
#pragma unroll
                    for (int h = 0; h < 4; ++h) o[j][h] = 0.0f;
                top[0] = top[1] = -INFINITY;
                sum[0] = sum[1] = 0.0f;
                fresh = false;
            }
            cp_async_wait<S - 1>();
            __syncwarp();
            const uint32_t ks = base + stage * stage_bytes(DP), vs = ks + kAttendTile * DP * 2;
            const uint32_t there = seen[warp][stage];

            float s[2][4] = {};
            {
                const int r = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
                const uint32_t row = ks + r * (DP * 2);
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    uint32_t b[4];
                    ldmatrix4(b, row + (((2 * k + half) ^ (r & 7)) << 4));
                    mma_16816<BF16>(s[0], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b[0], b[1]);
                    mma_16816<BF16>(s[1], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b[2], b[3]);
                }
            }
            float high[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    s[n][h] = (there >> (n * 8 + 2 * t + (h & 1))) & 1u ? s[n][h] * a.scale2 : -INFINITY;
                    high[h >> 1] = fmaxf(high[h >> 1], s[n][h]);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                high[h] = fmaxf(high[h], __shfl_xor_sync(0xffffffffu, high[h], 1));
                high[h] = fmaxf(high[h], __shfl_xor_sync(0xffffffffu, high[h], 2));
            }
            if (__any_sync(0xffffffffu, high[0] > top[0] || high[1] > top[1])) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float to = fmaxf(top[h], high[h]);
                    const float by = to == top[h] ? 1.0f : exp2f(top[h] - to);
                    top[h] = to;
                    sum[h] *= by;
#pragma unroll
                    for (int j = 0; j < kCols; ++j) {
                        o[j][2 * h] *= by;
                        o[j][2 * h + 1] *= by;
                    }
                }
            }
            // (nothing seen so far: exp2(-inf - 0) = 0)
            const float off[2] = {top[0] == -INFINITY ? 0.0f : top[0], top[1] == -INFINITY ? 0.0f : top[1]};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    s[n][h] = exp2f(s[n][h] - off[h >> 1]);
                    sum[h >> 1] += s[n][h];
                }
            // The weights go to the second product in the inputs' type: half
            // a step off each, as independent roundings that average out
            // (their sum above is of the unrounded ones).
            const uint32_t p0 = pack16<BF16>(s[0][0], s[0][1]), p1 = pack16<BF16>(s[0][2], s[0][3]);
            const uint32_t p2 = pack16<BF16>(s[1][0], s[1][1]), p3 = pack16<BF16>(s[1][2], s[1][3]);
            {
                const int r = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
                const uint32_t row = vs + r * (DP * 2);
#pragma unroll
                for (int j = 0; j < kCols; j += 2) {
                    uint32_t b[4];
                    ldmatrix4_t(b, row + (((j + half) ^ (r & 7)) << 4));
                    mma_16816<BF16>(o[j], p0, p1, p2, p3, b[0], b[1]);
                    mma_16816<BF16>(o[j + 1], p0, p1, p2, p3, b[2], b[3]);
                }
            }
            __syncwarp();
            if (i + S < count) issue(entry, slot, stage);
            cp_async_commit();
            stage = stage + 1 == S ? 0 : stage + 1;

            const bool ends = c.tile + 1 == c.s.tiles;
            if (ends || i + 1 == count) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
                    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
                }
                if (ends && whole) {
                    if (c.s.used) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = g + 8 * h;
                            if (r >= rows) continue;
                            const float by = sum[h] == 0.0f ? 0.0f : 1.0f / sum[h];
                            const int64_t at = static_cast<int64_t>(c.b) * a.H + head + r;
                            uint16_t *out = static_cast<uint16_t *>(a.out) + at * a.D;
#pragma unroll
                            for (int j = 0; j < kCols; ++j)
                                if (j * 8 < a.D)
                                    *reinterpret_cast<uint32_t *>(out + j * 8 + 2 * t) =
                                        pack16<BF16>(o[j][2 * h] * by, o[j][2 * h + 1] * by);
                            if (a.lse && t == 0)
                                a.lse[at] = sum[h] == 0.0f ? -INFINITY : top[h] * kLn2 + logf(sum[h]);
                        }
                    }
                    if (a.slot_by_item && lane == 0)
                        a.jobs[static_cast<int64_t>(c.b) * items + c.item] = AttendJob{-1, -1, 0, 0};
                } else {
                    const int64_t part = (static_cast<int64_t>(worker) * 2 + (whole ? 1 : 0)) * a.part_rows;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = g + 8 * h;
                        if (r >= rows) continue;
                        if (t == 0) a.part_ml[part + r] = make_float2(top[h], sum[h]);
                        float *po = a.part_o + (part + r) * DP;
#pragma unroll
                        for (int j = 0; j < kCols; ++j)
                            *reinterpret_cast<float2 *>(po + j * 8 + 2 * t) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
                    }
                    if (whole) {      // the others' parts follow
                        const long long end = first + i + (c.s.tiles - c.tile);
                        job = AttendJob{worker, static_cast<int>((end - 1) / share), c.b, c.item};
                        if (a.slot_by_item && lane == 0) a.jobs[static_cast<int64_t>(c.b) * items + c.item] = job;
                    }
                }
                fresh = whole = true;
            }
            advance(a, c, &bad);
        }
        cp_async_wait<0>();
    }
    if (!a.slot_by_item && lane == 0) a.jobs[worker] = job;
    const bool any = __any_sync(0xffffffffu, bad);
    if (lane == 0) a.flags[worker] = any;
}

// The parts of an item that several workers share, a block for each job and
// row: the parts' weights first, then their sums, kJoinWarps parts at a time.
constexpr int kJoinWarps = 16;

template <bool BF16, int DP>
__global__ void __launch_bounds__(32 * kJoinWarps) attend_join_kernel(const __grid_constant__ AttendArgs a)
{
    extern __shared__ float weight[];     // [workers]
    __shared__ float sums[kJoinWarps][DP];
    __shared__ float red[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        int bad = 0;
        for (int w = threadIdx.x; w < a.workers; w += 32 * kJoinWarps) bad |= a.flags[w];
        const int any = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.err = any ? kDevErrPage : 0;
    }
    const AttendJob job = a.jobs[blockIdx.x];
    const int row = blockIdx.y;
    if (job.first < 0) return;
    const int kv_head = job.item / a.blocks, block = job.item - kv_head * a.blocks;
    if (row >= a.group - block * kAttendRows) return;
    const int parts = job.last - job.first + 1;
    auto part = [&](int i) { return (static_cast<int64_t>(job.first + i) * 2 + (i == 0 ? 1 : 0)) * a.part_rows + row; };

    float top = -INFINITY;
    for (int i = threadIdx.x; i < parts; i += 32 * kJoinWarps) top = fmaxf(top, a.part_ml[part(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) red[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, red[w]);
    const float off = top == -INFINITY ? 0.0f : top;
    for (int i = threadIdx.x; i < parts; i += 32 * kJoinWarps) weight[i] = exp2f(a.part_ml[part(i)].x - off);
    __syncthreads();
    // (every warp sums the denominators the same way)
    float total = 0.0f;
    for (int i = lane; i < parts; i += 32) total += weight[i] * a.part_ml[part(i)].y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);

    constexpr int kEach = DP / 32;
    float acc[kEach] = {};
#pragma unroll 4
    for (int i = warp; i < parts; i += kJoinWarps) {
        const float *po = a.part_o + part(i) * DP;
        const float w = weight[i];
#pragma unroll
        for (int e = 0; e < kEach; ++e) acc[e] += w * po[e * 32 + lane];
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) sums[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    const int64_t at = static_cast<int64_t>(job.row) * a.H + kv_head * a.group + block * kAttendRows + row;
    const float by = total == 0.0f ? 0.0f : 1.0f / total;
    if (threadIdx.x < DP / 2 && static_cast<int>(threadIdx.x) * 2 < a.D) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            x += sums[w][2 * threadIdx.x];
            y += sums[w][2 * threadIdx.x + 1];
        }
        *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at * a.D + 2 * threadIdx.x) =
            pack16<BF16>(x * by, y * by);
    }
    if (a.lse && threadIdx.x == 0) a.lse[at] = total == 0.0f ? -INFINITY : top * kLn2 + logf(total);
}

template <bool BF16, int DP>
cudaError_t attend(const AttendArgs &a, cudaStream_t stream)
{
    constexpr int kWarps = DP == 256 ? 4 : 8;
    constexpr int kSmem = kWarps * warp_bytes(DP);
    // (an attribute of the device's copy of the function: set at every call,
    // as the current device may be another)
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<BF16, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attend_kernel<BF16, DP><<<a.workers / kWarps, 32 * kWarps, kSmem, stream>>>(a);
    return cudaGetLastError();
}

template <bool BF16, int DP>
cudaError_t join(const AttendArgs &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.slots), static_cast<unsigned>(a.part_rows));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.workers) * sizeof(float);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_join_kernel<BF16, DP>, a);
}

template <bool BF16>
cudaError_t by_dim(bool joining, const AttendArgs &a, cudaStream_t stream)
{
    switch (attend_dim(a.D)) {
    case 64: return joining ? join<BF16, 64>(a, stream) : attend<BF16, 64>(a, stream);
    case 128: return joining ? join<BF16, 128>(a, stream) : attend<BF16, 128>(a, stream);
    default: return joining ? join<BF16, 256>(a, stream) : attend<BF16, 256>(a, stream);
    }
}

}  // namespace

int launch_attend(bool bf16, const AttendArgs &a, cudaStream_t stream)
{
    const cudaError_t e = bf16 ? by_dim<true>(false, a, stream) : by_dim<false>(false, a, stream);
    return e == cudaSuccess ? 0 : record_cuda_error("paged attention launch", e, cudaGetErrorString(e));
}

int launch_attend_join(bool bf16, const AttendArgs &a, cudaStream_t stream)
{
    const cudaError_t e = bf16 ? by_dim<true>(true, a, stream) : by_dim<false>(true, a, stream);
    return e == cudaSuccess ? 0 : record_cuda_error("paged attention join launch", e, cudaGetErrorString(e));
}

}  // namespace ngr
