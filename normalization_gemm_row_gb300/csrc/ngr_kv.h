// ngr_kv.h -- argument blocks of the paged key-value cache's kernels: the
// rotated append (ngr_append.cu) and the attention of one new token
// (ngr_attend.cuh).  Not installed.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace ngr {

// The caches [pages, page_size, heads, dim] by their strides in elements, and
// the block table [rows, table_stride] whose rows' first table_pages entries
// are pages.
struct KvView {
    void *k, *v;
    int64_t k_page, k_token, k_head, v_page, v_token, v_head;
    const int *table;
    int64_t table_stride;
    int64_t capacity;     // tokens that a row of the table has room for
    int pages, page_size, rows;
    // token / page_size for 31-bit tokens: the high word of the product with
    // page_mul shifted down by page_sh (page_mul 0: pages of one token)
    uint32_t page_mul, page_sh;
};

struct AppendArgs {
    KvView kv;
    const void *q, *k, *v;    // q may be null
    void *q_out;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head, qo_token, qo_head;
    const int *positions, *rows;   // rows null: token t's is t
    const float *inv_freq;
    int *err;                 // null: nothing is reported
    int T, H, G, D, rot;
    int units, blocks_per_token, threads, each;     // units of a head; of `each` heads a thread
};
constexpr int kAppendThreads = 256;    // a block, at most
constexpr int kAppendEach = 4;         // heads a thread of a large call
// vec: elements that one access moves (8, 4, 2 or 1).
int launch_append(bool bf16, int vec, bool interleaved, const AppendArgs &a, cudaStream_t stream);
// Units (pairs of accesses) of a head, at most kAppendThreads.
int append_units(int vec, bool interleaved, int64_t D, int64_t rot);

constexpr int kAttendMaxDim = 256;
constexpr int kAttendRows = 16;    // query heads of one key head that a warp takes at once
constexpr int kAttendTile = 16;    // tokens a warp takes at once
constexpr int kAttendSms = 152;    // sizing must not ask a device
// Query heads of a key head: their blocks have a warp each, of four an SM at
// 256 dimensions.
constexpr int kAttendMaxGroup = kAttendRows * kAttendSms * 4;

// An item whose tokens several workers (warps) share.  Each leaves its part
// of it, [part_rows] (maximum, sum) and [part_rows][dim padded] sums in FP32:
// in the second of a worker's two places if the part begins the item.  An
// item's parts lie one after the other (a group's together: the join took 18
// instead of 12 us at 512 items).
struct AttendJob {
    int first, last;     // the workers' groups; first < 0: no job
    int row, item;       // sequence, (key head, block of query heads)
};

struct AttendArgs {
    KvView kv;
    // the view's strides in 16-byte units: no offset passes 32 bits
    uint32_t k_page, k_token, k_head, v_page, v_token, v_head;
    bool alike;               // v's are k's
    const void *q;
    int64_t q_row, q_head;
    const int *lengths;
    void *out;                // [B, H, D]
    float *lse;               // [B, H] or null
    float scale2;             // softmax scale x log2 e
    int window;               // 0: none
    int B, H, G, D;
    int group, blocks;        // query heads of a key head; blocks of kAttendRows of them
    int workers, groups, min_share;
    int part_rows;            // query heads in a part: at most kAttendRows
    int slots;                // jobs: one an item, or one a worker if there are fewer
    bool slot_by_item;
    float2 *part_ml;          // [items of a row][groups][2][rows]
    float *part_o;            // [items of a row][groups][2][rows][dim padded]
    AttendJob *jobs;
    int *flags;               // [workers]
    int *err;
    bool err_keep;            // what an earlier launch of the call reported stays
};

// The padded head dimension (the kernels are built for these), the blocks of 8
// query heads a warp takes at once, and the warps of a CTA: as many as their
// registers (64 for the sums of 8 heads and 256 dimensions) leave room for.
inline int attend_dim(int64_t D)
{
    return D == 80 || D == 96 || D == 192 ? static_cast<int>(D) : D <= 64 ? 64 : D <= 128 ? 128 : 256;
}
inline int attend_heads(int64_t group) { return group <= 8 ? 1 : 2; }
constexpr int attend_warps(int dim, int heads) { return dim * heads <= 128 ? 16 : dim * heads <= 256 ? 8 : 4; }
int launch_attend_bf16(const AttendArgs &a, cudaStream_t stream);
int launch_attend_f16(const AttendArgs &a, cudaStream_t stream);
int launch_attend_solo_bf16(const AttendArgs &a, cudaStream_t stream);
int launch_attend_solo_f16(const AttendArgs &a, cudaStream_t stream);
int launch_attend_join_bf16(const AttendArgs &a, cudaStream_t stream);
int launch_attend_join_f16(const AttendArgs &a, cudaStream_t stream);

}  // namespace ngr
