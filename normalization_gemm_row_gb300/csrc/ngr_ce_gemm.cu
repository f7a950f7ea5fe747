// ngr_ce_gemm.cu -- the products of the linear cross entropy on CTA pairs
// (tcgen05 cta_group::2), 256 x 256 output tiles, with the softmax's work in
// the epilogue:
//
//   kCeLse   z = x W^T by tiles; a tile leaves (max, sum exp) of each row's
//            columns and the target's logit, so no logit reaches HBM;
//   kCeGrad  the same product again over a piece of the vocabulary, turned
//            into dz = weight_p p - weight_t [v = target] with p = exp(z - lse);
//   kCeDx    dx (+)= dz W over the piece;
//   kCeDw    dW = dz^T x for the piece's rows of W.
//
// Operands are read as they lie: x and W rows are K-major for z; W's rows
// are the contracted index of dx, dz's and x's rows that of dW, so those
// operands are MN-major, which the tensor core reads through a transposed
// shared-memory descriptor; nothing is transposed in memory.
//
// The tensor core adds each step's products to the FP32 accumulator without
// rounding to nearest, so over a long contracted length an element loses up
// to a part in 2^24 a step, always towards zero (measured: 6e-5 of a logit
// after the 256 steps of K = 4096).  Every kChunk k blocks the accumulator is
// therefore handed to the epilogue, which keeps the output in registers
// (a row of up to 128 columns a thread) and adds the pieces there, rounding to nearest; the
// loss's error against 64 bits falls from 5e-6 to below 1e-6, and the reads
// hide under the products of the next piece.
//
// Bound by the tensor cores for batches of tokens, by reading W (or writing
// dW) for a few tokens.  Per CTA a stage is 16 KB of A and 16 KB of B, six
// stages deep; the two 256-column accumulators take turns, so the epilogue (8
// warps, two per tensor-memory lane quarter; 16 were 10 % slower) runs under
// the next products.
//
// Warp roles: 0 TMA producer (and tensor memory), 1 MMA issuer (even CTA),
// 4-11 epilogue.  Barriers as in the CTA-pair tile kernel without a norm: full[s]
// on the leader, on which both CTAs' copies complete; empty[s] the leader's
// commit to both; acc_full[a] the same at a tile's end; acc_empty[a] on the
// leader, one arrival per epilogue warp of both CTAs.
#include "ngr_ce.h"
#include "ngr_ce_ptx.cuh"
#include "ngr_entry.h"
#include "ngr_gemm_kernel.cuh"

#include <cstdio>

namespace ngr {

namespace {

constexpr int kCeEpilogueWarp0 = 4;
constexpr int kCeEpilogueWarps = 8;
constexpr int kCeThreads = 32 * (kCeEpilogueWarp0 + kCeEpilogueWarps);
constexpr int kCePart = 128;                              // columns of a tile an epilogue warp takes at most
// k blocks per accumulator: short for the logits, whose error shows in the
// loss and, through the exponential, in dz; dx and dW are rounded to 16 bits.
template <int MODE>
__device__ __forceinline__ constexpr int ce_chunk() { return MODE == kCeLse || MODE == kCeGrad ? 8 : 32; }
constexpr int kCeOperand = kBM * kBK * 2;                 // 16 KB: a CTA's half of A or B
constexpr int kCeBox = 64 * kBK * 2;                      // an MN-major box of 64 x 64
constexpr int kCeOutBox = 64 * 32 * 2;                    // 64 columns of a warp's 32 rows of the output
constexpr int kCeOut = kCeEpilogueWarps * 2 * kCeOutBox;
// Pipeline stages of 32 KB a CTA: reading W for a few tokens takes six (177
// us at 33 x 8192 x 65536, 208 with four); dW, which reads little then and
// is bound by its writes, gives two of them to its output boxes.
template <int MODE>
__host__ __device__ constexpr int ce_stages() { return MODE == kCeDw ? 4 : 6; }
template <int MODE>
constexpr int ce_smem()
{
    return ce_stages<MODE>() * 2 * kCeOperand + (MODE == kCeDw ? kCeOut : 0) + 8 * (2 * ce_stages<MODE>() + 5) + 16 + 1024;
}

__device__ __forceinline__ float exp2_approx(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ void ld_global_v8(const float *p, float (&v)[8])
{
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                   "=f"(v[7])
                 : "l"(p)
                 : "memory");
}

// The first `n` of 128 values into a row of 16-bit values at `p`: whole
// sectors, 16-byte pieces or single elements by the address and n.
template <bool BF16>
__device__ __forceinline__ void store16(const float (&v)[kCePart], uint16_t *p, int n)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (n == kCePart && (at & 31u) == 0) {   // nearly always
#pragma unroll
        for (int c = 0; c < kCePart; c += 16) {
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = from_float2<BF16>(v[c + 2 * j], v[c + 2 * j + 1]);
            st_global_v8(p + c, o);
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < kCePart; c += 16) {
        if (c >= n) break;
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = from_float2<BF16>(v[c + 2 * j], v[c + 2 * j + 1]);
        if (c + 16 <= n && (at & 31u) == 0) {
            st_global_v8(p + c, o);
        } else if (n % 8 == 0 && (at & 15u) == 0) {
            *reinterpret_cast<uint4 *>(p + c) = make_uint4(o[0], o[1], o[2], o[3]);
            if (c + 16 <= n) *reinterpret_cast<uint4 *>(p + c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < n) p[c + j] = static_cast<uint16_t>(o[j >> 1] >> (16 * (j & 1)));
        }
    }
}

// A warp's 32 rows of 128 values to the output at row0, column c, by way of
// its own two 4 KB boxes of 64 columns in shared memory (the 128-byte
// swizzle), so that whole lines go to memory: stores by rows from 32 lanes
// write a sector of 32 lines each (dW of 33 tokens, 65536 x 8192: 317 us so,
// 217 through the boxes).  With a tensor map one lane stores the boxes; where
// the output's rows start at any element the warp writes row after row, two
// elements a lane on 4-byte boundaries.
template <bool BF16>
__device__ __forceinline__ void store_boxes(const float (&v)[kCePart], uint8_t *box, const CeGemmArgs &args, int c,
                                            int row0, int lane)
{
    if (lane == 0) tma_store_wait_read();   // the last tile's stores have read it
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kCePart / 8; ++i) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = from_float2<BF16>(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
        *reinterpret_cast<uint4 *>(box + (i >> 3) * kCeOutBox + lane * 128 + (((i & 7) ^ (lane & 7)) << 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (args.boxes) fence_proxy_async_smem();
    __syncwarp();
    if (args.boxes) {
        if (lane == 0) {
            if (row0 < args.rows) {
                tma_store_2d(&args.map_out, box, c, row0);
                if (c + 64 < args.cols) tma_store_2d(&args.map_out, box + kCeOutBox, c + 64, row0);
            }
            tma_store_commit();
        }
        return;
    }
    const int n = min(kCePart, args.cols - c);
#pragma unroll 1
    for (int r = 0; r < 32 && row0 + r < args.rows; ++r) {
        uint16_t *p = static_cast<uint16_t *>(args.out) + static_cast<int64_t>(row0 + r) * args.pitch + c;
        auto at = [&](int k) {
            return *reinterpret_cast<const uint16_t *>(box + (k >> 6) * kCeOutBox + r * 128 +
                                                       ((((k & 63) >> 3) ^ (r & 7)) << 4) + (k & 7) * 2);
        };
        const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
        if (odd && lane == 0) p[0] = at(0);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = odd + 2 * (32 * j + lane);
            if (k + 1 < n) *reinterpret_cast<uint32_t *>(p + k) = at(k) | (static_cast<uint32_t>(at(k + 1)) << 16);
            else if (k < n) p[k] = at(k);
        }
    }
}

// The output tiles of a call and the order they run in.
template <int MODE>
struct CeUnits {
    int tiles, slow, kb_all, splits, kb_per_split;   // `fast` dimension first
    int fast, width;
    __device__ __forceinline__ CeUnits(const CeGemmArgs &a)
    {
        // (no counted token: one tile of zero rows, so that dW is written)
        const int n = max(a.info->count, 1);
        const int m_tiles = ((MODE == kCeDw ? a.rows : n) + kCeTile - 1) / kCeTile;
        width = a.width;
        const int n_tiles = (a.cols + width - 1) / width;
        // z: the row tiles of one column tile run together, so W is read
        // once; dx, dW: the column tiles of one row tile, so dz is.
        constexpr bool kRowsFast = MODE == kCeLse || MODE == kCeGrad;
        fast = kRowsFast ? m_tiles : n_tiles;
        slow = kRowsFast ? n_tiles : m_tiles;
        tiles = m_tiles * n_tiles;
        kb_all = ((MODE == kCeDw ? n : a.depth) + kBK - 1) / kBK;
        splits = MODE == kCeDx ? a.splits : 1;
        kb_per_split = (kb_all + splits - 1) / splits;
    }
    __device__ __forceinline__ int count() const { return tiles * splits; }
    __device__ __forceinline__ int m0(int u) const
    {
        const int t = u / splits;
        return ((MODE == kCeLse || MODE == kCeGrad) ? t % fast : t / fast) * kCeTile;
    }
    __device__ __forceinline__ int n0(int u) const
    {
        const int t = u / splits;
        return ((MODE == kCeLse || MODE == kCeGrad) ? t / fast : t % fast) * width;
    }
    __device__ __forceinline__ int split(int u) const { return u % splits; }
    __device__ __forceinline__ int kb0(int u) const { return min(kb_all, split(u) * kb_per_split); }
    __device__ __forceinline__ int kb1(int u) const { return min(kb_all, (split(u) + 1) * kb_per_split); }
};

template <int MODE, bool BF16>
__global__ void __launch_bounds__(kCeThreads, 1) ce_gemm_kernel(const __grid_constant__ CeGemmArgs args)
{
    constexpr bool kAMn = MODE == kCeDw;
    constexpr bool kBMn = MODE == kCeDx || MODE == kCeDw;
    const int width = args.width;                            // columns of a tile
    const uint32_t idesc = idesc_f16_major(BF16, kCeTile, width, kAMn, kBMn);
    // both CTAs' copies of a stage (an MN-major B is copied in boxes of 64)
    const uint32_t stage_bytes = 2u * (kCeOperand + (kBMn ? (width / 2 + 63) / 64 * kCeBox : width / 2 * kBK * 2));
    constexpr int kChunk = ce_chunk<MODE>();

    constexpr int kCeStages = ce_stages<MODE>();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sA = smem;
    uint8_t *sB = smem + kCeStages * kCeOperand;
    uint8_t *sOut = smem + 2 * kCeStages * kCeOperand;
    uint64_t *full = reinterpret_cast<uint64_t *>(sOut + (MODE == kCeDw ? kCeOut : 0));
    uint64_t *empty = full + kCeStages;
    uint64_t *acc_full = empty + kCeStages;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    __shared__ int abort_flag;
    const WaitCtx wc{&abort_flag, args.err, args.timeout_ns};

    if (threadIdx.x == 0) {
        abort_flag = 0;
        prefetch_tmap(&args.map_a);
        prefetch_tmap(&args.map_b);
        for (int s = 0; s < kCeStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kCeEpilogueWarps);
        }
        mbar_init(drain, 1);
        fence_mbarrier_init();
    }
    if (warp == 0) {
        __syncwarp();
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // Launched as a programmatic dependent of the kernel before it.  dW reads
    // nothing that dx writes, and dz is complete once dx has begun its work:
    // launched behind dx it fills the SMs that dx's last tiles leave free and
    // waits for dx only at its end.  (So dx lets its dependent start after its
    // own wait for dz and not before.)
    if constexpr (MODE == kCeDx) pdl_wait();
    pdl_launch_dependents();
    if constexpr (MODE == kCeLse || MODE == kCeGrad) pdl_wait();

    const CeUnits<MODE> units(args);
    const int n_units = units.count();
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
    const uint32_t acc_empty_leader = mapa_shared(smem_u32(acc_empty), 0);

    if (warp == 0) {
        if (elect_one()) {
            // z: x stays in L2, W streams through.  dx: W's piece stays, unless
            // one row tile reads it once, and dz is read again by every column
            // tile (3 % faster than streaming it); dW: x stays.
            const uint64_t keep = policy_evict_last(), stream = policy_evict_first();
            constexpr bool kZ = MODE == kCeLse || MODE == kCeGrad;
            const uint64_t pol_a = kZ ? keep : MODE == kCeDx ? policy_evict_normal() : stream;
            const uint64_t pol_b = kZ || (MODE == kCeDx && units.slow == 1) ? stream : keep;
            int stage = 0;
            uint32_t phase = 0;
            long long fills = 0;
            bool ok = true;
            for (int u = first; ok && u < n_units; u += step) {
                const int m0 = units.m0(u) + static_cast<int>(rank) * kBM;
                const int n0 = units.n0(u) + static_cast<int>(rank) * (width / 2);
                for (int kb = units.kb0(u), end = units.kb1(u); kb < end; ++kb) {
                    if (!mbar_wait_ahead(&empty[stage], phase ^ 1u, wc)) { ok = false; break; }
                    const int kc = kb * kBK;
                    uint8_t *a = sA + stage * kCeOperand, *b = sB + stage * kCeOperand;
                    const uint32_t fb = full_leader + 8u * static_cast<uint32_t>(stage);
                    if (leader) mbar_arrive_expect_tx(&full[stage], stage_bytes);
                    if constexpr (kAMn) {
                        tma_load_2d_pair(a, &args.map_a, fb, m0, kc, pol_a);
                        tma_load_2d_pair(a + kCeBox, &args.map_a, fb, m0 + 64, kc, pol_a);
                    } else {
                        tma_load_2d_pair(a, &args.map_a, fb, kc, m0, pol_a);
                    }
                    if constexpr (kBMn) {
                        tma_load_2d_pair(b, &args.map_b, fb, n0, kc, pol_b);
                        if (width > 128) tma_load_2d_pair(b + kCeBox, &args.map_b, fb, n0 + 64, kc, pol_b);
                    } else {
                        tma_load_2d_pair(b, &args.map_b, fb, kc, n0, pol_b);
                    }
                    ++fills;
                    if (++stage == kCeStages) { stage = 0; phase ^= 1u; }
                }
            }
            // All copies complete on the leader's barriers: it waits for the
            // last fills before the pair leaves.
            if (leader) {
                const int outstanding = fills < kCeStages ? static_cast<int>(fills) : kCeStages;
                for (int j = 1; j <= outstanding; ++j) {
                    int s = stage - j;
                    uint32_t p = phase;
                    if (s < 0) { s += kCeStages; p ^= 1u; }
                    mbar_wait(&full[s], p, wc);
                }
            }
        }
    } else if (warp == 1) {
        if (leader && elect_one()) {
            // descriptors of stage 0; further stages and k steps add to the
            // address field (16-byte units)
            const uint64_t a0 = kAMn ? sdesc_mnmajor_sw128(smem_u32(sA), kCeBox) : sdesc_kmajor_sw128(smem_u32(sA));
            const uint64_t b0 = kBMn ? sdesc_mnmajor_sw128(smem_u32(sB), kCeBox) : sdesc_kmajor_sw128(smem_u32(sB));
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int u = first; ok && u < n_units; u += step) {
                int left = 0;   // k blocks until the accumulator is handed over
                for (int kb = units.kb0(u), end = units.kb1(u); kb < end; ++kb) {
                    const bool fresh = left == 0;
                    if (fresh) {
                        if (!mbar_wait_spin(&acc_empty[acc], acc_phase ^ 1u, wc)) { ok = false; break; }
                        left = min(kChunk, end - kb);
                    }
                    if (!mbar_wait_spin(&full[stage], phase, wc)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kCeTile);
                    const uint64_t a = a0 + static_cast<uint32_t>(stage * (kCeOperand >> 4));
                    const uint64_t b = b0 + static_cast<uint32_t>(stage * (kCeOperand >> 4));
#pragma unroll
                    for (int k = 0; k < kBK / kUmmaK; ++k) {
                        // (16 k on: 2048 bytes in an MN-major tile, 32 in a K-major one)
                        umma_f16_ss_pair(d, a + static_cast<uint32_t>(k * (kAMn ? 128 : 2)),
                                         b + static_cast<uint32_t>(k * (kBMn ? 128 : 2)), idesc,
                                         (!fresh || k != 0) ? 1u : 0u);
                    }
                    umma_commit_pair(&empty[stage], 0x3);
                    if (++stage == kCeStages) { stage = 0; phase ^= 1u; }
                    if (--left == 0) {
                        umma_commit_pair(&acc_full[acc], 0x3);
                        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
                    }
                }
            }
            umma_commit_pair(drain, 0x1);
            mbar_wait_long(drain, 0, wc);
        }
    } else if (warp >= kCeEpilogueWarp0) {
        const int q = warp & 3;                               // tensor-memory lane quarter
        const int piece = (warp - kCeEpilogueWarp0) >> 2;     // columns [piece width / 2, + width / 2)
        const int n_piece = width >> 1;
        uint8_t *const out_box = sOut + (warp - kCeEpilogueWarp0) * 2 * kCeOutBox;
        const int count = args.info->count;
        const float down = args.info->down;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int u = first; u < n_units; u += step) {
            const int row = units.m0(u) + static_cast<int>(rank) * kBM + q * 32 + lane;
            const int c0 = units.n0(u) + piece * n_piece;
            CeRow cr{0.0f, 0.0f, 0.0f, -1};
            int target = -1;
            if constexpr (MODE == kCeGrad) {
                if (row < count) cr = args.row[row];
                target = cr.target - args.v0 - c0;
            }
            if constexpr (MODE == kCeLse) {
                if (row < count) target = args.target[row] - c0;
            }
            float v[kCePart];
#pragma unroll
            for (int j = 0; j < kCePart; ++j) v[j] = 0.0f;
            bool ok = true;
            for (int kb = units.kb0(u), end = units.kb1(u); kb < end; kb += kChunk) {
                if (!mbar_wait_warp_long(&acc_full[acc], acc_phase, wc)) { ok = false; break; }
                tc_fence_after();
                // (columns past the piece are read along and not used)
                const uint32_t t0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                    static_cast<uint32_t>(acc * kCeTile + piece * n_piece);
#pragma unroll
                for (int c = 0; c < kCePart; c += 16) {
                    uint32_t r[16];
                    tmem_ld16(t0 + static_cast<uint32_t>(c), r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[c + j] += __uint_as_float(r[j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(acc_empty_leader + 8u * static_cast<uint32_t>(acc));
                if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
            }
            if (!ok) break;
            const int cols = min(n_piece, args.cols - c0);   // this warp's columns (may be <= 0)
            // (kCeLse: a piece past the vocabulary leaves the pair of an empty sum)
            if (MODE != kCeLse && cols <= 0) continue;
            if constexpr (MODE == kCeLse) {
                if (target >= 0 && target < cols) {
                    float z = 0.0f;
#pragma unroll
                    for (int j = 0; j < kCePart; ++j) z = target == j ? v[j] : z;
                    args.z_target[row] = z * args.scale;
                }
                float m[4], e[4];
#pragma unroll
                for (int j = 0; j < kCePart; ++j) {
                    v[j] = cols < kCePart && j >= cols ? -INFINITY : v[j] * args.scale2;
                    m[j & 3] = j < 4 ? v[j] : fmaxf(m[j & 3], v[j]);
                }
                const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                // (every logit -inf: their sum stays zero; one +inf: inf, not NaN)
                const float base = fabsf(top) == INFINITY ? 0.0f : top;
#pragma unroll
                for (int j = 0; j < kCePart; ++j) {
                    const float x = exp2_approx(v[j] - base);
                    e[j & 3] = j < 4 ? x : e[j & 3] + x;
                }
                if (row < count)
                    args.part[static_cast<int64_t>(units.n0(u) / width * 2 + piece) * args.part_pitch + row] =
                        make_float2(top, (e[0] + e[1]) + (e[2] + e[3]));
            } else if constexpr (MODE == kCeGrad) {
#pragma unroll
                for (int j = 0; j < kCePart; ++j) {
                    v[j] = exp2_approx(fmaf(v[j], args.scale2, -cr.lse2)) * cr.weight_p;
                    if (target == j) v[j] -= cr.weight_t;
                    // rows behind the counted tokens: x there may be anything
                    if (row >= count) v[j] = 0.0f;
                }
                store16<BF16>(v, static_cast<uint16_t *>(args.out) + static_cast<int64_t>(row) * args.pitch + c0, cols);
            } else if constexpr (MODE == kCeDw) {
#pragma unroll
                for (int j = 0; j < kCePart; ++j) v[j] *= down;
                store_boxes<BF16>(v, out_box, args, c0, row - lane, lane);
            } else if (row < count) {
                // (rows of sums are padded: whole sectors always)
                float *s = args.sums + (units.split(u) * args.sums_rows + row) * args.sums_pitch + c0;
#pragma unroll
                for (int c = 0; c < kCePart; c += 8) {
                    if (c >= cols || !args.add) break;
                    float o[8];
                    ld_global_v8(s + c, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[c + i] += o[i];
                }
                if (args.finish) {
#pragma unroll
                    for (int j = 0; j < kCePart; ++j) v[j] *= down;
                    store16<BF16>(v, static_cast<uint16_t *>(args.out) +
                                         static_cast<int64_t>(args.index[row]) * args.pitch + c0, cols);
                } else {
#pragma unroll
                    for (int c = 0; c < kCePart; c += 8) {
                        if (c >= cols) break;
                        uint32_t o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(v[c + i]);
                        st_global_v8(s + c, o);
                    }
                }
            }
        }
    }

    // The boxes of the last tiles are written out before the shared memory goes.
    if (MODE == kCeDw && lane == 0 && warp >= kCeEpilogueWarp0) tma_store_wait();
    if (MODE == kCeDw) pdl_wait();
    // Neither CTA frees its tensor memory or leaves while the pair may still
    // touch it.
    tc_fence_before();
    cluster_sync_all();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

template <int MODE, bool BF16>
int run(const CeGemmArgs &a, int grid, cudaStream_t stream)
{
    auto kern = ce_gemm_kernel<MODE, BF16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (ce_smem<MODE>()));
    if (e != cudaSuccess)
        return record_cuda_error("cudaFuncSetAttribute(max dynamic smem)", e, cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kCeThreads);
    cfg.dynamicSmemBytes = ce_smem<MODE>();
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.after_dx || MODE != kCeDw ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    return e == cudaSuccess ? 0 : record_cuda_error("cudaLaunchKernelEx (cross entropy)", e, cudaGetErrorString(e));
}

// Resident CTA pairs of the product kernels.
int ce_clusters()
{
    auto kern = ce_gemm_kernel<kCeLse, true>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (ce_smem<kCeLse>())) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kCeThreads);
    cfg.dynamicSmemBytes = ce_smem<kCeLse>();
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess ? n : 0;
}

}  // namespace

int launch_ce_gemm(int mode, bool bf16, const CeGemmArgs &a, int64_t units, cudaStream_t stream)
{
    // The kernel is persistent and its CTA pairs wait for nothing of one
    // another, so any number of them is right; as many as fit are fastest.
    static thread_local int clusters = 0;
    if (clusters == 0) clusters = ce_clusters();
    const int64_t most = clusters > 0 ? clusters : 64;
    const int grid = 2 * static_cast<int>(units < most ? units : most);
    if (trace_mode())
        std::fprintf(stderr, "ngr: cross entropy %s: %d columns, width=%d splits=%d grid=%d\n",
                     mode == kCeLse ? "z" : mode == kCeGrad ? "dz" : mode == kCeDx ? "dx" : "dW", a.cols, a.width,
                     a.splits, grid);
#define NGR_CE(M_)      \
    case M_: return bf16 ? run<M_, true>(a, grid, stream) : run<M_, false>(a, grid, stream);
    switch (mode) {
        NGR_CE(kCeLse)
        NGR_CE(kCeGrad)
        NGR_CE(kCeDx)
        NGR_CE(kCeDw)
    }
#undef NGR_CE
    return -9;
}

}  // namespace ngr
