// ngr_ce_ptx.cuh -- inline-PTX wrappers that the cross entropy's products use
// beside those of ngr_ptx.cuh: one elected lane, MN-major operands, tiled
// stores, another L2 policy.
#pragma once

#include "ngr_ptx.cuh"

namespace ngr {

// True in one lane of a converged warp.  A role that issues tcgen05 or TMA
// instructions from one thread is entered through this and not through
// "lane == 0": the compiler then knows the thread to be one, and the
// instructions take their descriptors without a detour (measured on the
// cross entropy's products: 500 clocks a k block to issue with lane == 0,
// about what its products take, and 16 % off the kernel's time without).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Shared-memory matrix descriptor for an MN-major operand tile (the rows or
// columns of the output are contiguous, K strides) in the 128-byte swizzle
// layout: each TMA box is 64 output rows (128 bytes) x 64 k, k rows 128
// bytes apart, so 8-k groups lie 1024 bytes apart (the stride byte offset)
// and the boxes of further 64 output rows `box_bytes` apart (the leading
// byte offset).  Advancing K by 16 adds 2048 bytes to the start address.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr, uint32_t box_bytes)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(box_bytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// Instruction descriptor of idesc_f16 with A and/or B MN-major (the transpose
// bits 15 and 16).
__host__ __device__ constexpr uint32_t idesc_f16_major(bool bf16, int M, int N, bool a_mn, bool b_mn)
{
    return idesc_f16(bf16, M, N) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16);
}

// 2-D tiled store of the box at (c0, c1) from shared memory; elements past
// the tensor's end are not written.  The thread's stores so far form a group
// (commit); `wait_read`: their shared memory may be written again; `wait`:
// they are complete.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, const void *src, int c0, int c1)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void tma_store_commit()
{
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait()
{
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// The default L2 eviction priority as a policy for the cache_hint operand.
__device__ __forceinline__ uint64_t policy_evict_normal()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
}  // namespace ngr
