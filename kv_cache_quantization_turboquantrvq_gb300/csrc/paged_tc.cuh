// paged_tc.cuh - 128 x 128 x 128 products of query and key tiles on the 5th-generation
// tensor cores, shared by the kernels over chunks (paged_chunk.cu, paged_weigh.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "paged.h"
#include "tcgen05.cuh"

namespace vq {
namespace {

constexpr int TILE_B = PG_TILE * 128 * 2;  // a 16-bit tile of 128 rows: two halves of 64 columns
constexpr int HALF_B = TILE_B / 2;
constexpr int RAW_B = PG_TILE * 128;       // a tile of codes

// Instruction descriptor: fp32 accumulator, M = N = 128, both operands fp16 or
// both bf16; `b_mn`: B has its N dimension contiguous.
__host__ __device__ constexpr uint32_t ck_idesc(bool bf16, bool b_mn)
{
    return qt_idesc(128) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u);
}

// The products of one 128 x 128 x 128 tile, eight K = 16 steps, by one elected
// thread of the (whole, converged) warp.  One block of PTX each, so that the
// operands' addresses stay in uniform registers: issued one by one from a
// branch on the lane number, an instruction took 107 cycles to issue where the
// tensor core needs 64.  `bar` (shared) gets an arrival when they are done.

// D = A B, both from shared memory, rows of 64 entries: steps 32 bytes apart,
// the second half of K HALF_B further.
__device__ __forceinline__ void ck_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t bar)
{
    static_assert(HALF_B == 16384, "the descriptors' steps below");
    asm volatile(
        "{\n\t.reg .pred q, f, t;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 t, 1, 0;\n\tsetp.ne.b32 f, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\tadd.s64 a4, %1, 1024;\n\t"
        "add.s64 a5, %1, 1026;\n\tadd.s64 a6, %1, 1028;\n\tadd.s64 a7, %1, 1030;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\tadd.s64 b4, %2, 1024;\n\t"
        "add.s64 b5, %2, 1026;\n\tadd.s64 b6, %2, 1028;\n\tadd.s64 b7, %2, 1030;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, t;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(bar)
        : "memory");
}

// An arrival on `bar` when every product that this warp's elected thread issued
// is done.
__device__ __forceinline__ void ck_commit(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// L2 policy of the cache's tiles: other CTAs read them too.
__device__ __forceinline__ uint64_t ck_policy()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

__device__ __forceinline__ float2 ck_f2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

// A word with its n lowest bits set (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t ck_below(int n) { return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u; }

template <class T> __device__ __forceinline__ uint32_t ck_pack(float a, float b);
template <> __device__ __forceinline__ uint32_t ck_pack<__half>(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t ck_pack<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace
}  // namespace vq
